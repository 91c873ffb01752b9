// attention_ex_kernel.cuh -- attention forward with capped scores, a distance
// bias, causal / document / prefix masks, shared key/value heads and strided
// tensors (the formulas stand in attention_common.cuh):
//
//     O_i = sum_j w_ij V_j,   w_ij = exp(y_ij - lse_i),   lse_i = log sum_j exp(y_ij)
//
// One CTA computes two 128-row query tiles of one head against one stream of
// 128-key blocks, the tiles in ping-pong: while one warpgroup turns a tile's
// scores into weights, the tensor core works on the other tile.  Tensor
// Memory holds, per tile, S_i (128 fp32 columns; the 16-bit weights P_i are
// written over its first 64) and O_i (D columns).  Each tile visits only the
// blocks that some of its rows see; inside, only blocks that cut a row's
// interval pay for masking.
//
// What bounds it: 4 D multiply-adds a pair at the tensor core's 8192 a clock
// and SM against one 2^x a pair at 16 a clock: 1024 clocks a tile and block each
// with D = 128; capped scores add the multiply-adds of tanh_scores.
//
// Warp roles (384 threads): warp 0 TMA producer, warp 1 TMEM allocator and MMA
// issuer, warps 2..3 idle, warps 4..7 softmax of tile 0, 8..11 of tile 1.
// Every wait is bounded.
#pragma once

#include "attention_common.cuh"

namespace tl {

struct AttnExParams {
    MaskParams mask;
    ScoreParams score;
    int32_t B, H, group;     // batch, query heads, query heads per key/value head
    int32_t num_pairs;       // pairs of 128-row query tiles
    uint16_t *O;
    int64_t o_batch, o_head, o_row;  // O's strides in elements
    float *lse;              // [B][H][Sq] natural log, or null
    uint64_t timeout_ns;
};

template <int D_>
struct AttnExConfig {
    static constexpr int D = D_;
    static constexpr int BM = 128, BN = 128;
    static constexpr int KS = D == 128 ? 2 : 4;            // K and V ring depth
    static constexpr int ATOM_BYTES = 128 * 128;           // 128 rows x 64 16-bit values
    static constexpr int D_ATOMS = D / 64;
    static constexpr int Q_BYTES = D_ATOMS * ATOM_BYTES;
    static constexpr int KV_BYTES = D_ATOMS * ATOM_BYTES;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + KS * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + KS * KV_BYTES;
    static constexpr int BAR_Q = 0, BAR_KF = 1, BAR_KE = 1 + KS, BAR_VF = 1 + 2 * KS, BAR_VE = 1 + 3 * KS;
    static constexpr int BAR_SF = 1 + 4 * KS;   // [tile]: S_i in Tensor Memory
    static constexpr int BAR_PF = BAR_SF + 2;   // [tile]: P_i in Tensor Memory (4 warps arrive)
    static constexpr int BAR_PV = BAR_PF + 2;   // [tile]: O_i += P_i V completed
    static constexpr int BAR_DRAIN = BAR_PV + 2;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;  // TMEM address, abort flag, the tiles' key ranges
    static constexpr int OFF_DOCS = OFF_MISC + 32;
    static constexpr int SMEM_BYTES = OFF_DOCS + kDocsInSmem * 4 + 1024;
    static constexpr int THREADS = 384;
    static constexpr int FIRST_SOFTMAX_WARP = 4;
    static constexpr int REGS_CONTROL = 64, REGS_SOFTMAX = 216;
    static constexpr int LAUNCH_REGS = (128 * REGS_CONTROL + 256 * REGS_SOFTMAX + THREADS - 1) / THREADS;
    static constexpr int TMEM_S = 0, TMEM_O = 256;  // S_i at 128 i, O_i at 256 + D i
    static constexpr float RESCALE_LOG2 = 8.0f;     // m moves when a row maximum exceeds it by 2^8
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

template <class CF, int DT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1)
    attention_ex_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const AttnExParams p)
{
    constexpr int D = CF::D;
    constexpr int KS = CF::KS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // blocks start in the order of blockIdx.x.  Causal: every head's last
    // (heaviest) pair of tiles first; else the pairs of one head together, so
    // that the CTAs running side by side share its K and V in L2.
    const int BH = p.B * p.H;
    const int bx = static_cast<int>(blockIdx.x);
    const int qp = p.mask.causal ? p.num_pairs - 1 - bx / BH : bx % p.num_pairs;
    const int bh = p.mask.causal ? bx % BH : bx / p.num_pairs;
    const int b = bh / p.H, h = bh % p.H, hk = h / p.group;
    const int q0 = qp * 2 * CF::BM;

    const uint32_t sQ = smem_addr(smem + CF::OFF_Q);
    const uint32_t sK = smem_addr(smem + CF::OFF_K);
    const uint32_t sV = smem_addr(smem + CF::OFF_V);
    const uint32_t bar0 = smem_addr(smem + CF::OFF_BAR);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + CF::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *range = reinterpret_cast<int *>(tmem_slot + 2);  // [tile][first key, end key]
    int32_t *docs_smem = reinterpret_cast<int32_t *>(smem + CF::OFF_DOCS);

    if (threadIdx.x == 0) {
        mbar_init(bar(CF::BAR_Q), 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(bar(CF::BAR_KF + s), 1);
            mbar_init(bar(CF::BAR_KE + s), 1);
            mbar_init(bar(CF::BAR_VF + s), 1);
            mbar_init(bar(CF::BAR_VE + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_SF + i), 1);
            mbar_init(bar(CF::BAR_PF + i), 4);
            mbar_init(bar(CF::BAR_PV + i), 1);
            range[2 * i] = 0x7FFFFFFF;
            range[2 * i + 1] = 0;
        }
        mbar_init(bar(CF::BAR_DRAIN), 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmap_q);
        tma_prefetch_map(&tmap_k);
        tma_prefetch_map(&tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t *docs = p.mask.doc_offsets
                              ? p.mask.doc_offsets + static_cast<int64_t>(b) * (p.mask.num_docs + 1) : nullptr;
    if (docs && p.mask.num_docs < kDocsInSmem) {
        for (int i = threadIdx.x; i <= p.mask.num_docs; i += CF::THREADS)
            docs_smem[i] = docs[i];
        docs = docs_smem;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // each softmax thread's row and the keys it sees; the tiles' key ranges
    const int tile = warp >= CF::FIRST_SOFTMAX_WARP ? (warp - CF::FIRST_SOFTMAX_WARP) >> 2 : 0;
    const int row = q0 + tile * CF::BM + (warp & 3) * 32 + lane;  // query index (softmax warps)
    int2 seen = make_int2(0, 0);
    if (warp >= CF::FIRST_SOFTMAX_WARP) {
        seen = visible_keys(p.mask, docs, b, row);
        const int lo = __reduce_min_sync(0xffffffffu, seen.y > seen.x ? seen.x : 0x7FFFFFFF);
        const int hi = __reduce_max_sync(0xffffffffu, seen.y);
        if (lane == 0) {
            atomicMin(&range[2 * tile], lo);
            atomicMax(&range[2 * tile + 1], hi);
        }
    }
    __syncthreads();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t timeout = p.timeout_ns;
    // key blocks tile i visits: [first(i), end(i)); empty when no row sees a key
    int first_b[2], end_b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool any = range[2 * i + 1] > 0;
        first_b[i] = any ? range[2 * i] / CF::BN : 0;
        end_b[i] = any ? (range[2 * i + 1] + CF::BN - 1) / CF::BN : 0;
    }
    // the stream of blocks both tiles are fed from
    const bool e0 = end_b[0] > first_b[0], e1 = end_b[1] > first_b[1];
    const int j0 = e0 && e1 ? min(first_b[0], first_b[1]) : e0 ? first_b[0] : first_b[1];
    const int j1 = max(end_b[0], end_b[1]);
    auto visits = [&](int i, int j) { return i ? j >= first_b[1] && j < end_b[1] : j >= first_b[0] && j < end_b[0]; };

    uint32_t q_issued = 0, k_issued = 0, k_par = 0, v_issued = 0, v_par = 0;
    if (warp < CF::FIRST_SOFTMAX_WARP) {
        regs_decrease<CF::REGS_CONTROL>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            if (lane == 0 && j0 < j1) {
                mbar_arrive_expect_tx(bar(CF::BAR_Q), 2 * CF::Q_BYTES);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_4d(sQ + i * CF::Q_BYTES + a * CF::ATOM_BYTES, &tmap_q, bar(CF::BAR_Q), 64 * a,
                                    q0 + i * CF::BM, h, b);
                q_issued = 1;
                int st = 0;
                uint32_t ph = 0;
                for (int j = j0; j < j1; ++j) {
                    if (!wait_bounded(bar(CF::BAR_KE + st), ph ^ 1u, abort_flag, timeout, ERR_PRODUCER))
                        break;
                    mbar_arrive_expect_tx(bar(CF::BAR_KF + st), CF::KV_BYTES);
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_4d(sK + st * CF::KV_BYTES + a * CF::ATOM_BYTES, &tmap_k, bar(CF::BAR_KF + st),
                                    64 * a, j * CF::BN, hk, b);
                    k_issued |= 1u << st;
                    k_par = (k_par & ~(1u << st)) | (ph << st);
                    if (!wait_bounded(bar(CF::BAR_VE + st), ph ^ 1u, abort_flag, timeout, ERR_PRODUCER))
                        break;
                    mbar_arrive_expect_tx(bar(CF::BAR_VF + st), CF::KV_BYTES);
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_4d(sV + st * CF::KV_BYTES + a * CF::ATOM_BYTES, &tmap_v, bar(CF::BAR_VF + st),
                                    64 * a, j * CF::BN, hk, b);
                    v_issued |= 1u << st;
                    v_par = (v_par & ~(1u << st)) | (ph << st);
                    if (++st == KS) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0 && j0 < j1) {
                constexpr uint32_t IDESC_QK = mma_idesc_f16(DT, 128, 128, 0, 0);  // Q, K both K-major
                constexpr uint32_t IDESC_PV = mma_idesc_f16(DT, 128, D, 0, 1);    // P K-major (TMEM), V N-major
                const uint64_t k_desc0 = smem_desc_sw128(sK, 16, 1024);
                const uint64_t v_desc0 = smem_desc_sw128(sV, CF::ATOM_BYTES, 1024);
                auto kmaj = [](int k) { return static_cast<uint64_t>(((k >> 2) * CF::ATOM_BYTES + (k & 3) * 32) >> 4); };
                int kst = 0, vst = 0;
                uint32_t kph = 0, vph = 0;
                bool ok = wait_bounded(bar(CF::BAR_Q), 0, abort_flag, timeout, ERR_MMA_DATA);
                auto issue_s = [&](int i) {  // S_i = Q_i K^T from the current K slot
                    const uint64_t q_desc = smem_desc_sw128(sQ + i * CF::Q_BYTES, 16, 1024);
                    const uint64_t kd = k_desc0 + ((kst * CF::KV_BYTES) >> 4);
                    const uint32_t d_s = tmem_base + static_cast<uint32_t>(CF::TMEM_S + i * 128);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma_f16(d_s, q_desc + kmaj(k), kd + kmaj(k), IDESC_QK, k != 0 ? 1u : 0u);
                    tc_commit(bar(CF::BAR_SF + i));
                };
                auto issue_pv = [&](int i, bool first) {  // O_i (+)= P_i V from the current V slot
                    const uint32_t d_o = tmem_base + static_cast<uint32_t>(CF::TMEM_O + i * D);
                    const uint32_t a_p = tmem_base + static_cast<uint32_t>(CF::TMEM_S + i * 128);
                    const uint64_t vd = v_desc0 + ((vst * CF::KV_BYTES) >> 4);
#pragma unroll
                    for (int k = 0; k < CF::BN / 16; ++k)
                        tc_mma_f16_ts(d_o, a_p + 8 * k, vd + ((2048 * k) >> 4), IDESC_PV,
                                      (!first || k > 0) ? 1u : 0u);
                    tc_commit(bar(CF::BAR_PV + i));
                };
                // j counts one ahead for S: S_i(j) for the stream's first block, then in the loop S_i(j + 1)
                for (int j = j0 - 1; ok && j < j1; ++j) {
                    bool k_ready = false;  // K(j + 1) waited for
                    if (j >= j0 && !wait_bounded(bar(CF::BAR_VF + vst), vph, abort_flag, timeout, ERR_MMA_DATA)) {
                        ok = false;
                        break;
                    }
                    for (int i = 0; ok && i < 2; ++i) {
                        const bool here = j >= j0 && visits(i, j);
                        const uint32_t jp = static_cast<uint32_t>(j - first_b[i]) & 1u;
                        if (here) {
                            if (!wait_bounded(bar(CF::BAR_PF + i), jp, abort_flag, timeout, ERR_MMA_DATA)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after_sync();
                            issue_pv(i, j == first_b[i]);
                        }
                        if (j >= j0 && i == 1)
                            tc_commit(bar(CF::BAR_VE + vst));  // V(j) free once the last P V of block j is done
                        if (j + 1 < j1) {
                            if (!k_ready && !wait_bounded(bar(CF::BAR_KF + kst), kph, abort_flag, timeout,
                                                          ERR_MMA_DATA)) {
                                ok = false;
                                break;
                            }
                            k_ready = true;
                            if (visits(i, j + 1)) {
                                // S_i(j + 1) overwrites the P_i(j) that PV_i(j) reads: wait for it
                                if (here && !wait_bounded(bar(CF::BAR_PV + i), jp, abort_flag, timeout, ERR_MMA_ACC)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after_sync();
                                issue_s(i);
                            }
                        }
                    }
                    if (!ok)
                        break;
                    if (j >= j0 && ++vst == KS) {
                        vst = 0;
                        vph ^= 1u;
                    }
                    if (k_ready) {
                        tc_commit(bar(CF::BAR_KE + kst));
                        if (++kst == KS) {
                            kst = 0;
                            kph ^= 1u;
                        }
                    }
                }
                tc_commit(bar(CF::BAR_DRAIN));
                wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
            }
            __syncwarp();
        }
    } else {
        regs_increase<CF::REGS_SOFTMAX>();
        // ------------------------------------------------------------ softmax and output of one tile
        const int fb = tile ? first_b[1] : first_b[0], eb = tile ? end_b[1] : end_b[0];
        check_ok(CF::TMEM_O + tile * D + D <= 512 && eb <= (p.mask.Sk + CF::BN - 1) / CF::BN && bh < BH);
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_S + tile * 128);
        const uint32_t o_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_O + tile * D);
        auto wait_warp = [&](int id, uint32_t parity) -> bool {
            const bool w = wait_bounded(bar(id), parity, abort_flag, timeout, ERR_EPILOGUE);
            return __all_sync(0xffffffffu, w);
        };
        const float slope2 = BIAS ? p.score.slopes[h] * 1.4426950408889634f : 0.0f;
        const int pos = p.mask.q_offset + row;
        // m: the reference maximum of the row's weights (log2 units); l: sum of the weights against m
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = fb; ok && j < eb; ++j) {
            const uint32_t jp = static_cast<uint32_t>(j - fb) & 1u;
            if (!(ok = wait_warp(CF::BAR_SF + tile, jp)))
                break;
            tc_fence_after_sync();
            const int key0 = j * CF::BN;
            uint32_t sv[128];
            tmem_load_32cols(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
            tmem_load_32cols(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
            tmem_load_wait();
            tmem_load_32cols(s_addr + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
            tmem_load_32cols(s_addr + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
            // tanh of the capped scores, or biased scores in log2 units, in place of the raw ones
            const float dist0 = static_cast<float>(pos - key0);
            auto transform = [&](int half) {
                if constexpr (CAP)
                    tanh_scores<64>(sv + 64 * half, p.score.cap_arg);
                if constexpr (!BIAS)
                    return;
#pragma unroll
                for (int e = 64 * half; e < 64 * half + 64; e += 2) {
                    float2 x = fmul2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                     splat2(CAP ? p.score.cap_log2 : p.score.scale_log2));
                    if constexpr (BIAS) {
                        const float2 dist = fadd2(splat2(dist0), make_float2(-static_cast<float>(e), -static_cast<float>(e + 1)));
                        x = ffma2(make_float2(fabsf(dist.x), fabsf(dist.y)), splat2(-slope2), x);
                    }
                    sv[e] = __float_as_uint(x.x);
                    sv[e + 1] = __float_as_uint(x.y);
                }
            };
            if constexpr (CAP || BIAS)
                transform(0);
            float t[16];  // maxima of groups of 8 scores
            auto maxima = [&](int g0, int g1) {
#pragma unroll
                for (int g = g0; g < g1; ++g) {
                    const float *f = reinterpret_cast<const float *>(&sv[8 * g]);
                    t[g] = fmax3(fmax3(f[0], f[1], f[2]), fmax3(f[3], f[4], f[5]), fmaxf(f[6], f[7]));
                }
            };
            maxima(0, 8);
            tmem_load_wait();
            if constexpr (CAP || BIAS)
                transform(1);
            const int nlo = seen.x - key0, nhi = seen.y - key0;
            if (!__all_sync(0xffffffffu, nlo <= 0 && nhi >= CF::BN)) {
                // keys outside the row's interval count neither in the maximum nor in the weights
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    if (e < nlo || e >= nhi)
                        sv[e] = __float_as_uint(-INFINITY);
                maxima(0, 8);
            }
            maxima(8, 16);
#pragma unroll
            for (int g = 0; g < 8; ++g)
                t[g] = fmaxf(t[g], t[g + 8]);
            float mx = fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
            const float to_log2 = CAP ? p.score.cap_log2 : p.score.scale_log2;  // of a score without a bias
            if constexpr (!BIAS)
                mx *= to_log2;
            // move the reference maximum only when the weights would exceed 2^8
            const bool resc = mx > m + CF::RESCALE_LOG2;
            const float m_new = resc ? mx : m;
            const float m_ref = m_new == -INFINITY ? 0.0f : m_new;  // no visible key yet: all weights 0
            const float alpha = resc ? exp2_approx_ftz(m - m_ref) : 1.0f;  // 0 when m is -inf
            const float2 negm2 = splat2(-m_ref);
            float2 part[4] = {splat2(0.0f), splat2(0.0f), splat2(0.0f), splat2(0.0f)};
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t pk[32];
#pragma unroll
                for (int e2 = 0; e2 < 32; ++e2) {
                    const int e = 64 * g + 2 * e2;
                    const float2 s = make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    const float2 x = BIAS ? fadd2(s, negm2) : ffma2(s, splat2(to_log2), negm2);
                    const float2 w = make_float2(exp2_approx_ftz(x.x), exp2_approx_ftz(x.y));
                    part[e2 & 3] = fadd2(part[e2 & 3], w);
                    pk[e2] = pack2<DT>(w.x, w.y);  // keys 2 e2, 2 e2 + 1 of this half: one 32-bit column
                }
                tmem_store_32cols(s_addr + 32 * g, pk);
            }
            const float2 ps = fadd2(fadd2(part[0], part[1]), fadd2(part[2], part[3]));
            l = l * alpha + (ps.x + ps.y);
            m = m_new;
            // rows whose maximum moved take O_i down by alpha (O_i holds the
            // blocks before j, so their P V has to be complete)
            if (j > fb && __any_sync(0xffffffffu, resc)) {
                if (!(ok = wait_warp(CF::BAR_PV + tile, jp ^ 1u)))
                    break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_load_32cols(o_addr + 32 * c, o);
                    tmem_load_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_store_32cols(o_addr + 32 * c, o);
                }
            }
            tmem_store_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(CF::BAR_PF + tile));
        }
        // output: O_i / l once the last P V has landed; rows that see no key get 0 and lse -inf
        if (ok && eb > fb)
            ok = wait_warp(CF::BAR_PV + tile, static_cast<uint32_t>(eb - fb - 1) & 1u);
        if (ok) {
            tc_fence_after_sync();
            const bool live = row < p.mask.Sq;
            const bool empty = seen.y <= seen.x || l == 0.0f;
            const float inv = empty ? 0.0f : 1.0f / l;
            uint16_t *orow = p.O + b * p.o_batch + h * p.o_head + static_cast<int64_t>(row) * p.o_row;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (eb > fb) {
                    tmem_load_32cols(o_addr + 32 * c, o);
                    tmem_load_wait();
                }
                if (live) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (!empty) {
                            w.x = pack2<DT>(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
                            w.y = pack2<DT>(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
                            w.z = pack2<DT>(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
                            w.w = pack2<DT>(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
                        }
                        reinterpret_cast<uint4 *>(orow + 32 * c)[v] = w;
                    }
                }
            }
            if (p.lse && live)
                p.lse[static_cast<int64_t>(bh) * p.mask.Sq + row] =
                    empty ? -INFINITY : m * 0.69314718055994531f + logf(l);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        if (q_issued)
            wait_drain(bar(CF::BAR_Q), 0, timeout);
        for (int s = 0; s < KS; ++s) {
            if (k_issued & (1u << s))
                wait_drain(bar(CF::BAR_KF + s), (k_par >> s) & 1u, timeout);
            if (v_issued & (1u << s))
                wait_drain(bar(CF::BAR_VF + s), (v_par >> s) & 1u, timeout);
        }
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

} // namespace tl
