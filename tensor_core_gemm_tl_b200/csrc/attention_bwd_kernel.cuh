// attention_bwd_kernel.cuh -- the gradients of attention_ex_kernel.cuh:
//
//     P_ij  = exp(y_ij - lse_i)                 (0 outside the row's interval)
//     dV_j  = sum_i P_ij dO_i
//     delta_i = sum_j P_ij dP_ij,               dP_ij = dO_i . V_j
//     dX_ij = P_ij (dP_ij - delta_i) c_ij,      c = 1, or 1 - tanh^2 with capped scores
//     dQ_i  = scale sum_j dX_ij K_j,   dK_j = scale sum_i dX_ij Q_i
//
// with i running over every query head that shares the key/value head.  Three
// launches, none of which adds with atomics, so results repeat bit for bit:
//
//   attention_bwd_rows_kernel      delta from O, lse in log2 units, each row's interval
//   attention_bwd_kernel<!DKV>     a CTA holds 128 queries and runs over the keys:
//                                  S = Q K^T, dP = dO V^T, dQ += dX K; delta again, exactly
//   attention_bwd_kernel<DKV>      a CTA holds 128 keys and runs over the queries:
//                                  S^T = K Q^T, dP^T = V dO^T (keys along the Tensor
//                                  Memory lanes), dV += P^T dO, dK += dX^T Q
//
// delta_i = dO_i . O_i carries the rounding of O to 16 bits, which is all that
// is left of dP - delta where one weight is nearly 1.  So it only serves as a
// first value: the dQ pass also sums e_i = sum_j P_ij (dP_ij - delta_i) in fp32
// and B_i = sum_j P_ij c_ij K_j on the tensor cores, takes
// dQ_i = scale (sum_j dX_ij K_j - e_i B_i), and leaves delta_i + e_i for the
// dK and dV pass.  A query that sees one key has weight 1 whatever its score,
// and gets exactly 0.
//
// Recomputing S and dP in the second pass costs 8 products where 5 would do
// with atomics or an ordered exchange of dQ; it keeps every sum in Tensor
// Memory and the order of every sum fixed.  P and dX go back to Tensor Memory
// as 16-bit values over the scores they came from and feed the second products
// from there; nothing of size queries x keys leaves the SM.
//
// Pipeline: blocks of 64 columns alternate between two sets of Tensor Memory
// columns, so the first products of block n + 1 run while block n is turned
// into P and dX.  Two warpgroups share each set, 32 columns a thread: sixteen
// warps hide the latencies of one another's loads, exponentials and
// conversions, which with two warpgroups of 64 columns a thread set the pace
// (2560 clocks a block of 128 x 64 against 1280 of products).
//
// 16-bit range: bf16 takes P and dX as they are.  fp16 holds P times 2^10 and
// dX times 2^4 over the power of two above the largest |dO| (P of long rows
// and gradients of small losses lie below fp16's normal range); the factors
// are powers of two and leave with the fp32 sums.
#pragma once

#include <type_traits>

#include "attention_common.cuh"

namespace tl {

constexpr int kBwdCols = 64;  // queries (DKV) or keys a step takes
template <int DT>
constexpr float kPShift = DT == 0 ? 10.0f : 0.0f;  // fp16 holds P times 2^10

struct AttnBwdParams {
    MaskParams mask;
    ScoreParams score;
    int32_t B, H, Hk, group;
    int32_t nqb;               // blocks of 64 queries
    int32_t tiles;             // 128-row tiles a CTA each: of the keys (DKV) or of the queries
    float scale;               // softmax scale
    float *rows;               // [B][H][nqb][2][64]: -lse in log2 units (-inf where the row sees nothing) plus the
                               // exponent of P's factor, -delta
    const int32_t *intervals;  // [B][nqb][3][64]: first and end key of each query; 0.0f where it sees one key, else 1.0f
    const int4 *ranges;        // [B][nqb]: least first, largest end, largest first, least end of the block's queries
    const unsigned *amax;      // fp16: bits of the largest |dO|, else null
    uint16_t *out0, *out1;     // dK, dV (DKV) or dQ, null
    int64_t s0[3], s1[3];      // their strides (batch, head, row) in elements
    uint64_t timeout_ns;
};

struct AttnBwdRowsParams {
    MaskParams mask;
    int32_t B, H, D, nqb;
    const uint16_t *O, *dO;
    int64_t so[3], sdo[3];
    const float *lse;          // [B][H][Sq]
    float *rows;
    int32_t *intervals;
    int4 *ranges;
    unsigned *amax;
};

// One CTA (256 threads) per 64 queries of a head: 8 lanes a row.  Bound by
// reading O and dO once.
template <int DT, int D>
__global__ void __launch_bounds__(256) attention_bwd_rows_kernel(const AttnBwdRowsParams p)
{
    __shared__ int32_t docs_smem[kDocsInSmem];
    __shared__ int red[4];
    grid_dependency_wait();
    grid_launch_dependents();
    const int qb = static_cast<int>(blockIdx.x % p.nqb);
    const int bh = static_cast<int>(blockIdx.x / p.nqb);
    const int b = bh / p.H, h = bh % p.H;
    const int32_t *docs = p.mask.doc_offsets
                              ? p.mask.doc_offsets + static_cast<int64_t>(b) * (p.mask.num_docs + 1) : nullptr;
    if (h == 0) {
        if (docs && p.mask.num_docs < kDocsInSmem) {
            for (int i = threadIdx.x; i <= p.mask.num_docs; i += 256)
                docs_smem[i] = docs[i];
            docs = docs_smem;
        }
        if (threadIdx.x == 0) {
            red[0] = red[3] = 0x7FFFFFFF;
            red[1] = red[2] = 0;
        }
        __syncthreads();
        if (threadIdx.x < kBwdCols) {
            const int2 seen = visible_keys(p.mask, docs, b, qb * kBwdCols + threadIdx.x);
            int32_t *iv = p.intervals + (static_cast<int64_t>(b) * p.nqb + qb) * 3 * kBwdCols;
            iv[threadIdx.x] = seen.x;
            iv[kBwdCols + threadIdx.x] = seen.y;
            iv[2 * kBwdCols + threadIdx.x] = __float_as_int(seen.y - seen.x == 1 ? 0.0f : 1.0f);
            if (seen.y > seen.x) {
                atomicMin(&red[0], seen.x);
                atomicMax(&red[1], seen.y);
            }
            atomicMax(&red[2], seen.x);
            atomicMin(&red[3], seen.y);
        }
        __syncthreads();
        if (threadIdx.x == 0)
            p.ranges[static_cast<int64_t>(b) * p.nqb + qb] = make_int4(red[0], red[1], red[2], red[3]);
    }
    float top = 0.0f;
    const int sub = threadIdx.x & 7;
#pragma unroll
    for (int r = threadIdx.x >> 3; r < kBwdCols; r += 32) {
        const int i = qb * kBwdCols + r;
        float sum = 0.0f;
        if (i < p.mask.Sq) {
            const uint16_t *o = p.O + b * p.so[0] + h * p.so[1] + static_cast<int64_t>(i) * p.so[2];
            const uint16_t *g = p.dO + b * p.sdo[0] + h * p.sdo[1] + static_cast<int64_t>(i) * p.sdo[2];
#pragma unroll
            for (int c = sub * 8; c < D; c += 64) {
                const uint4 wo = __ldg(reinterpret_cast<const uint4 *>(o + c));
                const uint4 wg = __ldg(reinterpret_cast<const uint4 *>(g + c));
                const uint32_t ao[4] = {wo.x, wo.y, wo.z, wo.w}, ag[4] = {wg.x, wg.y, wg.z, wg.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float g0 = to_float<DT>(static_cast<uint16_t>(ag[e] & 0xFFFFu));
                    const float g1 = to_float<DT>(static_cast<uint16_t>(ag[e] >> 16));
                    sum = fmaf(g0, to_float<DT>(static_cast<uint16_t>(ao[e] & 0xFFFFu)), sum);
                    sum = fmaf(g1, to_float<DT>(static_cast<uint16_t>(ao[e] >> 16)), sum);
                    if constexpr (DT == 0)
                        top = fmaxf(top, fmaxf(fabsf(g0), fabsf(g1)));
                }
            }
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (sub == 0) {
            const float l = i < p.mask.Sq ? p.lse[static_cast<int64_t>(bh) * p.mask.Sq + i] : -INFINITY;
            float *rows = p.rows + (static_cast<int64_t>(bh) * p.nqb + qb) * 2 * kBwdCols;
            rows[r] = l == -INFINITY ? -INFINITY : kPShift<DT> - l * 1.4426950408889634f;
            rows[kBwdCols + r] = l == -INFINITY ? 0.0f : -sum;
        }
    }
    if constexpr (DT == 0) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if ((threadIdx.x & 31) == 0)
            atomicMax(p.amax, __float_as_uint(top));  // non-negative floats order like their bits
    }
}

template <int D_>
struct AttnBwdConfig {
    static constexpr int D = D_;
    static constexpr int BM = 128, BN = kBwdCols;
    static constexpr int D_ATOMS = D / 64;
    static constexpr int XATOM = 128 * 128, YATOM = BN * 128;  // bytes of 64 columns of a tile
    static constexpr int X_BYTES = D_ATOMS * XATOM, Y_BYTES = D_ATOMS * YATOM;
    static constexpr int ROWS_BYTES = 2 * BN * 4, INTERVAL_BYTES = 3 * BN * 4;  // of a block of queries
    static constexpr int STAGES = 4;
    static constexpr int STAGE_BYTES = 2 * Y_BYTES + 2048;  // Y1, Y2, rows, intervals
    static constexpr int OFF_X = 0;
    static constexpr int OFF_Y = 2 * X_BYTES;
    static constexpr int OFF_BAR = OFF_Y + STAGES * STAGE_BYTES;
    static constexpr int BAR_X = 0, BAR_YF = 1, BAR_YE = 1 + STAGES;
    static constexpr int BAR_SF = 1 + 2 * STAGES;  // [buffer]: S and dP in Tensor Memory
    static constexpr int BAR_PF = BAR_SF + 2;      // [buffer]: P and dX in Tensor Memory (8 warps arrive)
    static constexpr int BAR_DONE = BAR_PF + 2;    // [buffer]: the second products have read them
    static constexpr int BAR_EPS = BAR_DONE + 2;   // dQ: the warpgroups' parts of e are in shared memory (16 warps)
    static constexpr int BAR_DRAIN = BAR_EPS + 1;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int OFF_EPS = OFF_MISC + 32;   // [warpgroup][128] floats
    static constexpr int SMEM_BYTES = OFF_EPS + 2048 + 1024;
    static constexpr int THREADS = 640;  // 4 control warps, 4 warpgroups for P and dX
    static constexpr int REGS_CONTROL = 64, REGS_SOFTMAX = 104;
    static constexpr int LAUNCH_REGS = (128 * REGS_CONTROL + 512 * REGS_SOFTMAX + THREADS - 1) / THREADS;
    // Tensor Memory columns: S and dP of buffer w, the accumulators
    static constexpr int TMEM_S = 0, TMEM_DP = 128, TMEM_A0 = 256, TMEM_A1 = 256 + D;
    static_assert(ROWS_BYTES + INTERVAL_BYTES <= 2048 && SMEM_BYTES <= 232448, "shared memory");
};

// X1, X2: the CTA's 128 rows (K and V, or Q and dO); Y1, Y2: the blocks of 64
// it runs over (Q and dO, or K and V)
template <class CF, int DT, bool DKV, bool CAP, bool BIAS>
__global__ void __launch_bounds__(640, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                         const __grid_constant__ CUtensorMap map_y1, const __grid_constant__ CUtensorMap map_y2,
                         const AttnBwdParams p)
{
    constexpr int D = CF::D, STAGES = CF::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);  // uniform for the compiler too
    const int lane = threadIdx.x & 31;
    // the tile and its head.  Causal: the heaviest tiles first (the first keys,
    // the last queries); else one head's tiles together.
    const int heads = DKV ? p.Hk : p.H;
    const int BH = p.B * heads;
    const int bx = static_cast<int>(blockIdx.x);
    const int tile = p.mask.causal ? (DKV ? bx / BH : p.tiles - 1 - bx / BH) : bx % p.tiles;
    const int bh = p.mask.causal ? bx % BH : bx / p.tiles;
    const int b = bh / heads, head = bh % heads;
    const int x0 = tile * CF::BM;

    const uint32_t sX = smem_addr(smem + CF::OFF_X);
    const uint32_t sY = smem_addr(smem + CF::OFF_Y);
    const uint32_t bar0 = smem_addr(smem + CF::OFF_BAR);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + CF::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *range = reinterpret_cast<int *>(tmem_slot + 2);  // first and end block of 64

    if (threadIdx.x == 0) {
        mbar_init(bar(CF::BAR_X), 1);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(CF::BAR_YF + s), 1);
            mbar_init(bar(CF::BAR_YE + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_SF + i), 1);
            mbar_init(bar(CF::BAR_PF + i), 8);
            mbar_init(bar(CF::BAR_DONE + i), 1);
        }
        mbar_init(bar(CF::BAR_EPS), 16);
        mbar_init(bar(CF::BAR_DRAIN), 1);
        *abort_flag = 0;
        range[0] = 0x7FFFFFFF;
        range[1] = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_x1);
        tma_prefetch_map(&map_x2);
        tma_prefetch_map(&map_y1);
        tma_prefetch_map(&map_y2);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const int group = warp >= 4 ? (warp - 4) >> 2 : 0;    // warpgroup
    const int wg = group & 1, half = group >> 1;          // its buffer, and which 32 of the 64 columns
    const int r = (warp & 3) * 32 + lane;                 // row of the tile (Tensor Memory lane)
    int2 seen = make_int2(0, 0);                          // dQ: the row's interval
    if constexpr (DKV) {
        // the blocks of queries that see some key of the tile
        const int4 *rg = p.ranges + static_cast<int64_t>(b) * p.nqb;
        int first = 0x7FFFFFFF, end = 0;
        for (int q = threadIdx.x; q < p.nqb; q += CF::THREADS) {
            const int4 v = __ldg(rg + q);
            if (v.x < x0 + CF::BM && v.y > x0) {
                first = min(first, q);
                end = max(end, q + 1);
            }
        }
        first = __reduce_min_sync(0xffffffffu, first);
        end = __reduce_max_sync(0xffffffffu, end);
        if (lane == 0) {
            atomicMin(&range[0], first);
            atomicMax(&range[1], end);
        }
    } else if (warp >= 4) {
        const int i = x0 + r;
        if (i < p.mask.Sq) {
            const int32_t *iv = p.intervals + (static_cast<int64_t>(b) * p.nqb + i / CF::BN) * 3 * CF::BN + i % CF::BN;
            seen = make_int2(iv[0], iv[CF::BN]);
        }
        const int lo = __reduce_min_sync(0xffffffffu, seen.y > seen.x ? seen.x / CF::BN : 0x7FFFFFFF);
        const int hi = __reduce_max_sync(0xffffffffu, (seen.y + CF::BN - 1) / CF::BN);
        if (lane == 0) {
            atomicMin(&range[0], lo);
            atomicMax(&range[1], hi);
        }
    }
    __syncthreads();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t timeout = p.timeout_ns;
    const int y_first = range[0];
    const int y_count = range[1] > y_first ? range[1] - y_first : 0;
    const int n_total = DKV ? y_count * p.group : y_count;  // DKV: over the heads that share the keys, one after another

    uint32_t x_issued = 0, y_issued = 0, y_par = 0;
    if (warp < 4) {
        regs_decrease<CF::REGS_CONTROL>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            if (lane == 0 && n_total > 0) {
                mbar_arrive_expect_tx(bar(CF::BAR_X), 2 * CF::X_BYTES);
#pragma unroll
                for (int a = 0; a < CF::D_ATOMS; ++a) {
                    tma_load_4d(sX + a * CF::XATOM, &map_x1, bar(CF::BAR_X), 64 * a, x0, head, b);
                    tma_load_4d(sX + CF::X_BYTES + a * CF::XATOM, &map_x2, bar(CF::BAR_X), 64 * a, x0, head, b);
                }
                x_issued = 1;
                int st = 0, yb = y_first, yh = DKV ? head * p.group : head / p.group;
                uint32_t ph = 0;
                for (int n = 0; n < n_total; ++n) {
                    if (!wait_bounded(bar(CF::BAR_YE + st), ph ^ 1u, abort_flag, timeout, ERR_PRODUCER))
                        break;
                    const uint32_t full = bar(CF::BAR_YF + st);
                    const uint32_t dst = sY + st * CF::STAGE_BYTES;
                    mbar_arrive_expect_tx(full, 2 * CF::Y_BYTES + (DKV ? CF::ROWS_BYTES + CF::INTERVAL_BYTES : 0));
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_4d(dst + a * CF::YATOM, &map_y1, full, 64 * a, yb * CF::BN, yh, b);
                    if constexpr (DKV) {
                        bulk_load_g2s(dst + 2 * CF::Y_BYTES,
                                      p.rows + ((static_cast<int64_t>(b) * p.H + yh) * p.nqb + yb) * 2 * CF::BN,
                                      CF::ROWS_BYTES, full);
                        bulk_load_g2s(dst + 2 * CF::Y_BYTES + CF::ROWS_BYTES,
                                      p.intervals + (static_cast<int64_t>(b) * p.nqb + yb) * 3 * CF::BN,
                                      CF::INTERVAL_BYTES, full);
                    }
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_4d(dst + CF::Y_BYTES + a * CF::YATOM, &map_y2, full, 64 * a, yb * CF::BN, yh, b);
                    y_issued |= 1u << st;
                    y_par = (y_par & ~(1u << st)) | (ph << st);
                    if (++yb == y_first + y_count) {
                        yb = y_first;
                        ++yh;
                    }
                    if (++st == STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            // the whole warp walks the loop and one elected lane issues: what the
            // instructions are made from stays uniform across the warp
            if (n_total > 0) {
                constexpr uint32_t IDESC_1 = mma_idesc_f16(DT, 128, CF::BN, 0, 0);  // both K-major
                constexpr uint32_t IDESC_2 = mma_idesc_f16(DT, 128, D, 0, 1);       // A from Tensor Memory, Y N-major
                const uint64_t x_desc = smem_desc_sw128(sX, 16, 1024);
                const uint64_t y_desc = smem_desc_sw128(sY, 16, 1024);
                const uint64_t yt_desc = smem_desc_sw128(sY, CF::YATOM, 1024);
                auto first_products = [&](int w, int st) {
                    const uint64_t yd = y_desc + ((st * CF::STAGE_BYTES) >> 4);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t d = tmem_base + static_cast<uint32_t>((m ? CF::TMEM_DP : CF::TMEM_S) + CF::BN * w);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16(d, x_desc + ((m * CF::X_BYTES + (k >> 2) * CF::XATOM + (k & 3) * 32) >> 4),
                                       yd + ((m * CF::Y_BYTES + (k >> 2) * CF::YATOM + (k & 3) * 32) >> 4), IDESC_1,
                                       k != 0 ? 1u : 0u);
                    }
                    tc_commit(bar(CF::BAR_SF + w));
                };
                // 16 values of P or dX take 8 columns; each half of the block's lies where its half of the scores was
                auto p_col = [](int k) { return (k >> 1) * (CF::BN / 2) + (k & 1) * 8; };
                auto second_products = [&](int w, int st, bool first) {
                    const uint64_t yd = yt_desc + ((st * CF::STAGE_BYTES) >> 4);
#pragma unroll
                    for (int k = 0; k < CF::BN / 16; ++k)  // dV += P^T dO, or B += P c K
                        tc_mma_f16_ts(tmem_base + CF::TMEM_A0, tmem_base + CF::TMEM_S + CF::BN * w + p_col(k),
                                      yd + (((DKV ? CF::Y_BYTES : 0) + 2048 * k) >> 4), IDESC_2,
                                      (!first || k > 0) ? 1u : 0u);
#pragma unroll
                    for (int k = 0; k < CF::BN / 16; ++k)  // dK += dX^T Q, or dQ += dX K
                        tc_mma_f16_ts(tmem_base + CF::TMEM_A1, tmem_base + CF::TMEM_DP + CF::BN * w + p_col(k),
                                      yd + ((2048 * k) >> 4), IDESC_2, (!first || k > 0) ? 1u : 0u);
                    tc_commit(bar(CF::BAR_DONE + w));
                    tc_commit(bar(CF::BAR_YE + st));
                };
                int st = 0, st1 = 0;  // stages of block n and of block n + 1
                uint32_t ph1 = 0;
                auto wait = [&](int id, uint32_t par, unsigned code) {
                    return __all_sync(0xffffffffu, wait_bounded(bar(id), par, abort_flag, timeout, code)) != 0;
                };
                bool ok = wait(CF::BAR_X, 0, ERR_MMA_DATA);
                for (int n = -1; ok && n < n_total; ++n) {
                    if (n + 1 < n_total) {
                        const int w1 = (n + 1) & 1;
                        // the buffer's previous P and dX (block n - 1) have been read
                        if (!wait(CF::BAR_YF + st1, ph1, ERR_MMA_DATA) ||
                            (n >= 1 && !wait(CF::BAR_DONE + w1, static_cast<uint32_t>((n - 1) >> 1) & 1u, ERR_MMA_ACC)))
                            break;
                        tc_fence_after_sync();
                        if (elect_one())
                            first_products(w1, st1);
                        __syncwarp();
                        if (++st1 == STAGES) {
                            st1 = 0;
                            ph1 ^= 1u;
                        }
                    }
                    if (n >= 0) {
                        if (!wait(CF::BAR_PF + (n & 1), static_cast<uint32_t>(n >> 1) & 1u, ERR_MMA_ACC))
                            break;
                        tc_fence_after_sync();
                        if (elect_one())
                            second_products(n & 1, st, n == 0);
                        __syncwarp();
                        if (++st == STAGES)
                            st = 0;
                    }
                }
                if (elect_one())
                    tc_commit(bar(CF::BAR_DRAIN));
                __syncwarp();
                wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
            }
            __syncwarp();
        }
    } else {
        regs_increase<CF::REGS_SOFTMAX>();
        // ------------------------------------------------------------ P and dX, one row a thread
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_S + CF::BN * wg);
        const uint32_t dp_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_DP + CF::BN * wg);
        constexpr int HN = CF::BN / 2;  // columns a thread
        auto wait_warp = [&](int id, uint32_t parity) -> bool {
            const bool w = wait_bounded(bar(id), parity, abort_flag, timeout, ERR_EPILOGUE);
            return __all_sync(0xffffffffu, w);
        };
        // fp16: P times 2^p_shift, dX times x_mul over P's factor; x_undo takes dX's factor out again
        constexpr float p_shift = kPShift<DT>;
        float x_mul = 1.0f, x_undo = CAP ? 4.0f : 1.0f;  // capped: 1 - tanh^2 = 4 r (1 - r), bf16 leaves the 4 for the end
        if constexpr (DT == 0) {
            const unsigned bits = __ldg(p.amax);
            // 2^-e with 2^(e-1) <= largest |dO| < 2^e, kept where both 2^e and 2^-e are normal; 1 for 0, inf, NaN
            int e = static_cast<int>(bits >> 23) - 126;
            e = bits == 0 || bits >= 0x7F800000u ? 0 : min(max(e, -100), 100);
            x_mul = exp2f(static_cast<float>(-e) + 4.0f - p_shift) * x_undo;  // the capped 4 goes in here
            x_undo = exp2f(static_cast<float>(e) - 4.0f);
        }
        float row_nlse = -INFINITY, row_ndelta = 0.0f;
        float2 eps[2] = {splat2(0.0f), splat2(0.0f)};  // dQ: this warpgroup's part of e (times P's factor)
        if constexpr (!DKV) {
            const int i = x0 + r;
            if (i < p.mask.Sq) {
                const float *rows = p.rows + ((static_cast<int64_t>(b) * p.H + head) * p.nqb + i / CF::BN) * 2 * CF::BN +
                                    i % CF::BN;
                row_nlse = rows[0];
                row_ndelta = rows[CF::BN];
            }
        }
        bool ok = true;
        int yb = y_first, yh = DKV ? head * p.group : 0;  // block and head of step n
        auto advance = [&]() {
            if (++yb == y_first + y_count) {
                yb = y_first;
                ++yh;
            }
        };
        if (wg && n_total > 0)
            advance();
        float slope2 = 0.0f;
        if constexpr (BIAS && !DKV)
            slope2 = p.score.slopes[head] * 1.4426950408889634f;
        for (int n = wg; n < n_total; n += 2) {
            const int st = n % STAGES;
            int4 rg = make_int4(0, 0, 0, 0);
            if constexpr (DKV) {
                rg = __ldg(p.ranges + static_cast<int64_t>(b) * p.nqb + yb);
                if constexpr (BIAS)
                    slope2 = __ldg(p.score.slopes + yh) * 1.4426950408889634f;
                // the info beside the stage's tiles: seen through the copy's own barrier
                if (!(ok = wait_warp(CF::BAR_YF + st, static_cast<uint32_t>(n / STAGES) & 1u)))
                    break;
            }
            if (!(ok = wait_warp(CF::BAR_SF + wg, static_cast<uint32_t>(n >> 1) & 1u)))
                break;
            tc_fence_after_sync();
            uint32_t sv[HN], dp[HN];
            tmem_load_32cols(s_addr + HN * half, sv);
            tmem_load_32cols(dp_addr + HN * half, dp);
            // DKV: -lse, -delta, first key, end key and "sees more than one key" of the block's queries
            const float4 *info = reinterpret_cast<const float4 *>(smem + CF::OFF_Y + st * CF::STAGE_BYTES + 2 * CF::Y_BYTES) +
                                 half * (HN / 4);
            const int4 *iv = reinterpret_cast<const int4 *>(info + 2 * CF::BN / 4);
            const float4 *many = info + 4 * CF::BN / 4;
            // |p_i - j|: the column's step away from the first column's distance
            const int y0 = yb * CF::BN + HN * half;  // the thread's first column
            const float dist0 = DKV ? static_cast<float>(p.mask.q_offset + y0 - (x0 + r))
                                    : static_cast<float>(p.mask.q_offset + x0 + r - y0);
            const int key = x0 + r;                             // DKV
            const int nlo = seen.x - y0, nhi = seen.y - y0;     // dQ
            bool whole = DKV ? rg.z <= x0 && rg.w >= x0 + CF::BM : nlo <= 0 && nhi >= HN;
            whole = __all_sync(0xffffffffu, whole);
            tmem_load_wait();
            // scores and dP to P and dX, in place and packed in pairs; only blocks that cut an interval are masked
            auto block = [&](auto masked) {
                constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
                for (int e = 0; e < HN; e += 4) {
                    float4 l4 = make_float4(row_nlse, row_nlse, row_nlse, row_nlse);
                    float4 d4 = make_float4(row_ndelta, row_ndelta, row_ndelta, row_ndelta);
                    float4 m4 = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    int4 lo4 = make_int4(0, 0, 0, 0), hi4 = lo4;
                    if constexpr (DKV) {
                        l4 = info[e / 4];
                        d4 = info[CF::BN / 4 + e / 4];
                        if constexpr (MASKED) {
                            lo4 = iv[e / 4];
                            hi4 = iv[CF::BN / 4 + e / 4];
                            m4 = many[e / 4];
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const float2 s = make_float2(__uint_as_float(sv[e + c]), __uint_as_float(sv[e + c + 1]));
                        const float2 nl = c ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                        const float2 nd = c ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                        float2 x, cap_r;
                        if constexpr (CAP) {
                            cap_r = cap_reciprocals(s, p.score.cap_arg);
                            x = ffma2(cap_r, splat2(-2.0f * p.score.cap_log2), fadd2(nl, splat2(p.score.cap_log2)));
                        } else {
                            x = ffma2(s, splat2(p.score.scale_log2), nl);
                        }
                        if constexpr (BIAS) {
                            const float f = static_cast<float>(e + c);
                            const float2 dist = DKV ? fadd2(splat2(dist0), make_float2(f, f + 1.0f))
                                                    : fadd2(splat2(dist0), make_float2(-f, -f - 1.0f));
                            x = ffma2(make_float2(fabsf(dist.x), fabsf(dist.y)), splat2(-slope2), x);
                        }
                        float2 w = make_float2(exp2_approx_ftz(x.x), exp2_approx_ftz(x.y));
                        const float2 dpv = make_float2(__uint_as_float(dp[e + c]), __uint_as_float(dp[e + c + 1]));
                        float2 g;
                        if constexpr (MASKED && DKV) {
                            w.x = key >= (c ? lo4.z : lo4.x) && key < (c ? hi4.z : hi4.x) ? w.x : 0.0f;
                            w.y = key >= (c ? lo4.w : lo4.y) && key < (c ? hi4.w : hi4.y) ? w.y : 0.0f;
                            // a query that sees one key gets dX = 0 exactly
                            const float2 m = c ? make_float2(m4.z, m4.w) : make_float2(m4.x, m4.y);
                            g = fmul2(fadd2(dpv, nd), m);
                        } else {
                            if constexpr (MASKED) {
                                w.x = e + c >= nlo && e + c < nhi ? w.x : 0.0f;
                                w.y = e + c + 1 >= nlo && e + c + 1 < nhi ? w.y : 0.0f;
                            }
                            g = fadd2(dpv, nd);
                        }
                        float2 ds = fmul2(w, g);
                        if constexpr (!DKV)
                            eps[c / 2] = fadd2(eps[c / 2], ds);
                        if constexpr (CAP) {
                            const float2 t = ffma2(make_float2(-cap_r.x, -cap_r.y), cap_r, cap_r);
                            ds = fmul2(ds, t);
                            if constexpr (!DKV)
                                w = fmul2(w, t);
                        }
                        if constexpr (DT == 0)
                            ds = fmul2(ds, splat2(x_mul));
                        sv[(e + c) / 2] = pack2<DT>(w.x, w.y);
                        dp[(e + c) / 2] = pack2<DT>(ds.x, ds.y);
                    }
                }
            };
            if (whole)
                block(std::false_type{});
            else
                block(std::true_type{});
            // over the first half of the columns this thread read itself (the other warpgroup may still read its own)
            tmem_store_16cols(s_addr + HN * half, sv);
            tmem_store_16cols(dp_addr + HN * half, dp);
            tmem_store_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(CF::BAR_PF + wg));
            advance();
            if (n + 1 < n_total)
                advance();
        }
        // all products complete, then the sums out
        if (ok && n_total > 0)
            ok = wait_warp(CF::BAR_DRAIN, 0);
        float e_row = 0.0f;  // dQ: the row's e
        if constexpr (!DKV) {
            float *eps_smem = reinterpret_cast<float *>(smem + CF::OFF_EPS);
            const float2 mine = fadd2(eps[0], eps[1]);
            eps_smem[group * 128 + r] = mine.x + mine.y;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(CF::BAR_EPS));
            ok = ok && wait_warp(CF::BAR_EPS, 0);
            if (ok)
                e_row = ((eps_smem[r] + eps_smem[128 + r]) + (eps_smem[256 + r] + eps_smem[384 + r])) *
                        (DT == 0 ? 1.0f / 1024.0f : 1.0f);
        }
        if (ok) {
            tc_fence_after_sync();
            const int row = x0 + r;
            const bool live = row < (DKV ? p.mask.Sk : p.mask.Sq);
            constexpr float p_undo = DT == 0 ? 1.0f / 1024.0f : 1.0f;
            // DKV: buffer 0's warpgroups write dK, buffer 1's dV, half the columns each; dQ: a quarter each
            uint16_t *out = DKV && wg ? p.out1 : p.out0;  // (batch, head, row) strides below
            const int64_t *sd = DKV && wg ? p.s1 : p.s0;
            const float mul = DKV && wg ? p_undo : p.scale * x_undo;
            out += b * sd[0] + head * sd[1] + static_cast<int64_t>(row) * sd[2];
            const uint32_t acc0 = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_A0);
            const uint32_t acc = DKV && wg ? acc0 : tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_A1);
            const float e_mul = -e_row * p.scale * p_undo * (CAP ? 4.0f : 1.0f);
            const bool none = n_total == 0 || (!DKV && seen.y - seen.x <= 1);  // nothing comes through
            if constexpr (!DKV) {
                if (group == 0 && live)
                    p.rows[((static_cast<int64_t>(b) * p.H + head) * p.nqb + row / CF::BN) * 2 * CF::BN + CF::BN +
                           row % CF::BN] = row_ndelta - e_row;
            }
            const int c0 = DKV ? half * (D / 32) : group * (D / 64), c1 = c0 + (DKV ? D / 32 : D / 64);  // of 16 columns
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                uint32_t o[16];
                if (n_total > 0) {
                    tmem_load_16cols(acc + 16 * c, o);
                    if constexpr (!DKV) {
                        uint32_t o0[16];
                        tmem_load_16cols(acc0 + 16 * c, o0);
                        tmem_load_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o0[e]), e_mul, __uint_as_float(o[e]) * mul));
                    } else {
                        tmem_load_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * mul);
                    }
                }
                if (none) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = 0;
                }
                if (live) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint4 w;
                        w.x = pack2<DT>(__uint_as_float(o[8 * v]), __uint_as_float(o[8 * v + 1]));
                        w.y = pack2<DT>(__uint_as_float(o[8 * v + 2]), __uint_as_float(o[8 * v + 3]));
                        w.z = pack2<DT>(__uint_as_float(o[8 * v + 4]), __uint_as_float(o[8 * v + 5]));
                        w.w = pack2<DT>(__uint_as_float(o[8 * v + 6]), __uint_as_float(o[8 * v + 7]));
                        reinterpret_cast<uint4 *>(out + 16 * c)[v] = w;
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        if (x_issued)
            wait_drain(bar(CF::BAR_X), 0, timeout);
        for (int s = 0; s < STAGES; ++s)
            if (y_issued & (1u << s))
                wait_drain(bar(CF::BAR_YF + s), (y_par >> s) & 1u, timeout);
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

} // namespace tl
