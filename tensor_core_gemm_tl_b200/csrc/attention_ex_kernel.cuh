// attention_ex_kernel.cuh -- attention forward with capped scores, a distance
// bias, causal / document / prefix masks, shared key/value heads and strided
// tensors (the formulas stand in attention_common.cuh):
//
//     O_i = sum_j w_ij V_j,   w_ij = exp(y_ij - lse_i),   lse_i = log sum_j exp(y_ij)
//
// An item is a pair of 128-row query tiles of one head against one stream of
// 128-key blocks.  A warpgroup turns a tile's scores into weights, a row a thread
// and 64 keys a step: Tensor Memory holds, per tile, two sets of 64 score columns
// (the 16-bit weights P are written over the first half of a set) and the sums O
// (D columns).  While step n becomes weights, the tensor core computes step n + 1's
// scores and adds step n - 1's P V, so the warpgroup never waits for a product;
// with one set of 128 columns a tile it did, each block: 1970 clocks a tile and
// block (and 2500 with two warpgroups a tile, which have to agree on the row's
// maximum).  With D = 64 Tensor Memory has room for sums of each set: each has a
// warpgroup of its own (TWIN), which keep maxima of their own and join at the
// item's end, so twice as many warps cover one another's latency (causal 2 x 16
// heads x 4096: 111 -> 106 us, capped 191 -> 174, with cap and bias 237 -> 201).
// Each tile visits only the steps that some of its rows see; inside,
// only steps that cut a row's interval pay for masking.
//
// CTAs are persistent: a CTA whose item's loads are out takes over one that has
// not started yet (cluster launch control), so set-up, the masks' ranges and
// the next item's loads pass beside the work; a CTA an item spent 6 us on them,
// more than a short document's attention takes.
//
// Where items are few (a short chunk of a long prompt) the blocks of each are split
// over several CTAs, which leave fp32 sums with their maxima and
// attention_join_kernel adds in the order of the keys: 8 heads, 77 queries x 1101
// keys, went from 30 to 15 us.
//
// What bounds it: 2 products of 128 x 128 x D a tile and block, with D = 128 1024
// clocks at 4096 multiply-adds a clock and SM (1376, as S in steps of 64 keys reads
// 48 bytes of operands for every 32 clocks' worth of products), against one 2^x a
// pair at 16 a clock (1024 clocks); capped scores add the multiply-adds of
// tanh_scores.  Measured, 4 x 16 heads x 4096 x 4096, bf16: D = 128 435 us, 1265
// TFLOP/s (causal 260); D = 64, 2 x 16 heads, 211 us, 652 TFLOP/s.  The chains' own
// latency bounds: scores, 2^x, sum, pack, P V and the next scores follow one
// another in each set (the tensor pipe 32..75 % busy, the special-function pipe
// 32..56 %).
//
// Warps: 0 items and TMA loads, 1 issues S (and allocates Tensor Memory), 2 issues
// P V, 3 idle, 4..7 softmax of tile 0, 8..11 of tile 1 (TWIN: of set 0; 12..19 of
// set 1).  Every wait is bounded.
#pragma once

#include "attention_common.cuh"

namespace tl {

struct AttnExParams {
    MaskParams mask;
    ScoreParams score;
    int32_t B, H, group;     // batch, query heads, query heads per key/value head
    int32_t num_pairs;       // pairs of 128-row query tiles
    int32_t splits;          // CTAs the keys of an item are split over
    float4 *part_o;          // splits > 1: [item][split][tile][D / 4][128]
    float2 *part_ml;         // [item][split][tile][128]: maximum (log2 units), sum
    float *lse;              // [B][H][Sq] natural log, or null
    uint64_t timeout_ns;
};

template <int D_>
struct AttnExConfig {
    static constexpr int D = D_;
    static constexpr bool TWIN = D == 64;                  // a warpgroup for each set of a tile
    static constexpr int WARPS = TWIN ? 16 : 8;            // of the softmax
    static constexpr int BM = 128, BN = 128;
    static constexpr int KS = D == 128 ? 2 : 4;            // K and V ring depth
    static constexpr int ATOM_BYTES = 128 * 128;           // 128 rows x 64 16-bit values
    static constexpr int D_ATOMS = D / 64;
    static constexpr int Q_BYTES = D_ATOMS * ATOM_BYTES;
    static constexpr int KV_BYTES = D_ATOMS * ATOM_BYTES;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + KS * KV_BYTES;
    static constexpr int OFF_OUT = OFF_V + KS * KV_BYTES;  // [warp] 32 rows x 32 columns on their way out
    static constexpr int OFF_ML = OFF_OUT + WARPS * 2048;  // TWIN: [item & 1][tile][set][128] float2
    static constexpr int OFF_BAR = OFF_ML + (TWIN ? 2 * 2 * 2 * 128 * 8 : 0);
    static constexpr int BAR_QF = 0, BAR_QE = 1;
    static constexpr int BAR_KF = 2, BAR_KE = 2 + KS, BAR_VF = 2 + 2 * KS, BAR_VE = 2 + 3 * KS;
    static constexpr int BAR_SF = 2 + 4 * KS;   // [tile][set]: S in Tensor Memory
    static constexpr int BAR_PF = BAR_SF + 4;   // [tile][set]: P in Tensor Memory (4 warps)
    static constexpr int BAR_PV = BAR_PF + 4;   // [tile][set]: O += P V completed
    static constexpr int BAR_OE = BAR_PV + 4;   // [tile]: O has been read (its warps)
    static constexpr int BAR_TF = BAR_OE + 2;   // [slot]: an item's description is in shared memory
    static constexpr int BAR_TE = BAR_TF + 2;   // [slot]: and has been read (two MMA issuers, the softmax warps)
    static constexpr int BAR_CLC = BAR_TE + 2;  // the answer to a request for another item
    static constexpr int BAR_DRAIN = BAR_CLC + 1;
    static constexpr int BAR_ML = BAR_DRAIN + 1;  // TWIN: [tile]: both sets are complete, their statistics in shared memory (8 warps)
    static constexpr int NUM_BARS = BAR_ML + 2;
    static constexpr int OFF_MISC = OFF_BAR + (NUM_BARS * 8 + 15) / 16 * 16;  // TMEM address, abort flag
    static constexpr int OFF_CLC = OFF_MISC + 16;
    static constexpr int OFF_ITEMS = OFF_CLC + 16;      // [slot] pair, head, first and end step of each tile
    static constexpr int SMEM_BYTES = OFF_ITEMS + 2 * 32 + 1024;
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr int REGS_CONTROL = TWIN ? 64 : 104, REGS_SOFTMAX = TWIN ? 104 : 200;
    static constexpr int LAUNCH_REGS = (128 * REGS_CONTROL + 32 * WARPS * REGS_SOFTMAX + THREADS - 1) / THREADS;
    static constexpr int BS = 64;               // keys a step
    // set h of tile i at 128 i + 64 h, its O at 256 + 128 i, TWIN: + 64 h (else one for both sets)
    static constexpr int TMEM_S = 0, TMEM_O = 256;
    static constexpr float RESCALE_LOG2 = 8.0f;     // m moves when a row maximum exceeds it by 2^8
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// Asks for a CTA of this grid that has not started: its index arrives at `dst`
// (16 bytes), counted as 16 bytes on `bar`.
__device__ __forceinline__ void clc_request(uint32_t dst, uint32_t bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}

// The answer at `src`: the blockIdx.x taken over, or -1 when none is left
__device__ __forceinline__ int clc_answer(uint32_t src)
{
    uint32_t taken, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(taken), "=r"(x)
        : "r"(src)
        : "memory");
    return taken ? static_cast<int>(x) : -1;
}

template <class CF, int DT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(CF::THREADS, 1)
    attention_ex_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                        const AttnExParams p)
{
    constexpr int D = CF::D;
    constexpr int KS = CF::KS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);  // uniform for the compiler too
    const int lane = threadIdx.x & 31;
    const uint32_t sQ = smem_addr(smem + CF::OFF_Q);
    const uint32_t sK = smem_addr(smem + CF::OFF_K);
    const uint32_t sV = smem_addr(smem + CF::OFF_V);
    const uint32_t bar0 = smem_addr(smem + CF::OFF_BAR);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + CF::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int4 *item_slots = reinterpret_cast<int4 *>(smem + CF::OFF_ITEMS);

    if (threadIdx.x == 0) {
        mbar_init(bar(CF::BAR_QF), 1);
        mbar_init(bar(CF::BAR_QE), 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(bar(CF::BAR_KF + s), 1);
            mbar_init(bar(CF::BAR_KE + s), 1);
            mbar_init(bar(CF::BAR_VF + s), 1);
            mbar_init(bar(CF::BAR_VE + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_OE + i), CF::WARPS / 2);
            mbar_init(bar(CF::BAR_ML + i), CF::WARPS / 2);
            mbar_init(bar(CF::BAR_TF + i), 1);
            mbar_init(bar(CF::BAR_TE + i), 2 + CF::WARPS);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(CF::BAR_SF + i), 1);
            mbar_init(bar(CF::BAR_PF + i), 4);
            mbar_init(bar(CF::BAR_PV + i), 1);
        }
        mbar_init(bar(CF::BAR_CLC), 1);
        mbar_init(bar(CF::BAR_DRAIN), 2);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 96) {
        tma_prefetch_map(&tmap_q);
        tma_prefetch_map(&tmap_k);
        tma_prefetch_map(&tmap_v);
        tma_prefetch_map(&tmap_o);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t timeout = p.timeout_ns;
    grid_dependency_wait();
    grid_launch_dependents();

    // An item as every role sees it: the pair and head, the steps of 64 keys
    // [fs, es) each tile visits (empty: 0, 0) and the blocks of 128 that hold them
    struct Item {
        int b, h, q0, slot, fs[2], es[2], j0, j1;  // slot: of its partial sums
        __device__ bool visits(int i, int n) const { return i ? n >= fs[1] && n < es[1] : n >= fs[0] && n < es[0]; }
    };
    auto unpack = [&](const int4 &x, const int4 &y) {
        Item it;
        it.b = x.y / p.H;
        it.h = x.y - it.b * p.H;
        it.q0 = x.x * 2 * CF::BM;
        it.fs[0] = x.z;
        it.es[0] = x.w;
        it.fs[1] = y.x;
        it.es[1] = y.y;
        it.slot = y.z;
        const bool e0 = x.w > x.z, e1 = y.y > y.x;
        it.j0 = (e0 && e1 ? min(x.z, y.x) : e0 ? x.z : y.x) >> 1;
        it.j1 = (max(x.w, y.y) + 1) >> 1;
        return it;
    };
    auto take_item = [&](int t, Item *out) {
        const bool w = __all_sync(0xffffffffu, wait_bounded(bar(CF::BAR_TF + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u,
                                                            abort_flag, timeout, ERR_EPILOGUE));
        if (!w)
            return false;
        const int4 x = item_slots[2 * (t & 1)], y = item_slots[2 * (t & 1) + 1];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(CF::BAR_TE + (t & 1)));
        if (x.x < 0)
            return false;
        *out = unpack(x, y);
        return true;
    };

    uint32_t issued = 0, parity = 0;  // bit 0: Q, bits 8..: K slots, bits 16..: V slots
    if (warp < 4) {
        regs_decrease<CF::REGS_CONTROL>();
        if (warp == 0) {
            // ------------------------------------------------------------ items and loads
            const int BH = p.B * p.H;
            const uint32_t clc_dst = smem_addr(smem + CF::OFF_CLC);
            auto wait = [&](int id, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_PRODUCER)) != 0;
            };
            // Item `index` (-1: none) as the t-th: which steps its tiles visit, for the others
            auto publish = [&](int t, int index, Item *out) {
                if (t >= 2 && !wait(CF::BAR_TE + (t & 1), static_cast<uint32_t>(t >> 1) - 1))
                    return false;
                int4 x = make_int4(-1, 0, 0, 0), y = make_int4(0, 0, 0, 0);
                if (index >= 0) {
                    y.z = index;
                    const int split = index % p.splits;
                    index /= p.splits;
                    // CTAs start in the order of their index.  Causal: every head's last (heaviest) pair of tiles
                    // first; else the pairs of one head together, so that those running side by side share its K and V.
                    x.x = p.mask.causal ? p.num_pairs - 1 - index / BH : index % p.num_pairs;
                    x.y = p.mask.causal ? index % BH : index / p.num_pairs;
                    const int b = x.y / p.H;
                    const int32_t *docs = p.mask.doc_offsets
                                              ? p.mask.doc_offsets + static_cast<int64_t>(b) * (p.mask.num_docs + 1) : nullptr;
                    // Intervals move on from row to row, so a tile's keys reach from its first row's first key to its last
                    // row's end: lanes 2 i and 2 i + 1 look up tile i's first and last row that lie in a document.
                    int i0 = x.x * 2 * CF::BM + ((lane >> 1) & 1) * CF::BM, i1 = min(i0 + CF::BM, p.mask.Sq) - 1;
                    if (docs) {
                        i0 = max(i0, max(docs[0], 0) - p.mask.q_offset);
                        i1 = min(i1, max(docs[p.mask.num_docs], 0) - 1 - p.mask.q_offset);
                    }
                    // A row of a document that begins past the keys sees none of them, and stands for their end: a
                    // tile that begins there has none, one that ends there has rows that see them to the end.
                    int2 seen = make_int2(0, 0);
                    if (lane < 4 && i0 <= i1) {
                        seen = visible_keys(p.mask, docs, b, lane & 1 ? i1 : i0);
                        if (seen.y <= seen.x)
                            seen = make_int2(p.mask.Sk, p.mask.Sk);
                    }
                    const int lo0 = __shfl_sync(0xffffffffu, seen.x, 0), hi0 = __shfl_sync(0xffffffffu, seen.y, 1);
                    const int lo1 = __shfl_sync(0xffffffffu, seen.x, 2), hi1 = __shfl_sync(0xffffffffu, seen.y, 3);
                    if (hi0 > lo0) {
                        x.z = lo0 / CF::BS;
                        x.w = (hi0 + CF::BS - 1) / CF::BS;
                    }
                    if (hi1 > lo1) {
                        y.x = lo1 / CF::BS;
                        y.y = (hi1 + CF::BS - 1) / CF::BS;
                    }
                    if (p.splits > 1) {
                        // this CTA's share of the blocks that hold either tile's steps
                        const Item all = unpack(x, y);
                        const int blocks = all.j1 - all.j0;
                        const int first = 2 * (all.j0 + static_cast<int>(static_cast<int64_t>(split) * blocks / p.splits));
                        const int end = 2 * (all.j0 + static_cast<int>(static_cast<int64_t>(split + 1) * blocks / p.splits));
                        auto clip = [&](int &a, int &b) {
                            a = max(a, first);
                            b = min(b, end);
                            if (b <= a)
                                a = b = 0;
                        };
                        clip(x.z, x.w);
                        clip(y.x, y.y);
                    }
                    // checked build: heads, tiles, steps and the place of partial sums
                    const int steps = (p.mask.Sk + CF::BS - 1) / CF::BS;
                    if (check_ok(x.x >= 0 && x.x < p.num_pairs && x.y >= 0 && x.y < BH && x.z >= 0 && x.w <= steps &&
                                 y.x >= 0 && y.y <= steps && y.z < p.num_pairs * BH * p.splits)) {
                        *out = unpack(x, y);
                        index = 0;
                    } else {
                        x.x = index = -1;
                    }
                }
                if (lane == 0) {
                    item_slots[2 * (t & 1)] = x;
                    item_slots[2 * (t & 1) + 1] = y;
                    mbar_arrive(bar(CF::BAR_TF + (t & 1)));
                }
                __syncwarp();
                return index >= 0;
            };
            Item it;
            int st = 0;
            uint32_t ph = 0, qph = 0;
            bool ok = publish(0, static_cast<int>(blockIdx.x), &it);
            for (int t = 0; ok; ++t) {
                if (it.j0 < it.j1) {
                    const int hk = it.h / p.group;
                    if (lane == 0) {
                        ok = wait_bounded(bar(CF::BAR_QE), qph ^ 1u, abort_flag, timeout, ERR_PRODUCER);
                        if (ok) {
                            mbar_arrive_expect_tx(bar(CF::BAR_QF), 2 * CF::Q_BYTES);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int a = 0; a < CF::D_ATOMS; ++a)
                                    tma_load_4d(sQ + i * CF::Q_BYTES + a * CF::ATOM_BYTES, &tmap_q, bar(CF::BAR_QF), 64 * a,
                                                it.q0 + i * CF::BM, it.h, it.b);
                            issued |= 1u;
                            parity = (parity & ~1u) | qph;
                        }
                        for (int j = it.j0; ok && j < it.j1; ++j) {
#pragma unroll
                            for (int kv = 0; kv < 2; ++kv) {
                                const int full = (kv ? CF::BAR_VF : CF::BAR_KF) + st;
                                if (!(ok = ok && wait_bounded(bar((kv ? CF::BAR_VE : CF::BAR_KE) + st), ph ^ 1u, abort_flag,
                                                              timeout, ERR_PRODUCER)))
                                    break;
                                mbar_arrive_expect_tx(bar(full), CF::KV_BYTES);
#pragma unroll
                                for (int a = 0; a < CF::D_ATOMS; ++a)
                                    tma_load_4d((kv ? sV : sK) + st * CF::KV_BYTES + a * CF::ATOM_BYTES,
                                                kv ? &tmap_v : &tmap_k, bar(full), 64 * a, j * CF::BN, hk, it.b);
                                const int bit = (kv ? 16 : 8) + st;
                                issued |= 1u << bit;
                                parity = (parity & ~(1u << bit)) | (ph << bit);
                            }
                            if (++st == KS) {
                                st = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                    qph ^= 1u;
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                }
                if (!ok)
                    break;
                // The next item is asked for when this one's last loads are out: the ring's depth before its end, which
                // covers the answer.  Asked for at its start, items would be dealt out regardless of who finishes first
                // (16 capped causal heads x 4096 on 148 CTAs: 162 us against 120).
                if (lane == 0) {
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(bar(CF::BAR_CLC), 16);
                    clc_request(clc_dst, bar(CF::BAR_CLC));
                }
                __syncwarp();
                const bool answered = __all_sync(0xffffffffu, wait_drain(bar(CF::BAR_CLC), static_cast<uint32_t>(t) & 1u, timeout));
                if (!answered)
                    break;
                const int next = clc_answer(clc_dst);
                ok = publish(t + 1, next, &it);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ S = Q K^T
            // The two issuers' waits pass while the other's products run.  The whole
            // warp walks the loop and one elected lane issues: what the instructions
            // are made from stays uniform across the warp.
            constexpr uint32_t IDESC_QK = mma_idesc_f16(DT, 128, CF::BS, 0, 0);  // Q, K both K-major
            const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024), k_desc = smem_desc_sw128(sK, 16, 1024);
            auto kmaj = [](int k) { return static_cast<uint64_t>(((k >> 2) * CF::ATOM_BYTES + (k & 3) * 32) >> 4); };
            auto wait = [&](int id, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_MMA_DATA)) != 0;
            };
            Item it;
            uint32_t count[2][2] = {{0, 0}, {0, 0}}, busy = 0, kg = 0;  // steps of each tile and set, items with blocks, blocks of K so far
            bool ok = true;
            for (int t = 0; ok && take_item(t, &it); ++t) {
                if (it.j0 >= it.j1)
                    continue;
                ok = wait(CF::BAR_QF, busy);
                for (int j = it.j0; ok && j < it.j1; ++j, ++kg) {
                    const int st = static_cast<int>(kg % KS);
                    ok = wait(CF::BAR_KF + st, kg / KS);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int set = q >> 1, i = q & 1;
                        if (!ok || !it.visits(i, 2 * j + set))
                            continue;
                        // its columns are free: the P over them has been read by P V
                        const uint32_t c = count[i][set];
                        if (c > 0 && !(ok = wait(CF::BAR_PV + 2 * i + set, c - 1)))
                            continue;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint64_t qd = q_desc + ((i * CF::Q_BYTES) >> 4);
                            const uint64_t kd = k_desc + ((st * CF::KV_BYTES + set * CF::BS * 128) >> 4);
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                tc_mma_f16(tmem_base + static_cast<uint32_t>(CF::TMEM_S + i * 128 + set * CF::BS), qd + kmaj(k),
                                           kd + kmaj(k), IDESC_QK, k != 0 ? 1u : 0u);
                            tc_commit(bar(CF::BAR_SF + 2 * i + set));
                        }
                        __syncwarp();
                        count[i][set] = c + 1;
                    }
                    if (ok && elect_one()) {
                        tc_commit(bar(CF::BAR_KE + st));
                        if (j + 1 == it.j1)
                            tc_commit(bar(CF::BAR_QE));
                    }
                    __syncwarp();
                }
                ++busy;
            }
            if (elect_one())
                tc_commit(bar(CF::BAR_DRAIN));
            __syncwarp();
            wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
        } else if (warp == 2) {
            // ------------------------------------------------------------ O += P V
            constexpr uint32_t IDESC_PV = mma_idesc_f16(DT, 128, D, 0, 1);  // P K-major (TMEM), V N-major
            const uint64_t v_desc = smem_desc_sw128(sV, CF::ATOM_BYTES, 1024);
            auto wait = [&](int id, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_MMA_ACC)) != 0;
            };
            Item it;
            uint32_t count[2][2] = {{0, 0}, {0, 0}}, busy[2] = {0, 0}, vg = 0;  // steps and items of each tile, blocks of V so far
            bool ok = true;
            for (int t = 0; ok && take_item(t, &it); ++t) {
                for (int j = it.j0; ok && j < it.j1; ++j, ++vg) {
                    const int st = static_cast<int>(vg % KS);
                    ok = wait(CF::BAR_VF + st, vg / KS);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int set = q >> 1, i = q & 1;
                        if (!ok || !it.visits(i, 2 * j + set))
                            continue;
                        const uint32_t c = count[i][set];
                        // its sums begin here: those of both sets, or (TWIN) of this one
                        const bool first = CF::TWIN ? 2 * j + set < it.fs[i] + 2 : 2 * j + set == it.fs[i];
                        // the last item's O has been read before this one's begins
                        if ((first && busy[i] > 0 && !(ok = wait(CF::BAR_OE + i, busy[i] - 1))) ||
                            !(ok = wait(CF::BAR_PF + 2 * i + set, c)))
                            continue;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint64_t vd = v_desc + ((st * CF::KV_BYTES + set * CF::BS * 128) >> 4);
#pragma unroll
                            for (int k = 0; k < CF::BS / 16; ++k)
                                tc_mma_f16_ts(tmem_base + static_cast<uint32_t>(CF::TMEM_O + i * 128 + (CF::TWIN ? set * D : 0)),
                                              tmem_base + static_cast<uint32_t>(CF::TMEM_S + i * 128 + set * CF::BS + 8 * k),
                                              vd + ((2048 * k) >> 4), IDESC_PV, (!first || k > 0) ? 1u : 0u);
                            tc_commit(bar(CF::BAR_PV + 2 * i + set));
                        }
                        __syncwarp();
                        count[i][set] = c + 1;
                    }
                    if (ok && elect_one())
                        tc_commit(bar(CF::BAR_VE + st));
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    busy[i] += it.es[i] > it.fs[i] ? 1u : 0u;
            }
            if (elect_one())
                tc_commit(bar(CF::BAR_DRAIN));
            __syncwarp();
            wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
        }
        __syncwarp();
    } else {
        regs_increase<CF::REGS_SOFTMAX>();
        // ------------------------------------------------------------ softmax and output of one tile
        constexpr int HN = CF::TWIN ? CF::BS / 2 : CF::BS;  // columns in registers at a time
        const int tile = ((warp - 4) >> 2) & 1;
        const int own = CF::TWIN ? (warp - 4) >> 3 : 0;  // TWIN: the set
        const int r = (warp & 3) * 32 + lane;  // row of the tile (Tensor Memory lane)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr0 = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_S + tile * 128);
        const uint32_t o_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_O + tile * 128);
        const uint32_t o_own = o_addr + static_cast<uint32_t>(own * D);
        uint4 *out_buf = reinterpret_cast<uint4 *>(smem + CF::OFF_OUT + (warp - 4) * 2048);
        auto wait_warp = [&](int id, uint32_t par) -> bool {
            return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_EPILOGUE));
        };
        uint32_t count[2] = {0, 0};  // steps of this tile so far, by set
        Item it;
        bool ok = true;
        for (int t = 0; ok && take_item(t, &it); ++t) {
            const int fs = tile ? it.fs[1] : it.fs[0], es = tile ? it.es[1] : it.es[0];
            const int row = it.q0 + tile * CF::BM + r;  // query index
            const int32_t *docs = p.mask.doc_offsets
                                      ? p.mask.doc_offsets + static_cast<int64_t>(it.b) * (p.mask.num_docs + 1) : nullptr;
            const int2 seen = visible_keys(p.mask, docs, it.b, row);
            const float slope2 = BIAS ? __ldg(p.score.slopes + it.h) * 1.4426950408889634f : 0.0f;
            const int pos = p.mask.q_offset + row;
            // m: the reference maximum of the row's weights (log2 units); l: sum of the weights against m
            float m = -INFINITY, l = 0.0f;
            const int n_first = CF::TWIN ? fs + ((fs ^ own) & 1) : fs;
            for (int n = n_first; n < es; n += CF::TWIN ? 2 : 1) {
                const int set = CF::TWIN ? own : n & 1;
                const uint32_t c = set ? count[1] : count[0];
                if (!(ok = wait_warp(CF::BAR_SF + 2 * tile + set, c)))
                    break;
                tc_fence_after_sync();
                const uint32_t s_addr = s_addr0 + static_cast<uint32_t>(CF::BS * set);
                const int key0 = n * CF::BS;
                const float to_log2 = CAP ? p.score.cap_log2 : p.score.scale_log2;  // of a score without a bias
                const int nlo = seen.x - key0, nhi = seen.y - key0;
                const bool cut = !__all_sync(0xffffffffu, nlo <= 0 && nhi >= CF::BS);
                // keys outside the row's interval count neither in the maximum nor in the weights
                auto hide = [&](uint32_t (&sv)[HN], int e0) {
                    if (cut && CF::TWIN) {  // by bits: fewer registers
                        const int lo = min(max(nlo - e0, 0), 32), hi = min(max(nhi - e0, 0), 32);
                        const uint32_t see = static_cast<uint32_t>((1ull << hi) - 1ull) & ~static_cast<uint32_t>((1ull << lo) - 1ull);
#pragma unroll
                        for (int e = 0; e < HN; ++e)
                            if (!(see & (1u << (e & 31))))
                                sv[e] = __float_as_uint(-INFINITY);
                    } else if (cut) {
#pragma unroll
                        for (int e = 0; e < HN; ++e)
                            if (e0 + e < nlo || e0 + e >= nhi)
                                sv[e] = __float_as_uint(-INFINITY);
                    }
                };
                // columns e0 ..: tanh of the capped scores, or biased scores in log2 units, in place of the raw ones
                auto scores = [&](uint32_t (&sv)[HN], int e0) {
                    if constexpr (CAP)
                        tanh_scores<HN>(sv, p.score.cap_arg);
                    if constexpr (BIAS) {
                        const float dist0 = static_cast<float>(pos - key0 - e0);
#pragma unroll
                        for (int e = 0; e < HN; e += 2) {
                            float2 x = fmul2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), splat2(to_log2));
                            const float2 dist = fadd2(splat2(dist0), make_float2(-static_cast<float>(e), -static_cast<float>(e + 1)));
                            x = ffma2(make_float2(fabsf(dist.x), fabsf(dist.y)), splat2(-slope2), x);
                            sv[e] = __float_as_uint(x.x);
                            sv[e + 1] = __float_as_uint(x.y);
                        }
                    }
                    hide(sv, e0);
                };
                auto top = [&](const uint32_t (&sv)[HN]) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < HN / 8; ++i) {
                        const float *f = reinterpret_cast<const float *>(&sv[8 * i]);
                        mx = fmax3(mx, fmax3(fmax3(f[0], f[1], f[2]), f[3], f[4]), fmax3(f[5], f[6], f[7]));
                    }
                    return mx;
                };
                uint32_t sv[HN], p1[CF::TWIN ? HN / 2 : 1];
                float mx;
                if constexpr (CF::TWIN) {
                    // 32 columns at a time: the first half waits in Tensor Memory for its second reading
                    tmem_load_32cols(s_addr, sv);
                    tmem_load_wait();
                    scores(sv, 0);
                    mx = top(sv);
                    if constexpr (CAP || BIAS)
                        tmem_store_32cols(s_addr, sv);
                    tmem_load_32cols(s_addr + HN, sv);
                    tmem_load_wait();
                    scores(sv, HN);
                    mx = fmaxf(mx, top(sv));
                    if constexpr (CAP || BIAS)
                        tmem_store_wait();
                } else {
                    tmem_load_32cols(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    tmem_load_32cols(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[HN - 32]));
                    tmem_load_wait();
                    scores(sv, 0);
                    mx = top(sv);
                }
                if constexpr (!BIAS)
                    mx *= to_log2;
                // move the reference maximum only when the weights would exceed 2^8
                const bool resc = mx > m + CF::RESCALE_LOG2;
                const float m_new = resc ? mx : m;
                const float m_ref = m_new == -INFINITY ? 0.0f : m_new;  // no visible key yet: all weights 0
                const float alpha = resc ? exp2_approx_ftz(m - m_ref) : 1.0f;  // 0 when m is -inf
                const float2 negm2 = splat2(-m_ref);
                float2 part[4] = {splat2(0.0f), splat2(0.0f), splat2(0.0f), splat2(0.0f)};
                auto weights = [&](const uint32_t (&sv)[HN], uint32_t *out) {
#pragma unroll
                    for (int e = 0; e < HN; e += 2) {
                        const float2 s = make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                        const float2 x = BIAS ? fadd2(s, negm2) : ffma2(s, splat2(to_log2), negm2);
                        const float2 w = make_float2(exp2_approx_ftz(x.x), exp2_approx_ftz(x.y));
                        part[(e >> 1) & 3] = fadd2(part[(e >> 1) & 3], w);
                        out[e / 2] = pack2<DT>(w.x, w.y);  // keys e, e + 1: one 32-bit column
                    }
                };
                if constexpr (CF::TWIN) {
                    weights(sv, p1);
                    tmem_load_32cols(s_addr, sv);
                    tmem_load_wait();
                    if constexpr (!(CAP || BIAS))
                        hide(sv, 0);
                    uint32_t p0[HN / 2];
                    weights(sv, p0);
                    tmem_store_16cols(s_addr, p0);
                    tmem_store_16cols(s_addr + HN / 2, p1);
                } else {
                    weights(sv, sv);
                    tmem_store_32cols(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                }
                const float2 ps = fadd2(fadd2(part[0], part[1]), fadd2(part[2], part[3]));
                l = l * alpha + (ps.x + ps.y);
                m = m_new;
                // rows whose maximum moved take O down by alpha once it holds all steps before n (those before
                // n - 1 are in it: S(n - 1) was issued behind the P V of n - 3, S(n) behind that of n - 2; TWIN: that
                // was the set's last)
                if (n > n_first && __any_sync(0xffffffffu, resc)) {
                    if (!CF::TWIN && !(ok = wait_warp(CF::BAR_PV + 2 * tile + (set ^ 1), (set ? count[0] : count[1]) - 1)))
                        break;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tmem_load_32cols(o_own + 32 * k, o);
                        tmem_load_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_store_32cols(o_own + 32 * k, o);
                    }
                }
                tmem_store_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(CF::BAR_PF + 2 * tile + set));
                if (set)
                    ++count[1];
                else
                    ++count[0];
            }
            // output: O / l once the last P V of both sets have landed; rows that see no key get 0 and lse -inf
#pragma unroll
            for (int set = 0; set < 2; ++set)
                if (ok && count[set] > 0)
                    ok = wait_warp(CF::BAR_PV + 2 * tile + set, count[set] - 1);
            if (!ok)
                break;
            tc_fence_after_sync();
            // TWIN: the sets' sums are joined, half the columns by each of their warpgroups
            float f0 = 1.0f, f1 = 0.0f;
            bool has0 = true, has1 = false;
            if constexpr (CF::TWIN) {
                float2 *ml = reinterpret_cast<float2 *>(smem + CF::OFF_ML) + ((t & 1) * 2 + tile) * 256 + r;
                ml[own * 128] = make_float2(m, l);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(CF::BAR_ML + tile));
                if (!(ok = wait_warp(CF::BAR_ML + tile, static_cast<uint32_t>(t))))
                    break;
                tc_fence_after_sync();
                const float2 a = ml[0], c = ml[128];
                m = fmaxf(a.x, c.x);
                f0 = a.x == -INFINITY ? 0.0f : exp2_approx_ftz(a.x - m);
                f1 = c.x == -INFINITY ? 0.0f : exp2_approx_ftz(c.x - m);
                l = a.y * f0 + c.y * f1;
                has0 = es - fs >= 2 || (fs & 1) == 0;
                has1 = es - fs >= 2 || (fs & 1) == 1;
            }
            const int k0 = CF::TWIN ? own : 0, k1 = CF::TWIN ? own + 1 : D / 32;  // of 32 columns
            auto load_sums = [&](int k, uint32_t (&o)[32]) {
                if constexpr (CF::TWIN) {
                    tmem_load_32cols(o_addr + 32 * k, o);
                    tmem_load_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = has0 ? __float_as_uint(__uint_as_float(o[e]) * f0) : 0u;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t other[16];
                        tmem_load_16cols(o_addr + D + 32 * k + 16 * c, other);
                        tmem_load_wait();
                        if (has1) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[16 * c + e] = __float_as_uint(fmaf(__uint_as_float(other[e]), f1, __uint_as_float(o[16 * c + e])));
                        }
                    }
                } else {
                    tmem_load_32cols(o_addr + 32 * k, o);
                    tmem_load_wait();
                }
            };
            if (p.splits > 1) {
                const int64_t at = (static_cast<int64_t>(it.slot) * 2 + tile) * 128 + r;
                if (own == 0)
                    p.part_ml[at] = make_float2(m, l);
                float4 *part = p.part_o + (static_cast<int64_t>(it.slot) * 2 + tile) * (D / 4) * 128 + r;
#pragma unroll 1
                for (int k = k0; k < k1 && es > fs; ++k) {
                    uint32_t o[32];
                    load_sums(k, o);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        part[(8 * k + v) * 128] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                              __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
                if (es > fs) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(CF::BAR_OE + tile));
                }
                continue;
            }
            const bool empty = seen.y <= seen.x || l == 0.0f;
            const float inv = empty ? 0.0f : 1.0f / l;
            const int row0 = it.q0 + tile * CF::BM + (warp & 3) * 32;  // this warp's first row
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                uint32_t o[32];
                if (es > fs) {
                    load_sums(k, o);
                    if (k + 1 == k1) {  // in registers: the next item's O may begin
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(CF::BAR_OE + tile));
                    }
                }
                if (row0 >= p.mask.Sq)
                    continue;
                // 32 rows x 32 columns through this warp's buffer; rows behind the tensor's are not written
                if (lane == 0)
                    bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (!empty) {
                        w.x = pack2<DT>(__uint_as_float(o[8 * v]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
                        w.y = pack2<DT>(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
                        w.z = pack2<DT>(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
                        w.w = pack2<DT>(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
                    }
                    out_buf[4 * lane + v] = w;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_4d(&tmap_o, smem_addr(out_buf), 32 * k, row0, it.h, it.b);
                    bulk_commit_group();
                }
            }
            if (p.lse && own == 0 && row < p.mask.Sq)
                p.lse[(static_cast<int64_t>(it.b) * p.H + it.h) * p.mask.Sq + row] =
                    empty ? -INFINITY : m * 0.69314718055994531f + logf(l);
        }
        if (lane == 0)
            bulk_wait_group<0>();
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        if (issued & 1u)
            wait_drain(bar(CF::BAR_QF), parity & 1u, timeout);
        for (int s = 0; s < KS; ++s) {
            if (issued & (1u << (8 + s)))
                wait_drain(bar(CF::BAR_KF + s), (parity >> (8 + s)) & 1u, timeout);
            if (issued & (1u << (16 + s)))
                wait_drain(bar(CF::BAR_VF + s), (parity >> (16 + s)) & 1u, timeout);
        }
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

struct AttnJoinParams {
    int32_t H, Sq, num_pairs, BH, splits, causal;
    const float4 *part_o;
    const float2 *part_ml;
    uint16_t *O;
    int64_t o_batch, o_head, o_row;
    float *lse;
};

// Adds the splits of each row in the order of the keys: a row a lane, D / 8
// columns a warp (256 threads), a CTA for 32 rows.
template <int DT, int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnJoinParams p)
{
    constexpr int C4 = D / 32;  // groups of four columns a warp
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bx = static_cast<int>(blockIdx.x);
    const int quarter = bx & 3, tile = (bx >> 2) & 1, item = bx >> 3;
    if (!check_ok(item < p.num_pairs * p.BH))
        return;
    // the item's pair and head, as the forward numbers them
    const int pair = p.causal ? p.num_pairs - 1 - item / p.BH : item % p.num_pairs;
    const int bh = p.causal ? item % p.BH : item / p.num_pairs;
    const int r = 32 * quarter + lane;
    const int row = (2 * pair + tile) * 128 + r;
    if (row >= p.Sq)
        return;
    auto slot = [&](int s) { return (static_cast<int64_t>(item) * p.splits + s) * 2 + tile; };
    float M = -INFINITY, L = 0.0f, acc[4 * C4];
#pragma unroll
    for (int v = 0; v < 4 * C4; ++v)
        acc[v] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s)
        M = fmaxf(M, p.part_ml[slot(s) * 128 + r].x);
#pragma unroll 2
    for (int s = 0; s < p.splits; ++s) {
        const float2 x = p.part_ml[slot(s) * 128 + r];
        if (x.x == -INFINITY && x.y == 0.0f)
            continue;  // saw no key: its sums may not even be there
        const float f = exp2_approx_ftz(x.x - M);
        L = fmaf(x.y, f, L);
        const float4 *part = p.part_o + (slot(s) * (D / 4) + warp * C4) * 128 + r;
#pragma unroll
        for (int v = 0; v < C4; ++v) {
            const float4 w = part[v * 128];
            acc[4 * v] = fmaf(w.x, f, acc[4 * v]);
            acc[4 * v + 1] = fmaf(w.y, f, acc[4 * v + 1]);
            acc[4 * v + 2] = fmaf(w.z, f, acc[4 * v + 2]);
            acc[4 * v + 3] = fmaf(w.w, f, acc[4 * v + 3]);
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int b = bh / p.H, h = bh - b * p.H;
    uint16_t *orow = p.O + b * p.o_batch + h * p.o_head + static_cast<int64_t>(row) * p.o_row + warp * 4 * C4;
#pragma unroll
    for (int v = 0; v < C4; v += 2)
        *reinterpret_cast<uint4 *>(orow + 4 * v) =
            make_uint4(pack2<DT>(acc[4 * v] * inv, acc[4 * v + 1] * inv), pack2<DT>(acc[4 * v + 2] * inv, acc[4 * v + 3] * inv),
                       pack2<DT>(acc[4 * v + 4] * inv, acc[4 * v + 5] * inv),
                       pack2<DT>(acc[4 * v + 6] * inv, acc[4 * v + 7] * inv));
    if (p.lse && warp == 0)
        p.lse[static_cast<int64_t>(bh) * p.Sq + row] = L == 0.0f ? -INFINITY : M * 0.69314718055994531f + logf(L);
}

} // namespace tl
