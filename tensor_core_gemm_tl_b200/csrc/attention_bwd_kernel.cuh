// attention_bwd_kernel.cuh -- the gradients of attention_ex_kernel.cuh:
//
//     P_ij  = exp(y_ij - lse_i)                 (0 outside the row's interval)
//     dV_j  = sum_i P_ij dO_i
//     delta_i = sum_j P_ij dP_ij,               dP_ij = dO_i . V_j
//     dX_ij = P_ij (dP_ij - delta_i) c_ij,      c = 1, or 1 - tanh^2 with capped scores
//     dQ_i  = scale sum_j dX_ij K_j,   dK_j = scale sum_i dX_ij Q_i
//
// with i running over every query head that shares the key/value head.  Three
// launches (and two that join pieces), none of which adds with atomics, so results repeat bit for bit:
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
// Pipeline: a block is 128 x 64 scores; blocks alternate between two sets of
// Tensor Memory columns (S and dP) and two teams of eight warps, 32 columns a
// thread, so that one team's exponentials run beside the other's second step and
// the products of both.  The products of a block go out as dV(n), dK(n), S(n + 2),
// dP(n + 2): S(n + 2) takes the columns dV(n) has read P(n) from and dP(n + 2) those
// of dX(n), each wait covered by the product in between.  (Blocks of 128 x 128 in
// one set, which D = 128 leaves room for, need 2080 instead of 2800 clocks of
// products a 128 x 128 but left warps and products waiting for one another:
// 3300, and 5700 with capped scores.)
//
// The CTAs are persistent and take tiles from a counter; the next tile's operands
// load while this one's sums leave through shared memory and TMA stores (stores
// of a row a thread held up every other memory operation of the SM, the products'
// issue included: 5000 clocks a tile).
//
// Few tiles of many blocks are cut into pieces along the blocks (attention_bwd.cu
// says when): each piece leaves fp32 sums, and attention_bwd_join_kernel adds them
// in their order, taking dQ's correction by the whole e.
//
// What bounds it: 4 products of 128 x 64 x D a block, with D = 128 1024 clocks at
// 4096 multiply-adds a clock and SM, 1400 as S and dP read 48 bytes of shared
// memory operands for every 32 clocks' worth of products, against one 2^x a score
// (512 clocks; 2.5 times that with capped scores).  Measured, 4 x 16 heads on 4 x 4096
// x 4096 x 128, bf16: all three launches 1740 us, causal 900; with six documents a
// sequence rows 25, dQ 171, dK and dV 215 us, the tensor pipe 50..53 % busy, the
// warps waiting for Tensor Memory loads and barriers.
//
// 16-bit range: bf16 takes P and dX as they are.  fp16 holds P times 2^10 and
// dX times 2^15 over a power of two that no |dX| exceeds (P of long rows and
// gradients of small losses lie below fp16's normal range, dX of large values
// above it).  O being a mean of rows of V, |dX_ij| <= |dO_i . (V_j - O_i)| <=
// 2 max |dO_i| max |V_j|, 2-norms of the queries and keys that count: the rows
// kernel takes them, those of V in CTAs of their own (3 x 8 heads x 1001 x 1001 x
// 64, with its forward: 70 -> 72 us; 4 x 16 heads on 4 x 4096 x 4096 x 128 with
// documents: 552 -> 560).  The factors are powers of two and leave with the fp32
// sums.
#pragma once

#include <type_traits>

#include "attention_common.cuh"

namespace tl {

constexpr int kBwdCols = 64;  // columns of a block of scores
template <int DT>
constexpr float kPShift = DT == 0 ? 10.0f : 0.0f;  // fp16 holds P times 2^10

struct AttnBwdParams {
    MaskParams mask;
    ScoreParams score;
    int32_t B, H, Hk, group;
    int32_t nqb;               // blocks of 64 queries
    int32_t tiles;             // 128-row tiles of the keys (DKV) or of the queries
    float scale;               // softmax scale
    float *rows;               // [B][H][nqb][2][64]: -lse in log2 units (-inf where the row sees nothing) plus the
                               // exponent of P's factor, -delta
    const int32_t *intervals;  // [B][nqb][3][64]: first and end key of each query; 0.0f where it sees one key, else 1.0f
    const int4 *ranges;        // [B][nqb]: least first, largest end, largest first, least end of the block's queries
    const float *norms;        // fp16: the largest |dO_i|^2 of queries that see some key and |V_j|^2 of keys that some see
    int32_t *next;             // counter that pieces are taken from, 0 at the start
    int32_t chunk, splits;     // a piece is up to `chunk` blocks of a tile, a tile `splits` pieces at most
    int32_t *pieces;           // [tiles of all heads]: how many a tile has; null where every tile is one
    float4 *part;              // [tiles][splits][2][D / 4][128]: a row a lane, so a warp's rows lie side by side
    float *part_e;             // dQ: [tiles][splits][128]: e
    uint64_t timeout_ns;
};

struct AttnBwdJoinParams {
    MaskParams mask;
    int32_t H, heads, tiles, BH, splits, nqb;  // heads: of the tiles
    const int32_t *pieces;
    const float4 *part;
    const float *part_e;
    float *rows;               // dQ: as the passes'
    const int32_t *intervals;
    uint16_t *out0, *out1;     // dQ, or dK and dV
    int64_t s0[3], s1[3];
};

// The tile and batch * heads index of item i: causal: the heaviest tiles first (the first keys, the last queries);
// else one head's tiles together
template <bool DKV>
__device__ __forceinline__ int2 bwd_tile(int i, int tiles, int BH, bool causal)
{
    return causal ? make_int2(DKV ? i / BH : tiles - 1 - i / BH, i % BH) : make_int2(i % tiles, i / tiles);
}

struct AttnBwdRowsParams {
    MaskParams mask;
    int32_t B, H, Hk, D, nqb;
    int32_t query_ctas, nkb;   // CTAs for queries; blocks of 64 keys
    const uint16_t *O, *dO, *V;
    int64_t so[3], sdo[3], sv[3];
    const float *lse;          // [B][H][Sq]
    float *rows;
    int32_t *intervals;
    int4 *ranges;
    float *norms;              // fp16: as the passes', 0 at the start
    int32_t *next;             // the two passes' tile counters
};

// The largest of the warp's finite norms (inf and NaN spoil their own rows only) into `to`, of floats that are not
// negative and so order like their bits
__device__ __forceinline__ void raise_norm(float *to, float norm)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        norm = fmaxf(norm, __shfl_xor_sync(0xffffffffu, norm, off));
    if ((threadIdx.x & 31) == 0)
        atomicMax(reinterpret_cast<unsigned *>(to), __float_as_uint(norm));
}

// One CTA (256 threads) per 64 queries of a head: 8 lanes a row.  Bound by
// reading O and dO once.  fp16: then one per 64 keys of a head, for V's norms.
template <int DT, int D>
__global__ void __launch_bounds__(256) attention_bwd_rows_kernel(const AttnBwdRowsParams p)
{
    __shared__ int32_t docs_smem[kDocsInSmem];
    __shared__ int red[4];
    grid_dependency_wait();
    grid_launch_dependents();
    if (DT == 0 && static_cast<int>(blockIdx.x) >= p.query_ctas) {
        const int at = static_cast<int>(blockIdx.x) - p.query_ctas;
        const int bhk = at / p.nkb, b = bhk / p.Hk, hk = bhk - b * p.Hk, sub = threadIdx.x & 7;
        const int32_t *docs = p.mask.doc_offsets
                                  ? p.mask.doc_offsets + static_cast<int64_t>(b) * (p.mask.num_docs + 1) : nullptr;
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < kBwdCols / 32; ++k) {
            const int j = (at - bhk * p.nkb) * kBwdCols + (threadIdx.x >> 3) + 32 * k;
            float norm = 0.0f;
            if (key_is_seen(p.mask, docs, b, j)) {
                const uint16_t *v = p.V + b * p.sv[0] + hk * p.sv[1] + static_cast<int64_t>(j) * p.sv[2];
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(v + 64 * c + 8 * sub));
                    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v0 = to_float<DT>(static_cast<uint16_t>(a[e] & 0xFFFFu));
                        const float v1 = to_float<DT>(static_cast<uint16_t>(a[e] >> 16));
                        norm = fmaf(v0, v0, fmaf(v1, v1, norm));
                    }
                }
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1)
                norm += __shfl_xor_sync(0xffffffffu, norm, off);
            top = norm < INFINITY ? fmaxf(top, norm) : top;
        }
        raise_norm(p.norms + 1, top);
        return;
    }
    const int qb = static_cast<int>(blockIdx.x % p.nqb);
    const int bh = static_cast<int>(blockIdx.x / p.nqb);
    const int b = bh / p.H, h = bh % p.H;
    if (blockIdx.x == 0 && threadIdx.x < 2)
        p.next[threadIdx.x] = 0;
    // all of a thread's words first: 2 rows x D / 64 words of O and of dO in flight
    constexpr int RN = kBwdCols / 32, WN = D / 64;
    float top = 0.0f;
    const int sub = threadIdx.x & 7;
    uint4 wo[RN][WN], wg[RN][WN];
    float l[RN];
#pragma unroll
    for (int k = 0; k < RN; ++k) {
        const int i = qb * kBwdCols + (threadIdx.x >> 3) + 32 * k;
        l[k] = -INFINITY;
        if (i < p.mask.Sq) {
            const uint16_t *o = p.O + b * p.so[0] + h * p.so[1] + static_cast<int64_t>(i) * p.so[2];
            const uint16_t *g = p.dO + b * p.sdo[0] + h * p.sdo[1] + static_cast<int64_t>(i) * p.sdo[2];
#pragma unroll
            for (int c = 0; c < WN; ++c) {
                wo[k][c] = __ldg(reinterpret_cast<const uint4 *>(o + 64 * c + 8 * sub));
                wg[k][c] = __ldg(reinterpret_cast<const uint4 *>(g + 64 * c + 8 * sub));
            }
            if (sub == 0)
                l[k] = p.lse[static_cast<int64_t>(bh) * p.mask.Sq + i];
        } else {
#pragma unroll
            for (int c = 0; c < WN; ++c)
                wo[k][c] = wg[k][c] = make_uint4(0, 0, 0, 0);
        }
    }
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
#pragma unroll
    for (int k = 0; k < RN; ++k) {
        float sum = 0.0f, norm = 0.0f;
#pragma unroll
        for (int c = 0; c < WN; ++c) {
            const uint32_t ao[4] = {wo[k][c].x, wo[k][c].y, wo[k][c].z, wo[k][c].w};
            const uint32_t ag[4] = {wg[k][c].x, wg[k][c].y, wg[k][c].z, wg[k][c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float g0 = to_float<DT>(static_cast<uint16_t>(ag[e] & 0xFFFFu));
                const float g1 = to_float<DT>(static_cast<uint16_t>(ag[e] >> 16));
                sum = fmaf(g0, to_float<DT>(static_cast<uint16_t>(ao[e] & 0xFFFFu)), sum);
                sum = fmaf(g1, to_float<DT>(static_cast<uint16_t>(ao[e] >> 16)), sum);
                if constexpr (DT == 0)
                    norm = fmaf(g0, g0, fmaf(g1, g1, norm));
            }
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if constexpr (DT == 0)
                norm += __shfl_xor_sync(0xffffffffu, norm, off);
        }
        if (sub == 0) {
            if (DT == 0 && l[k] != -INFINITY && norm < INFINITY)  // queries that see nothing have no part in it
                top = fmaxf(top, norm);
            float *rows = p.rows + (static_cast<int64_t>(bh) * p.nqb + qb) * 2 * kBwdCols + (threadIdx.x >> 3) + 32 * k;
            rows[0] = l[k] == -INFINITY ? -INFINITY : kPShift<DT> - l[k] * 1.4426950408889634f;
            rows[kBwdCols] = l[k] == -INFINITY ? 0.0f : -sum;
        }
    }
    if constexpr (DT == 0)
        raise_norm(p.norms, top);
}

template <int D_>
struct AttnBwdConfig {
    static constexpr int D = D_;
    static constexpr int BM = 128, BN = kBwdCols;
    static constexpr int D_ATOMS = D / 64;
    static constexpr int XATOM = BM * 128, YATOM = BN * 128;  // bytes of 64 columns
    static constexpr int X_BYTES = D_ATOMS * XATOM, Y_BYTES = D_ATOMS * YATOM;
    static constexpr int ROWS_BYTES = 2 * BN * 4, INTERVAL_BYTES = 3 * BN * 4;  // of a block of queries
    static constexpr int STAGES = 4;
    static constexpr int STAGE_BYTES = 2 * Y_BYTES + 2048;  // Y1, Y2, rows, intervals
    static constexpr int OFF_X = 0;
    static constexpr int OFF_Y = 2 * X_BYTES;
    static constexpr int OFF_BAR = OFF_Y + STAGES * STAGE_BYTES;
    static constexpr int BAR_XF = 0, BAR_XE = 1, BAR_YF = 2, BAR_YE = 2 + STAGES;
    static constexpr int BAR_SF = 2 + 2 * STAGES;  // [set]: S in Tensor Memory
    static constexpr int BAR_DPF = BAR_SF + 2;     // [set]: dP in Tensor Memory
    static constexpr int BAR_PF = BAR_DPF + 2;     // [set]: P in Tensor Memory (8 warps arrive)
    static constexpr int BAR_DXF = BAR_PF + 2;     // [set]: dX in Tensor Memory (8 warps)
    static constexpr int BAR_PE = BAR_DXF + 2;     // [set]: P has been read
    static constexpr int BAR_DXE = BAR_PE + 2;     // [set]: dX has been read
    static constexpr int BAR_ACCF = BAR_DXE + 2;   // a tile's sums are complete
    static constexpr int BAR_ACCE = BAR_ACCF + 1;  // and have been read (16 warps)
    static constexpr int BAR_EPS = BAR_ACCE + 1;   // dQ: the warpgroups' parts of e are in shared memory (16 warps)
    static constexpr int BAR_TF = BAR_EPS + 1;     // [slot]: a tile's description is in shared memory
    static constexpr int BAR_TE = BAR_TF + 2;      // [slot]: and has been read (19: three MMA issuers, 16 warps)
    static constexpr int BAR_DRAIN = BAR_TE + 2;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + (NUM_BARS * 8 + 15) / 16 * 16;  // TMEM address, abort flag
    // [slot] x0, batch entry * heads + head, first block, blocks of a head; then the piece: its first block, its
    // blocks, where its sums go (-1: to the result)
    static constexpr int OFF_TILES = OFF_MISC + 16;
    static constexpr int OFF_EPS = OFF_TILES + 64;   // [tile & 1][warpgroup][128] floats
    static constexpr int OFF_OUT = (OFF_EPS + 4096 + 127) / 128 * 128;  // [warp] 32 rows x 16 columns on their way out
    static constexpr int SMEM_BYTES = OFF_OUT + 16 * 1024 + 1024;
    static constexpr int THREADS = 640;  // 4 control warps, 4 warpgroups for P and dX
    static constexpr int REGS_CONTROL = 64, REGS_SOFTMAX = 104;
    static constexpr int LAUNCH_REGS = (128 * REGS_CONTROL + 512 * REGS_SOFTMAX + THREADS - 1) / THREADS;
    // Tensor Memory columns: S and dP of set w at 64 w beyond these, the sums
    static constexpr int TMEM_S = 0, TMEM_DP = 128, TMEM_A0 = 256, TMEM_A1 = 256 + D;
    static_assert(TMEM_A1 + D <= 512, "Tensor Memory columns");
    static_assert(ROWS_BYTES + INTERVAL_BYTES <= 2048 && SMEM_BYTES <= 232448, "shared memory");
};

// X1, X2: the CTA's 128 rows (K and V, or Q and dO); Y1, Y2: the blocks it runs
// over (Q and dO, or K and V); out0, out1: dK and dV, or dQ twice
template <class CF, int DT, bool DKV, bool CAP, bool BIAS>
__global__ void __launch_bounds__(640, 1)
    attention_bwd_kernel(const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                         const __grid_constant__ CUtensorMap map_y1, const __grid_constant__ CUtensorMap map_y2,
                         const __grid_constant__ CUtensorMap map_out0, const __grid_constant__ CUtensorMap map_out1,
                         const AttnBwdParams p)
{
    constexpr int D = CF::D, STAGES = CF::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);  // uniform for the compiler too
    const int lane = threadIdx.x & 31;
    const int heads = DKV ? p.Hk : p.H;
    const int BH = p.B * heads;
    const int items = p.tiles * BH * p.splits;

    const uint32_t sX = smem_addr(smem + CF::OFF_X);
    const uint32_t sY = smem_addr(smem + CF::OFF_Y);
    const uint32_t bar0 = smem_addr(smem + CF::OFF_BAR);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + CF::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int4 *tile_slots = reinterpret_cast<int4 *>(smem + CF::OFF_TILES);
    float *eps_smem = reinterpret_cast<float *>(smem + CF::OFF_EPS);

    if (threadIdx.x == 0) {
        mbar_init(bar(CF::BAR_XF), 1);
        mbar_init(bar(CF::BAR_XE), 2);  // S and dP of a tile complete
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(CF::BAR_YF + s), 1);
            mbar_init(bar(CF::BAR_YE + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_SF + i), 1);
            mbar_init(bar(CF::BAR_DPF + i), 1);
            mbar_init(bar(CF::BAR_PF + i), 8);
            mbar_init(bar(CF::BAR_DXF + i), 8);
            mbar_init(bar(CF::BAR_PE + i), 1);
            mbar_init(bar(CF::BAR_DXE + i), 1);
        }
        mbar_init(bar(CF::BAR_ACCF), 1);
        mbar_init(bar(CF::BAR_ACCE), 16);
        mbar_init(bar(CF::BAR_EPS), 16);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_TF + i), 1);
            mbar_init(bar(CF::BAR_TE + i), 19);
        }
        mbar_init(bar(CF::BAR_DRAIN), 3);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_x1);
        tma_prefetch_map(&map_x2);
        tma_prefetch_map(&map_y1);
        tma_prefetch_map(&map_y2);
        tma_prefetch_map(&map_out0);
        tma_prefetch_map(&map_out1);
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

    // The tiles this CTA takes, one after another: every role reads the same
    // descriptions, two of them ahead at most.
    auto take_tile = [&](int t, int4 *out, int4 *piece) {
        const bool w = __all_sync(0xffffffffu, wait_bounded(bar(CF::BAR_TF + (t & 1)), static_cast<uint32_t>(t >> 1) & 1u,
                                                            abort_flag, timeout, ERR_EPILOGUE));
        if (!w)
            return false;
        *out = tile_slots[2 * (t & 1)];
        *piece = tile_slots[2 * (t & 1) + 1];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(CF::BAR_TE + (t & 1)));
        return out->x >= 0;
    };

    uint32_t issued = 0, parity = 0;  // bit 0: X, bits 8..: stages
    if (warp < 4) {
        regs_decrease<CF::REGS_CONTROL>();
        if (warp == 0) {
            // ------------------------------------------------------------ tiles and loads
            // Takes tile t from the counter, works out which blocks it visits and
            // leaves its description for the others.
            auto next_tile = [&](int t, int4 *out, int4 *piece) {
                if (t >= 2 && !__all_sync(0xffffffffu, wait_bounded(bar(CF::BAR_TE + (t & 1)),
                                                                    static_cast<uint32_t>((t >> 1) - 1) & 1u, abort_flag,
                                                                    timeout, ERR_PRODUCER)))
                    return false;
                int4 tl, pc;
                do {
                    int item = 0;
                    if (lane == 0)
                        item = atomicAdd(p.next, 1);
                    item = __shfl_sync(0xffffffffu, item, 0);
                    tl = make_int4(-1, 0, 0, 0);
                    pc = make_int4(0, 0, -1, 0);
                    if (item >= items)
                        break;
                    const int i = item / p.splits, s = item - i * p.splits;
                    const int2 at = bwd_tile<DKV>(i, p.tiles, BH, p.mask.causal);
                    const int tile = at.x, bh = at.y;
                    const int b = bh / heads, x0 = tile * CF::BM;
                    const int4 *rg = p.ranges + static_cast<int64_t>(b) * p.nqb;
                    int first = 0x7FFFFFFF, end = 0;
                    if constexpr (DKV) {
                        // the blocks of queries that see some key of the tile
                        for (int q = lane; q < p.nqb; q += 32) {
                            const int4 v = __ldg(rg + q);
                            if (v.x < x0 + CF::BM && v.y > x0) {
                                first = min(first, q);
                                end = max(end, q + 1);
                            }
                        }
                        first = __reduce_min_sync(0xffffffffu, first);
                        end = __reduce_max_sync(0xffffffffu, end);
                    } else {
                        // the blocks of keys that some query of the tile sees
                        for (int q = tile * (CF::BM / CF::BN); q < min(p.nqb, (tile + 1) * (CF::BM / CF::BN)); ++q) {
                            const int4 v = __ldg(rg + q);
                            first = min(first, v.x / CF::BN);
                            end = max(end, (v.y + CF::BN - 1) / CF::BN);
                        }
                    }
                    // a piece of the blocks, those of the heads that share the keys one after another; a tile
                    // without blocks is one empty piece
                    const int blocks = end > first ? end - first : 0, all = DKV ? blocks * p.group : blocks;
                    const int n0 = s * p.chunk;
                    if (n0 >= all && s > 0)
                        continue;  // (tl.x is -1: the next one)
                    tl = make_int4(x0, bh, first, blocks);
                    pc = make_int4(n0, min(p.chunk, all - n0), all > p.chunk ? item : -1, 0);
                    if (p.pieces && s == 0 && lane == 0)
                        p.pieces[i] = (all + p.chunk - 1) / p.chunk;
                    // checked build: heads, tiles, blocks and the place of partial sums
                    const int limit = DKV ? p.nqb : (p.mask.Sk + CF::BN - 1) / CF::BN;
                    if (!check_ok(tile >= 0 && tile < p.tiles && bh < BH && (blocks == 0 || (first >= 0 && end <= limit)) &&
                                  pc.y >= 0 && n0 + pc.y <= all && s < p.splits && all <= static_cast<int64_t>(p.splits) * p.chunk)) {
                        tl = make_int4(-1, 0, 0, 0);
                        break;
                    }
                    if (!DKV) {
                        tl.z += n0;
                        tl.w = pc.y;
                        pc.x = 0;
                    }
                } while (tl.x < 0);
                if (lane == 0) {
                    tile_slots[2 * (t & 1)] = tl;
                    tile_slots[2 * (t & 1) + 1] = pc;
                    mbar_arrive(bar(CF::BAR_TF + (t & 1)));
                }
                __syncwarp();
                *out = tl;
                *piece = pc;
                return true;
            };
            int st = 0;
            uint32_t ph = 0, xph = 0;
            int4 tl, pc;
            bool ok = next_tile(0, &tl, &pc);
            // The next tile is taken when this one's last loads are out: taken at its start, tiles would be dealt out
            // regardless of who finishes first.
            for (int t = 0; ok && tl.x >= 0; ok = ok && next_tile(t + 1, &tl, &pc), ++t) {
                if (pc.y == 0)
                    continue;
                const int b = tl.y / heads, head = tl.y - b * heads;
                if (lane == 0) {
                    ok = wait_bounded(bar(CF::BAR_XE), xph ^ 1u, abort_flag, timeout, ERR_PRODUCER);
                    if (ok) {
                        mbar_arrive_expect_tx(bar(CF::BAR_XF), 2 * CF::X_BYTES);
#pragma unroll
                        for (int a = 0; a < CF::D_ATOMS; ++a) {
                            tma_load_4d(sX + a * CF::XATOM, &map_x1, bar(CF::BAR_XF), 64 * a, tl.x, head, b);
                            tma_load_4d(sX + CF::X_BYTES + a * CF::XATOM, &map_x2, bar(CF::BAR_XF), 64 * a, tl.x, head, b);
                        }
                        issued |= 1u;
                        parity = (parity & ~1u) | xph;
                    }
                    // DKV: over the heads that share the keys, one after another
                    int yb = DKV ? tl.z + pc.x % tl.w : tl.z;
                    int yh = DKV ? head * p.group + pc.x / tl.w : head / p.group;
                    const int n_total = pc.y;
                    for (int n = 0; ok && n < n_total; ++n) {
                        if (!(ok = wait_bounded(bar(CF::BAR_YE + st), ph ^ 1u, abort_flag, timeout, ERR_PRODUCER)))
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
                        issued |= 256u << st;
                        parity = (parity & ~(256u << st)) | (ph << (8 + st));
                        if (++yb == tl.z + tl.w) {
                            yb = tl.z;
                            ++yh;
                        }
                        if (++st == STAGES) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                }
                xph ^= 1u;
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            }
        } else {
            // ------------------------------------------------------------ MMA issuers
            // Warp 1 issues S, warp 2 dP, warp 3 dV and dK: one's waits (some 150
            // clocks each even on a completed barrier) pass while the others'
            // products run (one issuer for all: 2350 clocks a block; two: 1750).
            // What one needs of another comes through the barriers.  A whole warp
            // walks the loop and one elected lane issues: what the instructions
            // are made from stays uniform across the warp.
            constexpr uint32_t IDESC_1 = mma_idesc_f16(DT, 128, CF::BN, 0, 0);  // both K-major
            constexpr uint32_t IDESC_2 = mma_idesc_f16(DT, 128, D, 0, 1);       // A from Tensor Memory, Y N-major
            const uint64_t x_desc = smem_desc_sw128(sX, 16, 1024);
            const uint64_t y_desc = smem_desc_sw128(sY, 16, 1024);
            const uint64_t yt_desc = smem_desc_sw128(sY, CF::YATOM, 1024);
            // S (m = 0) or dP (m = 1) of the block in stage `st` into set `set`, from X1, Y1 or X2, Y2
            auto first_product = [&](int m, int st, int set) {
                if (elect_one()) {
                    const uint64_t yd = y_desc + ((st * CF::STAGE_BYTES + m * CF::Y_BYTES) >> 4);
                    const uint64_t xd = x_desc + ((m * CF::X_BYTES) >> 4);
                    const uint32_t d = tmem_base + static_cast<uint32_t>((m ? CF::TMEM_DP : CF::TMEM_S) + CF::BN * set);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma_f16(d, xd + (((k >> 2) * CF::XATOM + (k & 3) * 32) >> 4),
                                   yd + (((k >> 2) * CF::YATOM + (k & 3) * 32) >> 4), IDESC_1, k != 0 ? 1u : 0u);
                    tc_commit(bar((m ? CF::BAR_DPF : CF::BAR_SF) + set));
                }
                __syncwarp();
            };
            // 16 values of P or dX take 8 columns; each 32 of the block's lie where their scores were
            auto p_col = [](int k) { return (k >> 1) * 32 + (k & 1) * 8; };
            // dV += P^T dO, or B += P c K (m = 0); dK += dX^T Q, or dQ += dX K (m = 1)
            auto second_product = [&](int m, int st, int set, bool first) {
                if (elect_one()) {
                    const uint64_t yd = yt_desc + ((st * CF::STAGE_BYTES + (DKV && m == 0 ? CF::Y_BYTES : 0)) >> 4);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(m ? CF::TMEM_A1 : CF::TMEM_A0);
                    const uint32_t a = tmem_base + static_cast<uint32_t>((m ? CF::TMEM_DP : CF::TMEM_S) + CF::BN * set);
#pragma unroll
                    for (int k = 0; k < CF::BN / 16; ++k)
                        tc_mma_f16_ts(d, a + p_col(k), yd + ((2048 * k) >> 4), IDESC_2, (!first || k > 0) ? 1u : 0u);
                    tc_commit(bar((m ? CF::BAR_DXE : CF::BAR_PE) + set));
                    if (m)
                        tc_commit(bar(CF::BAR_YE + st));
                }
                __syncwarp();
            };
            auto wait = [&](int id, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_MMA_DATA)) != 0;
            };
            auto commit = [&](int id) {
                if (elect_one())
                    tc_commit(bar(id));
                __syncwarp();
            };
            uint32_t g = 0, busy = 0;  // blocks and tiles with blocks so far
            int4 tl, pc;
            bool ok = true;
            // Every wait follows each phase of its barrier in turn, so no two phases
            // can be mistaken.
            for (int t = 0; ok && take_tile(t, &tl, &pc); ++t) {
                const int n_total = pc.y;
                if (n_total == 0)
                    continue;
                if (warp < 3) {
                    // S takes the columns that dV has read P of two blocks before from, dP those of dX
                    const int m = warp - 1, free_bar = m ? CF::BAR_DXE : CF::BAR_PE;
                    ok = wait(CF::BAR_XF, busy);
                    for (int n = 0; ok && n < n_total; ++n, ++g) {
                        const int st = static_cast<int>(g % STAGES), set = static_cast<int>(g & 1u);
                        if (!(ok = wait(CF::BAR_YF + st, g / STAGES)) ||
                            (g >= 2 && !(ok = wait(free_bar + set, (g >> 1) - 1))))
                            break;
                        tc_fence_after_sync();
                        first_product(m, st, set);
                    }
                    if (ok)
                        commit(CF::BAR_XE);
                } else {
                    for (int n = 0; ok && n < n_total; ++n, ++g) {
                        const int st = static_cast<int>(g % STAGES), set = static_cast<int>(g & 1u);
                        // the last tile's sums have been read before this one's begin
                        if (!(ok = wait(CF::BAR_PF + set, g >> 1)) ||
                            (n == 0 && busy > 0 && !(ok = wait(CF::BAR_ACCE, busy - 1))))
                            break;
                        tc_fence_after_sync();
                        second_product(0, st, set, n == 0);
                        if (!(ok = wait(CF::BAR_DXF + set, g >> 1)))
                            break;
                        tc_fence_after_sync();
                        second_product(1, st, set, n == 0);
                    }
                    if (ok)
                        commit(CF::BAR_ACCF);
                }
                ++busy;
            }
            commit(CF::BAR_DRAIN);
            wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
        }
        __syncwarp();
    } else {
        regs_increase<CF::REGS_SOFTMAX>();
        // ------------------------------------------------------------ P and dX: one row and 32 columns a thread
        constexpr int HN = 32;
        const int group = (warp - 4) >> 2;         // warpgroup: its team (and set) and which 32 of the 64 columns
        const int team = group & 1, half = group >> 1;
        const int r = (warp & 3) * 32 + lane;      // row of the tile (Tensor Memory lane)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_S + CF::BN * team + HN * half);
        const uint32_t dp_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_DP + CF::BN * team + HN * half);
        auto wait_warp = [&](int id, uint32_t par) -> bool {
            return __all_sync(0xffffffffu, wait_bounded(bar(id), par & 1u, abort_flag, timeout, ERR_EPILOGUE));
        };
        auto arrive = [&](int id) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(id));
        };
        // fp16: dX times x_mul over P's factor; x_undo takes dX's factor out again
        float x_mul = 1.0f, x_undo = 1.0f;
        if constexpr (DT == 0) {
            // the least e with 4 |dO|^2 |V|^2 < 2^(2 e), so that |dX| < 2^e; 0 where one of them is 0.  The norms of
            // finite fp16 rows keep e between -47 and 42.
            const unsigned bits = __float_as_uint(4.0f * __ldg(p.norms) * __ldg(p.norms + 1));
            const int e = bits == 0 ? 0 : (static_cast<int>(bits >> 23) - 126 + 1) >> 1;
            auto power = [](int n) { return __uint_as_float(static_cast<unsigned>(n + 127) << 23); };
            x_mul = power(15 - e - static_cast<int>(kPShift<DT>));
            x_undo = power(e - 15);
        }
        constexpr float p_undo = DT == 0 ? 1.0f / 1024.0f : 1.0f;
        uint4 *out_buf = reinterpret_cast<uint4 *>(smem + CF::OFF_OUT + (warp - 4) * 1024);
        uint32_t g0 = 0, busy = 0;  // blocks and tiles with blocks so far
        int4 tl, pc;
        bool ok = true;
        for (int t = 0; ok && take_tile(t, &tl, &pc); ++t) {
            const int b = tl.y / heads, head = tl.y - b * heads, x0 = tl.x;
            const int row = x0 + r;
            const int n_total = pc.y;
            int2 seen = make_int2(0, 0);                   // dQ: the row's interval
            float row_nlse = -INFINITY, row_ndelta = 0.0f;
            float2 eps = splat2(0.0f);                     // dQ: this thread's part of e (times P's factor)
            float *row_stats = nullptr;
            if constexpr (!DKV) {
                if (row < p.mask.Sq) {
                    const int64_t block = row / CF::BN;
                    const int32_t *iv = p.intervals + (static_cast<int64_t>(b) * p.nqb + block) * 3 * CF::BN + row % CF::BN;
                    seen = make_int2(iv[0], iv[CF::BN]);
                    row_stats = p.rows + ((static_cast<int64_t>(b) * p.H + head) * p.nqb + block) * 2 * CF::BN + row % CF::BN;
                    row_nlse = row_stats[0];
                    row_ndelta = row_stats[CF::BN];
                }
            }
            float slope2 = 0.0f;
            if constexpr (BIAS && !DKV)
                slope2 = __ldg(p.score.slopes + head) * 1.4426950408889634f;
            // this team's blocks; where they lie, and DKV: in which head
            const int n_first = static_cast<int>((static_cast<uint32_t>(team) - g0) & 1u);
            int yb = tl.z + (DKV ? pc.x : 0) + n_first, yh = head * p.group;
            auto carry = [&]() {
                while (yb >= tl.z + tl.w) {
                    yb -= tl.w;
                    ++yh;
                }
            };
            for (int n = n_first; n < n_total; n += 2, yb += 2) {
                if constexpr (DKV)
                    carry();
                const uint32_t g = g0 + static_cast<uint32_t>(n);
                const int st = static_cast<int>(g % STAGES);
                int4 rg = make_int4(0, 0, 0, 0);
                if constexpr (DKV) {
                    rg = __ldg(p.ranges + static_cast<int64_t>(b) * p.nqb + yb);
                    if constexpr (BIAS)
                        slope2 = __ldg(p.score.slopes + yh) * 1.4426950408889634f;
                    // what lies beside the stage's tiles is seen through the copy's own barrier
                    if (!(ok = wait_warp(CF::BAR_YF + st, g / STAGES)))
                        break;
                }
                if (!(ok = wait_warp(CF::BAR_SF + team, g >> 1)))
                    break;
                tc_fence_after_sync();
                uint32_t sv[HN];
                tmem_load_32cols(s_addr, sv);
                // DKV: -lse, -delta, first key, end key and "sees more than one key" of the block's queries
                const float4 *info = reinterpret_cast<const float4 *>(smem + CF::OFF_Y + st * CF::STAGE_BYTES +
                                                                      2 * CF::Y_BYTES) + half * (HN / 4);
                const int4 *iv = reinterpret_cast<const int4 *>(info + 2 * CF::BN / 4);
                const float4 *many = info + 4 * CF::BN / 4;
                const int y0 = yb * CF::BN + HN * half;  // the thread's first column
                // |p_i - j|: the column's step away from the first column's distance
                const float dist0 = DKV ? static_cast<float>(p.mask.q_offset + y0 - row)
                                        : static_cast<float>(p.mask.q_offset + row - y0);
                const int nlo = seen.x - y0, nhi = seen.y - y0;  // dQ
                bool whole = DKV ? rg.z <= x0 && rg.w >= x0 + CF::BM : nlo <= 0 && nhi >= HN;
                whole = __all_sync(0xffffffffu, whole);
                tmem_load_wait();
                float2 w[HN / 2];        // P
                float2 c[CAP ? HN / 2 : 1];  // 1 - tanh^2
                // scores to P; only blocks that cut an interval are masked
                auto weights = [&](auto masked) {
                    constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
                    for (int e = 0; e < HN; e += 4) {
                        float4 l4 = make_float4(row_nlse, row_nlse, row_nlse, row_nlse);
                        int4 lo4 = make_int4(0, 0, 0, 0), hi4 = lo4;
                        if constexpr (DKV) {
                            l4 = info[e / 4];
                            if constexpr (MASKED) {
                                lo4 = iv[e / 4];
                                hi4 = iv[CF::BN / 4 + e / 4];
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 4; h += 2) {
                            const int i = e + h;
                            const float2 s = make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
                            const float2 nl = h ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                            float2 x;
                            if constexpr (CAP) {
                                x = ffma2(s, splat2(p.score.cap_log2), nl);
                                c[i / 2] = ffma2(make_float2(-s.x, -s.y), s, splat2(1.0f));
                            } else {
                                x = ffma2(s, splat2(p.score.scale_log2), nl);
                            }
                            if constexpr (BIAS) {
                                const float f = static_cast<float>(i);
                                const float2 dist = DKV ? fadd2(splat2(dist0), make_float2(f, f + 1.0f))
                                                        : fadd2(splat2(dist0), make_float2(-f, -f - 1.0f));
                                x = ffma2(make_float2(fabsf(dist.x), fabsf(dist.y)), splat2(-slope2), x);
                            }
                            float2 v = make_float2(exp2_approx_ftz(x.x), exp2_approx_ftz(x.y));
                            if constexpr (MASKED && DKV) {
                                v.x = row >= (h ? lo4.z : lo4.x) && row < (h ? hi4.z : hi4.x) ? v.x : 0.0f;
                                v.y = row >= (h ? lo4.w : lo4.y) && row < (h ? hi4.w : hi4.y) ? v.y : 0.0f;
                            } else if constexpr (MASKED) {
                                v.x = i >= nlo && i < nhi ? v.x : 0.0f;
                                v.y = i + 1 >= nlo && i + 1 < nhi ? v.y : 0.0f;
                            }
                            w[i / 2] = v;
                            if constexpr (CAP && !DKV)
                                v = fmul2(v, c[i / 2]);
                            sv[i / 2] = pack2<DT>(v.x, v.y);
                        }
                    }
                };
                if constexpr (CAP)
                    tanh_scores<HN>(sv, p.score.cap_arg);
                if (whole)
                    weights(std::false_type{});
                else
                    weights(std::true_type{});
                // over the first half of the columns this thread read itself (others may still read theirs)
                tmem_store_16cols(s_addr, sv);
                tmem_store_wait();
                arrive(CF::BAR_PF + team);
                if (!(ok = wait_warp(CF::BAR_DPF + team, g >> 1)))
                    break;
                tc_fence_after_sync();
                // dP to dX, 16 columns at a time
                uint32_t dx[HN / 2];
                auto gradients = [&](auto masked) {
                    constexpr bool MASKED = decltype(masked)::value;
#pragma unroll
                    for (int e0 = 0; e0 < HN; e0 += 16) {
                        uint32_t dp[16];
                        tmem_load_16cols(dp_addr + e0, dp);
                        tmem_load_wait();
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            float4 d4 = make_float4(row_ndelta, row_ndelta, row_ndelta, row_ndelta);
                            float4 m4 = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                            if constexpr (DKV) {
                                d4 = info[(CF::BN + e0 + e) / 4];
                                if constexpr (MASKED)
                                    m4 = many[(e0 + e) / 4];
                            }
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                const int i = e0 + e + h;
                                const float2 nd = h ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                                float2 v = fadd2(make_float2(__uint_as_float(dp[e + h]), __uint_as_float(dp[e + h + 1])), nd);
                                if constexpr (MASKED && DKV)  // a query that sees one key gets dX = 0 exactly
                                    v = fmul2(v, h ? make_float2(m4.z, m4.w) : make_float2(m4.x, m4.y));
                                v = fmul2(v, w[i / 2]);
                                if constexpr (!DKV)
                                    eps = fadd2(eps, v);
                                if constexpr (CAP)
                                    v = fmul2(v, c[i / 2]);
                                if constexpr (DT == 0)
                                    v = fmul2(v, splat2(x_mul));
                                dx[i / 2] = pack2<DT>(v.x, v.y);
                            }
                        }
                    }
                };
                if (!DKV || whole)
                    gradients(std::false_type{});
                else
                    gradients(std::true_type{});
                tmem_store_16cols(dp_addr, dx);
                tmem_store_wait();
                arrive(CF::BAR_DXF + team);
            }
            g0 += static_cast<uint32_t>(n_total);
            // all products of the tile complete, then the sums out
            if (ok && n_total > 0)
                ok = wait_warp(CF::BAR_ACCF, busy);
            float e_row = 0.0f;  // dQ: the row's e
            if constexpr (!DKV) {
                if (ok) {
                    float *parts = eps_smem + (t & 1) * 512;
                    parts[group * 128 + r] = eps.x + eps.y;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(CF::BAR_EPS));
                    ok = wait_warp(CF::BAR_EPS, static_cast<uint32_t>(t));
                    e_row = ((parts[r] + parts[128 + r]) + (parts[256 + r] + parts[384 + r])) * p_undo;
                }
            }
            if (!ok)
                break;
            tc_fence_after_sync();
            // DKV: two warpgroups write dK, two dV, half the columns each; dQ: a quarter each
            const bool second = DKV && (group & 1);
            const CUtensorMap *map_out = second ? &map_out1 : &map_out0;
            const float mul = second ? p_undo : p.scale * x_undo;
            const uint32_t acc0 = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_A0);
            const uint32_t acc = second ? acc0 : tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_A1);
            const float e_mul = -e_row * p.scale * p_undo;
            const bool none = n_total == 0 || (!DKV && seen.y - seen.x <= 1);  // nothing comes through
            if constexpr (!DKV) {
                if (group == 0) {
                    if (pc.z >= 0)
                        p.part_e[static_cast<int64_t>(pc.z) * 128 + r] = e_row;
                    else if (row_stats)
                        row_stats[CF::BN] = row_ndelta - e_row;
                }
            }
            const int c0 = DKV ? (group >> 1) * (D / 32) : group * (D / 64), c1 = c0 + (DKV ? D / 32 : D / 64);  // of 16 columns
            if (pc.z >= 0) {
                // one of several pieces: its sums as they are; dQ's B beside them
                float4 *part = p.part + static_cast<int64_t>(pc.z) * (2 * D / 4) * 128 + r;
#pragma unroll 1
                for (int k = DKV ? c0 : 2 * c0; k < (DKV ? c1 : 2 * c1); ++k) {
                    const int m = DKV ? (second ? 1 : 0) : k & 1, col = 16 * (DKV ? k : k >> 1);
                    uint32_t o[16];
                    tmem_load_16cols((DKV || m == 0 ? acc : acc0) + col, o);
                    tmem_load_wait();
                    const float by = DKV || m == 0 ? mul : p.scale * p_undo;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        part[(m * (D / 4) + col / 4 + v) * 128] =
                            make_float4(__uint_as_float(o[4 * v]) * by, __uint_as_float(o[4 * v + 1]) * by,
                                        __uint_as_float(o[4 * v + 2]) * by, __uint_as_float(o[4 * v + 3]) * by);
                }
                arrive(CF::BAR_ACCE);
                ++busy;
                continue;
            }
#pragma unroll 1
            for (int cc = c0; cc < c1; ++cc) {
                uint32_t o[16];
                if (n_total > 0) {
                    tmem_load_16cols(acc + 16 * cc, o);
                    if constexpr (!DKV) {
                        uint32_t o0[16];
                        tmem_load_16cols(acc0 + 16 * cc, o0);
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
                if (cc + 1 == c1 && n_total > 0)
                    arrive(CF::BAR_ACCE);  // in registers: the next tile's sums may begin
                if (none) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = 0;
                }
                // 32 rows x 16 columns through this warp's buffer; rows behind the tensor's are not written
                const int row0 = x0 + (warp & 3) * 32;
                if (row0 >= (DKV ? p.mask.Sk : p.mask.Sq))
                    continue;
                if (lane == 0)
                    bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint4 x;
                    x.x = pack2<DT>(__uint_as_float(o[8 * v]), __uint_as_float(o[8 * v + 1]));
                    x.y = pack2<DT>(__uint_as_float(o[8 * v + 2]), __uint_as_float(o[8 * v + 3]));
                    x.z = pack2<DT>(__uint_as_float(o[8 * v + 4]), __uint_as_float(o[8 * v + 5]));
                    x.w = pack2<DT>(__uint_as_float(o[8 * v + 6]), __uint_as_float(o[8 * v + 7]));
                    out_buf[2 * lane + v] = x;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_4d(map_out, smem_addr(out_buf), 16 * cc, row0, head, b);
                    bulk_commit_group();
                }
            }
            if (n_total > 0)
                ++busy;
        }
        if (lane == 0)
            bulk_wait_group<0>();
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        if (issued & 1u)
            wait_drain(bar(CF::BAR_XF), parity & 1u, timeout);
        for (int s = 0; s < STAGES; ++s)
            if (issued & (256u << s))
                wait_drain(bar(CF::BAR_YF + s), (parity >> (8 + s)) & 1u, timeout);
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

// Adds the pieces of each tile that has several, in their order: a row a lane,
// D / 8 columns a warp, a CTA for 32 rows.
template <int DT, int D, bool DKV>
__global__ void __launch_bounds__(256) attention_bwd_join_kernel(const AttnBwdJoinParams p)
{
    constexpr int C4 = D / 32;  // groups of four columns a warp
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = static_cast<int>(blockIdx.x >> 2);
    const int pieces = p.pieces[item];
    if (pieces <= 1 || !check_ok(pieces <= p.splits && item < p.tiles * p.BH))
        return;
    const int2 at = bwd_tile<DKV>(item, p.tiles, p.BH, p.mask.causal);
    const int r = 32 * static_cast<int>(blockIdx.x & 3) + lane, row = at.x * 128 + r;
    if (row >= (DKV ? p.mask.Sk : p.mask.Sq))
        return;
    const int b = at.y / p.heads, h = at.y - b * p.heads;
    const int64_t slot0 = static_cast<int64_t>(item) * p.splits;
    float4 sum[2][C4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int v = 0; v < C4; ++v)
            sum[m][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float e = 0.0f;
    const float4 *part = p.part + (slot0 * (2 * D / 4) + warp * C4) * 128 + r;
#pragma unroll 2
    for (int s = 0; s < pieces; ++s) {
        if constexpr (!DKV)
            e += p.part_e[(slot0 + s) * 128 + r];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int v = 0; v < C4; ++v) {
                const float4 x = part[(static_cast<int64_t>(s) * (2 * D / 4) + m * (D / 4) + v) * 128];
                sum[m][v].x += x.x;
                sum[m][v].y += x.y;
                sum[m][v].z += x.z;
                sum[m][v].w += x.w;
            }
    }
    if constexpr (!DKV) {
        const int64_t block = row / kBwdCols;
        const int32_t *iv = p.intervals + (static_cast<int64_t>(b) * p.nqb + block) * 3 * kBwdCols + row % kBwdCols;
        const bool none = iv[kBwdCols] - iv[0] <= 1;
#pragma unroll
        for (int v = 0; v < C4; ++v) {
            float4 &x = sum[0][v];
            const float4 y = sum[1][v];
            x = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                     : make_float4(fmaf(-e, y.x, x.x), fmaf(-e, y.y, x.y), fmaf(-e, y.z, x.z), fmaf(-e, y.w, x.w));
        }
        if (warp == 0) {
            float *stats = p.rows + ((static_cast<int64_t>(b) * p.H + h) * p.nqb + block) * 2 * kBwdCols + row % kBwdCols;
            stats[kBwdCols] -= e;
        }
    }
#pragma unroll
    for (int m = 0; m < (DKV ? 2 : 1); ++m) {
        const int64_t *st = m ? p.s1 : p.s0;
        uint16_t *out = (m ? p.out1 : p.out0) + b * st[0] + h * st[1] + row * st[2] + warp * 4 * C4;
#pragma unroll
        for (int v = 0; v < C4; v += 2) {
            const float4 x = sum[m][v], y = sum[m][v + 1];
            reinterpret_cast<uint4 *>(out)[v / 2] =
                make_uint4(pack2<DT>(x.x, x.y), pack2<DT>(x.z, x.w), pack2<DT>(y.x, y.y), pack2<DT>(y.z, y.w));
        }
    }
}

} // namespace tl
