// tree_attention_kernel.cuh -- one or several drafted tokens of each request
// against its paged key/value cache.
//
// Request b has context_b keys in the cache and, behind them, those of its
// drafted tokens; token t sees every key of the context, itself and the tokens
// it hangs below (its ancestors in the draft's tree):
//
//     O_t = sum_j w_tj V_j,  w_tj = exp(y_tj - lse_t)   over the keys j that t sees
//
// with y as in attention_common.cuh; a context key lies at its index, a drafted
// token at context_b + its depth in the tree.
//
// Bound by reading the cache once (4 D bytes a key and key/value head).  All
// query heads that share a key/value head and all tokens become rows of one
// 128-row tile (token-major), so the cache is read once for all of them; the
// products are those of 128 rows whatever the number of rows is, which costs
// nothing while the reads bound: a 128-key block is 64 KB (D = 128), about
// 2800 clocks of one SM's share of the HBM, against about 512 for the products.
//
// Split over the keys: the blocks of all requests and heads are laid end to
// end and cut into equal runs, one for each CTA, from the lengths on the device
// (the host never reads them).  A run that holds all blocks of a tile writes
// the result; the others leave fp32 sums with their maximum, which
// tree_combine_kernel joins.  A CTA prefetches across the ends of its pieces.
//
// Measured, 32 requests of 8192 keys, 8 key/value heads of 128, bf16, pages of 64:
// 178 to 181 us, 6.0 TB/s (D = 64: 146 to 156 us, 3.4 to 3.7 TB/s: one warp holds
// the few rows, and its latency bounds; capped, D = 128: 229 to 240 us); pages of
// 16: 204 to 213 us, with four times the copies.  One request of 900 keys: 11 us,
// of which its block takes 2; the rest is two launches and the reads of length,
// table and page one after another.
//
// Shared memory goes to the K and V slots: a Q tile keeps only the rows it has
// (rounded up to 8).  The products still read 128 rows and find other tiles'
// bytes behind them, which only reaches Tensor Memory lanes that are never
// looked at.  With 16 rows that leaves three slots of each instead of two, and V,
// which waits for its block's weights, needs the third.
//
// Inside a CTA consecutive blocks alternate between two sets of Tensor Memory
// columns (scores and sums) and two softmax warpgroups, joined at the end of
// the piece, so that one block's exponentials overlap the next one's products.
//
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2..3 the tree's
// masks and zeros for V rows behind the last key (a page's unused rows may
// hold anything, and 0 times NaN is NaN), 4..7 and 8..11 softmax.
#pragma once

#include "attention_common.cuh"

namespace tl {

constexpr int kTreeMaxTokens = 64;
constexpr int kTreeMaxBatch = 4096;

struct TreeParams {
    ScoreParams score;
    int32_t B, H, Hk, group, T;
    int32_t tile_tokens, row_tiles;   // tokens a 128-row tile holds, tiles a request
    int32_t units;                    // Hk * row_tiles
    int32_t page_size, box_rows;      // box_rows: rows a TMA box loads, a divisor of page_size and of 128
    int32_t capacity;                 // keys a block table row covers
    int64_t table_row;                // block table's row stride in entries
    const int32_t *block_table, *context, *parents, *tree_lens;  // parents, tree_lens: may be null
    uint16_t *O;
    int64_t o_batch, o_head, o_row;
    float *lse;                       // [B][H][T], or null
    float *part_o;                    // [2 CTAs][D / 4][128][4]: a row a lane, so a warp's rows lie side by side
    float2 *part_ml;                  // [2 CTAs][128]: maximum (log2 units), sum
    int32_t slots;                    // K and V slots
    int32_t q_bytes;                  // of one Q tile: D / 64 atoms of its rows
    uint64_t timeout_ns;
};

// A request's lengths: drafted tokens, keys of the context and all keys
struct TreeRequest {
    int tokens, context, keys;
    __device__ __forceinline__ int blocks() const { return tokens > 0 ? (keys + 127) / 128 : 0; }
};

__device__ __forceinline__ TreeRequest tree_request(const TreeParams &p, int b)
{
    TreeRequest r;
    r.tokens = p.tree_lens ? min(max(p.tree_lens[b], 0), p.T) : p.T;
    r.context = min(max(p.context[b], 0), p.capacity);
    r.keys = min(r.context, p.capacity - r.tokens) + r.tokens;
    r.keys = max(min(r.keys, p.capacity), 0);
    return r;
}

// How many CTAs share `work` blocks
__device__ __forceinline__ int tree_ctas(int grid, int work) { return min(grid, work); }

template <int D_>
struct TreeConfig {
    static constexpr int D = D_;
    static constexpr int BN = 128;
    static constexpr int KS = D == 128 ? 3 : 6;              // most K and V slots
    static constexpr int ATOM_BYTES = 128 * 128;
    static constexpr int D_ATOMS = D / 64;
    static constexpr int TILE_BYTES = D_ATOMS * ATOM_BYTES;  // a K block, a V block
    static constexpr int BAR_QF = 0, BAR_QE = 2, BAR_KF = 4, BAR_KE = 4 + KS, BAR_VF = 4 + 2 * KS, BAR_VE = 4 + 3 * KS;
    static constexpr int BAR_SF = 4 + 4 * KS;     // [stream]: scores in Tensor Memory
    static constexpr int BAR_PF = BAR_SF + 2;     // [stream]: weights in Tensor Memory (4 warps arrive)
    static constexpr int BAR_DONE = BAR_PF + 2;   // [stream]: O += P V completed
    static constexpr int BAR_OE = BAR_DONE + 2;   // [piece & 1]: the piece's sums have been read (8 warps)
    static constexpr int BAR_TF = BAR_OE + 2;     // [piece & 1]: the tree's masks are there (2 warps)
    static constexpr int BAR_VZ = BAR_TF + 2;     // [V slot]: rows behind the last key are zero (2 warps)
    static constexpr int BAR_ZR = BAR_VZ + KS;    // a block with rows behind the last key has landed
    static constexpr int BAR_ML = BAR_ZR + 1;     // both streams of a piece are complete, their statistics in shared memory (8 warps)
    static constexpr int BAR_DRAIN = BAR_ML + 1;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static_assert(2 * TILE_BYTES >= ATOM_BYTES, "what is read behind a Q tile's rows lies in the K slots");
    // behind the Q tiles, the K slots and the V slots:
    static constexpr int OFF_MISC = (NUM_BARS * 8 + 15) / 16 * 16;        // TMEM address, abort flag
    static constexpr int OFF_ML = OFF_MISC + 16;                          // [piece & 1][stream][128] float2
    static constexpr int OFF_TREE = OFF_ML + 2 * 2 * 128 * 8;             // [piece & 1][64] masks
    // [piece & 1][320] floats: where the keys around the context's end lie, counted from it
    static constexpr int PLACES = 320, PLACE0 = 128;
    static constexpr int OFF_PLACE = OFF_TREE + 2 * kTreeMaxTokens * 8;
    static constexpr int OFF_PARENT = OFF_PLACE + 2 * PLACES * 4;         // [warp][64]
    static constexpr int OFF_CUM = OFF_PARENT + 2 * kTreeMaxTokens * 4;   // [batch]: blocks of the requests before
    static constexpr int SMEM_FIXED = OFF_CUM + 1024;                     // + 4 (batch + 1), Q tiles, slots
    static constexpr int THREADS = 384;
    static constexpr int TMEM_S = 0, TMEM_O = 256;
    static constexpr float RESCALE_LOG2 = 8.0f;
    static constexpr int SMEM_MAX = 232448;
    static_assert(SMEM_FIXED + 4 * (kTreeMaxBatch + 1) + 6 * TILE_BYTES <= SMEM_MAX, "two whole Q tiles and two slots each");
};

// A piece: consecutive blocks of one tile (request, key/value head, row tile)
struct TreePiece {
    int b, unit, first, len, blocks;  // blocks: the tile's
};

// The piece of the run [g, g1) that begins at block g of the laid-out work
__device__ __forceinline__ TreePiece tree_piece(const int32_t *cum, int B, int units, int g, int g1)
{
    int lo = 0, hi = B - 1;  // the last request that begins at or before g (empty ones begin where the next does)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] * units <= g)
            lo = mid;
        else
            hi = mid - 1;
    }
    TreePiece s;
    s.b = lo;
    s.blocks = cum[lo + 1] - cum[lo];
    const int o = g - cum[lo] * units;
    s.unit = o / s.blocks;
    s.first = o - s.unit * s.blocks;
    s.len = min(s.blocks - s.first, g1 - g);
    return s;
}

// The lengths of a piece's request.  They are read again here, so they are held to what the work was laid out
// from: lengths that are written while the call runs (a caller's missing wait between streams) give wrong
// results, but no access out of bounds.
__device__ __forceinline__ TreeRequest tree_request(const TreeParams &p, const TreePiece &s)
{
    TreeRequest r = tree_request(p, s.b);
    r.keys = min(max(r.keys, (s.blocks - 1) * 128 + 1), s.blocks * 128);
    r.context = min(max(r.context, r.keys - kTreeMaxTokens), r.keys);
    return r;
}

template <class CF, int DT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v, const TreeParams p)
{
    constexpr int D = CF::D;
    const int KS = p.slots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // Q tiles first: what the products read behind their rows are the K slots, never past the allocation
    const int off_k = 2 * p.q_bytes, off_v = off_k + KS * CF::TILE_BYTES;
    uint8_t *fixed = smem + off_v + KS * CF::TILE_BYTES;
    const uint32_t sQ = smem_addr(smem);
    const uint32_t sK = sQ + static_cast<uint32_t>(off_k);
    const uint32_t sV = sQ + static_cast<uint32_t>(off_v);
    const uint32_t bar0 = smem_addr(fixed);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fixed + CF::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float2 *ml = reinterpret_cast<float2 *>(fixed + CF::OFF_ML);
    uint64_t *tree_mask = reinterpret_cast<uint64_t *>(fixed + CF::OFF_TREE);
    float *tree_place = reinterpret_cast<float *>(fixed + CF::OFF_PLACE);
    int32_t *parent_smem = reinterpret_cast<int32_t *>(fixed + CF::OFF_PARENT);
    int32_t *cum = reinterpret_cast<int32_t *>(fixed + CF::OFF_CUM);

    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(CF::BAR_QF + i), 1);
            mbar_init(bar(CF::BAR_QE + i), 1);
            mbar_init(bar(CF::BAR_SF + i), 1);
            mbar_init(bar(CF::BAR_PF + i), 4);
            mbar_init(bar(CF::BAR_DONE + i), 1);
            mbar_init(bar(CF::BAR_OE + i), 8);
            mbar_init(bar(CF::BAR_TF + i), 2);
        }
        for (int s = 0; s < KS; ++s) {
            mbar_init(bar(CF::BAR_KF + s), 1);
            mbar_init(bar(CF::BAR_KE + s), 1);
            mbar_init(bar(CF::BAR_VF + s), 1);
            mbar_init(bar(CF::BAR_VE + s), 1);
            mbar_init(bar(CF::BAR_VZ + s), 2);
        }
        mbar_init(bar(CF::BAR_ZR), 1);
        mbar_init(bar(CF::BAR_ML), 8);
        mbar_init(bar(CF::BAR_DRAIN), 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_map(&tmap_q);
        tma_prefetch_map(&tmap_k);
        tma_prefetch_map(&tmap_v);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        // blocks of the requests before each one
        int before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int x = b < p.B ? tree_request(p, b).blocks() : 0;
            const int own = x;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off)
                    x += y;
            }
            if (b < p.B)
                cum[b] = before + x - own;
            before += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0)
            cum[p.B] = before;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t timeout = p.timeout_ns;
    const int work = cum[p.B] * p.units;
    const int ctas = tree_ctas(static_cast<int>(gridDim.x), work);
    const int cta = static_cast<int>(blockIdx.x);
    const int g0 = cta < ctas ? static_cast<int>(static_cast<int64_t>(cta) * work / ctas) : 0;
    const int g1 = cta < ctas ? static_cast<int>(static_cast<int64_t>(cta + 1) * work / ctas) : 0;

    uint32_t issued = 0, parity = 0;  // bits: Q tiles 0..1, K slots 8.., V slots 16..
    if (warp < 4) {
        if (warp == 0) {
            // ------------------------------------------------------------ producer (the whole warp, a box a lane)
            const int boxes = CF::BN / p.box_rows;
            const uint32_t q_load = static_cast<uint32_t>(CF::D_ATOMS * 128 * p.group * p.tile_tokens);
            bool ok = true;
            int st = 0, seg = 0;
            uint32_t ph = 0;
            auto mark = [&](int bit, uint32_t par) {
                issued |= 1u << bit;
                parity = (parity & ~(1u << bit)) | (par << bit);
            };
            auto wait_w = [&](int id, uint32_t par) {
                return __all_sync(0xffffffffu, wait_bounded(bar(id), par, abort_flag, timeout, ERR_PRODUCER)) != 0;
            };
            for (int g = g0; ok && g < g1; ++seg) {
                const TreePiece s = tree_piece(cum, p.B, p.units, g, g1);
                const TreeRequest rq = tree_request(p, s);
                const int hk = s.unit / p.row_tiles, rt = s.unit - hk * p.row_tiles;
                const int32_t *table = p.block_table + s.b * p.table_row;
                // this lane's box of block j: its page and the row in it
                auto page_of = [&](int j) {
                    const int k = j * CF::BN + lane * p.box_rows;
                    return lane < boxes && k < rq.keys && check_ok(k >= 0 && k < p.capacity && s.b < p.B)
                               ? table[k / p.page_size] : -1;
                };
                int page = page_of(s.first);
                const int qi = seg & 1;
                const uint32_t qp = static_cast<uint32_t>(seg >> 1) & 1u;
                if (!(ok = wait_w(CF::BAR_QE + qi, qp ^ 1u)))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(CF::BAR_QF + qi), q_load);
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a)
                        tma_load_5d(sQ + (qi * CF::D_ATOMS + a) * (p.q_bytes / CF::D_ATOMS), &tmap_q, bar(CF::BAR_QF + qi), 64 * a,
                                    0, hk, rt * p.tile_tokens, s.b);
                }
                mark(qi, qp);
                for (int j = s.first; j < s.first + s.len; ++j) {
                    const int k = j * CF::BN + lane * p.box_rows;
                    const bool load = lane < boxes && k < rq.keys;
                    const int row = k % p.page_size;
                    const int this_page = page;
                    page = j + 1 < s.first + s.len ? page_of(j + 1) : -1;
                    const uint32_t bytes = static_cast<uint32_t>(
                        __popc(__ballot_sync(0xffffffffu, load)) * p.box_rows * 128 * CF::D_ATOMS);
                    const uint32_t off = static_cast<uint32_t>(lane * p.box_rows * 128);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int full = (kv ? CF::BAR_VF : CF::BAR_KF) + st;
                        if (!(ok = wait_w((kv ? CF::BAR_VE : CF::BAR_KE) + st, ph ^ 1u)))
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(bar(full), bytes);
                        __syncwarp();
                        if (load) {
#pragma unroll
                            for (int a = 0; a < CF::D_ATOMS; ++a)
                                tma_load_4d((kv ? sV : sK) + st * CF::TILE_BYTES + a * CF::ATOM_BYTES + off,
                                            kv ? &tmap_v : &tmap_k, bar(full), 64 * a, row, hk, this_page);
                        }
                        mark((kv ? 16 : 8) + st, ph);
                    }
                    if (!ok)
                        break;
                    if (++st == KS) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                g += s.len;
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0 && g0 < g1) {
                constexpr uint32_t IDESC_QK = mma_idesc_f16(DT, 128, 128, 0, 0);
                constexpr uint32_t IDESC_PV = mma_idesc_f16(DT, 128, D, 0, 1);
                const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
                const uint64_t k_desc = smem_desc_sw128(sK, 16, 1024);
                const uint64_t v_desc = smem_desc_sw128(sV, CF::ATOM_BYTES, 1024);
                auto kmaj = [](int k) { return static_cast<uint64_t>(((k >> 2) * CF::ATOM_BYTES + (k & 3) * 32) >> 4); };
                const int q_atom = p.q_bytes / CF::D_ATOMS;
                auto wait = [&](int id, uint32_t par) {
                    return wait_bounded(bar(id), par, abort_flag, timeout, ERR_MMA_DATA);
                };
                const int total = g1 - g0;
                TreePiece s1 = tree_piece(cum, p.B, p.units, g0, g1), s2 = s1;  // of block n + 1, of block n
                int seg1 = 0, seg2 = 0, i1 = 0, i2 = 0;                          // their numbers, blocks done in them
                int keys2 = tree_request(p, s2).keys;
                int st1 = 0, st2 = 0;
                uint32_t ph1 = 0, ph2 = 0, zeroed = 0;  // zeroed: parity of each V slot's zeroings
                for (int n = -1; n < total; ++n) {
                    if (n + 1 < total) {
                        const int w1 = (n + 1) & 1;
                        if (i1 == 0 && !wait(CF::BAR_QF + (seg1 & 1), static_cast<uint32_t>(seg1 >> 1) & 1u))
                            break;
                        if (!wait(CF::BAR_KF + st1, ph1))
                            break;
                        if (n >= 1 && !wait(CF::BAR_DONE + w1, static_cast<uint32_t>((n - 1) >> 1) & 1u))
                            break;
                        tc_fence_after_sync();
                        const uint64_t qd = q_desc + (((seg1 & 1) * p.q_bytes) >> 4);
                        const uint64_t kd = k_desc + ((st1 * CF::TILE_BYTES) >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_f16(tmem_base + CF::TMEM_S + 128 * w1, qd + (((k >> 2) * q_atom + (k & 3) * 32) >> 4),
                                       kd + kmaj(k), IDESC_QK,
                                       k != 0 ? 1u : 0u);
                        tc_commit(bar(CF::BAR_SF + w1));
                        tc_commit(bar(CF::BAR_KE + st1));
                        if (++st1 == KS) {
                            st1 = 0;
                            ph1 ^= 1u;
                        }
                        if (++i1 == s1.len) {
                            tc_commit(bar(CF::BAR_QE + (seg1 & 1)));
                            if (n + 2 < total)
                                s1 = tree_piece(cum, p.B, p.units, g0 + n + 2, g1);
                            ++seg1;
                            i1 = 0;
                        }
                    }
                    if (n >= 0) {
                        const int w = n & 1;
                        if (!wait(CF::BAR_VF + st2, ph2))
                            break;
                        if ((s2.first + i2 + 1) * CF::BN > keys2) {
                            mbar_arrive(bar(CF::BAR_ZR));
                            if (!wait(CF::BAR_VZ + st2, (zeroed >> st2) & 1u))
                                break;
                            zeroed ^= 1u << st2;
                        }
                        // the previous piece's sums have left Tensor Memory
                        if (i2 == 0 && seg2 > 0 &&
                            !wait(CF::BAR_OE + ((seg2 - 1) & 1), static_cast<uint32_t>((seg2 - 1) >> 1) & 1u))
                            break;
                        if (!wait(CF::BAR_PF + w, static_cast<uint32_t>(n >> 1) & 1u))
                            break;
                        tc_fence_after_sync();
                        const uint64_t vd = v_desc + ((st2 * CF::TILE_BYTES) >> 4);
#pragma unroll
                        for (int k = 0; k < CF::BN / 16; ++k)
                            tc_mma_f16_ts(tmem_base + CF::TMEM_O + D * w, tmem_base + CF::TMEM_S + 128 * w + 8 * k,
                                          vd + ((2048 * k) >> 4), IDESC_PV, (i2 >= 2 || k > 0) ? 1u : 0u);
                        tc_commit(bar(CF::BAR_DONE + w));
                        tc_commit(bar(CF::BAR_VE + st2));
                        if (++st2 == KS) {
                            st2 = 0;
                            ph2 ^= 1u;
                        }
                        if (++i2 == s2.len && n + 1 < total) {
                            s2 = tree_piece(cum, p.B, p.units, g0 + n + 1, g1);
                            keys2 = tree_request(p, s2).keys;
                            ++seg2;
                            i2 = 0;
                        }
                    }
                }
                tc_commit(bar(CF::BAR_DRAIN));
                wait_drain(bar(CF::BAR_DRAIN), 0, timeout);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ the tree's masks; zeros behind the last key
            const int t = threadIdx.x - 64;  // token
            bool ok = true;
            int seg = 0, n = 0;
            uint32_t tails = 0;
            for (int g = g0; ok && g < g1; ++seg) {
                const TreePiece s = tree_piece(cum, p.B, p.units, g, g1);
                const TreeRequest rq = tree_request(p, s);
                const int buf = seg & 1;
                if (seg >= 2 && !(ok = __all_sync(0xffffffffu, wait_bounded(bar(CF::BAR_OE + buf),
                                                                            static_cast<uint32_t>((seg >> 1) - 1) & 1u,
                                                                            abort_flag, timeout, ERR_EPILOGUE))))
                    break;
                // bit u: token t sees drafted token u; only tokens that have a key
                uint64_t mask = ~0ull >> (63 - t);
                int depth = t;
                if (p.parents) {
                    // each warp keeps its own copy, so neither waits for the other
                    int32_t *par = parent_smem + (warp - 2) * kTreeMaxTokens;
                    __syncwarp();
                    for (int i = lane; i < kTreeMaxTokens; i += 32)
                        par[i] = i < p.T ? p.parents[static_cast<int64_t>(s.b) * p.T + i] : -1;
                    __syncwarp();
                    mask = 1ull << t;
                    depth = 0;
                    for (int a = t, up = par[t]; up >= 0 && up < a; up = par[a]) {
                        a = up;
                        mask |= 1ull << a;
                        ++depth;
                    }
                }
                const int live = rq.keys - rq.context;  // drafted tokens with a key
                if (live < kTreeMaxTokens)
                    mask &= live > 0 ? (1ull << live) - 1 : 0ull;
                tree_mask[buf * kTreeMaxTokens + t] = mask;
                if constexpr (BIAS) {
                    // context keys at their index, drafted ones at their depth; what lies behind is hidden
                    float *place = tree_place + buf * CF::PLACES;
                    place[CF::PLACE0 + t] = static_cast<float>(depth);
                    place[t] = static_cast<float>(t - CF::PLACE0);
                    place[64 + t] = static_cast<float>(64 + t - CF::PLACE0);
                    place[CF::PLACE0 + 64 + t] = 0.0f;
                    place[CF::PLACE0 + 128 + t] = 0.0f;
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(CF::BAR_TF + buf));
                // the tile's last block, where the keys end inside it
                const int end = s.first + s.len;
                if (end * CF::BN > rq.keys) {
                    // the MMA warp says when it has landed: it follows every phase of the V slots, this warp does not
                    const int st = (n + s.len - 1) % KS;
                    if (!(ok = __all_sync(0xffffffffu, wait_bounded(bar(CF::BAR_ZR), tails & 1u, abort_flag, timeout,
                                                                    ERR_EPILOGUE))))
                        break;
                    ++tails;
                    const int from = rq.keys - (end - 1) * CF::BN;  // first row behind the keys
                    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int a = 0; a < CF::D_ATOMS; ++a) {
                        uint4 *dst = reinterpret_cast<uint4 *>(smem + off_v + st * CF::TILE_BYTES + a * CF::ATOM_BYTES);
                        for (int i = from * 8 + t; i < CF::BN * 8 && check_ok(i >= 0 && st < KS); i += 64)
                            dst[i] = zero;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar(CF::BAR_VZ + st));
                }
                n += s.len;
                g += s.len;
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax of every other block, output of a piece
        const int w = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const int r_token = r / p.group, r_head = r - r_token * p.group;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_S + 128 * w);
        const uint32_t o_addr = tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_O + D * w);
        auto wait_warp = [&](int id, uint32_t par) -> bool {
            return __all_sync(0xffffffffu, wait_bounded(bar(id), par, abort_flag, timeout, ERR_EPILOGUE));
        };
        bool ok = true;
        int seg = 0, n0 = 0;
        for (int g = g0; ok && g < g1; ++seg) {
            const TreePiece s = tree_piece(cum, p.B, p.units, g, g1);
            const TreeRequest rq = tree_request(p, s);
            const int hk = s.unit / p.row_tiles, rt = s.unit - hk * p.row_tiles;
            const int tok = rt * p.tile_tokens + r_token;
            const bool valid = r_token < p.tile_tokens && tok < rq.tokens &&
                               check_ok(tok < p.T && s.b < p.B && hk * p.group + r_head < p.H);
            const bool active = __any_sync(0xffffffffu, valid);  // warps without a row only keep the barriers going
            const int head = hk * p.group + r_head;
            const int buf = seg & 1;
            if (!(ok = wait_warp(CF::BAR_TF + buf, static_cast<uint32_t>(seg >> 1) & 1u)))
                break;
            const uint64_t mask = valid ? tree_mask[buf * kTreeMaxTokens + tok] : 0ull;
            float slope2 = 0.0f;
            float pos_f = 0.0f;  // the token's place, counted from the context's end: its depth
            if constexpr (BIAS) {
                if (valid) {
                    slope2 = __ldg(p.score.slopes + head) * 1.4426950408889634f;
                    pos_f = tree_place[buf * CF::PLACES + CF::PLACE0 + tok];
                }
            }
            float m = -INFINITY, l = 0.0f;
            const int i_first = (w - n0) & 1;  // first block of the piece that is this stream's
            for (int i = i_first; ok && i < s.len; i += 2) {
                const int n = n0 + i;
                if (!(ok = wait_warp(CF::BAR_SF + w, static_cast<uint32_t>(n >> 1) & 1u)))
                    break;
                tc_fence_after_sync();
                if (active) {
                    const int key0 = (s.first + i) * CF::BN;
                    const bool context_only = key0 + CF::BN <= rq.context;
                    const float to_log2 = CAP ? p.score.cap_log2 : p.score.scale_log2;  // of a score without a bias
                    // 32 columns at a time, in loops: a call visits few blocks, and straight-line code for 128
                    // columns spent its time on instruction fetches
                    uint32_t sv[32];
                    // put `value` in the place of the keys the row does not see, of columns 32 q ..
                    auto hide = [&](int q, float value) {
                        const int a = key0 + 32 * q - rq.context;  // the first key among the drafted
                        uint32_t see;
                        if (a <= -32)
                            see = 0xFFFFFFFFu;
                        else if (a < 0)
                            see = (static_cast<uint32_t>(mask) << -a) | ((1u << -a) - 1u);
                        else
                            see = a < 64 ? static_cast<uint32_t>(mask >> a) : 0u;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see & (1u << e)))
                                sv[e] = __float_as_uint(value);
                    };
                    // with a bias: the scores in log2 units, less slope2 times the distance
                    auto biased = [&](int q) {
                        if (!context_only && !check_ok(key0 + 32 * q - rq.context >= -CF::PLACE0 &&
                                                       key0 + 32 * q + 32 - rq.context <= CF::PLACES - CF::PLACE0))
                            return;
                        const float dist0 = pos_f - static_cast<float>(key0 + 32 * q - rq.context);
                        const float *place = tree_place + buf * CF::PLACES + CF::PLACE0 + (key0 + 32 * q - rq.context);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 dist;
                            if (context_only)
                                dist = fadd2(splat2(dist0), make_float2(-static_cast<float>(e), -static_cast<float>(e + 1)));
                            else
                                dist = make_float2(fabsf(pos_f - place[e]), fabsf(pos_f - place[e + 1]));
                            const float2 x = ffma2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                                   splat2(to_log2), fmul2(dist, splat2(-slope2)));
                            sv[e] = __float_as_uint(x.x);
                            sv[e + 1] = __float_as_uint(x.y);
                        }
                    };
                    // Columns 32 q .., hidden keys at -inf.  A page's unused rows may hold anything, and a
                    // reciprocal shared by two keys would spread it: they are 0 before the cap.
                    auto scores = [&](int q, bool cap) {
                        tmem_load_32cols(s_addr + 32 * q, sv);
                        tmem_load_wait();
                        if (cap) {
                            if (!context_only)
                                hide(q, 0.0f);
                            tanh_scores<32>(sv, p.score.cap_arg, valid);
                        }
                        if constexpr (BIAS)
                            biased(q);
                        if (!context_only)
                            hide(q, -INFINITY);
                    };
                    // the maximum; the cap is monotonic, so without a bias that of the raw scores serves
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        scores(q, CAP && BIAS);
                        if constexpr (BIAS)  // the second pass finds them as they are here
                            tmem_store_32cols(s_addr + 32 * q, sv);
                        const float *f = reinterpret_cast<const float *>(sv);
                        float t[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            t[i] = fmax3(fmax3(f[8 * i], f[8 * i + 1], f[8 * i + 2]),
                                         fmax3(f[8 * i + 3], f[8 * i + 4], f[8 * i + 5]), fmaxf(f[8 * i + 6], f[8 * i + 7]));
                        mx = fmax3(mx, fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                    }
                    if constexpr (CAP && !BIAS) {
                        if (mx != -INFINITY)
                            mx = 1.0f - 2.0f * rcp_approx(1.0f + exp2_approx_ftz(fminf(2.8853900817779268f * p.score.cap_arg * mx,
                                                                                      60.0f)));
                    }
                    if constexpr (!BIAS)
                        mx *= to_log2;
                    else
                        tmem_store_wait();
                    const bool resc = mx > m + CF::RESCALE_LOG2;
                    const float m_new = resc ? mx : m;
                    const float m_ref = m_new == -INFINITY ? 0.0f : m_new;
                    const float alpha = resc ? exp2_approx_ftz(m - m_ref) : 1.0f;
                    const float2 negm2 = splat2(-m_ref);
                    float2 part[2] = {splat2(0.0f), splat2(0.0f)};
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (BIAS) {
                            tmem_load_32cols(s_addr + 32 * q, sv);
                            tmem_load_wait();
                        } else {
                            scores(q, CAP);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 v = make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                            const float2 x = BIAS ? fadd2(v, negm2) : ffma2(v, splat2(to_log2), negm2);
                            const float2 w2 = make_float2(exp2_approx_ftz(x.x), exp2_approx_ftz(x.y));
                            part[(e >> 1) & 1] = fadd2(part[(e >> 1) & 1], w2);
                            sv[e / 2] = pack2<DT>(w2.x, w2.y);
                        }
                        tmem_store_16cols(s_addr + 16 * q, sv);  // over columns that have been read
                    }
                    const float2 ps = fadd2(part[0], part[1]);
                    l = l * alpha + (ps.x + ps.y);
                    m = m_new;
                    // S(n) was issued after this stream's last P V had completed, so O is whole here
                    if (i > i_first && __any_sync(0xffffffffu, resc)) {
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
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(CF::BAR_PF + w));
            }
            if (!ok)
                break;
            // the two streams' sums of the piece, joined: this warpgroup takes half the columns
            float2 *mls = ml + buf * 2 * 128;
            mls[w * 128 + r] = make_float2(m, l);
            const int n1 = n0 + s.len;
            // this stream's last P V (the ones before it have completed, S(n) being issued behind them), then the other's
            if (i_first < s.len)
                ok = wait_warp(CF::BAR_DONE + w, static_cast<uint32_t>((n1 - w + 1) / 2 - 1) & 1u);
            if (!ok)
                break;
            tc_fence_after_sync();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(CF::BAR_ML));
            if (!(ok = wait_warp(CF::BAR_ML, static_cast<uint32_t>(seg) & 1u)))
                break;
            tc_fence_after_sync();
            const bool whole = s.len == s.blocks;
            if (active) {
                const float2 a = mls[r], c = mls[128 + r];
                const float M = fmaxf(a.x, c.x);
                const float f0 = a.x == -INFINITY ? 0.0f : exp2_approx_ftz(a.x - M);
                const float f1 = c.x == -INFINITY ? 0.0f : exp2_approx_ftz(c.x - M);
                const float L = a.y * f0 + c.y * f1;
                const bool use0 = ((0 - n0) & 1) < s.len, use1 = ((1 - n0) & 1) < s.len;
                const float inv = whole ? (L == 0.0f ? 0.0f : 1.0f / L) : 1.0f;
                const int slot = 2 * cta + (s.first == 0 ? 1 : 0);
                uint16_t *orow = p.O + s.b * p.o_batch + head * p.o_head + static_cast<int64_t>(tok) * p.o_row;
                float4 *prow = reinterpret_cast<float4 *>(p.part_o) + static_cast<int64_t>(slot) * (D / 4) * 128 + r;
#pragma unroll 1
                for (int c0 = w * (D / 2); c0 < (w + 1) * (D / 2); c0 += 32) {
                    uint32_t o0[32], o1[32];
                    if (use0)
                        tmem_load_32cols(tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_O + c0), o0);
                    if (use1)
                        tmem_load_32cols(tmem_base + lane_base + static_cast<uint32_t>(CF::TMEM_O + D + c0), o1);
                    tmem_load_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float v = 0.0f;
                        if (use0)
                            v = __uint_as_float(o0[e]) * f0;
                        if (use1)
                            v = fmaf(__uint_as_float(o1[e]), f1, v);
                        o0[e] = __float_as_uint(v * inv);
                    }
                    if (valid) {
                        if (whole) {
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                uint4 x;
                                x.x = pack2<DT>(__uint_as_float(o0[8 * v]), __uint_as_float(o0[8 * v + 1]));
                                x.y = pack2<DT>(__uint_as_float(o0[8 * v + 2]), __uint_as_float(o0[8 * v + 3]));
                                x.z = pack2<DT>(__uint_as_float(o0[8 * v + 4]), __uint_as_float(o0[8 * v + 5]));
                                x.w = pack2<DT>(__uint_as_float(o0[8 * v + 6]), __uint_as_float(o0[8 * v + 7]));
                                reinterpret_cast<uint4 *>(orow + c0)[v] = x;
                            }
                        } else {
#pragma unroll
                            for (int v = 0; v < 8; ++v)
                                prow[(c0 / 4 + v) * 128] =
                                    make_float4(__uint_as_float(o0[4 * v]), __uint_as_float(o0[4 * v + 1]),
                                                __uint_as_float(o0[4 * v + 2]), __uint_as_float(o0[4 * v + 3]));
                        }
                    }
                }
                if (valid && w == 0) {
                    if (!whole)
                        p.part_ml[static_cast<int64_t>(slot) * 128 + r] = make_float2(M, L);
                    else if (p.lse)
                        p.lse[(static_cast<int64_t>(s.b) * p.H + head) * p.T + tok] =
                            L == 0.0f ? -INFINITY : M * 0.69314718055994531f + logf(L);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(CF::BAR_OE + buf));
            n0 = n1;
            g += s.len;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        for (int i = 0; i < 2; ++i)
            if (issued & (1u << i))
                wait_drain(bar(CF::BAR_QF + i), (parity >> i) & 1u, timeout);
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

// Joins the pieces of each tile whose blocks fell to several CTAs: a row a lane.
// The loads of one piece wait for the L2 (about half a microsecond), so what counts is how
// many pieces are read one after the other.  With W = 1 the block's 8 warps take
// D / 8 columns each and read every piece; with W = 8 a block takes D / 8 columns
// of the tile, its warps every eighth piece each, joined through shared memory
// (8000 keys of 4 heads, 37 pieces a tile: 34 -> 16 us for the whole call).
// The order of the sums depends on the lengths and the number of SMs only.
template <int DT, int D, int W>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeParams p, int grid)
{
    constexpr int C4 = D / 32;  // groups of four columns a warp
    __shared__ float4 join_o[W == 1 ? 1 : C4 * W * 32];
    __shared__ float2 join_ml[W == 1 ? 1 : W * 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row_groups = (p.tile_tokens * p.group + 31) / 32;
    const int tile_rows = static_cast<int>(W == 1 ? blockIdx.x : blockIdx.x / 8);
    const int columns = W == 1 ? warp : static_cast<int>(blockIdx.x % 8);  // which eighth of them
    const int rb = tile_rows % row_groups, bu = tile_rows / row_groups;
    const int unit = bu % p.units, b = bu / p.units;
    int before = 0, all = 0;
    TreeRequest rq{0, 0, 0};
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int i = b0 + lane;
        TreeRequest x{0, 0, 0};
        if (i < p.B)
            x = tree_request(p, i);
        all += x.blocks();
        before += i < b ? x.blocks() : 0;
        if (b >= b0 && b < b0 + 32) {
            rq.tokens = __shfl_sync(0xffffffffu, x.tokens, b - b0);
            rq.keys = __shfl_sync(0xffffffffu, x.keys, b - b0);
        }
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    const int blocks = rq.blocks();
    if (blocks == 0)
        return;
    const int work = all * p.units;
    const int first = before * p.units + unit * blocks;
    const int ctas = tree_ctas(grid, work);
    // the CTA whose run [c work / ctas, (c + 1) work / ctas) holds block g
    auto owner = [&](int g) { return static_cast<int>(((static_cast<int64_t>(g) + 1) * ctas - 1) / work); };
    const int c0 = owner(first), c1 = owner(first + blocks - 1);
    if (c0 == c1 || !check_ok(b < p.B && c0 >= 0 && c0 < c1 && c1 < grid))
        return;
    const int hk = unit / p.row_tiles, rt = unit - hk * p.row_tiles;
    const int rows = min(p.tile_tokens, rq.tokens - rt * p.tile_tokens) * p.group;
    const int r = 32 * rb + lane;
    if (32 * rb >= rows)
        return;
    const bool valid = r < rows;
    auto slot = [&](int c) { return static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0)); };
    const float4 *parts = reinterpret_cast<const float4 *>(p.part_o) + columns * C4 * 128 + r;
    float M = -INFINITY, L = 0.0f;
    float4 acc[C4];
#pragma unroll
    for (int v = 0; v < C4; ++v)
        acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float4 &to, const float4 &x, float f) {
        to.x = fmaf(x.x, f, to.x);
        to.y = fmaf(x.y, f, to.y);
        to.z = fmaf(x.z, f, to.z);
        to.w = fmaf(x.w, f, to.w);
    };
    const int own = W == 1 ? 0 : warp;
    if (valid) {
#pragma unroll 4
        for (int c = c0 + own; c <= c1; c += W)
            M = fmaxf(M, p.part_ml[slot(c) * 128 + r].x);
#pragma unroll 4
        for (int c = c0 + own; c <= c1; c += W) {
            const float2 x = p.part_ml[slot(c) * 128 + r];
            const float f = x.x == -INFINITY ? 0.0f : exp2_approx_ftz(x.x - M);
            L = fmaf(x.y, f, L);
#pragma unroll
            for (int v = 0; v < C4; ++v)
                add(acc[v], parts[(slot(c) * (D / 4) + v) * 128], f);
        }
    }
    if constexpr (W > 1) {
        // the warps' sums, joined by the first warps: a warp a group of four columns
        join_ml[warp * 32 + lane] = make_float2(M, L);
#pragma unroll
        for (int v = 0; v < C4; ++v)
            join_o[(v * W + warp) * 32 + lane] = acc[v];
        __syncthreads();
        if (warp >= C4)
            return;
        M = -INFINITY;
        L = 0.0f;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < W; ++i)
            M = fmaxf(M, join_ml[i * 32 + lane].x);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 x = join_ml[i * 32 + lane];
            const float f = x.x == -INFINITY ? 0.0f : exp2_approx_ftz(x.x - M);
            L = fmaf(x.y, f, L);
            add(sum, join_o[(warp * W + i) * 32 + lane], f);
        }
        acc[0] = sum;
    }
    if (!valid)
        return;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int tok = rt * p.tile_tokens + r / p.group, head = hk * p.group + r % p.group;
    uint16_t *orow = p.O + b * p.o_batch + head * p.o_head + static_cast<int64_t>(tok) * p.o_row + columns * 4 * C4;
    auto pack4 = [&](const float4 &x) { return make_uint2(pack2<DT>(x.x * inv, x.y * inv), pack2<DT>(x.z * inv, x.w * inv)); };
    if constexpr (W > 1) {
        reinterpret_cast<uint2 *>(orow)[warp] = pack4(acc[0]);
    } else {
#pragma unroll
        for (int v = 0; v < C4; v += 2) {
            const uint2 lo = pack4(acc[v]), hi = pack4(acc[v + 1]);
            reinterpret_cast<uint4 *>(orow)[v / 2] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
    if (p.lse && warp == 0 && columns == 0)
        p.lse[(static_cast<int64_t>(b) * p.H + head) * p.T + tok] =
            L == 0.0f ? -INFINITY : M * 0.69314718055994531f + logf(L);
}

} // namespace tl
