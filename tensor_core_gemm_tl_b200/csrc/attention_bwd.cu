// attention_bwd.cu -- host side of tl_attention_bwd: argument checks, the
// workspace, tensor maps and the launches.
#include "attention_host.h"
#include "attention_bwd_kernel.cuh"

#include <algorithm>

namespace tl {
namespace {

using BwdFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, AttnBwdParams);
using RowsFn = void (*)(AttnBwdRowsParams);
using JoinFn = void (*)(AttnBwdJoinParams);

struct BwdEntry {
    BwdFn fn[2][2][2][2];  // [dtype][dK and dV][capped][biased]
    RowsFn rows[2];        // [dtype]
    JoinFn join[2][2];     // [dtype][dK and dV]
    int smem, threads, launch_regs;
};

template <class CF, int DT>
void fill_bwd(BwdEntry &e)
{
    e.fn[DT][0][0][0] = attention_bwd_kernel<CF, DT, false, false, false>;
    e.fn[DT][0][0][1] = attention_bwd_kernel<CF, DT, false, false, true>;
    e.fn[DT][0][1][0] = attention_bwd_kernel<CF, DT, false, true, false>;
    e.fn[DT][0][1][1] = attention_bwd_kernel<CF, DT, false, true, true>;
    e.fn[DT][1][0][0] = attention_bwd_kernel<CF, DT, true, false, false>;
    e.fn[DT][1][0][1] = attention_bwd_kernel<CF, DT, true, false, true>;
    e.fn[DT][1][1][0] = attention_bwd_kernel<CF, DT, true, true, false>;
    e.fn[DT][1][1][1] = attention_bwd_kernel<CF, DT, true, true, true>;
    e.rows[DT] = attention_bwd_rows_kernel<DT, CF::D>;
    e.join[DT][0] = attention_bwd_join_kernel<DT, CF::D, false>;
    e.join[DT][1] = attention_bwd_join_kernel<DT, CF::D, true>;
}

template <int D>
BwdEntry make_bwd()
{
    using CF = AttnBwdConfig<D>;
    BwdEntry e;
    fill_bwd<CF, 0>(e);
    fill_bwd<CF, 1>(e);
    e.smem = CF::SMEM_BYTES;
    e.threads = CF::THREADS;
    e.launch_regs = CF::LAUNCH_REGS;
    return e;
}

const BwdEntry kBwd64 = make_bwd<64>();
const BwdEntry kBwd128 = make_bwd<128>();

// How a pass's tiles are cut.  A tile's blocks run one after another, so where there are few tiles, or causal ones
// of very different lengths, the longest decides.  In blocks (about 1 us each): a piece costs its own and about 8
// more, the joining of the pieces 8; an SM gets its share of the pieces and, as they end at different times, half a
// piece more (measured: 84 tiles of up to 98 blocks 125 -> 82 us, joining included; 150 tiles of up to 56 blocks
// 76 us either way).  The sums of eight pieces an SM are the most that is kept in memory.
struct Pieces {
    int32_t chunk, splits;
};

Pieces cut_tiles(int64_t items, int64_t longest, double seen, int num_sms)
{
    Pieces c{0x7FFFFFFF, 1};
    const double work = static_cast<double>(items) * longest * seen;
    double best = 0.85 * (std::max(static_cast<double>(longest), (work + 8.0 * items) / num_sms) + 8.0);
    for (int k = 2; k <= 32 && longest >= 4 * k && items * k <= 8ll * num_sms; ++k) {
        const int64_t chunk = ceil_div(longest, k);
        const double pieces = items * (seen * longest / chunk + 0.5);
        const double share = pieces <= num_sms ? 0.0 : (work + 8.0 * pieces) / num_sms + 0.5 * (chunk + 8);
        const double t = std::max(chunk + 8.0, share) + 8.0;
        if (t < best) {
            best = 0.97 * t;
            c.chunk = static_cast<int32_t>(chunk);
            c.splits = static_cast<int32_t>(ceil_div(longest, chunk));
        }
    }
    return c;
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

tl_status attention_bwd_impl(const void *dO, const void *Q, const void *K, const void *V, const void *O,
                             const float *lse, void *dQ, void *dK, void *dV, int64_t batch, int64_t heads,
                             int64_t seq_q, int64_t seq_k, int64_t head_dim, int dtype, cudaStream_t stream,
                             const tl_attention_options *opt)
{
    if (!dO || !dQ || !dK || !dV || !lse)
        return TL_ERR_INVALID_ARG;
    AttentionCall c;
    tl_status st = attention_call(Q, K, V, O, lse, batch, heads, seq_q, seq_k, head_dim, dtype, opt, &c);
    if (st != TL_OK)
        return st;
    if (!aligned(dO, 16) || !aligned(dQ, 16) || !aligned(dK, 16) || !aligned(dV, 16))
        return TL_ERR_MISALIGNED;
    static const int64_t dense[3] = {0, 0, 0};
    const int64_t sq[3] = {batch, heads, seq_q}, sk[3] = {batch, c.kv_heads, seq_k};
    Strides sdo, sdq, sdk, sdv;
    if ((st = take_strides(opt ? opt->do_strides : dense, sq, head_dim, &sdo)) != TL_OK ||
        (st = take_strides(opt ? opt->dq_strides : dense, sq, head_dim, &sdq)) != TL_OK ||
        (st = take_strides(opt ? opt->dk_strides : dense, sk, head_dim, &sdk)) != TL_OK ||
        (st = take_strides(opt ? opt->dv_strides : dense, sk, head_dim, &sdv)) != TL_OK)
        return st;
    DeviceState *d = nullptr;
    if ((st = device_state(&d)) != TL_OK)
        return st;
    if (d->cc_major != 10)
        return TL_ERR_UNSUPPORTED;
    const BwdEntry &e = head_dim == 64 ? kBwd64 : kBwd128;
    BwdFn dkv = e.fn[dtype][1][c.cap > 0.0f][c.slopes != nullptr];
    BwdFn dq = e.fn[dtype][0][c.cap > 0.0f][c.slopes != nullptr];
    if ((st = ready_kernel(d, dkv, e.smem, e.launch_regs)) != TL_OK ||
        (st = ready_kernel(d, dq, e.smem, e.launch_regs)) != TL_OK)
        return st;
    // tiles of 128 rows and blocks of 64: dK and dV hold the keys, dQ the queries
    CUtensorMap tk, tv, tq, tdo, bk, bv, bq, bdo, out_q, out_k, out_v;
    if (!encode_heads(&tk, K, dtype, batch, c.kv_heads, seq_k, head_dim, c.k, 128) ||
        !encode_heads(&tv, V, dtype, batch, c.kv_heads, seq_k, head_dim, c.v, 128) ||
        !encode_heads(&tq, Q, dtype, batch, heads, seq_q, head_dim, c.q, 128) ||
        !encode_heads(&tdo, dO, dtype, batch, heads, seq_q, head_dim, sdo, 128) ||
        !encode_heads(&bk, K, dtype, batch, c.kv_heads, seq_k, head_dim, c.k, kBwdCols) ||
        !encode_heads(&bv, V, dtype, batch, c.kv_heads, seq_k, head_dim, c.v, kBwdCols) ||
        !encode_heads(&bq, Q, dtype, batch, heads, seq_q, head_dim, c.q, kBwdCols) ||
        !encode_heads(&bdo, dO, dtype, batch, heads, seq_q, head_dim, sdo, kBwdCols) ||
        !encode_heads_out(&out_q, dQ, dtype, batch, heads, seq_q, head_dim, sdq, 32, 16) ||
        !encode_heads_out(&out_k, dK, dtype, batch, c.kv_heads, seq_k, head_dim, sdk, 32, 16) ||
        !encode_heads_out(&out_v, dV, dtype, batch, c.kv_heads, seq_k, head_dim, sdv, 32, 16))
        return TL_ERR_CUDA;

    const int64_t nqb = ceil_div(seq_q, kBwdCols);
    const int64_t rows_bytes = round256(batch * heads * nqb * 2 * kBwdCols * 4);
    const int64_t interval_bytes = round256(batch * nqb * 3 * kBwdCols * 4);
    const int64_t range_bytes = round256(batch * nqb * 16);
    if ((st = ensure_pool(d)) != TL_OK)
        return st;
    // both passes' tiles and the most blocks one has
    const int64_t q_tiles = ceil_div(seq_q, 128), k_tiles = ceil_div(seq_k, 128);
    const int64_t q_items = q_tiles * batch * heads, k_items = k_tiles * batch * c.kv_heads;
    const int64_t keys = c.mask.causal && !c.mask.prefix ? std::min(seq_k, c.mask.q_offset + seq_q) : seq_k;
    const double seen = c.mask.causal ? std::min(1.0, (c.mask.q_offset + 0.5 * seq_q) / keys) : 1.0;
    const Pieces cut_q = cut_tiles(q_items, ceil_div(keys, kBwdCols), seen, d->num_sms);
    const Pieces cut_k = cut_tiles(k_items, nqb * (heads / c.kv_heads), seen, d->num_sms);
    // what the pieces leave: the passes use the same memory one after the other
    const int64_t q_slots = cut_q.splits > 1 ? q_items * cut_q.splits : 0, k_slots = cut_k.splits > 1 ? k_items * cut_k.splits : 0;
    const int64_t slots = std::max(q_slots, k_slots);
    const int64_t piece_bytes = slots ? round256(std::max(q_items, k_items) * 4) : 0;
    const int64_t part_bytes = slots * 2 * head_dim * 128 * 4;
    const int64_t own_bytes = rows_bytes + interval_bytes + range_bytes + 256;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(own_bytes + piece_bytes + part_bytes + q_slots * 128 * 4), d->pool,
                                stream) != cudaSuccess)
        return TL_ERR_CUDA;
    uint8_t *at = static_cast<uint8_t *>(ws);
    AttnBwdRowsParams rp{};
    rp.mask = c.mask;
    rp.B = static_cast<int32_t>(batch);
    rp.H = static_cast<int32_t>(heads);
    rp.D = static_cast<int32_t>(head_dim);
    rp.nqb = static_cast<int32_t>(nqb);
    rp.O = static_cast<const uint16_t *>(O);
    rp.dO = static_cast<const uint16_t *>(dO);
    rp.lse = lse;
    rp.rows = reinterpret_cast<float *>(at);
    rp.intervals = reinterpret_cast<int32_t *>(at + rows_bytes);
    rp.ranges = reinterpret_cast<int4 *>(at + rows_bytes + interval_bytes);
    rp.next = reinterpret_cast<int32_t *>(at + rows_bytes + interval_bytes + range_bytes + 16);
    rp.norms = reinterpret_cast<float *>(at + rows_bytes + interval_bytes + range_bytes);
    rp.Hk = static_cast<int32_t>(c.kv_heads);
    rp.V = static_cast<const uint16_t *>(V);
    rp.query_ctas = static_cast<int32_t>(nqb * batch * heads);
    rp.nkb = static_cast<int32_t>(ceil_div(seq_k, kBwdCols));
    AttnBwdParams p{};
    p.mask = c.mask;
    p.score = score_params(c.scale, c.cap, c.slopes);
    p.B = rp.B;
    p.H = rp.H;
    p.Hk = static_cast<int32_t>(c.kv_heads);
    p.group = static_cast<int32_t>(heads / c.kv_heads);
    p.nqb = rp.nqb;
    p.scale = c.scale;
    p.rows = rp.rows;
    p.intervals = rp.intervals;
    p.ranges = rp.ranges;
    p.norms = rp.norms;
    p.timeout_ns = kDefaultTimeoutNs;
    AttnBwdParams pk = p, pq = p;
    pq.next = rp.next;
    pk.next = rp.next + 1;
    pk.tiles = static_cast<int32_t>(k_tiles);
    pq.tiles = static_cast<int32_t>(q_tiles);
    auto cut = [&](AttnBwdParams &a, const Pieces &by) {
        a.chunk = by.chunk;
        a.splits = by.splits;
        a.pieces = by.splits > 1 ? reinterpret_cast<int32_t *>(at + own_bytes) : nullptr;
        a.part = reinterpret_cast<float4 *>(at + own_bytes + piece_bytes);
        a.part_e = reinterpret_cast<float *>(at + own_bytes + piece_bytes + part_bytes);
    };
    cut(pq, cut_q);
    cut(pk, cut_k);
    for (int i = 0; i < 3; ++i) {
        rp.so[i] = c.o.s[i];
        rp.sdo[i] = sdo.s[i];
        rp.sv[i] = c.v.s[i];
    }
    // fp16: the norms that dX's factor comes from, those of V in CTAs behind the queries'
    int64_t rows_grid = nqb * batch * heads;
    if (dtype == TL_F16) {
        rows_grid += rp.nkb * batch * c.kv_heads;
        if (cudaMemsetAsync(rp.norms, 0, 2 * sizeof(float), stream) != cudaSuccess)
            st = TL_ERR_CUDA;
    }
    if (st == TL_OK)
        st = launch_overlapped(e.rows[dtype], rows_grid, 256, 0, stream, rp);
    // persistent CTAs, one an SM; they take pieces from the passes' counters
    auto launch = [&](int dkv_pass, const CUtensorMap &x1, const CUtensorMap &x2, const CUtensorMap &y1,
                      const CUtensorMap &y2, const CUtensorMap &o0, const CUtensorMap &o1, int64_t items,
                      const AttnBwdParams &a, void *out0, const Strides &s0, void *out1, const Strides &s1) {
        const int64_t pieces = items * a.splits;
        tl_status r = launch_overlapped(dkv_pass ? dkv : dq, pieces < d->num_sms ? pieces : d->num_sms, e.threads, e.smem,
                                        stream, x1, x2, y1, y2, o0, o1, a);
        if (r != TL_OK || a.splits == 1)
            return r;
        AttnBwdJoinParams j{};
        j.mask = a.mask;
        j.H = a.H;
        j.heads = dkv_pass ? a.Hk : a.H;
        j.tiles = a.tiles;
        j.BH = a.B * j.heads;
        j.splits = a.splits;
        j.nqb = a.nqb;
        j.pieces = a.pieces;
        j.part = a.part;
        j.part_e = a.part_e;
        j.rows = rp.rows;
        j.intervals = a.intervals;
        j.out0 = static_cast<uint16_t *>(out0);
        j.out1 = static_cast<uint16_t *>(out1);
        for (int i = 0; i < 3; ++i) {
            j.s0[i] = s0.s[i];
            j.s1[i] = s1.s[i];
        }
        return launch_overlapped(e.join[dtype][dkv_pass], items * 4, 256, 0, stream, j);
    };
    if (st == TL_OK)
        st = launch(0, tq, tdo, bk, bv, out_q, out_q, q_items, pq, dQ, sdq, dQ, sdq);
    if (st == TL_OK)
        st = launch(1, tk, tv, bq, bdo, out_k, out_v, k_items, pk, dK, sdk, dV, sdv);
    if (cudaFreeAsync(ws, stream) != cudaSuccess && st == TL_OK)
        st = TL_ERR_CUDA;
    return st;
}

} // namespace

bool take_error_attention_bwd(unsigned int *word) { return take_device_error(word); }

} // namespace tl

extern "C" tl_status tl_attention_bwd(const void *dO, const void *Q, const void *K, const void *V, const void *O,
                                      const float *lse, void *dQ, void *dK, void *dV, int64_t batch, int64_t heads,
                                      int64_t seq_q, int64_t seq_k, int64_t head_dim, tl_dtype dtype, tl_stream stream,
                                      const tl_attention_options *options)
{
    return tl::attention_bwd_impl(dO, Q, K, V, O, lse, dQ, dK, dV, batch, heads, seq_q, seq_k, head_dim, dtype,
                                  static_cast<cudaStream_t>(stream), options);
}
