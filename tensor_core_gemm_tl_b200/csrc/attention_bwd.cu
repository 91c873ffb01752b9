// attention_bwd.cu -- host side of tl_attention_bwd: argument checks, the
// workspace, tensor maps and the three launches.
#include "attention_host.h"
#include "attention_bwd_kernel.cuh"

namespace tl {
namespace {

using BwdFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, AttnBwdParams);
using RowsFn = void (*)(AttnBwdRowsParams);

struct BwdEntry {
    BwdFn fn[2][2][2][2];  // [dtype][dK and dV][capped][biased]
    RowsFn rows[2];        // [dtype]
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
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(rows_bytes + interval_bytes + range_bytes + 256), d->pool,
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
    rp.amax = dtype == TL_F16 ? reinterpret_cast<unsigned *>(at + rows_bytes + interval_bytes + range_bytes) : nullptr;
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
    p.amax = rp.amax;
    p.timeout_ns = kDefaultTimeoutNs;
    AttnBwdParams pk = p, pq = p;
    pq.next = rp.next;
    pk.next = rp.next + 1;
    pk.tiles = static_cast<int32_t>(ceil_div(seq_k, 128));
    pq.tiles = static_cast<int32_t>(ceil_div(seq_q, 128));
    for (int i = 0; i < 3; ++i) {
        rp.so[i] = c.o.s[i];
        rp.sdo[i] = sdo.s[i];
    }
    if (rp.amax && cudaMemsetAsync(rp.amax, 0, sizeof(unsigned), stream) != cudaSuccess)
        st = TL_ERR_CUDA;
    if (st == TL_OK)
        st = launch_overlapped(e.rows[dtype], nqb * batch * heads, 256, 0, stream, rp);
    // persistent CTAs, one an SM; they take tiles from the passes' counters
    auto launch = [&](BwdFn fn, const CUtensorMap &x1, const CUtensorMap &x2, const CUtensorMap &y1,
                      const CUtensorMap &y2, const CUtensorMap &o0, const CUtensorMap &o1, int64_t items,
                      const AttnBwdParams &a) {
        return launch_overlapped(fn, items < d->num_sms ? items : d->num_sms, e.threads, e.smem, stream, x1, x2, y1, y2,
                                 o0, o1, a);
    };
    if (st == TL_OK)
        st = launch(dq, tq, tdo, bk, bv, out_q, out_q, pq.tiles * batch * heads, pq);
    if (st == TL_OK)
        st = launch(dkv, tk, tv, bq, bdo, out_k, out_v, pk.tiles * batch * c.kv_heads, pk);
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
