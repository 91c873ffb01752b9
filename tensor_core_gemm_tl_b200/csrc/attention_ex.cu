// attention_ex.cu -- host side of tl_attention_ex: argument checks (shared with
// the backward), tensor maps and the launch.
#include "attention_host.h"
#include "attention_ex_kernel.cuh"

namespace tl {

tl_status attention_call(const void *Q, const void *K, const void *V, const void *O, const float *lse, int64_t batch,
                         int64_t heads, int64_t seq_q, int64_t seq_k, int64_t head_dim, int dtype,
                         const tl_attention_options *opt, AttentionCall *c)
{
    static const tl_attention_options none{};
    const tl_attention_options &o = opt ? *opt : none;
    if (!Q || !K || !V || !O)
        return TL_ERR_INVALID_ARG;
    if (batch < 1 || heads < 1 || seq_q < 1 || seq_k < 1)
        return TL_ERR_INVALID_ARG;
    if (dtype != TL_F16 && dtype != TL_BF16)
        return TL_ERR_INVALID_ARG;
    const int64_t kv = o.kv_heads == 0 ? heads : o.kv_heads;
    if (kv < 1 || heads % kv != 0)
        return TL_ERR_INVALID_ARG;
    if (!score_values_ok(o.softmax_scale, o.score_cap, head_dim))
        return TL_ERR_INVALID_ARG;
    if ((o.causal != 0 && o.causal != 1) || o.q_offset < 0 || o.num_docs < 0)
        return TL_ERR_INVALID_ARG;
    if ((o.doc_offsets != nullptr) != (o.num_docs > 0))
        return TL_ERR_INVALID_ARG;
    if (o.prefix_lens && !o.causal)
        return TL_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128)
        return TL_ERR_UNSUPPORTED;
    if (seq_k > kMaxLength || seq_q > kMaxLength || o.q_offset > kMaxLength - seq_q || o.num_docs > kMaxLength)
        return TL_ERR_UNSUPPORTED;
    // one CTA for 128 rows at least of each head: the grid and batch * heads stay inside 31 bits
    if (batch > 0x7FFFFFFFll || heads > 0x7FFFFFFFll / batch)
        return TL_ERR_UNSUPPORTED;
    const int64_t longest = seq_q > seq_k ? seq_q : seq_k;
    if (ceil_div(longest, 64) > 0x7FFFFFFFll / (batch * heads))
        return TL_ERR_UNSUPPORTED;
    if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 16) || (lse && !aligned(lse, 4)) ||
        (o.slopes && !aligned(o.slopes, 4)) || (o.doc_offsets && !aligned(o.doc_offsets, 4)) ||
        (o.prefix_lens && !aligned(o.prefix_lens, 4)))
        return TL_ERR_MISALIGNED;
    const int64_t sq[3] = {batch, heads, seq_q}, sk[3] = {batch, kv, seq_k};
    tl_status st;
    if ((st = take_strides(o.q_strides, sq, head_dim, &c->q)) != TL_OK ||
        (st = take_strides(o.k_strides, sk, head_dim, &c->k)) != TL_OK ||
        (st = take_strides(o.v_strides, sk, head_dim, &c->v)) != TL_OK ||
        (st = take_strides(o.o_strides, sq, head_dim, &c->o)) != TL_OK)
        return st;
    c->batch = batch;
    c->heads = heads;
    c->kv_heads = kv;
    c->seq_q = seq_q;
    c->seq_k = seq_k;
    c->head_dim = head_dim;
    c->dtype = dtype;
    c->scale = softmax_scale(o.softmax_scale, head_dim);
    c->cap = o.score_cap;
    c->slopes = o.slopes;
    c->mask = MaskParams{};
    c->mask.Sq = static_cast<int32_t>(seq_q);
    c->mask.Sk = static_cast<int32_t>(seq_k);
    c->mask.q_offset = static_cast<int32_t>(o.q_offset);
    c->mask.causal = o.causal;
    c->mask.doc_offsets = o.doc_offsets;
    c->mask.num_docs = static_cast<int32_t>(o.num_docs);
    c->mask.prefix = o.prefix_lens;
    return TL_OK;
}

namespace {

using ExFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, AttnExParams);

using JoinFn = void (*)(AttnJoinParams);

struct ExEntry {
    ExFn fn[2][2][2];  // [dtype][capped][biased]
    JoinFn join[2];    // [dtype]
    int smem, threads, launch_regs;
};

template <int D>
ExEntry make_ex()
{
    using CF = AttnExConfig<D>;
    return {{{{attention_ex_kernel<CF, 0, false, false>, attention_ex_kernel<CF, 0, false, true>},
              {attention_ex_kernel<CF, 0, true, false>, attention_ex_kernel<CF, 0, true, true>}},
             {{attention_ex_kernel<CF, 1, false, false>, attention_ex_kernel<CF, 1, false, true>},
              {attention_ex_kernel<CF, 1, true, false>, attention_ex_kernel<CF, 1, true, true>}}},
            {attention_join_kernel<0, D>, attention_join_kernel<1, D>},
            CF::SMEM_BYTES, CF::THREADS, CF::LAUNCH_REGS};
}

const ExEntry kEx64 = make_ex<64>();
const ExEntry kEx128 = make_ex<128>();

tl_status attention_ex_impl(const void *Q, const void *K, const void *V, void *O, float *lse, int64_t batch,
                            int64_t heads, int64_t seq_q, int64_t seq_k, int64_t head_dim, int dtype,
                            cudaStream_t stream, const tl_attention_options *opt)
{
    AttentionCall c;
    tl_status st = attention_call(Q, K, V, O, lse, batch, heads, seq_q, seq_k, head_dim, dtype, opt, &c);
    if (st != TL_OK)
        return st;
    DeviceState *d = nullptr;
    if ((st = device_state(&d)) != TL_OK)
        return st;
    if (d->cc_major != 10)
        return TL_ERR_UNSUPPORTED;
    const ExEntry &e = head_dim == 64 ? kEx64 : kEx128;
    ExFn fn = e.fn[dtype][c.cap > 0.0f][c.slopes != nullptr];
    if ((st = ready_kernel(d, fn, e.smem, e.launch_regs)) != TL_OK)
        return st;
    CUtensorMap tq, tk, tv, to;
    if (!encode_heads(&tq, Q, dtype, batch, heads, seq_q, head_dim, c.q, 128) ||
        !encode_heads(&tk, K, dtype, batch, c.kv_heads, seq_k, head_dim, c.k, 128) ||
        !encode_heads(&tv, V, dtype, batch, c.kv_heads, seq_k, head_dim, c.v, 128) ||
        !encode_heads_out(&to, O, dtype, batch, heads, seq_q, head_dim, c.o, 32, 32))
        return TL_ERR_CUDA;
    AttnExParams p{};
    p.mask = c.mask;
    p.score = score_params(c.scale, c.cap, c.slopes);
    p.B = static_cast<int32_t>(batch);
    p.H = static_cast<int32_t>(heads);
    p.group = static_cast<int32_t>(heads / c.kv_heads);
    p.num_pairs = static_cast<int32_t>(ceil_div(seq_q, 256));
    p.lse = lse;
    p.timeout_ns = kDefaultTimeoutNs;
    const int64_t items = p.num_pairs * batch * heads;
    // Split the keys where at most half the SMs would have an item and the longest has four blocks at least: a block
    // takes a CTA about 2 us, the joining of the splits about 4 (measured: 8 items of 9 blocks 30 -> 15 us; with one
    // item to two SMs and 4 blocks both ways take the same time).  Causal items differ in length and the longest decides
    // as long as there is one SM for each: two splits then (measured: 96 items of up to 8 blocks 31 -> 27 us).
    const int64_t blocks = ceil_div(seq_k, 128);
    p.splits = 1;
    if (2 * items <= d->num_sms && blocks >= 4) {
        const int64_t most = d->num_sms / items;
        p.splits = static_cast<int32_t>(most < blocks ? most : blocks);
    } else if (items <= d->num_sms && c.mask.causal && blocks >= 8) {
        p.splits = 2;
    }
    if (p.splits == 1)
        return launch_overlapped(fn, items, e.threads, e.smem, stream, tq, tk, tv, to, p);
    const int64_t slots = items * p.splits * 2;
    const int64_t o_bytes = slots * head_dim * 128 * 4;
    if ((st = ensure_pool(d)) != TL_OK)
        return st;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(o_bytes + slots * 128 * 8), d->pool, stream) != cudaSuccess)
        return TL_ERR_CUDA;
    p.part_o = static_cast<float4 *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + o_bytes);
    AttnJoinParams j{};
    j.H = p.H;
    j.Sq = c.mask.Sq;
    j.num_pairs = p.num_pairs;
    j.BH = static_cast<int32_t>(batch * heads);
    j.splits = p.splits;
    j.causal = c.mask.causal;
    j.part_o = p.part_o;
    j.part_ml = p.part_ml;
    j.O = static_cast<uint16_t *>(O);
    j.o_batch = c.o.s[0];
    j.o_head = c.o.s[1];
    j.o_row = c.o.s[2];
    j.lse = lse;
    st = launch_overlapped(fn, items * p.splits, e.threads, e.smem, stream, tq, tk, tv, to, p);
    if (st == TL_OK)
        st = launch_overlapped(e.join[dtype], items * 8, 256, 0, stream, j);
    if (cudaFreeAsync(ws, stream) != cudaSuccess && st == TL_OK)
        st = TL_ERR_CUDA;
    return st;
}

} // namespace

bool take_error_attention_ex(unsigned int *word) { return take_device_error(word); }

} // namespace tl

extern "C" tl_status tl_attention_ex(const void *Q, const void *K, const void *V, void *O, float *lse, int64_t batch,
                                     int64_t heads, int64_t seq_q, int64_t seq_k, int64_t head_dim, tl_dtype dtype,
                                     tl_stream stream, const tl_attention_options *options)
{
    return tl::attention_ex_impl(Q, K, V, O, lse, batch, heads, seq_q, seq_k, head_dim, dtype,
                                 static_cast<cudaStream_t>(stream), options);
}
