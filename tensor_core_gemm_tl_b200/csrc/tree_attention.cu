// tree_attention.cu -- host side of tl_tree_attention and tl_rotary: argument
// checks, tensor maps, the workspace and the launches.
#include "attention_host.h"
#include "rotary_kernel.cuh"
#include "tree_attention_kernel.cuh"

namespace tl {
namespace {

using TreeFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, TreeParams);
using CombineFn = void (*)(TreeParams, int);

struct TreeEntry {
    TreeFn fn[2][2][2];  // [dtype][capped][biased]
    CombineFn combine[2][2];  // [dtype][warps share a tile's pieces]
    int smem_fixed, smem_max, tile_bytes, most_slots;
};

template <int D>
TreeEntry make_tree()
{
    using CF = TreeConfig<D>;
    return {{{{tree_attention_kernel<CF, 0, false, false>, tree_attention_kernel<CF, 0, false, true>},
              {tree_attention_kernel<CF, 0, true, false>, tree_attention_kernel<CF, 0, true, true>}},
             {{tree_attention_kernel<CF, 1, false, false>, tree_attention_kernel<CF, 1, false, true>},
              {tree_attention_kernel<CF, 1, true, false>, tree_attention_kernel<CF, 1, true, true>}}},
            {{tree_combine_kernel<0, D, 1>, tree_combine_kernel<0, D, 8>},
             {tree_combine_kernel<1, D, 1>, tree_combine_kernel<1, D, 8>}},
            CF::SMEM_FIXED,
            CF::SMEM_MAX,
            CF::TILE_BYTES,
            CF::KS};
}

const TreeEntry kTree64 = make_tree<64>();
const TreeEntry kTree128 = make_tree<128>();

int gcd_int(int64_t a, int64_t b)
{
    while (b) {
        const int64_t t = a % b;
        a = b;
        b = t;
    }
    return static_cast<int>(a);
}

tl_status tree_attention_impl(const void *Q, const void *K, const void *V, const int32_t *block_table,
                              const int32_t *context, const int32_t *parents, const int32_t *tree_lens, void *O,
                              float *lse, int64_t batch, int64_t heads, int64_t kv_heads, int64_t tokens,
                              int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t head_dim, int dtype,
                              cudaStream_t stream, const tl_tree_options *opt)
{
    static const tl_tree_options none{};
    const tl_tree_options &o = opt ? *opt : none;
    if (!Q || !K || !V || !block_table || !context || !O)
        return TL_ERR_INVALID_ARG;
    if (batch < 1 || heads < 1 || kv_heads < 1 || tokens < 1 || num_pages < 1 || page_size < 1 || max_pages < 1)
        return TL_ERR_INVALID_ARG;
    if (heads % kv_heads != 0 || (dtype != TL_F16 && dtype != TL_BF16) ||
        !score_values_ok(o.softmax_scale, o.score_cap, head_dim) || o.table_stride < 0 ||
        (o.table_stride != 0 && batch > 1 && o.table_stride < max_pages))
        return TL_ERR_INVALID_ARG;
    const int64_t group = heads / kv_heads;
    if ((head_dim != 64 && head_dim != 128) || tokens > kTreeMaxTokens || batch > kTreeMaxBatch || group > 128 ||
        page_size % 8 != 0)
        return TL_ERR_UNSUPPORTED;
    if (num_pages > 0x7FFFFFFFll || page_size > kMaxLength || max_pages > kMaxLength / page_size ||
        kv_heads > 0x7FFFFFFFll / 128)
        return TL_ERR_UNSUPPORTED;
    const int64_t tile_tokens = 128 / group < tokens ? 128 / group : tokens;
    const int64_t row_tiles = ceil_div(tokens, tile_tokens);
    const int64_t units = kv_heads * row_tiles;
    // the blocks of all requests and tiles, laid end to end, count in 31 bits
    if (units > 0x7FFFFFFFll / batch || ceil_div(max_pages * page_size, 128) > 0x7FFFFFFFll / (batch * units))
        return TL_ERR_UNSUPPORTED;
    if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 16) || !aligned(block_table, 4) ||
        !aligned(context, 4) || !aligned(parents, 4) || !aligned(tree_lens, 4) || !aligned(lse, 4) ||
        !aligned(o.slopes, 4))
        return TL_ERR_MISALIGNED;
    const int64_t sq[3] = {batch, heads, tokens}, sc[3] = {num_pages, page_size, kv_heads};
    Strides q, k, v, out;
    tl_status st;
    if ((st = take_strides(o.q_strides, sq, head_dim, &q)) != TL_OK ||
        (st = take_strides(o.k_strides, sc, head_dim, &k)) != TL_OK ||
        (st = take_strides(o.v_strides, sc, head_dim, &v)) != TL_OK ||
        (st = take_strides(o.o_strides, sq, head_dim, &out)) != TL_OK)
        return st;
    DeviceState *d = nullptr;
    if ((st = device_state(&d)) != TL_OK)
        return st;
    if (d->cc_major != 10)
        return TL_ERR_UNSUPPORTED;
    const TreeEntry &e = head_dim == 64 ? kTree64 : kTree128;
    const float scale = softmax_scale(o.softmax_scale, head_dim);
    TreeFn fn = e.fn[dtype][o.score_cap > 0.0f][o.slopes != nullptr];
    if ((st = raise_smem_limit(d, reinterpret_cast<const void *>(fn), e.smem_max)) != TL_OK)
        return st;

    TreeParams p{};
    p.score = score_params(scale, o.score_cap, o.slopes);
    p.B = static_cast<int32_t>(batch);
    p.H = static_cast<int32_t>(heads);
    p.Hk = static_cast<int32_t>(kv_heads);
    p.group = static_cast<int32_t>(group);
    p.T = static_cast<int32_t>(tokens);
    p.tile_tokens = static_cast<int32_t>(tile_tokens);
    p.row_tiles = static_cast<int32_t>(row_tiles);
    p.units = static_cast<int32_t>(units);
    p.page_size = static_cast<int32_t>(page_size);
    p.box_rows = gcd_int(page_size, 128);
    p.capacity = static_cast<int32_t>(max_pages * page_size);
    p.table_row = o.table_stride ? o.table_stride : max_pages;
    p.block_table = block_table;
    p.context = context;
    p.parents = parents;
    p.tree_lens = tree_lens;
    p.O = static_cast<uint16_t *>(O);
    p.o_batch = out.s[0];
    p.o_head = out.s[1];
    p.o_row = out.s[2];
    p.lse = lse;
    p.timeout_ns = kDefaultTimeoutNs;
    // the Q tiles take what their rows need, the K and V slots as much of the rest as they can use
    p.q_bytes = static_cast<int32_t>(ceil_div(group * tile_tokens, 8) * 1024 * (head_dim / 64));
    const int fixed = e.smem_fixed + static_cast<int>(ceil_div(4 * (batch + 1), 16) * 16) + 2 * p.q_bytes;
    p.slots = (e.smem_max - fixed) / (2 * e.tile_bytes);
    p.slots = p.slots < e.most_slots ? p.slots : e.most_slots;
    const int smem = fixed + p.slots * 2 * e.tile_bytes;

    CUtensorMap tq, tk, tv;
    {
        // rows of a tile: the group's heads innermost, then the tokens
        const int64_t dims[5] = {head_dim, group, kv_heads, tokens, batch};
        const int64_t strides[4] = {q.s[1], heads == 1 ? q.s[1] : q.s[1] * group, q.s[2], q.s[0]};
        const int box[5] = {64, p.group, 1, p.tile_tokens, 1};
        if (!encode_rows(&tq, Q, dtype, 5, dims, strides, box))
            return TL_ERR_CUDA;
        const int64_t cdims[4] = {head_dim, page_size, kv_heads, num_pages};
        const int64_t ks[3] = {k.s[1], k.s[2], k.s[0]}, vs[3] = {v.s[1], v.s[2], v.s[0]};
        const int cbox[4] = {64, p.box_rows, 1, 1};
        if (!encode_rows(&tk, K, dtype, 4, cdims, ks, cbox) || !encode_rows(&tv, V, dtype, 4, cdims, vs, cbox))
            return TL_ERR_CUDA;
    }
    // one CTA an SM, fewer when the table cannot hold that many blocks
    const int64_t most = ceil_div(max_pages * page_size, 128) * batch * units;
    const int grid = static_cast<int>(most < d->num_sms ? most : d->num_sms);
    const int64_t o_bytes = 2ll * grid * 128 * head_dim * 4;
    if ((st = ensure_pool(d)) != TL_OK)
        return st;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(o_bytes + 2ll * grid * 128 * 8), d->pool, stream) != cudaSuccess)
        return TL_ERR_CUDA;
    p.part_o = static_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + o_bytes);
    st = launch_overlapped(fn, grid, 384, smem, stream, tq, tk, tv, p);
    // few tiles: many pieces each, so warps share them; with a tile an SM a tile has three pieces at most
    const int64_t rows32 = batch * units * ceil_div(tile_tokens * group, 32);
    const bool shared_pieces = batch * units * 4 <= d->num_sms;
    if (st == TL_OK)
        st = launch_overlapped(e.combine[dtype][shared_pieces], rows32 * (shared_pieces ? 8 : 1), 256, 0, stream, p, grid);
    if (cudaFreeAsync(ws, stream) != cudaSuccess && st == TL_OK)
        st = TL_ERR_CUDA;
    return st;
}

// ------------------------------------------------------------------ rotary positions
// Strides in elements; any positive ones (a dimension of one element: any)
tl_status plain_strides(const int64_t given[3], int64_t batch, int64_t heads, int64_t seq, int64_t dim, int64_t out[3])
{
    const int64_t sizes[3] = {batch, heads, seq}, dense[3] = {heads * seq * dim, seq * dim, dim};
    const bool all_zero = given[0] == 0 && given[1] == 0 && given[2] == 0;
    for (int i = 0; i < 3; ++i) {
        out[i] = all_zero ? dense[i] : given[i];
        if (sizes[i] == 1)
            out[i] = 0;
        else if (out[i] <= 0)
            return TL_ERR_INVALID_ARG;
    }
    return TL_OK;
}

tl_status rotary_impl(const void *Q, const void *K, void *Qout, void *Kout, const void *positions,
                      const float *inv_freq, int64_t batch, int64_t heads, int64_t kv_heads, int64_t seq,
                      int64_t head_dim, int64_t rot_dim, int dtype, cudaStream_t stream, const tl_rotary_options *opt)
{
    static const tl_rotary_options none{};
    const tl_rotary_options &o = opt ? *opt : none;
    if (!Q || !Qout || !positions || !inv_freq || (K == nullptr) != (Kout == nullptr))
        return TL_ERR_INVALID_ARG;
    if (batch < 1 || heads < 1 || seq < 1 || head_dim < 2 || (K ? kv_heads < 1 : kv_heads != 0))
        return TL_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim || (dtype != TL_F16 && dtype != TL_BF16))
        return TL_ERR_INVALID_ARG;
    if ((o.interleaved != 0 && o.interleaved != 1) || (o.inverse != 0 && o.inverse != 1) ||
        (o.positions_int64 != 0 && o.positions_int64 != 1) || (o.positions_shared != 0 && o.positions_shared != 1) ||
        !(o.scale >= 0.0f && o.scale < INFINITY))
        return TL_ERR_INVALID_ARG;
    const int64_t lim = 0x7FFFFFFFll;
    if (head_dim > 1024 || batch > lim || seq > lim / batch || heads > 65536 || kv_heads > 65536)
        return TL_ERR_UNSUPPORTED;
    if (!aligned(Q, 2) || !aligned(K, 2) || !aligned(Qout, 2) || !aligned(Kout, 2) || !aligned(inv_freq, 4) ||
        !aligned(positions, o.positions_int64 ? 8 : 4))
        return TL_ERR_MISALIGNED;
    RotaryParams p{};
    tl_status st;
    if ((st = plain_strides(o.q_strides, batch, heads, seq, head_dim, p.t[0].xs)) != TL_OK ||
        (st = plain_strides(o.qout_strides, batch, heads, seq, head_dim, p.t[0].ys)) != TL_OK)
        return st;
    p.t[0].x = static_cast<const uint16_t *>(Q);
    p.t[0].y = static_cast<uint16_t *>(Qout);
    p.t[0].heads = static_cast<int32_t>(heads);
    if (K) {
        if ((st = plain_strides(o.k_strides, batch, kv_heads, seq, head_dim, p.t[1].xs)) != TL_OK ||
            (st = plain_strides(o.kout_strides, batch, kv_heads, seq, head_dim, p.t[1].ys)) != TL_OK)
            return st;
        p.t[1].x = static_cast<const uint16_t *>(K);
        p.t[1].y = static_cast<uint16_t *>(Kout);
        p.t[1].heads = static_cast<int32_t>(kv_heads);
    }
    DeviceState *d = nullptr;
    if ((st = device_state(&d)) != TL_OK)
        return st;
    bool vec = head_dim % 8 == 0 && rot_dim % (o.interleaved ? 8 : 16) == 0;
    for (int i = 0; i < (K ? 2 : 1); ++i) {
        vec = vec && aligned(p.t[i].x, 16) && aligned(p.t[i].y, 16);
        for (int j = 0; j < 3; ++j)
            vec = vec && p.t[i].xs[j] % 8 == 0 && p.t[i].ys[j] % 8 == 0;
    }
    p.B = static_cast<int32_t>(batch);
    p.S = static_cast<int32_t>(seq);
    p.D = static_cast<int32_t>(head_dim);
    p.rot = static_cast<int32_t>(rot_dim);
    p.interleaved = o.interleaved;
    p.inverse = o.inverse;
    p.positions = positions;
    p.pos_batch = o.positions_shared ? 0 : seq;
    p.pos64 = o.positions_int64;
    p.inv_freq = inv_freq;
    p.scale = o.scale > 0.0f ? o.scale : 1.0f;
    // a warp a token; where tokens are few, up to eight, each with part of the heads
    const int items = vec ? static_cast<int>((o.interleaved ? rot_dim / 8 : rot_dim / 16) + (head_dim - rot_dim) / 8)
                          : static_cast<int>(rot_dim / 2 + head_dim - rot_dim);
    const int64_t goes = ceil_div(heads + kv_heads, items < 32 ? 32 / items : 1);  // of a warp alone over a token's heads
    int wpt = 1;
    while (wpt < 8 && 2 * wpt <= goes && batch * seq * wpt < 8 * static_cast<int64_t>(d->num_sms))
        wpt *= 2;
    p.warps_per_token = wpt;
    const int64_t grid = ceil_div(batch * seq * wpt, 8);
    const int smem = 8 * static_cast<int>((rot_dim / 2 + 1) / 2 * 2) * 8;
    if (vec)
        return launch_overlapped(dtype == TL_BF16 ? rotary_kernel<1, true> : rotary_kernel<0, true>, grid, 256, smem,
                                 stream, p);
    return launch_overlapped(dtype == TL_BF16 ? rotary_kernel<1, false> : rotary_kernel<0, false>, grid, 256, smem,
                             stream, p);
}

} // namespace

bool take_error_tree_attention(unsigned int *word) { return take_device_error(word); }

} // namespace tl

extern "C" {

tl_status tl_tree_attention(const void *Q, const void *K_cache, const void *V_cache, const int32_t *block_table,
                            const int32_t *context_lens, const int32_t *parents, const int32_t *tree_lens, void *O,
                            float *lse, int64_t batch, int64_t heads, int64_t kv_heads, int64_t tokens,
                            int64_t num_pages, int64_t page_size, int64_t max_pages, int64_t head_dim, tl_dtype dtype,
                            tl_stream stream, const tl_tree_options *options)
{
    return tl::tree_attention_impl(Q, K_cache, V_cache, block_table, context_lens, parents, tree_lens, O, lse, batch,
                                   heads, kv_heads, tokens, num_pages, page_size, max_pages, head_dim, dtype,
                                   static_cast<cudaStream_t>(stream), options);
}

tl_status tl_rotary(const void *Q, const void *K, void *Q_out, void *K_out, const void *positions,
                    const float *inv_freq, int64_t batch, int64_t heads, int64_t kv_heads, int64_t seq,
                    int64_t head_dim, int64_t rot_dim, tl_dtype dtype, tl_stream stream,
                    const tl_rotary_options *options)
{
    return tl::rotary_impl(Q, K, Q_out, K_out, positions, inv_freq, batch, heads, kv_heads, seq, head_dim, rot_dim,
                           dtype, static_cast<cudaStream_t>(stream), options);
}

} // extern "C"
