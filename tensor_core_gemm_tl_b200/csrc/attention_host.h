// attention_host.h -- host-side helpers of the masked attention, tree attention
// and rotary entry points: stride checks, tensor maps, launches.
#pragma once

#include <cmath>

#include "host_common.h"
#include "attention_common.cuh"

namespace tl {

// Largest length or end position: a block's rounding up stays inside 32 bits
constexpr int64_t kMaxLength = 0x7FFFFFFFll - 256;

// Strides of (outer, middle, row) of a 16-bit tensor with `dim` values a row:
// all zero means contiguous in that order.  A dimension of one element takes
// any stride.
struct Strides {
    int64_t s[3];
};

inline tl_status take_strides(const int64_t given[3], const int64_t sizes[3], int64_t dim, Strides *out)
{
    const int64_t dense[3] = {sizes[1] * sizes[2] * dim, sizes[2] * dim, dim};
    const bool all_zero = given[0] == 0 && given[1] == 0 && given[2] == 0;
    for (int i = 0; i < 3; ++i) {
        int64_t v = all_zero ? dense[i] : given[i];
        if (sizes[i] == 1)
            v = dim;
        else if (v <= 0)
            return TL_ERR_INVALID_ARG;
        if (v % 8 != 0)
            return TL_ERR_MISALIGNED;
        if (v >= (1ll << 39))
            return TL_ERR_UNSUPPORTED;
        out->s[i] = v;
    }
    return TL_OK;
}

// 16-bit tensor of `rank` dimensions (innermost first; strides in elements of
// dimensions 1..rank-1), 128-byte swizzle or none; what lies outside reads as zero.
inline bool encode_rows(CUtensorMap *map, const void *base, int dtype, int rank, const int64_t *dims,
                        const int64_t *strides, const int *box, bool swizzle = true)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t d[5], s[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        bx[i] = static_cast<cuuint32_t>(box[i]);
        es[i] = 1;
        if (i > 0)
            s[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
    }
    const CUtensorMapDataType dt = dtype == TL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(map, dt, static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, s, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (batch, heads, rows, dim) as a 4-D map whose box is 64 values of `box_rows` rows
inline bool encode_heads(CUtensorMap *map, const void *base, int dtype, int64_t batch, int64_t heads, int64_t rows,
                         int64_t dim, const Strides &st, int box_rows)
{
    const int64_t dims[4] = {dim, rows, heads, batch};
    const int64_t strides[3] = {st.s[2], st.s[1], st.s[0]};
    const int box[4] = {64, box_rows, 1, 1};
    return encode_rows(map, base, dtype, 4, dims, strides, box);
}

// The same tensor for stores of `box_cols` values of `box_rows` rows, rows side by side in shared memory
inline bool encode_heads_out(CUtensorMap *map, const void *base, int dtype, int64_t batch, int64_t heads, int64_t rows,
                             int64_t dim, const Strides &st, int box_rows, int box_cols)
{
    const int64_t dims[4] = {dim, rows, heads, batch};
    const int64_t strides[3] = {st.s[2], st.s[1], st.s[0]};
    const int box[4] = {box_cols, box_rows, 1, 1};
    return encode_rows(map, base, dtype, 4, dims, strides, box, false);
}

// A launch whose set-up may overlap the previous kernel on the stream (the
// kernels wait for it before they read global memory).
template <class... P, class... A>
tl_status launch_overlapped(void (*fn)(P...), int64_t grid, int threads, int smem, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...) != cudaSuccess)
        return TL_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ERR_CUDA;
}

// What a warp-specialised kernel needs once per device: its shared-memory
// limit, and enough registers a thread at launch for its warpgroups' split.
template <class Fn>
tl_status ready_kernel(DeviceState *d, Fn fn, int smem, int launch_regs)
{
    const void *f = reinterpret_cast<const void *>(fn);
    if (smem_limit_raised(d, f))  // done before, the registers included
        return TL_OK;
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess)
        return TL_ERR_CUDA;
    if (fa.numRegs < launch_regs)
        return TL_ERR_UNSUPPORTED;
    return raise_smem_limit(d, f, smem);
}

// The scale of a call: the given one, or 1 / sqrt(head_dim) for 0
inline float softmax_scale(float given, int64_t head_dim)
{
    return given > 0.0f ? given : 1.0f / sqrtf(static_cast<float>(head_dim));
}

inline bool score_values_ok(float scale, float cap, int64_t head_dim)
{
    // both are held in fp32 times log2 e, and so is scale / cap, times 2 log2 e
    if (!(scale >= 0.0f && scale < 1e38f && cap >= 0.0f && cap < 1e38f))
        return false;
    const float ratio = softmax_scale(scale, head_dim) / cap;
    return cap == 0.0f || (cap > 1e-30f && ratio > 1e-37f && ratio < 1e38f);
}

inline ScoreParams score_params(float scale, float cap, const float *slopes)
{
    ScoreParams s{};
    s.scale_log2 = scale * 1.4426950408889634f;
    s.cap_arg = cap > 0.0f ? scale / cap : 0.0f;
    s.cap_log2 = cap * 1.4426950408889634f;
    s.slopes = slopes;
    return s;
}

// Arguments that the masked forward and its backward share
struct AttentionCall {
    int64_t batch, heads, kv_heads, seq_q, seq_k, head_dim;
    int dtype;
    float scale, cap;
    const float *slopes;
    MaskParams mask;
    Strides q, k, v, o;
};

// Checks them and fills `c`; `opt` may be null
tl_status attention_call(const void *Q, const void *K, const void *V, const void *O, const float *lse, int64_t batch,
                         int64_t heads, int64_t seq_q, int64_t seq_k, int64_t head_dim, int dtype,
                         const tl_attention_options *opt, AttentionCall *c);

} // namespace tl
