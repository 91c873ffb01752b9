// attention_common.cuh -- what the masked attention kernels share: 4- and 5-D
// TMA loads, the interval of keys a query sees, and the score's capping and
// distance bias.
//
// With a = q . k and p_i = q_offset + i (the place of query i among the keys),
//
//   u_ij = scale a                          or   cap tanh(scale a / cap)
//   y_ij = u_ij - slope_h |p_i - j|
//
// and query i sees the keys lo_i <= j < hi_i: documents cut [0, seq_k) at
// their offsets, a causal query sees nothing after p_i, and a prefix opens the
// first keys of its document to everyone in it.  All three masks together are
// one interval a query, which is why no mask is read for each score.
#pragma once

#include "device_common.cuh"
#include "sm100.cuh"

namespace tl {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// 4-D tiled store shared -> global, tracked by the issuing thread's bulk groups;
// what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z,
                                             int32_t w)
{
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w, int32_t v)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns: thread t gets, or writes, lane (base + t)
__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_store_16cols(uint32_t taddr, const uint32_t (&r)[N])
{
    static_assert(N >= 16, "registers");
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// min that keeps a NaN
__device__ __forceinline__ float fmin_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct MaskParams {
    int32_t Sq, Sk, q_offset, causal;
    const int32_t *doc_offsets;  // [batch][num_docs + 1], or null
    int32_t num_docs;
    const int32_t *prefix;       // [batch][max(num_docs, 1)], or null
};

// Document offsets kept in shared memory while rows look theirs up
constexpr int kDocsInSmem = 512;

// The last document that begins at or before `pos` (empty documents end where they begin), or -1
__device__ __forceinline__ int last_document(const MaskParams &m, const int32_t *docs, int pos)
{
    int a = 0, n = m.num_docs;
    while (a < n) {
        const int mid = (a + n) >> 1;
        if (docs[mid] <= pos)
            a = mid + 1;
        else
            n = mid;
    }
    return a - 1;
}

// The keys query row `i` of batch entry `b` sees, [x, y); empty for rows past
// the queries or outside every document.  `docs` are the batch entry's
// offsets (shared or global memory).  Offsets out of order or out of range
// give some interval inside [0, Sk], never an access outside it.
__device__ __forceinline__ int2 visible_keys(const MaskParams &m, const int32_t *docs, int b, int i)
{
    if (i >= m.Sq)
        return make_int2(0, 0);
    const int pos = m.q_offset + i;
    int lo = 0, hi = m.Sk, d = 0;
    if (m.doc_offsets) {
        d = last_document(m, docs, pos);
        if (d < 0)
            return make_int2(0, 0);
        lo = docs[d];
        hi = docs[d + 1];
        if (pos >= hi)
            return make_int2(0, 0);
    }
    if (m.causal) {
        int64_t last = static_cast<int64_t>(pos) + 1;
        if (m.prefix) {
            const int64_t open = static_cast<int64_t>(lo) +
                                 m.prefix[static_cast<int64_t>(b) * max(m.num_docs, 1) + d];
            last = open > last ? open : last;
        }
        hi = static_cast<int>(last < hi ? last : hi);
    }
    lo = max(lo, 0);
    hi = min(hi, m.Sk);
    return hi > lo ? make_int2(lo, hi) : make_int2(0, 0);
}

// Whether some query sees key `j` of batch entry `b`: its document (the sequence) has queries and, causal, one of
// them stands at or behind the key, or the prefix reaches it.
__device__ __forceinline__ bool key_is_seen(const MaskParams &m, const int32_t *docs, int b, int j)
{
    if (j >= m.Sk)
        return false;
    int first = m.q_offset, end = m.q_offset + m.Sq, lo = 0, d = 0;  // the queries' places
    if (m.doc_offsets) {
        d = last_document(m, docs, j);
        if (d < 0 || j >= docs[d + 1])
            return false;
        lo = docs[d];
        first = max(first, lo);
        end = min(end, docs[d + 1]);
    }
    if (end <= first)
        return false;
    return !m.causal || j < end ||
           (m.prefix && j < static_cast<int64_t>(lo) + m.prefix[static_cast<int64_t>(b) * max(m.num_docs, 1) + d]);
}

struct ScoreParams {
    float scale_log2;  // scale * log2(e)
    float cap_arg;     // scale / cap
    float cap_log2;    // cap * log2(e)
    const float *slopes;  // [heads], or null
};

// t = x p(x^2) of N scores in place, p of degree M - 1 with coefficients c, x = arg v
template <int N, int M>
__device__ __forceinline__ void odd_polynomial(uint32_t *v, float arg, const float (&c)[M])
{
    float2 k[M];  // coefficients in powers of the raw score: c_i arg^(2 i + 1)
    float power = arg;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        k[i] = splat2(c[i] * power);
        power *= arg * arg;
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 x = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        const float2 u = fmul2(x, x);
        float2 t = ffma2(u, k[M - 1], k[M - 2]);
#pragma unroll
        for (int i = M - 3; i >= 0; --i)
            t = ffma2(u, t, k[i]);
        t = fmul2(t, x);
        v[e] = __float_as_uint(t.x);
        v[e + 1] = __float_as_uint(t.y);
    }
}

// The N raw scores v to tanh(arg v), in place, N a multiple of 4; arg > 0.
//
// Where the warp's |arg v| are all at most 1/2 -- scores well inside the cap, the
// usual case -- or at most 1, tanh x = x p(x^2) with p of degree 4 or 6, the
// minimax fits of csrc/fit_tanh.py (relative errors 1.3e-8 and 5e-8): 3 or 4
// multiply-adds a score, two to an instruction, and no special-function
// operation.  Otherwise tanh x = 1 - 2 / (1 + 2^(2 log2(e) x)), one 2^x a score and
// one reciprocal for two, of the product of their denominators; the exponent is
// held below 2^60 (tanh is 1 to 2^-59 there) so that the product stays finite.  All
// are absolutely exact to about 2^-22, which is what a score needs: a cap of 50
// leaves 1e-5.  (The polynomials' coefficients hold arg^13 at most: they are left to
// arg <= 64, far above any cap in use, and where arg^13 underflows tanh x = x,
// which the vanishing coefficients give.)
//
// The forms differ by 2^-22, so lanes whose scores belong to no row pass `counts`
// false and have no say in the choice: what they hold must not reach the others.
template <int N>
__device__ __forceinline__ void tanh_scores(uint32_t *v, float arg, bool counts = true)
{
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < N; e += 2)
        top = fmax3(top, fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
    top = !counts ? 0.0f : arg <= 64.0f ? top * arg : INFINITY;
    if (__all_sync(0xffffffffu, top <= 0.5f)) {
        const float c[5] = {0.9999999869f, -0.3333306939f, 0.1332477932f, -0.05298607529f, 0.01713500663f};
        odd_polynomial<N>(v, arg, c);
    } else if (__all_sync(0xffffffffu, top <= 1.0f)) {
        const float c[7] = {0.9999999502f, -0.3333283915f, 0.1332520408f, -0.05345702957f, 0.02028998043f,
                            -0.006203379112f, 0.001041022636f};
        odd_polynomial<N>(v, arg, c);
    } else {
        const float2 arg2 = splat2(2.8853900817779268f * arg);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 z = fmul2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), arg2);
            const float2 d = fadd2(make_float2(exp2_approx_ftz(fmin_nan(z.x, 60.0f)), exp2_approx_ftz(fmin_nan(z.y, 60.0f))),
                                   splat2(1.0f));
            const float r = -2.0f * rcp_approx(d.x * d.y);
            const float2 t = ffma2(splat2(r), make_float2(d.y, d.x), splat2(1.0f));
            v[e] = __float_as_uint(t.x);
            v[e + 1] = __float_as_uint(t.y);
        }
    }
}

} // namespace tl
