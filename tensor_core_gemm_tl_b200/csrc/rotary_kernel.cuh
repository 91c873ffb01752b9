// rotary_kernel.cuh -- rotary positions of q and k in one launch:
//
//     (a, b) -> scale (a cos f - b sin f, a sin f + b cos f),  f = +-position * inv_freq[i]
//
// over the pairs i of the first `rot` values of each head: (x_i, x_(i + rot/2))
// in the half layout, (x_2i, x_(2i+1)) interleaved; the other values pass
// through.  The negative angle is the inverse up to scale^2 and, the map being
// linear, its own backward.
//
// Bound by reading and writing q and k once.  The angles are taken once a token
// and frequency, not once a head: a CTA turns the positions of a few tokens
// into sines and cosines in shared memory and applies them to all their heads.
// position * inv_freq is multiplied and reduced to [-pi, pi] in double (a
// float product is off by 0.06 rad at position 10^6), the sine and cosine are
// fp32.
#pragma once

#include "device_common.cuh"

namespace tl {

struct RotaryTensor {
    const uint16_t *x;
    uint16_t *y;
    int64_t xs[3], ys[3];  // strides of batch, head, token in elements
    int32_t heads;         // 0: absent
};

struct RotaryParams {
    RotaryTensor t[2];
    int32_t B, S, D, rot;
    int32_t interleaved, inverse;
    int32_t tokens_per_cta;
    const void *positions;  // int32 or int64, [S] or [B][S]
    int64_t pos_batch;      // its batch stride (0: shared by the batch)
    int32_t pos64;
    const float *inv_freq;  // [rot / 2]
    float scale;
};

// Words of 16 bytes (VEC) or single values: VEC needs D, rot and the strides
// in whole words and, in the half layout, rot / 2 too.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryParams p)
{
    extern __shared__ float2 turn[];  // [token][frequency]: cos, sin
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = p.rot / 2;
    const int64_t total = static_cast<int64_t>(p.B) * p.S;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tokens_per_cta;
    const int toks = static_cast<int>(total - tok0 < p.tokens_per_cta ? total - tok0 : p.tokens_per_cta);
    for (int i = threadIdx.x; i < toks * n; i += 256) {
        const int64_t tok = tok0 + i / n;
        const int64_t at = tok / p.S * p.pos_batch + tok % p.S;
        const double pos = p.pos64 ? static_cast<double>(static_cast<const int64_t *>(p.positions)[at])
                                   : static_cast<double>(static_cast<const int32_t *>(p.positions)[at]);
        const double f = pos * static_cast<double>(p.inv_freq[i % n]);
        const double turns = rint(f * 0.15915494309189533577);
        // 2 pi in two parts: the product with the first is exact enough for |turns| < 2^27
        const float r = static_cast<float>(fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586232, f)));
        float s, c;
        sincosf(r, &s, &c);
        turn[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
    }
    __syncthreads();
    const int heads = p.t[0].heads + p.t[1].heads;
    constexpr int W = VEC ? 8 : 1;
    // work items of a head: pairs of words (half layout) or words of pairs, then words that pass through
    const int turned = VEC ? (p.interleaved ? p.rot / 8 : n / 8) : n;
    const int items = turned + (p.D - p.rot) / W;
    for (int i = threadIdx.x; i < toks * heads * items; i += 256) {
        const int item = i % items;
        const int th = i / items;
        const int head = th % heads, t = th / heads;
        const bool second = head >= p.t[0].heads;
        const RotaryTensor &q = p.t[second ? 1 : 0];
        const int h = second ? head - p.t[0].heads : head;
        const int64_t tok = tok0 + t;
        const int64_t b = tok / p.S, s = tok - b * p.S;
        const uint16_t *x = q.x + b * q.xs[0] + h * q.xs[1] + s * q.xs[2];
        uint16_t *y = q.y + b * q.ys[0] + h * q.ys[1] + s * q.ys[2];
        if (item >= turned) {
            const int c = p.rot + (item - turned) * W;
            if constexpr (VEC)
                *reinterpret_cast<uint4 *>(y + c) = *reinterpret_cast<const uint4 *>(x + c);
            else
                y[c] = x[c];
            continue;
        }
        const float2 *cs = turn + t * n;
        if constexpr (VEC) {
            auto lo = [](uint32_t v) { return to_float<DT>(static_cast<uint16_t>(v & 0xFFFFu)); };
            auto hi = [](uint32_t v) { return to_float<DT>(static_cast<uint16_t>(v >> 16)); };
            if (p.interleaved) {
                uint4 w = *reinterpret_cast<const uint4 *>(x + 8 * item);
                uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = cs[4 * item + e];
                    const float a = lo(u[e]), c = hi(u[e]);
                    u[e] = pack2<DT>(a * f.x - c * f.y, a * f.y + c * f.x);
                }
                *reinterpret_cast<uint4 *>(y + 8 * item) = w;
            } else {
                uint4 wa = *reinterpret_cast<const uint4 *>(x + 8 * item);
                uint4 wb = *reinterpret_cast<const uint4 *>(x + n + 8 * item);
                uint32_t *ua = reinterpret_cast<uint32_t *>(&wa), *ub = reinterpret_cast<uint32_t *>(&wb);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = cs[8 * item + 2 * e], g = cs[8 * item + 2 * e + 1];
                    const float a0 = lo(ua[e]), a1 = hi(ua[e]), b0 = lo(ub[e]), b1 = hi(ub[e]);
                    ua[e] = pack2<DT>(a0 * f.x - b0 * f.y, a1 * g.x - b1 * g.y);
                    ub[e] = pack2<DT>(a0 * f.y + b0 * f.x, a1 * g.y + b1 * g.x);
                }
                *reinterpret_cast<uint4 *>(y + 8 * item) = wa;
                *reinterpret_cast<uint4 *>(y + n + 8 * item) = wb;
            }
        } else {
            const int ia = p.interleaved ? 2 * item : item, ib = p.interleaved ? 2 * item + 1 : n + item;
            const float2 f = cs[item];
            const float a = to_float<DT>(x[ia]), c = to_float<DT>(x[ib]);
            const uint32_t w = pack2<DT>(a * f.x - c * f.y, a * f.y + c * f.x);
            y[ia] = static_cast<uint16_t>(w & 0xFFFFu);
            y[ib] = static_cast<uint16_t>(w >> 16);
        }
    }
}

} // namespace tl
