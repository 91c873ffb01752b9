// rotary_kernel.cuh -- rotary positions of q and k in one launch:
//
//     (a, b) -> scale (a cos f - b sin f, a sin f + b cos f),  f = +-position * inv_freq[i]
//
// over the pairs i of the first `rot` values of each head: (x_i, x_(i + rot/2))
// in the half layout, (x_2i, x_(2i+1)) interleaved; the other values pass
// through.  The negative angle is the inverse up to scale^2 and, the map being
// linear, its own backward.
//
// Bound by reading and writing q and k once.  A warp takes a token (or, where
// tokens are few, part of its heads): it works the angles out, two frequencies a
// lane, hands them round through its own shared memory and keeps those of its
// lanes' words in registers for all heads, the first heads' words already on
// their way meanwhile.  With the angles in shared memory for a whole CTA and read
// for every head the kernel issued 340 instructions for every 32 items and was
// bound by that (39 us for 16384 tokens of 20 heads of 128, 26 us of traffic; now
// 32.7 us, 0.78 of the rate of a plain copy).
// position * inv_freq is multiplied and reduced to half a turn in double (a
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
    int32_t warps_per_token;
    const void *positions;  // int32 or int64, [S] or [B][S]
    int64_t pos_batch;      // its batch stride (0: shared by the batch)
    int32_t pos64;
    const float *inv_freq;  // [rot / 2]
    float scale;
};

// (a cos - b sin, a sin + b cos), rounded the same way on every path
__device__ __forceinline__ float2 turn_pair(float a, float b, float cos, float sin)
{
    return make_float2(fmaf(a, cos, -__fmul_rn(b, sin)), fmaf(a, sin, __fmul_rn(b, cos)));
}

// Words of 16 bytes (VEC) or single values: VEC needs D, rot and the strides
// in whole words and, in the half layout, rot / 2 too.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256, 4) rotary_kernel(const RotaryParams p)
{
    extern __shared__ __align__(16) float2 turn_smem[];  // [warp][frequency]: cos, sin
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = p.rot / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    const int tok = static_cast<int>(w / p.warps_per_token);
    if (tok >= p.B * p.S)
        return;
    const int part = static_cast<int>(w - static_cast<int64_t>(tok) * p.warps_per_token);
    const int b = tok / p.S;
    const int64_t s = tok - b * p.S;
    float2 *turn = turn_smem + warp * ((n + 1) & ~1);

    // A lane keeps its item of a head (a pair of words in the half layout, a word
    // of pairs interleaved, or a word that passes through) and goes over heads; a
    // warp takes as many heads at a time as its lanes hold.  Heads of more than
    // 32 items are gone over once for every 32.
    constexpr int W = VEC ? 8 : 1, AHEAD = 2;
    const int heads = p.t[0].heads + p.t[1].heads;
    const int turned = VEC ? (p.interleaved ? p.rot / 8 : n / 8) : n;
    const int items = turned + (p.D - p.rot) / W;
    const int lanes = min(items, 32);
    const int warp_rows = 32 / lanes, sub = lane / lanes;
    const int step = warp_rows * p.warps_per_token, h0 = part * warp_rows + sub;
    const uint16_t *xq = p.t[0].x + b * p.t[0].xs[0] + s * p.t[0].xs[2];
    uint16_t *yq = p.t[0].y + b * p.t[0].ys[0] + s * p.t[0].ys[2];
    const uint16_t *xk = p.t[1].x + b * p.t[1].xs[0] + s * p.t[1].xs[2];
    uint16_t *yk = p.t[1].y + b * p.t[1].ys[0] + s * p.t[1].ys[2];
    auto lo = [](uint32_t v) { return to_float<DT>(static_cast<uint16_t>(v & 0xFFFFu)); };
    auto hi = [](uint32_t v) { return to_float<DT>(static_cast<uint16_t>(v >> 16)); };

    for (int item0 = 0; item0 < items; item0 += 32) {
        const int item = item0 + lane - sub * lanes;
        const bool turns = item < turned;
        // value offsets of the one or two words
        const int at = turns ? (!VEC && p.interleaved ? 2 * item : W * item) : p.rot + (item - turned) * W;
        const int second = !turns || (VEC && p.interleaved) ? 0 : p.interleaved ? at + 1 : at + n;
        const bool mine = sub < warp_rows && item < items && check_ok(at + W <= p.D && second + W <= p.D);
        uint4 va[AHEAD], vb[AHEAD];
        auto fetch = [&](int h, uint4 &a, uint4 &c) {
            if (!mine || h >= heads)
                return;
            const uint16_t *x = h < p.t[0].heads ? xq + h * p.t[0].xs[1] : xk + (h - p.t[0].heads) * p.t[1].xs[1];
            if constexpr (VEC) {
                a = *reinterpret_cast<const uint4 *>(x + at);
                if (second)
                    c = *reinterpret_cast<const uint4 *>(x + second);
            } else {
                a.x = x[at];
                if (second)
                    c.x = x[second];
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            fetch(h0 + i * step, va[i], vb[i]);
        if (item0 == 0) {
            const double pos = p.pos64 ? static_cast<double>(static_cast<const int64_t *>(p.positions)[b * p.pos_batch + s])
                                       : static_cast<double>(static_cast<const int32_t *>(p.positions)[b * p.pos_batch + s]);
            for (int i = lane; i < n; i += 32) {
                // whole turns go in double: what is left is exact to 2^-53 of the angle
                double t = pos * static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;
                t -= rint(t);
                float sn, cs;
                sincospif(static_cast<float>(2.0 * t), &sn, &cs);
                turn[i] = make_float2(cs * p.scale, (p.inverse ? -sn : sn) * p.scale);
            }
            __syncwarp();
        }
        float2 f[W];  // the lane's cos and sin
        if (mine && turns) {
            if constexpr (VEC) {
                const float4 *t4 = reinterpret_cast<const float4 *>(turn + (p.interleaved ? 4 * item : 8 * item));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e < 2 || !p.interleaved) {
                        const float4 v = t4[e];
                        f[2 * e] = make_float2(v.x, v.y);
                        f[2 * e + 1] = make_float2(v.z, v.w);
                    }
                }
            } else {
                f[0] = turn[item];
            }
        }
        for (int h = h0; h < heads; h += AHEAD * step) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int hh = h + i * step;
                if (!mine || hh >= heads)
                    continue;
                uint16_t *y = hh < p.t[0].heads ? yq + hh * p.t[0].ys[1] : yk + (hh - p.t[0].heads) * p.t[1].ys[1];
                uint4 a = va[i], c = vb[i];
                if constexpr (VEC) {
                    uint32_t *ua = reinterpret_cast<uint32_t *>(&a), *uc = reinterpret_cast<uint32_t *>(&c);
                    if (second) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v0 = turn_pair(lo(ua[e]), lo(uc[e]), f[2 * e].x, f[2 * e].y);
                            const float2 v1 = turn_pair(hi(ua[e]), hi(uc[e]), f[2 * e + 1].x, f[2 * e + 1].y);
                            ua[e] = pack2<DT>(v0.x, v1.x);
                            uc[e] = pack2<DT>(v0.y, v1.y);
                        }
                        *reinterpret_cast<uint4 *>(y + second) = c;
                    } else if (turns) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = turn_pair(lo(ua[e]), hi(ua[e]), f[e].x, f[e].y);
                            ua[e] = pack2<DT>(v.x, v.y);
                        }
                    }
                    *reinterpret_cast<uint4 *>(y + at) = a;
                } else {
                    uint32_t v = a.x;
                    if (second) {
                        const float2 t = turn_pair(lo(a.x), lo(c.x), f[0].x, f[0].y);
                        v = pack2<DT>(t.x, t.y);
                        y[second] = static_cast<uint16_t>(v >> 16);
                    }
                    y[at] = static_cast<uint16_t>(v & 0xFFFFu);
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                fetch(h + (AHEAD + i) * step, va[i], vb[i]);
        }
    }
}

} // namespace tl
