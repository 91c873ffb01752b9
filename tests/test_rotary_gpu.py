"""Rotary positions on the GPU against the 64-bit form: both layouts, part of the
head, strided and odd tensors, far positions, the inverse."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import close, rotate  # noqa: E402


def bound(x, want, inv_freq, scale):
    """One rounding of the result; before it fp32: two products and a sum (3 2^-24 of
    |a| + |b|), cos and sin off by 2^-23 and by the angle's rounding to fp32 (pi 2^-25)."""
    n = 2 * inv_freq.shape[0]
    size = x.double().abs()[..., :n].amax(-1, keepdim=True)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 1e-38
    return torch.finfo(x.dtype).eps / 2 * want.abs() * (1 + 2.0 ** -6) + scale * size * 2.0 ** -20 + tiny


def draw(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dt)


CASES = [
    # batch, seq, heads, kv heads, head_dim, rotated
    (2, 33, 4, 2, 128, 128),
    (1, 1, 1, 1, 64, 64),
    (3, 17, 5, 1, 128, 96),
    (2, 9, 3, 3, 64, 16),
    (2, 9, 3, 3, 64, 2),
    (1, 40, 2, 1, 80, 74),
    (2, 5, 2, 2, 7, 6),
    (1, 300, 32, 8, 128, 64),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("n", range(len(CASES)))
def test_rotary(n, interleaved, inverse, dt):
    import tensor_core_gemm_tl_b200 as tg
    B, S, H, Hk, D, rot = CASES[n]
    qkv = draw((B, S, H + 2 * Hk, D), dt, n)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    inv_freq, _ = tg.rotary_frequencies(rot, device="cuda")
    far = [0, 5000, 1000003][n % 3]
    pos = torch.arange(S, device="cuda", dtype=[torch.int32, torch.int64][n % 2]) + far
    pos = pos if n % 2 else (pos + 7 * torch.arange(B, device="cuda", dtype=pos.dtype)[:, None]).contiguous()
    oq, ok = tg.rotary(q, k, pos, inv_freq, interleaved=interleaved, inverse=inverse, scale=1.25)
    full = pos.expand(B, S)
    for name, x, y in (("q", q, oq), ("k", k, ok)):
        want = rotate(x, full, inv_freq, interleaved, 1.25, inverse)
        close(name, y, want, bound(x, want, inv_freq, 1.25))
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_in_place_alone_and_strided_outputs():
    import tensor_core_gemm_tl_b200 as tg
    q, k = draw((2, 4, 50, 64), torch.bfloat16, 1), draw((2, 2, 50, 64), torch.bfloat16, 2)
    inv_freq, _ = tg.rotary_frequencies(64, device="cuda")
    pos = torch.arange(50, device="cuda")
    oq, ok = tg.rotary(q, k, pos, inv_freq)
    alone, none = tg.rotary(q, None, pos, inv_freq)
    assert none is None and torch.equal(alone, oq)
    big = torch.zeros((2, 50, 9, 64), device="cuda", dtype=torch.bfloat16)
    tg.rotary(q, k, pos, inv_freq, out_q=big[:, :, :4].transpose(1, 2), out_k=big[:, :, 5:7].transpose(1, 2))
    assert torch.equal(big[:, :, :4].transpose(1, 2), oq) and torch.equal(big[:, :, 5:7].transpose(1, 2), ok)
    assert (big[:, :, 4] == 0).all() and (big[:, :, 7:] == 0).all()
    # a base off the 16-byte boundary, rows at an odd stride: element by element, the same values
    odd = torch.empty((2, 4, 50, 67), device="cuda", dtype=torch.bfloat16)[..., 1:65]
    odd.copy_(q)
    assert torch.equal(tg.rotary(odd, None, pos, inv_freq)[0], oq)
    q1, k1 = q.clone(), k.clone()
    tg.rotary(q1, k1, pos, inv_freq, out_q=q1, out_k=k1)
    assert torch.equal(q1, oq) and torch.equal(k1, ok)


def test_the_inverse_undoes_and_is_the_gradient():
    import tensor_core_gemm_tl_b200 as tg
    x, g = draw((1, 3, 200, 128), torch.bfloat16, 3), draw((1, 3, 200, 128), torch.bfloat16, 4)
    inv_freq, _ = tg.rotary_frequencies(128, base=500000.0, device="cuda")
    pos = torch.arange(200, device="cuda") + 70000
    y, _ = tg.rotary(x, None, pos, inv_freq)
    back, _ = tg.rotary(y, None, pos, inv_freq, inverse=True)
    # two roundings of values no larger than the pair's norm
    assert (back - x).abs().max() <= 2 * 2.0 ** -8 * 2 ** 0.5 * x.abs().max()
    # <rotate(d), g> = <d, inverse(g)> in 64 bits, and by differences, the map being linear
    gx, _ = tg.rotary(g, None, pos, inv_freq, inverse=True)
    d = torch.randn(x.shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(5))
    diff = (rotate(x.double() + d, pos[None], inv_freq) - rotate(x.double() - d, pos[None], inv_freq)) / 2
    lhs, rhs = (diff * g.double()).sum(), (d * gx.double()).sum()
    want = rotate(g, pos[None], inv_freq, inverse=True)
    assert abs(lhs - rhs) <= (bound(g, want, inv_freq, 1.0) * d.abs()).sum()


@pytest.mark.parametrize("first", [(1 << 24) - 3, (1 << 31) - 6])
def test_far_positions(first):
    import tensor_core_gemm_tl_b200 as tg
    x = draw((1, 1, 5, 64), torch.float16, 6)
    inv_freq, _ = tg.rotary_frequencies(64, device="cuda")
    pos = torch.arange(5, device="cuda", dtype=torch.int64) + first
    y, _ = tg.rotary(x, None, pos, inv_freq)
    want = rotate(x, pos[None], inv_freq)
    close("x", y, want, bound(x, want, inv_freq, 1.0))
