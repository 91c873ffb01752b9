"""Masked attention and its backward on the GPU against the plain 64-bit form:
caps, bias, causal / document / prefix masks, shared heads, strides, odd sizes,
rows that see nothing; streams, graphs, repeated runs."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import Plain, close, visible  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def tensors(B, H, Hk, Sq, Sk, D, dt, seed, q_scale=1.0, rows_first=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(h, s, f=1.0):
        if rows_first:
            return (torch.randn((B, s, h, D), generator=g, device="cuda") * f).to(DT[dt]).transpose(1, 2)
        return (torch.randn((B, h, s, D), generator=g, device="cuda") * f).to(DT[dt])

    return t(H, Sq, q_scale), t(Hk, Sk), t(Hk, Sk), t(H, Sq)


def problem(c, dt, seed=0):
    B, H, Hk, Sq, Sk, D = c["shape"]
    q, k, v, do = tensors(B, H, Hk, Sq, Sk, D, dt, seed, c.get("q_scale", 1.0), c.get("rows_first", False))
    off = c.get("offset", 0)
    how = dict(causal=c.get("causal", False), score_cap=c.get("cap", 0.0), q_offset=off)
    slopes = None
    if c.get("bias"):
        slopes = torch.pow(2.0, -torch.arange(1, H + 1, device="cuda", dtype=torch.float32) * 8 / H)
        how["slopes"] = slopes
    if "docs" in c:
        how["doc_offsets"] = torch.tensor(c["docs"], dtype=torch.int32, device="cuda")
    if "prefix" in c:
        how["prefix"] = torch.tensor(c["prefix"], dtype=torch.int32, device="cuda")
    see = visible(B, Sq, Sk, how["causal"], off, c.get("docs"), c.get("prefix"))
    pos_q = (off + torch.arange(Sq, device="cuda")).expand(B, Sq)
    pos_k = torch.arange(Sk, device="cuda").expand(B, Sk)
    p = Plain(q, k, v, see, 1.0 / math.sqrt(D), how["score_cap"], slopes, pos_q, pos_k)
    return q, k, v, do, how, p


CASES = {
    # shape: batch, heads, kv heads, queries, keys, head_dim
    "one": dict(shape=(1, 1, 1, 1, 1, 64)),
    "one_query": dict(shape=(2, 4, 2, 1, 300, 128), causal=True, offset=299, cap=30.0, q_scale=4.0),
    "plain_grouped": dict(shape=(2, 6, 2, 130, 257, 64)),
    "causal_grouped": dict(shape=(1, 5, 1, 300, 300, 128), causal=True, rows_first=True),
    "capped": dict(shape=(1, 4, 2, 333, 333, 128), causal=True, cap=20.0, q_scale=6.0),
    "biased": dict(shape=(2, 3, 3, 200, 200, 64), causal=True, bias=True),
    "biased_both_ways": dict(shape=(1, 2, 1, 257, 129, 128), bias=True),
    "capped_biased": dict(shape=(1, 4, 4, 140, 140, 64), causal=True, bias=True, cap=5.0, q_scale=3.0),
    "chunk": dict(shape=(1, 4, 2, 77, 400, 128), causal=True, offset=323, rows_first=True),
    "more_queries": dict(shape=(1, 2, 2, 400, 90, 64), causal=True),
    "documents": dict(shape=(2, 2, 1, 300, 300, 128), docs=[[0, 7, 7, 135, 256, 300], [0, 1, 2, 290, 290, 295]]),
    "documents_causal": dict(shape=(2, 4, 2, 517, 517, 64), causal=True, rows_first=True,
                             docs=[[0, 128, 256, 384, 512, 517], [0, 3, 200, 201, 450, 500]]),
    # rows before the first document and behind the last see nothing; whole tiles of them too
    "documents_gap": dict(shape=(2, 2, 2, 700, 700, 64), causal=True, docs=[[300, 310, 330], [0, 0, 0]]),
    "documents_single": dict(shape=(1, 2, 1, 260, 260, 128), causal=True, docs=[list(range(261))]),
    "documents_many": dict(shape=(1, 1, 1, 650, 650, 64), docs=[[0] + list(range(20, 651))]),
    "documents_offset": dict(shape=(1, 2, 2, 60, 260, 64), causal=True, offset=190, docs=[[0, 100, 210, 240]], bias=True),
    "prefix": dict(shape=(3, 2, 1, 290, 290, 128), causal=True, prefix=[[0], [150], [1000]]),
    "prefix_documents": dict(shape=(1, 4, 2, 400, 400, 64), causal=True, docs=[[0, 150, 390]], prefix=[[40, 500]], cap=30.0,
                             bias=True, q_scale=3.0),
    # more items than SMs: CTAs go on to further items; as many as SMs, causal: two splits of each
    "many_items": dict(shape=(2, 80, 40, 270, 640, 64), causal=True, offset=370, docs=[[0, 200, 500, 630], [0, 5, 640, 640]]),
    "many_items_128": dict(shape=(1, 160, 32, 200, 300, 128), bias=True),
    "as_many_items_as_sms": dict(shape=(1, 100, 50, 150, 1100, 64), causal=True, offset=950, cap=10.0, q_scale=4.0),
    # few tiles of many blocks: the backward cuts them into pieces, along the keys for dq, the queries of all heads for
    # dk and dv; pieces that see nothing of a document, rows that see one key or none
    "pieces_of_keys": dict(shape=(1, 2, 1, 300, 2300, 128), causal=True, offset=2000, docs=[[0, 5, 2001, 2002, 2290]], bias=True),
    "pieces_of_queries": dict(shape=(1, 6, 1, 900, 900, 64), causal=True, cap=10.0, q_scale=3.0, rows_first=True),
    "pieces_of_both": dict(shape=(2, 3, 1, 1500, 1500, 64), causal=True, docs=[[0, 1, 1400, 1490], [20, 700, 710, 1500]],
                           prefix=[[0, 900, 0], [50, 3, 2000]]),
    "pieces_all_keys": dict(shape=(1, 3, 1, 260, 2100, 128), cap=20.0, q_scale=4.0),
    "many_blocks": dict(shape=(1, 2, 1, 260, 1500, 128), causal=True, offset=1240, q_scale=3.0),
}


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name, dt):
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(CASES[name], dt, seed=len(name))
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    assert tg.check_device() == 0
    close("out", out, p.out, p.out_bound())
    close("lse", lse, p.lse, p.lse_bound())
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_gradient_against_differences(dt):
    """<gradient, direction> against central differences of the 64-bit forward."""
    import tensor_core_gemm_tl_b200 as tg
    c = CASES["prefix_documents"]
    q, k, v, do, how, p = problem(c, dt, seed=5)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    _, bounds = p.gradients(do)
    pos = torch.arange(q.shape[2], device="cuda").expand(1, -1)
    see = p.see.cpu()
    h = 1e-4
    for n, (name, g, b) in enumerate(zip(("q", "k", "v"), grads, bounds)):
        gen = torch.Generator(device="cuda").manual_seed(n)
        d = torch.randn(g.shape, generator=gen, device="cuda", dtype=torch.float64)
        loss = []
        for s in (h, -h):
            x = [t.double() for t in (q, k, v)]
            x[n] = x[n] + s * d
            f = Plain(*x, see, p.scale, p.cap, how["slopes"], pos, pos)
            loss.append((f.out.detach() * do.double()).sum())
        slope = (loss[0] - loss[1]) / (2 * h)
        # the difference is off by h^2 / 6 of the third derivative along d; scores move by about |d| |k| scale h,
        # a few percent of 1 at most here, so 1e-4 of the sum of absolute products holds it
        slack = (b * d.abs()).sum() + 1e-4 * (g.double() * d).abs().sum()
        assert abs((g.double() * d).sum() - slope) <= slack, name


@pytest.mark.parametrize("D", [64, 128])
def test_equals_the_plain_forward_without_options(D):
    """Without options attention_ex computes what attention does (the same bound)."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, _ = tensors(2, 3, 3, 260, 300, D, "bf16", 3)
    for causal in (False, True):
        see = visible(2, 260, 300, causal)
        p = Plain(q, k, v, see, 1 / math.sqrt(D))
        for f in (tg.attention, tg.attention_ex):
            close(f.__name__, f(q, k, v, causal=causal), p.out, p.out_bound())


def test_scale_strides_and_given_outputs():
    import tensor_core_gemm_tl_b200 as tg
    B, H, Hk, S, D = 2, 4, 2, 150, 64
    # q, k and v of a token side by side in one tensor, outputs inside larger ones
    qkv = torch.randn((B, S, H + 2 * Hk, D), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hk, Hk], dim=2))
    big = torch.full((B, S, H + 3, D), 5.0, device="cuda", dtype=torch.bfloat16)
    out = big[:, :, 1:1 + H].transpose(1, 2)
    lse = torch.empty((B, H, S), device="cuda")
    r = tg.attention_ex(q, k, v, causal=True, scale=0.2, out=out, lse=lse)
    assert r.data_ptr() == out.data_ptr()
    p = Plain(q, k, v, visible(B, S, S, True), 0.2)
    close("out", out, p.out, p.out_bound())
    assert (big[:, :, 0] == 5).all() and (big[:, :, 1 + H:] == 5).all()
    do = torch.randn_like(q)
    dqkv = torch.full_like(qkv, 9.0)
    dq, dk, dv = (t.transpose(1, 2) for t in dqkv.split([H, Hk, Hk], dim=2))
    tg.attention_backward(do, q, k, v, out, lse, causal=True, scale=0.2, dq=dq, dk=dk, dv=dv)
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), (dq, dk, dv), want, bounds):
        close(n, g, w, b)


@pytest.mark.parametrize("scale", [1e-6, 1.0, 3e4])
def test_gradients_of_small_and_large_losses(scale):
    """fp16 gradients far under and over 1: what the outputs can hold comes through."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(dict(shape=(1, 2, 1, 300, 300, 64), causal=True), "fp16", 2)
    v16, do = (v * 0.01).half(), (do * min(scale, 1.0)).half()
    if scale > 1:
        do, v16 = (do * 100).half(), (v * 1.0).half()
    p = Plain(q, k, v16, p.see.cpu(), p.scale)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v16, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v16, out, lse, **how)
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


@pytest.mark.parametrize("cap,scale,q_scale", [(1e-3, 1.0, 1e-4), (1e-3, 8.0, 1e-6), (2e6, 0.125, 1.0), (1e-6, 0.125, 1.0)])
def test_caps_far_from_the_scores(cap, scale, q_scale):
    """Caps thousands of times below or above what is usual, scores inside and outside them."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do = tensors(1, 2, 1, 140, 200, 64, "bf16", 9, q_scale)
    how = dict(score_cap=cap, scale=scale)
    p = Plain(q, k, v, visible(1, 140, 200, False), scale, cap)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    close("out", out, p.out, p.out_bound())
    close("lse", lse, p.lse, p.lse_bound())
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), tg.attention_backward(do, q, k, v, out, lse, **how), want, bounds):
        close(n, g, w, b)


def test_nan_stays_in_its_rows():
    """A NaN query spoils its own row, nothing else."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, _, how, p = problem(dict(shape=(1, 2, 1, 200, 200, 64), causal=True, cap=10.0), "bf16", 4)
    clean = tg.attention_ex(q, k, v, **how)
    q2 = q.clone()
    q2[0, 1, 50] = math.nan
    out = tg.attention_ex(q2, k, v, **how)
    bad = torch.isnan(out).any(-1)
    assert bad[0, 1, 50] and int(bad.sum()) == 1
    keep = ~bad
    assert torch.equal(out[keep], clean[keep])


def test_offsets_out_of_order_stay_inside():
    """Offsets and prefixes that make no sense give finite results and disturb nobody else."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do = tensors(2, 2, 2, 300, 300, 64, "bf16", 6)
    bad = torch.tensor([[250, -5, 1 << 30, -(1 << 30)], [0, 100, 200, 300]], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([[1 << 30, -7, 3], [0, 0, 0]], dtype=torch.int32, device="cuda")
    how = dict(causal=True, doc_offsets=bad, prefix=prefix)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    assert tg.check_device() == 0
    for t in (out, *grads):
        assert torch.isfinite(t).all()
    p = Plain(q[1:], k[1:], v[1:], visible(1, 300, 300, True, 0, [[0, 100, 200, 300]]), 1 / 8)
    close("out", out[1:], p.out, p.out_bound())


def test_repeats_bit_for_bit_on_busy_and_side_streams():
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, _ = problem(dict(shape=(2, 8, 2, 1000, 1000, 64), causal=True, bias=True, rows_first=True), "bf16", 7)

    def step():
        lse = torch.empty(q.shape[:3], device="cuda")
        out = tg.attention_ex(q, k, v, lse=lse, **how)
        return (out, lse, *tg.attention_backward(do, q, k, v, out, lse, **how))

    first = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = []
    for n in range(6):
        s = streams[n % 3]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            runs.append(step())
    torch.cuda.synchronize()
    assert tg.check_device() == 0
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_captured_and_replayed_with_other_values():
    import tensor_core_gemm_tl_b200 as tg
    c = dict(shape=(1, 4, 2, 300, 300, 64), causal=True, docs=[[0, 100, 250]])
    q, k, v, do, how, _ = problem(c, "fp16", 8)
    lse, out = torch.empty(q.shape[:3], device="cuda"), torch.empty_like(q)
    grads = [torch.empty_like(t) for t in (q, k, v)]

    def step():
        tg.attention_ex(q, k, v, out=out, lse=lse, **how)
        tg.attention_backward(do, q, k, v, out, lse, dq=grads[0], dk=grads[1], dv=grads[2], **how)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for n in range(3):
        q2, k2, v2, do2 = tensors(1, 4, 2, 300, 300, 64, "fp16", 20 + n)
        for a, b in zip((q, k, v, do), (q2, k2, v2, do2)):
            a.copy_(b)
        how["doc_offsets"].copy_(torch.tensor([[0, 50 + n, 299]], dtype=torch.int32))
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        p = Plain(q, k, v, visible(1, 300, 300, True, 0, [[0, 50 + n, 299]]), 1 / 8)
        close("out", out, p.out, p.out_bound())
        want, bounds = p.gradients(do)
        for name, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
            close(name, g, w, b)
    assert tg.check_device() == 0
