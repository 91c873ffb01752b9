"""The attention operators where their ranges end, on the GPU against the plain 64-bit
forms."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import Plain, close, rotate  # noqa: E402
from test_attention_ex_gpu import CASES, problem  # noqa: E402
from test_tree_attention_gpu import Cache  # noqa: E402

# Documents that begin at or behind the last key: their queries see nothing, those before them in the same tile do
PAST_THE_KEYS = {
    "inside_a_tile": dict(shape=(1, 2, 1, 200, 100, 64), causal=True, docs=[[0, 50, 120, 200]]),
    "at_the_end": dict(shape=(1, 2, 2, 130, 100, 128), docs=[[0, 100, 130]]),
    "several_tiles": dict(shape=(2, 2, 2, 700, 300, 128), causal=True, rows_first=True, bias=True,
                          docs=[[0, 100, 290, 310, 700], [0, 300, 301, 640, 700]]),
    "both_ways": dict(shape=(2, 4, 2, 400, 260, 64), docs=[[0, 255, 256, 280, 400], [0, 259, 260, 260, 1 << 30]]),
    "prefixes": dict(shape=(1, 2, 1, 390, 300, 64), causal=True, docs=[[0, 150, 299, 320, 390]], prefix=[[40, 500, 60, 9]]),
    # the keys of the few tiles are split over CTAs
    "split": dict(shape=(1, 1, 1, 200, 600, 128), causal=True, offset=500, docs=[[0, 550, 620, 700]], cap=20.0, q_scale=4.0),
    "none_left": dict(shape=(1, 2, 1, 140, 90, 64), docs=[[90, 140, 230]], offset=90),
}


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(PAST_THE_KEYS))
def test_documents_that_begin_past_the_keys(name, dt):
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(PAST_THE_KEYS[name], dt, seed=len(name))
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    assert tg.check_device() == 0
    close("out", out, p.out, p.out_bound())
    close("lse", lse, p.lse, p.lse_bound())
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


# ------------------------------------------------------------------ large counts
LARGE_COUNTS = {
    "heads": dict(shape=(300, 256, 128, 1, 3, 64), causal=True, offset=1),
    "a_long_context": dict(shape=(1, 2, 1, 1, 150001, 64), causal=True, offset=150000, bias=True),
    "a_long_context_128": dict(shape=(1, 3, 1, 5, 70003, 128), causal=True, offset=69998, cap=20.0, q_scale=3.0),
    "many_queries": dict(shape=(1, 2, 1, 70001, 2, 64)),
    "many_documents": dict(shape=(1, 1, 1, 6000, 6000, 64), docs=[list(range(0, 6001, 3))]),
}


@pytest.mark.parametrize("name", list(LARGE_COUNTS))
def test_large_counts(name):
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(LARGE_COUNTS[name], "bf16", seed=len(name))
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    assert tg.check_device() == 0
    close("out", out, p.out, p.out_bound())
    close("lse", lse, p.lse, p.lse_bound())
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


# ------------------------------------------------------------------ fp16 gradients
def held_gradients(p, do):
    """The gradients and bounds of `Plain`, with the step of what fp16 holds dX in.

    |dX| <= |dP - delta| <= 2 m, m = max |dO_i| max |V_j| (2-norms; O is a mean of V rows), and dX is held
    times 2^15 over the power of two above 2 m at least: half of fp16's smallest step 2^-24 is then at most
    2^-25 2^-15 4 m = 2^-38 m of dX."""
    want, (bq, bk, bv) = p.gradients(do)
    m = do.double().norm(dim=-1).amax() * p.v.detach().norm(dim=-1).amax()
    step = 2.0 ** -38 * m * (1 + 2.0 ** -6) * p.scale * p.see[:, None].double()
    bq = bq + torch.einsum("bhij,bhjd->bhid", step.expand(-1, do.shape[1], -1, -1), p.kk.detach().abs())
    by_head = torch.einsum("bhij,bhid->bhjd", step.expand(-1, do.shape[1], -1, -1), p.q.detach().abs())
    bk = bk + by_head.view(by_head.shape[0], -1, p.G, *by_head.shape[2:]).sum(2)
    return want, (bq, bk, bv)


LARGE = {
    # two values of opposite sign share the weight, gradients of a sum: dX is about 12, the sums behind it of order 1
    "a_sum": dict(shape=(1, 1, 1, 130, 2, 128), v=100.0, do=1.9e-3, even=True),
    "a_sum_64": dict(shape=(1, 2, 1, 130, 300, 64), v=100.0, do=1.9e-3, even=True, causal=True),
    "values": dict(shape=(1, 4, 2, 333, 300, 128), v=300.0, do=1e-3, causal=True),
    "small_values": dict(shape=(1, 2, 1, 200, 260, 64), v=1e-3, do=1.0, causal=True),
    "largest_values": dict(shape=(1, 2, 2, 150, 270, 64), v=15000.0, do=1e-5),
    "capped": dict(shape=(2, 2, 1, 140, 140, 128), v=500.0, do=1e-3, causal=True, cap=10.0, q_scale=3.0),
    "pieces": dict(shape=(1, 3, 1, 900, 900, 64), v=400.0, do=1e-3, causal=True, bias=True),
}


@pytest.mark.parametrize("name", list(LARGE))
def test_fp16_gradients_over_large_values(name):
    """Values far from 1: dX would leave fp16's range where the gradients do not."""
    import tensor_core_gemm_tl_b200 as tg
    c = LARGE[name]
    q, k, v, do, how, p = problem(c, "fp16", seed=3)
    if c.get("even"):
        sign = 1 - 2 * (torch.arange(v.shape[2], device="cuda") % 2)
        v = (c["v"] * sign[:, None].half()).expand_as(v).contiguous()
        do = torch.full_like(do, c["do"])
    else:
        v, do = (v.clamp(-4, 4) * c["v"]).half(), (do * c["do"]).half()
    slopes = how.get("slopes")
    at = [torch.arange(n, device="cuda").expand(q.shape[0], n) for n in (q.shape[2], k.shape[2])]
    p = Plain(q, k, v, p.see.cpu(), p.scale, p.cap, slopes, *at)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    want, bounds = held_gradients(p, do)
    assert all(w.abs().max() < 60000 for w in want)  # the gradients themselves fit
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


def test_an_infinite_gradient_spoils_its_own_query():
    """fp16 dout with an infinite and a NaN row: dq of every other query as if those rows were 0."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, _ = problem(dict(shape=(1, 2, 1, 300, 300, 64), causal=True), "fp16", seed=2)
    do = (do * 40).half()
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    do[0, 1, 50:52] = 0
    want = tg.attention_backward(do, q, k, v, out, lse, **how)[0]
    do[0, 1, 50, 3], do[0, 1, 51, 60] = math.inf, math.nan
    dq = tg.attention_backward(do, q, k, v, out, lse, **how)[0]
    bad = ~torch.isfinite(dq).all(-1)
    assert bad[0, 1, 50:52].all() and int(bad.sum()) == 2
    assert torch.equal(dq[~bad], want[~bad])


@pytest.mark.parametrize("how", [dict(docs=[[20, 150, 260]]), dict(docs=[[20, 150, 260]], causal=True),
                                 dict(docs=[[20, 21, 150, 260]], causal=True, prefix=[[0, 30, 200]]),
                                 dict(causal=True, offset=5, queries=140)])
def test_fp16_gradients_beside_rows_that_do_not_count(how):
    """Queries that see nothing and keys that nobody sees, left with large finite numbers, take nothing of the small
    gradients' precision."""
    import tensor_core_gemm_tl_b200 as tg
    how = dict(how)
    sq = how.pop("queries", 300)
    q, k, v, do, how, p = problem(dict(shape=(1, 4, 2, sq, 300, 64), **how), "fp16", seed=8)
    do = (do * 1e-3).half()
    see = p.see.cpu()
    queries, keys = see.any(2)[0].cuda(), see.any(1)[0].cuda()
    assert not (queries.all() and keys.all())
    p = Plain(q, k, v, see, p.scale)
    want, bounds = p.gradients(do * queries[:, None])
    q[:, :, ~queries], do[:, :, ~queries] = 1000.0, 60000.0
    k[:, :, ~keys], v[:, :, ~keys] = 100.0, 60000.0
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


# ------------------------------------------------------------------ tree attention
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bias", [False, True])
def test_capped_tokens_do_not_depend_on_how_many_heads_share(D, dt, bias):
    """One token of two query heads, and the same two among 32: bit for bit the same, whatever the tile's rows behind
    them hold (the first leaves 30 lanes of a warp without a row; keys far larger than the queries take those lanes'
    products past the cap, the rows' own lie well inside it)."""
    import tensor_core_gemm_tl_b200 as tg
    g = torch.Generator(device="cuda").manual_seed(D)
    for contexts in ([5, 300, 1000], [4000]):
        B, page = len(contexts), 16
        per = (max(contexts) + page) // page
        kc, vc = (torch.randn((B * per, page, 1, D), generator=g, device="cuda") * f for f in (10.0, 1.0))
        kc, vc = kc.to(dt), vc.to(dt)
        table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        context = torch.tensor(contexts, dtype=torch.int32, device="cuda")
        two = (torch.randn((B, 2, 1, D), generator=g, device="cuda") * 0.2).to(dt)
        many = two.repeat(1, 16, 1, 1)
        slopes = torch.tensor([0.01, 0.002], device="cuda")
        res = []
        for q in (two, many, two):
            lse = torch.empty(q.shape[:3], device="cuda")
            how = dict(score_cap=50.0, slopes=slopes.repeat(q.shape[1] // 2) if bias else None)
            res.append((tg.tree_attention(q, kc, vc, table, context, lse=lse, **how), lse))
        assert tg.check_device() == 0
        for out, lse in res[1:]:
            for n in range(0, out.shape[1], 2):
                assert torch.equal(out[:, n:n + 2], res[0][0]) and torch.equal(lse[:, n:n + 2], res[0][1])


def test_capped_trees_repeat_bit_for_bit():
    """Drafted trees with a cap, some rows of a warp without a token, run again and again among other calls."""
    import tensor_core_gemm_tl_b200 as tg
    g = torch.Generator(device="cuda").manual_seed(1)
    B, T, H, Hk, D, page, keys = 8, 31, 16, 4, 128, 32, 4096
    per = (keys + T + page - 1) // page
    kc, vc = (torch.randn((B * per, page, Hk, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    context = torch.randint(keys // 4, keys + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    parents = (torch.rand((B, T), generator=g, device="cuda") * (torch.arange(T, device="cuda") + 1)).to(torch.int32) - 1
    q = (torch.randn((B, T, H, D), generator=g, device="cuda") * 4).bfloat16().transpose(1, 2)
    first = None
    for n in range(12):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        tg.tree_attention(q, kc, vc, table, context, parents, tree_lens=lens, score_cap=30.0, out=out, lse=lse)
        first = (out, lse) if first is None else first
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), n
        tg.tree_attention((q * (n % 3)).contiguous(), vc, kc, table, context, score_cap=3.0)  # other bytes in shared memory
    assert tg.check_device() == 0


@pytest.mark.parametrize("tokens,lens", [(1, False), (3, True)])
def test_as_many_requests_as_are_allowed(tokens, lens):
    import tensor_core_gemm_tl_b200 as tg
    B = 4096
    g = torch.Generator().manual_seed(tokens)
    contexts = torch.randint(0, 300, (B,), generator=g).tolist()
    live = torch.randint(0, tokens + 1, (B,), generator=g).tolist() if lens else [tokens] * B
    c = Cache(contexts, tokens, 4, 2, 64, 16, "bf16", seed=B, live=live)
    how = dict(tree_lens=torch.tensor(live, dtype=torch.int32, device="cuda")) if lens else {}
    out, lse = torch.full_like(c.q, 3.0), torch.full(c.q.shape[:3], 3.0, device="cuda")
    tg.tree_attention(c.q, c.k, c.v, c.table, c.context, out=out, lse=lse, **how)
    assert tg.check_device() == 0
    for b in range(B):
        assert not lens or (out[b, :, live[b]:] == 3).all()
    few = set(range(0, B, 67)) | {B - 1}
    c.live = [n if b in few else 0 for b, n in enumerate(live)]
    c.check(out, lse)


@pytest.mark.parametrize("page", [8, 1000, 4096])
def test_pages_of_many_rows_and_of_few(page):
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([900, 2500, 5000, 0], 5, 8, 2, 128, page, "fp16", seed=page)
    lse = torch.empty(c.q.shape[:3], device="cuda")
    out = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, lse=lse)
    assert tg.check_device() == 0
    c.check(out, lse)


# ------------------------------------------------------------------ gradients against differences
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["prefix_documents", "capped", "biased"])
def test_gradients_along_themselves_against_differences(name, dt):
    """<gradient, d> against central differences of the 64-bit forward, d along the exact gradient, where nothing
    cancels: the slope is many times what the roundings may add up to, so a gradient that is off shows."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(CASES[name], dt, seed=5)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    want, bounds = p.gradients(do)
    at = [torch.arange(n, device="cuda").expand(q.shape[0], n) for n in (q.shape[2], k.shape[2])]
    see = p.see.cpu()
    h = 1e-3
    for n, (t, g, w, b) in enumerate(zip("qkv", grads, want, bounds)):
        d = w / w.norm()
        loss = []
        for s in (h, -h):
            x = [y.double() for y in (q, k, v)]
            x[n] = x[n] + s * d
            f = Plain(*x, see, p.scale, p.cap, how.get("slopes"), *at)
            loss.append((f.out.detach() * do.double()).sum())
        slope = (loss[0] - loss[1]) / (2 * h)
        # the difference is off by h^2 / 6 of the third derivative along d: 2e-9 of the slope at most on such draws
        # (h = 1e-2, 1e-3 and 1e-4 agree to that), 1e-6 of it holds that
        slack = (b * d.abs()).sum() + 1e-6 * slope.abs()
        assert slope > 20 * slack, t  # so neither 0 nor a gradient 5 % off passes
        assert abs((g.double() * d).sum() - slope) <= slack, t


# ------------------------------------------------------------------ rotary positions
def rotary_bound(x, want):
    """As in the rotary tests, for scale 1: one rounding, and fp32 before it."""
    size = x.double().abs().amax(-1, keepdim=True)
    return torch.finfo(x.dtype).eps / 2 * want.abs() * (1 + 2.0 ** -6) + size * 2.0 ** -20 + 1e-38


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient_along_itself(interleaved):
    """<rotate(d), g> = <d, inverse(g)> for d along the exact inverse, where nothing cancels."""
    import tensor_core_gemm_tl_b200 as tg
    g = torch.randn((1, 3, 200, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    inv_freq, _ = tg.rotary_frequencies(128, base=500000.0, device="cuda")
    pos = torch.arange(200, device="cuda") + 70000
    gx, _ = tg.rotary(g, None, pos, inv_freq, interleaved=interleaved, inverse=True)
    want = rotate(g, pos[None], inv_freq, interleaved, inverse=True)
    d = want / want.norm()
    lhs, rhs = (rotate(d, pos[None], inv_freq, interleaved) * g.double()).sum(), (d * gx.double()).sum()
    slack = (rotary_bound(g, want) * d.abs()).sum()
    assert lhs > 100 * slack
    assert abs(lhs - rhs) <= slack


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_windows_that_overlap(interleaved):
    """Positive strides of any size, rows that lie inside one another among them: the output is laid out on its own."""
    import tensor_core_gemm_tl_b200 as tg
    x = torch.randn(4096, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).bfloat16()
    inv_freq, _ = tg.rotary_frequencies(8, device="cuda")
    for shape, strides in (((1, 2, 4, 8), (100, 32, 1, 1)), ((2, 3, 4, 8), (1, 1, 1, 1)), ((2, 2, 5, 8), (40, 3, 8, 1))):
        q = torch.as_strided(x, shape, strides)
        pos = torch.arange(shape[2], device="cuda")
        out, _ = tg.rotary(q, None, pos, inv_freq, interleaved=interleaved)
        want, _ = tg.rotary(q.contiguous(), None, pos, inv_freq, interleaved=interleaved)
        assert torch.equal(out, want)


# ------------------------------------------------------------------ autograd
def test_outputs_carry_no_graph():
    """Inputs that require grad give the values they give otherwise, and outputs without a graph."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, _ = problem(dict(shape=(1, 4, 2, 50, 50, 64), causal=True), "bf16", seed=1)
    inv_freq, _ = tg.rotary_frequencies(64, device="cuda")
    pos, table = torch.arange(50, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    context = torch.full((1,), 40, dtype=torch.int32, device="cuda")

    def run(q, k, v):
        lse = torch.empty(q.shape[:3], device="cuda")
        out = tg.attention_ex(q, k, v, lse=lse, **how)
        kc, vc = (t[0, :, :48].transpose(0, 1)[None] for t in (k, v))
        return [out, lse, *tg.attention_backward(do, q, k, v, out, lse, **how), *tg.rotary(q, k, pos, inv_freq),
                tg.tree_attention(q[:, :, :3], kc, vc, table, context)]

    want = run(q, k, v)
    got = run(*(t.requires_grad_() for t in (q, k, v)))
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not a.requires_grad
