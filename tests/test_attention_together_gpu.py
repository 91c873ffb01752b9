"""The operators as a model runs them: rotary positions into the masked attention
and back through both; then the same layer served token by token and as a drafted
tree from a paged cache."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import Plain, close, rotate, visible  # noqa: E402

B, S, H, HK, D, CAP = 2, 230, 6, 2, 64, 20.0


def layer(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn((B, S, H + 2 * HK, D), generator=g, device="cuda").bfloat16()


def split(qkv):
    return [t.transpose(1, 2) for t in qkv.split([H, HK, HK], dim=2)]


def test_a_training_step():
    import tensor_core_gemm_tl_b200 as tg
    qkv = layer(1)
    q0, k0, v = split(qkv)
    inv_freq, scale = tg.rotary_frequencies(D, scaling="yarn", factor=4.0, original_length=64, device="cuda")
    pos = torch.arange(S, device="cuda")
    docs = [[0, 100, 220], [0, 30, 230]]
    how = dict(causal=True, score_cap=CAP, doc_offsets=torch.tensor(docs, dtype=torch.int32, device="cuda"))
    q, k = tg.rotary(q0, k0, pos, inv_freq, scale=scale)
    lse = torch.empty((B, H, S), device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    dout = torch.randn_like(out)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = split(dqkv)
    tg.attention_backward(dout, q, k, v, out, lse, dq=dq, dk=dk, dv=dv, **how)
    p = Plain(q, k, v, visible(B, S, S, True, 0, docs), 1 / math.sqrt(D), CAP)
    close("out", out, p.out, p.out_bound())
    want, bounds = p.gradients(dout)
    for n, g, w, b in zip(("dq", "dk", "dv"), (dq, dk, dv), want, bounds):
        close(n, g, w, b)
    before = dq.clone(), dk.clone()
    tg.rotary(dq, dk, pos, inv_freq, scale=scale, inverse=True, out_q=dq, out_k=dk)
    assert tg.check_device() == 0
    for g, was in zip((dq, dk), before):
        w = rotate(was, pos.expand(B, S), inv_freq, scale=scale, inverse=True)
        size = scale * was.double().abs().amax(-1, keepdim=True)
        close("through the positions", g, w, 2.0 ** -8 * w.abs() * (1 + 2.0 ** -6) + size * 2.0 ** -20 + 1e-38)


def test_serving_gives_the_prefill_rows():
    """A prompt by attention_ex in one go, its last tokens again from the cache: one at a time, as a
    chain, and as a tree of two branches of which one is the prompt's."""
    import tensor_core_gemm_tl_b200 as tg
    page, T = 16, 5
    qkv = layer(2)
    inv_freq, _ = tg.rotary_frequencies(D, device="cuda")
    q0, k0, v = split(qkv)
    pos = torch.arange(S, device="cuda", dtype=torch.int32)
    q, k = tg.rotary(q0, k0, pos, inv_freq)
    lse = torch.empty((B, H, S), device="cuda")
    out = tg.attention_ex(q, k, v, causal=True, score_cap=CAP, lse=lse)
    p = Plain(q, k, v, visible(B, S, S, True), 1 / math.sqrt(D), CAP)
    # the two kernels' sums differ in order: each is within the bound of the exact rows
    per = -(-(S + T) // page)
    table = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    kc, vc = (torch.full((B * per, page, HK, D), math.nan, device="cuda").bfloat16() for _ in range(2))

    def write(b, first, kk, vv):  # (heads, n, D) at key `first`
        at = first + torch.arange(kk.shape[1], device="cuda")
        kc[table[b].long()[at // page], at % page] = kk.transpose(0, 1)
        vc[table[b].long()[at // page], at % page] = vv.transpose(0, 1)

    n0 = S - T
    for b in range(B):
        write(b, 0, k[b, :, :n0], v[b, :, :n0])
    context = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    for t in range(T):
        for b in range(B):
            write(b, n0 + t, k[b, :, n0 + t:n0 + t + 1], v[b, :, n0 + t:n0 + t + 1])
        one = tg.tree_attention(q[:, :, n0 + t:n0 + t + 1], kc, vc, table, context + t, score_cap=CAP)
        close("one token", one, p.out[:, :, n0 + t:n0 + t + 1], p.out_bound()[:, :, n0 + t:n0 + t + 1])
    chain = tg.tree_attention(q[:, :, n0:], kc, vc, table, context, score_cap=CAP)
    close("chain", chain, p.out[:, :, n0:], p.out_bound()[:, :, n0:])
    # the tree: tokens 0, 2, 4, 5, 6 are the prompt's last ones, 1 and 3 another branch below token 0
    parents = torch.tensor([[-1, 0, 0, 1, 2, 4, 5]] * B, dtype=torch.int32, device="cuda")
    mine = [0, 2, 4, 5, 6]
    noise = torch.randn((3, B, 7, H + HK, D), device="cuda").bfloat16()
    tq, tk, tv = noise[0, :, :, :H].transpose(1, 2).contiguous(), noise[1, :, :, H:].transpose(1, 2).contiguous(), \
        noise[2, :, :, H:].transpose(1, 2).contiguous()
    tq[:, :, mine], tk[:, :, mine], tv[:, :, mine] = q[:, :, n0:], k[:, :, n0:], v[:, :, n0:]
    for b in range(B):
        write(b, n0, tk[b], tv[b])
    tree = tg.tree_attention(tq, kc, vc, table, context, parents, score_cap=CAP)
    assert tg.check_device() == 0
    close("tree", tree[:, :, mine], p.out[:, :, n0:], p.out_bound()[:, :, n0:])


def test_split_and_cut_calls_at_once_and_in_two_graphs():
    """Calls whose work is split over CTAs and joined (few items, few tiles, one long request) on several streams at
    once, then captured twice and replayed side by side: bit for bit the results of the same calls one at a time."""
    import tensor_core_gemm_tl_b200 as tg
    g = torch.Generator(device="cuda").manual_seed(11)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, k, v, do = rand(1, 6, 900, 64), rand(1, 1, 900, 64), rand(1, 1, 900, 64), rand(1, 6, 900, 64)
    qt, cache = rand(2, 8, 3, 128), rand(2 * 160, 16, 2, 128)
    table = torch.randperm(320, generator=g, device="cuda").to(torch.int32).view(2, 160)
    context = torch.tensor([2500, 700], device="cuda", dtype=torch.int32)

    def step(stream=None):
        lse = torch.empty((1, 6, 900), device="cuda")
        if stream is not None:
            lse.record_stream(stream)
        o = tg.attention_ex(q, k, v, causal=True, lse=lse, stream=stream)
        grads = tg.attention_backward(do, q, k, v, o, lse, causal=True, stream=stream)
        few = tg.attention_ex(q[:, :2, :50], k, v, q_offset=850, causal=True, stream=stream)
        t = tg.tree_attention(qt, cache, cache, table, context, stream=stream)
        return [o, lse, *grads, few, t]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [step(streams[i % 3]) for i in range(12)]
    torch.cuda.synchronize()
    assert tg.check_device() == 0
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graphs, outs = [], []
    for s in streams[:2]:
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(step())
        graphs.append(graph)
    for n in range(5):
        for r in outs:
            for t in r:
                t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for r in outs:
            assert all(torch.equal(a, b) for a, b in zip(r, want)), n
    assert tg.check_device() == 0
