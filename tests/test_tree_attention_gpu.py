"""Tree attention over a paged cache on the GPU against the plain 64-bit form:
one token to 64, chains and trees, page sizes, ragged lengths, shared heads,
unused rows that hold NaN, pages out of range, streams and graphs."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import Plain, close, tree_visible  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Cache:
    """A paged cache with every row no request owns set to NaN, and the new tokens' queries."""

    def __init__(self, contexts, T, H, Hk, D, page, dt, seed, q_scale=1.0, extra_pages=0, heads_first=False, live=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(contexts)
        self.live = [T] * B if live is None else live
        per = max(-(-(c + T) // page) for c in contexts) + extra_pages
        n = B * per + 3
        order = torch.randperm(n, generator=g, device="cuda")[:B * per].to(torch.int32).view(B, per)
        shape = (n, Hk, page, D) if heads_first else (n, page, Hk, D)
        self.k, self.v = (torch.full(shape, math.nan, device="cuda", dtype=DT[dt]) for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.keys = []
        for b, c in enumerate(contexts):
            m = c + self.live[b]
            kk, vv = (torch.randn((m, Hk, D), generator=g, device="cuda").to(DT[dt]) for _ in range(2))
            at = torch.arange(m, device="cuda")
            self.k[order[b].long()[at // page], at % page] = kk
            self.v[order[b].long()[at // page], at % page] = vv
            self.keys.append((kk, vv))
            order[b, -(-m // page):] = (1 << 30) if b % 2 else -1  # entries behind the last key: never read
        self.table = order
        self.context = torch.tensor(contexts, dtype=torch.int32, device="cuda")
        self.q = (torch.randn((B, T, H, D), generator=g, device="cuda") * q_scale).to(DT[dt]).transpose(1, 2)

    def check(self, out, lse=None, parents=None, cap=0.0, slopes=None, scale=None):
        B, H, T, D = self.q.shape
        for b in range(B):
            live, c = self.live[b], int(self.context[b])
            if live == 0:
                continue
            kk, vv = (t.transpose(0, 1)[None] for t in self.keys[b])
            see, depth = tree_visible(c, T, c + live, None if parents is None else parents[b].tolist(), live)
            pos_k = torch.cat([torch.arange(c), c + torch.tensor(depth[:live])])[None].cuda()
            pos_q = (c + torch.tensor(depth))[None].cuda()
            p = Plain(self.q[b:b + 1, :, :live], kk, vv, see[None, :live], scale or 1 / math.sqrt(D), cap, slopes,
                      pos_q[:, :live], pos_k)
            close(f"out[{b}]", out[b:b + 1, :, :live], p.out, p.out_bound())
            if lse is not None:
                close(f"lse[{b}]", lse[b:b + 1, :, :live], p.lse, p.lse_bound())


def random_parents(B, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand((B, T), generator=g, device="cuda")
    return ((u * (torch.arange(T, device="cuda") + 1)).to(torch.int32) - 1).contiguous()


CASES = [
    # contexts, tokens, heads, kv heads, head_dim, page
    ([0], 1, 1, 1, 64, 8),
    ([1, 0, 127, 128, 129], 1, 4, 4, 128, 16),
    ([900], 1, 16, 8, 128, 16),
    ([5000, 3, 0, 777, 2048, 130], 1, 8, 2, 64, 64),
    ([300, 1000, 64], 7, 8, 1, 128, 24),
    ([40, 250], 64, 10, 2, 64, 32),        # five heads share: 25 tokens a tile, three tiles
    ([120, 121, 64], 64, 4, 2, 128, 256),  # drafted tokens across a block's end
    ([700], 5, 128, 1, 64, 128),           # 128 heads share: a tile a token
    ([20000], 3, 8, 1, 128, 64),           # one tile over every CTA
    ([256] * 40, 1, 8, 8, 128, 16),        # more tiles than CTAs
    ([17 * n % 400 for n in range(70)], 2, 6, 3, 64, 8),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", range(len(CASES)))
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_tree_attention(n, dt, kind):
    import tensor_core_gemm_tl_b200 as tg
    contexts, T, H, Hk, D, page = CASES[n]
    c = Cache(contexts, T, H, Hk, D, page, dt, seed=n)
    parents = random_parents(len(contexts), T, n) if kind == "tree" else None
    lse = torch.empty(c.q.shape[:3], device="cuda")
    out = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, lse=lse)
    assert tg.check_device() == 0
    c.check(out, lse, parents)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (8.0, True)])
def test_tree_caps_and_bias(D, cap, bias):
    import tensor_core_gemm_tl_b200 as tg
    H = 6
    c = Cache([0, 100, 1500, 127], 33, H, 2, D, 16, "bf16", seed=3, q_scale=4.0)
    parents = random_parents(4, 33, 9)
    slopes = torch.linspace(0.5, 0.004, H, device="cuda") if bias else None
    lse = torch.empty(c.q.shape[:3], device="cuda")
    out = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, score_cap=cap, slopes=slopes, lse=lse, scale=0.1)
    assert tg.check_device() == 0
    c.check(out, lse, parents, cap, slopes, scale=0.1)


def test_shorter_trees_leave_the_rest_alone():
    import tensor_core_gemm_tl_b200 as tg
    live = [0, 3, 9, 1]
    c = Cache([100, 128, 3000, 0], 9, 4, 2, 64, 16, "fp16", seed=4, live=live)
    parents = random_parents(4, 9, 1)
    out, lse = torch.full_like(c.q, 3.0), torch.full(c.q.shape[:3], 3.0, device="cuda")
    lens = torch.tensor(live, dtype=torch.int32, device="cuda")
    tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, tree_lens=lens, out=out, lse=lse)
    assert tg.check_device() == 0
    c.check(out, lse, parents)
    for b, n in enumerate(live):
        assert (out[b, :, n:] == 3).all() and (lse[b, :, n:] == 3).all()
    # nobody has a token: nothing is written
    before = out.clone()
    tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, tree_lens=torch.zeros_like(lens), out=out, lse=lse)
    assert tg.check_device() == 0 and torch.equal(out, before)


def test_caches_with_heads_before_rows_and_outputs_inside_others():
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([200, 400], 3, 8, 2, 128, 32, "bf16", seed=5, heads_first=True, extra_pages=4)
    big = torch.full((2, 3, 12, 128), 1.5, device="cuda", dtype=torch.bfloat16)
    out = big[:, :, 2:10].transpose(1, 2)
    tg.tree_attention(c.q, c.k, c.v, c.table, c.context, out=out)
    c.check(out)
    assert (big[:, :, :2] == 1.5).all() and (big[:, :, 10:] == 1.5).all()


def test_pages_out_of_range_read_as_zeros():
    """A bad page index in the middle of a context: its keys and values count as zeros."""
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([200], 1, 2, 1, 64, 16, "bf16", seed=6)
    for bad in (-1, c.k.shape[0], (1 << 31) - 1, -(1 << 31)):
        table = c.table.clone()
        table[0, 4] = bad
        kk, vv = (t.clone() for t in c.keys[0])
        kk[64:80], vv[64:80] = 0, 0
        out = tg.tree_attention(c.q, c.k, c.v, table, c.context)
        assert tg.check_device() == 0
        see, _ = tree_visible(200, 1, 201)
        p = Plain(c.q, kk.transpose(0, 1)[None], vv.transpose(0, 1)[None], see[None], 0.125)
        close("out", out, p.out, p.out_bound())


def test_lengths_past_the_table_are_held_to_it():
    """A context that the table cannot hold: only what it holds is read, new tokens without a key see the context."""
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([60], 4, 2, 1, 64, 16, "bf16", seed=7)  # 64 keys in 4 pages
    for n in (61, 64, 1000, (1 << 31) - 1):
        ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
        out = tg.tree_attention(c.q, c.k, c.v, c.table, ctx)
        assert tg.check_device() == 0
        see, _ = tree_visible(min(n, 64), 4, 64)
        p = Plain(c.q, *(t.transpose(0, 1)[None] for t in c.keys[0]), see[None], 0.125)
        close("out", out, p.out, p.out_bound())
    neg = tg.tree_attention(c.q, c.k, c.v, c.table, torch.tensor([-5], dtype=torch.int32, device="cuda"))
    zero = tg.tree_attention(c.q, c.k, c.v, c.table, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert torch.equal(neg, zero)


def test_parents_that_are_no_tree_end():
    """A parent that is not earlier counts as the context."""
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([50], 6, 2, 2, 64, 16, "bf16", seed=8)
    odd = torch.tensor([[0, 5, 1, 3, 1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    out = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, odd)
    assert tg.check_device() == 0
    c.check(out, parents=odd)


def test_repeats_on_several_streams_and_in_graphs():
    import tensor_core_gemm_tl_b200 as tg
    c = Cache([3000, 10, 777], 5, 8, 2, 128, 16, "bf16", seed=9, extra_pages=2)
    parents = random_parents(3, 5, 2)
    first = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for n in range(9):
        s = streams[n % 3]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    # captured once, replayed with other lengths: the host reads none of them
    out, lens = torch.empty_like(c.q), torch.full((3,), 5, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, tree_lens=lens, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    live = c.context.clone()
    for short in (2900, 127, 128):
        c.context.copy_(live)
        c.context[0] = short
        eager = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    assert tg.check_device() == 0
