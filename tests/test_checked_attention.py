"""The masked attention, its gradients, the tree attention and rotary positions through
the checked build (libtlgemm_checked.so), whose kernels test heads, tiles, blocks,
page-table entries, rows and the places of partial sums at run time and set bit 7
of the device error word on a violation: results as ever, and no check fires."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import test_attention_limits_gpu as limits  # noqa: E402
import test_rotary_gpu as turned  # noqa: E402
import test_tree_attention_gpu as tree  # noqa: E402
from test_attention_ex_gpu import CASES, problem  # noqa: E402
from test_checked_build import checked_lib  # noqa: E402

from attention_plain import close  # noqa: E402


@pytest.fixture(autouse=True)
def checked(monkeypatch):
    """The package's calls go to the checked library; its error word is clean before and after."""
    import tensor_core_gemm_tl_b200 as tg
    monkeypatch.setattr(tg._binding, "_lib", checked_lib())
    assert tg.check_device() == 0
    yield
    assert tg.check_device() == 0


MASKED = {**CASES, **limits.PAST_THE_KEYS}


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(MASKED))
def test_masked_attention(name, dt):
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, p = problem(MASKED[name], dt, seed=len(name))
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, v, lse=lse, **how)
    grads = tg.attention_backward(do, q, k, v, out, lse, **how)
    close("out", out, p.out, p.out_bound())
    want, bounds = p.gradients(do)
    for n, g, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        close(n, g, w, b)


def test_offsets_out_of_order():
    """Whatever the offsets hold, every index stays inside."""
    import tensor_core_gemm_tl_b200 as tg
    q, k, v, do, how, _ = problem(dict(shape=(2, 2, 2, 300, 300, 64)), "bf16", 6)
    big = 1 << 30
    for first in ([250, -5, big, -big], [-(1 << 31), (1 << 31) - 1, 0, 5], [300, 200, 100, 0], [-7, -7, -7, -7]):
        docs = torch.tensor([first, [0, 100, 200, 300]], dtype=torch.int32, device="cuda")
        prefix = torch.tensor([[big, -7, 3], [0, (1 << 31) - 1, -(1 << 31)]], dtype=torch.int32, device="cuda")
        for how in (dict(doc_offsets=docs), dict(doc_offsets=docs, causal=True, prefix=prefix),
                    dict(doc_offsets=docs, q_offset=200, causal=True)):
            lse = torch.empty(q.shape[:3], device="cuda")
            out = tg.attention_ex(q, k, v, lse=lse, **how)
            tg.attention_backward(do, q, k, v, out, lse, **how)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (8.0, True)])
@pytest.mark.parametrize("n", range(len(tree.CASES)))
def test_tree_attention(n, cap, bias):
    import tensor_core_gemm_tl_b200 as tg
    contexts, T, H, Hk, D, page = tree.CASES[n]
    c = tree.Cache(contexts, T, H, Hk, D, page, "bf16", seed=n)
    parents = tree.random_parents(len(contexts), T, n)
    slopes = torch.linspace(0.5, 0.004, H, device="cuda") if bias else None
    out = tg.tree_attention(c.q, c.k, c.v, c.table, c.context, parents, score_cap=cap, slopes=slopes)
    c.check(out, None, parents, cap, slopes)


def test_lengths_that_the_table_cannot_hold():
    import tensor_core_gemm_tl_b200 as tg
    c = tree.Cache([60, 33], 4, 2, 1, 64, 16, "bf16", seed=7)
    slopes = torch.tensor([0.5, 0.01], device="cuda")
    for n in (61, 64, 1000, (1 << 31) - 1, -1, -(1 << 31)):
        context = torch.tensor([n, 33], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n, 4], dtype=torch.int32, device="cuda")
        for how in (dict(), dict(slopes=slopes), dict(tree_lens=lens), dict(slopes=slopes, tree_lens=lens, score_cap=5.0)):
            tg.tree_attention(c.q, c.k, c.v, c.table, context, out=torch.zeros_like(c.q), **how)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", range(len(turned.CASES)))
def test_rotary(n, interleaved):
    turned.test_rotary(n, interleaved, False, torch.bfloat16)
