"""The attention operators where their ranges end, on the GPU against the plain 64-bit
forms."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from attention_plain import Plain, close  # noqa: E402
from test_attention_ex_gpu import problem  # noqa: E402

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


# ------------------------------------------------------------------ fp16 gradients
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
