"""How the attention operators may be called: from several host threads at once,
captured into a graph by the first call of a process, after a call that failed, and
on tensors whose offsets pass 32 bits."""
import os
import subprocess
import sys
import threading

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def inputs(seed, dt, D):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    return dict(q=rand(1, 6, 700, D), k=rand(1, 2, 700, D), v=rand(1, 2, 700, D), do=rand(1, 6, 700, D),
                qt=rand(2, 4, 3, D), cache=rand(2 * 70, 16, 2, D), inv_freq=torch.rand(D // 2, generator=g, device="cuda"),
                table=torch.randperm(140, generator=g, device="cuda").to(torch.int32).view(2, 70),
                context=torch.tensor([1000, 77], device="cuda", dtype=torch.int32), pos=torch.arange(700, device="cuda"))


def step(x):
    """Rotary, forward and backward, a chunk and a chain from the cache: split calls and whole ones, all workspaces."""
    import tensor_core_gemm_tl_b200 as tg
    q, k = tg.rotary(x["q"], x["k"], x["pos"], x["inv_freq"])
    lse = torch.empty(q.shape[:3], device="cuda")
    out = tg.attention_ex(q, k, x["v"], causal=True, score_cap=20.0, lse=lse)
    grads = tg.attention_backward(x["do"], q, k, x["v"], out, lse, causal=True, score_cap=20.0)
    few = tg.attention_ex(q[:, :2, :50], k, x["v"], q_offset=650, causal=True)
    tree = tg.tree_attention(x["qt"], x["cache"], x["cache"], x["table"], x["context"], score_cap=20.0)
    return [q, k, out, lse, *grads, few, tree]


def test_threads_on_their_own_streams():
    import tensor_core_gemm_tl_b200 as tg
    work = [inputs(n, [torch.bfloat16, torch.float16][n % 2], [64, 128][n // 2 % 2]) for n in range(8)]
    want = [step(x) for x in work]
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(work))

    def run(n):
        try:
            stream = torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(5):
                    got = step(work[n])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        failures.append((n, "differs"))
        except Exception as e:
            failures.append((n, repr(e)))

    threads = [threading.Thread(target=run, args=(n,)) for n in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
    assert tg.check_device() == 0


CAPTURED_FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
import tensor_core_gemm_tl_b200 as tg
from test_attention_calls_gpu import inputs, step
x = inputs(1, torch.%s, %d)
a, b = x["q"][0, 0, :100].reshape(-1)[:300 * 21].view(300, 21), x["k"][0, 0, :100].reshape(-1)[:21 * 77].view(21, 77)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step(x) + [tg.gemm(a, b)]  # the product's operands are copied into padded temporaries
graph.replay()
torch.cuda.synchronize()
want = step(x) + [tg.gemm(a, b)]
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert tg.check_device() == 0
print("same")
"""


@pytest.mark.parametrize("dt,D", [("bfloat16", 128), ("float16", 64)])
def test_captured_by_the_first_call(dt, D):
    done = subprocess.run([sys.executable, "-c", CAPTURED_FIRST % (os.path.dirname(HERE), HERE, dt, D)],
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]


def test_a_call_after_one_that_ran_out_of_memory():
    """A workspace of a terabyte is refused with nothing launched, and is forgotten: the next call of any kind succeeds."""
    import tensor_core_gemm_tl_b200 as tg
    x = inputs(3, torch.bfloat16, 64)
    want = step(x)
    a, b = torch.ones((2, 128, 128), device="cuda", dtype=torch.float16)
    f = torch.ones(1000, device="cuda")
    calls = [lambda: step(x), lambda: [tg.gemm(a, b)], lambda: [tg.gemm(a[:, :77].contiguous(), b[:77, :55].contiguous())],
             lambda: [tg.attention(x["q"], x["q"], x["q"])], lambda: [tg.softmax(a)], lambda: [tg.vector_add(f, f)],
             lambda: tg.rotary(x["q"], x["k"], x["pos"], x["inv_freq"]),
             lambda: [tg.tree_attention(x["qt"], x["cache"], x["cache"], x["table"], x["context"])]]
    before = [c() for c in calls]
    p, stream = x["q"].data_ptr(), torch.cuda.current_stream().cuda_stream
    for call, was in zip(calls, before):
        # 500 heads of 2^28 queries: 8 bytes each for the row statistics alone
        assert tg.tl_attention_bwd(*[p] * 9, 1, 500, 1 << 28, 64, 64, tg.TL_BF16, stream) == tg.Status.CUDA
        assert all(torch.equal(i, j) for i, j in zip(call(), was))
    assert all(torch.equal(i, j) for i, j in zip(step(x), want))
    assert tg.check_device() == 0


def far_apart(t, gap):
    """`t` in a buffer of its own where its first dimension's entries lie `gap` values apart."""
    big = torch.empty(gap * (t.shape[0] - 1) + t[0].numel(), dtype=t.dtype, device="cuda")
    y = big.as_strided(t.shape, (gap, *t[0].contiguous().stride()))
    y.copy_(t)
    return y


def test_offsets_that_pass_32_bits():
    """Batch entries and cache pages more than 2^31 values apart: the results of the same tensors close together."""
    import tensor_core_gemm_tl_b200 as tg
    gap = (1 << 31) + 8 * 1000
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").half()

    q, k, v, do = rand(2, 4, 300, 64), rand(2, 2, 600, 64), rand(2, 2, 600, 64), rand(2, 4, 300, 64)
    pos, inv_freq = torch.arange(300, device="cuda"), torch.rand(32, generator=g, device="cuda")
    qt, kc, vc = rand(2, 4, 3, 64), rand(2, 32, 2, 64), rand(2, 32, 2, 64)
    table = torch.tensor([[1, 0], [0, 1]], device="cuda", dtype=torch.int32)
    context = torch.tensor([50, 29], device="cuda", dtype=torch.int32)

    def run(place, empty):
        lse = torch.empty((2, 4, 300), device="cuda")
        rq, _ = tg.rotary(place(q), None, pos, inv_freq, out_q=empty(q))
        o = tg.attention_ex(rq, place(k), place(v), causal=True, q_offset=300, score_cap=20.0, out=empty(q), lse=lse)
        grads = tg.attention_backward(place(do), rq, place(k), place(v), o, lse, causal=True, q_offset=300, score_cap=20.0,
                                      dq=empty(q), dk=empty(k), dv=empty(v))
        t = tg.tree_attention(qt, place(kc), place(vc), table, context)
        return [x.contiguous() for x in (rq, o, lse, *grads, t)]

    want = run(lambda t: t, torch.empty_like)
    got = run(lambda t: far_apart(t, gap), lambda t: far_apart(torch.zeros_like(t), gap))
    assert tg.check_device() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
