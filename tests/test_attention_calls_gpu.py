"""How the attention operators may be called: from several host threads at once, and
captured into a graph by the first call of a process."""
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
