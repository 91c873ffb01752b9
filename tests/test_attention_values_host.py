"""Scales and caps that float32 does not hold are refused, on the CPU: 0 has a meaning
of its own (the default scale, no cap), so a value may not become it."""
import math
import os
import struct
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch  # noqa: E402

import tensor_core_gemm_tl_b200 as tg  # noqa: E402
from test_attention_ops_host import NO_GPU, Fake, I32, backward, call_attention, call_tree, forward  # noqa: E402

OUT = (1e-46, 1e-300, 1e39, 1e300, math.inf, math.nan, -1e-46)
SMALLEST, LARGEST = 2.0 ** -149, (2 - 2.0 ** -23) * 2.0 ** 127


def tree(scale=0.0, score_cap=0.0):
    tg.tree_attention(Fake((2, 4, 3, 64)), Fake((9, 16, 2, 64)), Fake((9, 16, 2, 64)), Fake((2, 4), I32), Fake((2,), I32),
                      scale=scale, score_cap=score_cap, out=Fake((2, 4, 3, 64)))


def masked(f):
    def call(**kw):
        f(Fake((2, 4, 50, 64)), Fake((2, 2, 60, 64)), Fake((2, 2, 60, 64)), **kw)
    return call


def turned(scale):
    tg.rotary(Fake((2, 4, 50, 64)), None, Fake((2, 50), I32), Fake((32,), torch.float32), scale=scale,
              out_q=Fake((2, 4, 50, 64)))


CALLS = {
    "forward": lambda **kw: masked(forward)(out=Fake((2, 4, 50, 64)), **kw),
    "backward": lambda **kw: masked(backward)(dq=Fake((2, 4, 50, 64)), dk=Fake((2, 2, 60, 64)), dv=Fake((2, 2, 60, 64)), **kw),
    "tree": tree,
}


@pytest.fixture
def launches(monkeypatch):
    """The option structs that reach the C ABI."""
    seen = []
    for name in ("tl_attention_ex", "tl_attention_bwd", "tl_tree_attention", "tl_rotary"):
        monkeypatch.setattr(tg, name, name)
    monkeypatch.setattr(tg, "_launch", lambda torch, device, stream, options, *a: seen.append(options))
    return seen


@pytest.mark.parametrize("value", OUT)
@pytest.mark.parametrize("what", ["scale", "score_cap"])
@pytest.mark.parametrize("call", list(CALLS))
def test_scores(call, what, value, launches):
    with pytest.raises(ValueError):
        CALLS[call](**{what: value})
    assert not launches


@pytest.mark.parametrize("value", OUT + (0.0,))
def test_rotary(value, launches):
    with pytest.raises(ValueError):
        turned(value)
    assert not launches


@pytest.mark.parametrize("value", [SMALLEST, 1e-40, 1.0, LARGEST])
def test_what_float32_holds_arrives(value, launches):
    as_float32 = struct.unpack("f", struct.pack("f", value))[0]
    for call, at in (("forward", 1), ("tree", 0)):
        CALLS[call](scale=value)
        o = (tg.ATTENTION_OPTIONS if call == "forward" else tg.TREE_OPTIONS).unpack(launches.pop())
        assert o[at] == as_float32 > 0
    turned(value)
    assert tg.ROTARY_OPTIONS.unpack(launches.pop())[2] == as_float32 > 0


# softmax_scale, score_cap: their product with log2 e, or their quotient, leaves fp32's normal range
PAST_FP32 = [(2.4e38, 0.0), (1e38, 0.0), (0.0, 3e38), (1.0, 1.5e38), (1e-20, 1e30), (0.0, 9e37), (1e-38, 1.0)]


@pytest.mark.parametrize("scale,cap", PAST_FP32)
def test_the_library_refuses_scores_past_fp32(scale, cap):
    o = dict(softmax_scale=scale, score_cap=cap)
    for st in (call_attention({}, o, False), call_attention({}, o, True), call_tree({}, o)):
        assert st == tg.Status.INVALID_ARG


@NO_GPU
@pytest.mark.parametrize("scale,cap", [(9e37, 0.0), (1e-38, 0.0), (0.0, 1e35), (1e-6, 1e-29), (1e30, 1e-7)])
def test_scores_inside_fp32_reach_the_device(scale, cap):
    o = dict(softmax_scale=scale, score_cap=cap)
    for st in (call_attention({}, o, False), call_attention({}, o, True), call_tree({}, o)):
        assert st == tg.Status.CUDA
