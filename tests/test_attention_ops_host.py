"""Refusals of the masked attention, its backward, the tree attention and the
rotary positions, on the CPU: the C ABI's checks before any CUDA call, the
binding's checks of tensors before any pointer is taken, the frequencies."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import tensor_core_gemm_tl_b200 as tg

P = 1 << 20  # an aligned "device pointer" that is never followed
BAD, UNSUP, MISAL = tg.Status.INVALID_ARG, tg.Status.UNSUPPORTED, tg.Status.MISALIGNED
# with valid arguments the first CUDA call is reached, and fails where there is no GPU
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a GPU")


def attention_options(**over):
    return tg.AttentionOptions(**over)


ATTENTION = [
    (dict(Q=0), {}, BAD), (dict(K=0), {}, BAD), (dict(V=0), {}, BAD), (dict(O=0), {}, BAD),
    (dict(batch=0), {}, BAD), (dict(heads=0), {}, BAD), (dict(seq_q=0), {}, BAD), (dict(seq_k=-1), {}, BAD),
    (dict(dtype=2), {}, BAD), (dict(head_dim=96), {}, UNSUP), (dict(head_dim=0), {}, UNSUP),
    ({}, dict(kv_heads=3), BAD), ({}, dict(kv_heads=-1), BAD), ({}, dict(kv_heads=16), BAD),
    ({}, dict(softmax_scale=-1.0), BAD), ({}, dict(softmax_scale=math.inf), BAD), ({}, dict(softmax_scale=math.nan), BAD),
    ({}, dict(score_cap=1e-20, softmax_scale=1e30), BAD), ({}, dict(score_cap=1e-35), BAD),
    ({}, dict(score_cap=-1.0), BAD), ({}, dict(score_cap=math.nan), BAD), ({}, dict(score_cap=math.inf), BAD),
    ({}, dict(causal=2), BAD), ({}, dict(q_offset=-1), BAD), ({}, dict(num_docs=-1), BAD),
    ({}, dict(num_docs=2), BAD), ({}, dict(doc_offsets=P), BAD),
    ({}, dict(prefix_lens=P), BAD),  # a prefix without causal
    ({}, dict(doc_offsets=P + 2, num_docs=1), MISAL), ({}, dict(slopes=P + 1), MISAL),
    ({}, dict(causal=1, prefix_lens=P + 1), MISAL),
    (dict(seq_k=(1 << 31) - 1), {}, UNSUP), (dict(seq_q=1 << 33), {}, UNSUP), ({}, dict(q_offset=(1 << 31) - 200), UNSUP),
    (dict(batch=1 << 20, heads=1 << 12), {}, UNSUP), (dict(batch=1 << 14, heads=1 << 8, seq_q=1 << 20), {}, UNSUP),
    (dict(Q=P + 8), {}, MISAL), (dict(K=P + 2), {}, MISAL), (dict(O=P + 4), {}, MISAL), (dict(lse=P + 2), {}, MISAL),
    ({}, dict(q_strides=(8192, 0, 64)), BAD), ({}, dict(k_strides=(8192, -64, 64)), BAD),
    ({}, dict(v_strides=(8192, 1024, 60)), MISAL), ({}, dict(o_strides=(1 << 40, 1024, 64)), UNSUP),
]


def call_attention(a, o, backward):
    f = dict(Q=P, K=P, V=P, O=P, lse=P, batch=2, heads=8, seq_q=100, seq_k=100, head_dim=64, dtype=1)
    f.update(a)
    opt = attention_options(**o)
    tail = (f["batch"], f["heads"], f["seq_q"], f["seq_k"], f["head_dim"], f["dtype"], 0, opt)
    if backward:
        return tg.tl_attention_bwd(P, f["Q"], f["K"], f["V"], f["O"], f["lse"], P, P, P, *tail)
    return tg.tl_attention_ex(f["Q"], f["K"], f["V"], f["O"], f["lse"], *tail)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("n", range(len(ATTENTION)))
def test_attention_refusals(n, backward):
    a, o, status = ATTENTION[n]
    assert call_attention(a, o, backward) == status


def test_backward_needs_its_own_arguments():
    shape = (2, 8, 100, 100, 64, 1, 0, None)
    for i in (0, 5, 6, 7, 8):  # dO, lse, dQ, dK, dV
        args = [P] * 9
        args[i] = 0
        assert tg.tl_attention_bwd(*args, *shape) == BAD
    for i in (0, 6, 7, 8):
        args = [P] * 9
        args[i] = P + 2
        assert tg.tl_attention_bwd(*args, *shape) == MISAL
    for name in ("do", "dq", "dk", "dv"):
        opt = attention_options(**{name + "_strides": (8192, 1024, 4)})
        assert tg.tl_attention_bwd(*[P] * 9, *shape[:-1], opt) == MISAL


@NO_GPU
def test_valid_calls_reach_the_device():
    CUDA = tg.Status.CUDA
    assert call_attention({}, {}, False) == CUDA and call_attention({}, dict(kv_heads=2, causal=1), True) == CUDA
    # a dimension of one element takes any stride, three zeros mean contiguous
    assert call_attention(dict(batch=1, seq_q=1), dict(q_strides=(3, 64, -5)), False) == CUDA
    assert call_tree({}, {}) == CUDA and call_tree(dict(parents=P, tree_lens=P), dict(slopes=P)) == CUDA
    assert call_rotary({}, {}) == CUDA and call_rotary(dict(K=0, Kout=0, kv_heads=0), {}) == CUDA


TREE = [
    (dict(Q=0), {}, BAD), (dict(K=0), {}, BAD), (dict(table=0), {}, BAD), (dict(context=0), {}, BAD), (dict(O=0), {}, BAD),
    (dict(batch=0), {}, BAD), (dict(heads=7), {}, BAD), (dict(kv_heads=0), {}, BAD), (dict(tokens=0), {}, BAD),
    (dict(num_pages=0), {}, BAD), (dict(page_size=0), {}, BAD), (dict(max_pages=0), {}, BAD), (dict(dtype=-1), {}, BAD),
    ({}, dict(softmax_scale=-0.5), BAD), ({}, dict(score_cap=math.nan), BAD),
    ({}, dict(table_stride=-1), BAD), ({}, dict(table_stride=9), BAD),
    (dict(tokens=65), {}, UNSUP), (dict(batch=4097), {}, UNSUP), (dict(heads=258, kv_heads=2), {}, UNSUP),
    (dict(head_dim=80), {}, UNSUP), (dict(page_size=12), {}, UNSUP), (dict(page_size=1 << 30, max_pages=4), {}, UNSUP),
    (dict(num_pages=1 << 32), {}, UNSUP), (dict(batch=4096, heads=4096, kv_heads=4096, max_pages=1 << 20), {}, UNSUP),
    (dict(Q=P + 2), {}, MISAL), (dict(V=P + 8), {}, MISAL), (dict(table=P + 2), {}, MISAL),
    (dict(parents=P + 1), {}, MISAL), (dict(tree_lens=P + 2), {}, MISAL), (dict(lse=P + 2), {}, MISAL),
    ({}, dict(k_strides=(4096, 1024, 0)), BAD), ({}, dict(v_strides=(4096, 1028, 64)), MISAL),
]


def call_tree(a, o):
    f = dict(Q=P, K=P, V=P, table=P, context=P, parents=0, tree_lens=0, O=P, lse=0, batch=2, heads=8, kv_heads=2,
             tokens=4, num_pages=100, page_size=16, max_pages=10, head_dim=64, dtype=0)
    f.update(a)
    return tg.tl_tree_attention(f["Q"], f["K"], f["V"], f["table"], f["context"], f["parents"], f["tree_lens"], f["O"],
                                f["lse"], f["batch"], f["heads"], f["kv_heads"], f["tokens"], f["num_pages"],
                                f["page_size"], f["max_pages"], f["head_dim"], f["dtype"], 0, tg.TreeOptions(**o))


@pytest.mark.parametrize("n", range(len(TREE)))
def test_tree_refusals(n):
    a, o, status = TREE[n]
    assert call_tree(a, o) == status


ROTARY = [
    (dict(Q=0), {}, BAD), (dict(Qout=0), {}, BAD), (dict(K=0), {}, BAD), (dict(Kout=0), {}, BAD),
    (dict(positions=0), {}, BAD), (dict(inv_freq=0), {}, BAD), (dict(K=0, Kout=0), {}, BAD), (dict(kv_heads=0), {}, BAD),
    (dict(batch=0), {}, BAD), (dict(seq=0), {}, BAD), (dict(rot=0), {}, BAD), (dict(rot=7), {}, BAD), (dict(rot=66), {}, BAD),
    (dict(dtype=3), {}, BAD), ({}, dict(interleaved=2), BAD), ({}, dict(inverse=-1), BAD), ({}, dict(scale=-1.0), BAD),
    ({}, dict(scale=math.nan), BAD), ({}, dict(positions_int64=3), BAD), ({}, dict(q_strides=(64, 0, 64)), BAD),
    ({}, dict(kout_strides=(64, 64, -64)), BAD),
    (dict(head_dim=2048, rot=64), {}, UNSUP), (dict(batch=1 << 16, seq=1 << 16), {}, UNSUP), (dict(heads=1 << 17), {}, UNSUP),
    (dict(Q=P + 1), {}, MISAL), (dict(positions=P + 4), dict(positions_int64=1), MISAL), (dict(inv_freq=P + 2), {}, MISAL),
]


def call_rotary(a, o):
    f = dict(Q=P, K=P, Qout=P, Kout=P, positions=P, inv_freq=P, batch=2, heads=4, kv_heads=2, seq=30, head_dim=64, rot=64,
             dtype=1)
    f.update(a)
    return tg.tl_rotary(f["Q"], f["K"], f["Qout"], f["Kout"], f["positions"], f["inv_freq"], f["batch"], f["heads"],
                        f["kv_heads"], f["seq"], f["head_dim"], f["rot"], f["dtype"], 0, tg.RotaryOptions(**o))


@pytest.mark.parametrize("n", range(len(ROTARY)))
def test_rotary_refusals(n):
    a, o, status = ROTARY[n]
    assert call_rotary(a, o) == status


class Fake:
    """Stands in for a CUDA tensor where there is none: it carries what the binding's checks read."""

    def __init__(self, shape, dtype=torch.bfloat16, device="cuda:0", stride=None, ptr=P, requires_grad=False):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda, self.ptr, self.requires_grad = self.device.type == "cuda", ptr, requires_grad
        dense = [int(np.prod(shape[i + 1:])) for i in range(len(shape))]
        self._stride = tuple(dense if stride is None else stride)
        self._dense = stride is None

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return self._dense

    def data_ptr(self):
        return self.ptr


def qkv(**k):
    return Fake((2, 4, 50, 64), **k), Fake((2, 2, 60, 64)), Fake((2, 2, 60, 64))


I32 = torch.int32


def attention_cases(f):
    q, k, v = qkv()
    return [
        lambda: f(Fake((2, 4, 50, 64), device="cpu"), k, v),
        lambda: f(q, Fake((2, 3, 60, 64)), Fake((2, 3, 60, 64))),
        lambda: f(q, k, Fake((2, 2, 61, 64))),
        lambda: f(q, Fake((2, 2, 60, 64), device="cuda:1"), v),
        lambda: f(q, Fake((2, 2, 60, 64), torch.float16), v),
        lambda: f(Fake((2, 4, 50, 64), stride=(12800, 3200, 64, 2)), k, v),
        lambda: f(Fake((2, 4, 50, 64), stride=(12800, 3200, 60, 1)), k, v),
        lambda: f(Fake((2, 4, 50, 64), stride=(0, 3200, 64, 1)), k, v),
        lambda: f(Fake((2, 4, 50, 64), ptr=P + 2), k, v),
        lambda: f(q, k, v, slopes=Fake((3,), torch.float32)),
        lambda: f(q, k, v, slopes=Fake((4,), torch.float16)),
        lambda: f(q, k, v, slopes=Fake((4,), torch.float32, requires_grad=True)),
        lambda: f(q, k, v, doc_offsets=Fake((2, 1), I32)),
        lambda: f(q, k, v, doc_offsets=Fake((3, 4), I32)),
        lambda: f(q, k, v, doc_offsets=Fake((2, 4), torch.int64)),
        lambda: f(q, k, v, doc_offsets=torch.zeros((2, 4), dtype=I32)),
        lambda: f(q, k, v, prefix=Fake((2, 1), I32)),
        lambda: f(q, k, v, causal=True, prefix=Fake((2, 2), I32)),
        lambda: f(q, k, v, causal=True, doc_offsets=Fake((2, 4), I32), prefix=Fake((2, 1), I32)),
        lambda: f(q, k, v, q_offset=-1),
        lambda: f(q, k, v, score_cap=-2.0),
        lambda: f(q, k, v, scale=math.nan),
    ]


def forward(q, k, v, **kw):
    return tg.attention_ex(q, k, v, **kw)


def backward(q, k, v, **kw):
    return tg.attention_backward(Fake(q.shape), q, k, v, Fake(q.shape), Fake(q.shape[:3], torch.float32), **kw)


def other_cases():
    q, k, v = qkv()
    do, lse = Fake((2, 4, 50, 64)), Fake((2, 4, 50), torch.float32)
    tq, kc = Fake((2, 4, 3, 64)), Fake((9, 16, 2, 64))
    table, ctx = Fake((2, 4), I32), Fake((2,), I32)
    pos, inv = Fake((2, 50), I32), Fake((32,), torch.float32)
    F32 = torch.float32
    return [
        lambda: tg.attention_ex(q, k, v, out=Fake((2, 4, 50, 64), torch.float16)),
        lambda: tg.attention_ex(q, k, v, out=Fake((2, 4, 50, 64), device="cuda:1")),
        lambda: tg.attention_ex(q, k, v, lse=Fake((2, 4, 51), F32)),
        lambda: tg.attention_ex(q, k, v, lse=torch.zeros(2, 4, 50)),
        lambda: tg.attention_backward(Fake((2, 4, 51, 64)), q, k, v, do, lse),
        lambda: tg.attention_backward(do, q, k, v, do, Fake((2, 4, 50))),
        lambda: tg.attention_backward(do, q, k, v, do, lse, dk=Fake((2, 4, 50, 64))),
        lambda: tg.attention_backward(do, q, k, v, do, lse, dv=torch.zeros((2, 2, 60, 64), dtype=torch.bfloat16)),
        lambda: tg.tree_attention(tq, kc, Fake((9, 16, 2, 32)), table, ctx),
        lambda: tg.tree_attention(tq, Fake((9, 16, 3, 64)), Fake((9, 16, 3, 64)), table, ctx),
        lambda: tg.tree_attention(tq, kc, kc, Fake((3, 4), I32), ctx),
        lambda: tg.tree_attention(tq, kc, kc, Fake((2, 4), torch.int64), ctx),
        lambda: tg.tree_attention(tq, kc, kc, Fake((2, 4), I32, stride=(8, 1)), ctx),
        lambda: tg.tree_attention(tq, kc, kc, table, Fake((3,), I32)),
        lambda: tg.tree_attention(tq, kc, kc, table, torch.zeros(2, dtype=I32)),
        lambda: tg.tree_attention(tq, kc, kc, table, ctx, Fake((2, 4), I32)),
        lambda: tg.tree_attention(tq, kc, kc, table, ctx, tree_lens=Fake((2,), torch.int64)),
        lambda: tg.tree_attention(tq, kc, kc, table, ctx, out=Fake((2, 4, 4, 64))),
        lambda: tg.tree_attention(tq, kc, kc, table, ctx, slopes=Fake((2,), F32)),
        lambda: tg.rotary(Fake((4, 50, 64)), None, pos, inv),
        lambda: tg.rotary(q, Fake((2, 2, 49, 64)), pos, inv),
        lambda: tg.rotary(q, None, Fake((2, 49), I32), inv),
        lambda: tg.rotary(q, None, Fake((2, 50), F32), inv),
        lambda: tg.rotary(q, None, torch.zeros((2, 50), dtype=I32), inv),
        lambda: tg.rotary(q, None, pos, Fake((33,), F32)),
        lambda: tg.rotary(q, None, pos, Fake((32,), torch.float64)),
        lambda: tg.rotary(q, None, pos, inv, scale=0.0),
        lambda: tg.rotary(q, None, pos, inv, out_k=q),
        lambda: tg.rotary(q, None, pos, inv, out_q=Fake((2, 4, 50, 64), stride=(12800, 3200, 64, 2))),
    ]


@pytest.mark.parametrize("n", range(22 + 22 + 29))
def test_the_binding_refuses_before_any_launch(n, monkeypatch):
    cases = attention_cases(forward) + attention_cases(backward) + other_cases()
    assert len(cases) == 73

    def no_launch(*a, **k):
        raise AssertionError("the C ABI was called with arguments the binding should have refused")

    for name in ("tl_attention_ex", "tl_attention_bwd", "tl_tree_attention", "tl_rotary"):
        monkeypatch.setattr(tg, name, no_launch)
    with pytest.raises(ValueError):
        cases[n]()


def test_types_are_refused():
    q = Fake((2, 4, 50, 64), torch.float32)
    with pytest.raises(TypeError):
        tg.attention_ex(q, q, q)
    with pytest.raises(TypeError):
        tg.rotary(q, None, Fake((2, 50), I32), Fake((32,), torch.float32))


def test_structs_match_the_header():
    """Sizes by the C compiler's own layout rules (natural alignment, 64-bit)."""
    assert ctypes.sizeof(tg.AttentionOptions) == 16 + 6 * 8 + 8 * 24
    assert ctypes.sizeof(tg.TreeOptions) == 8 + 2 * 8 + 4 * 24
    assert ctypes.sizeof(tg.RotaryOptions) == 24 + 4 * 24
    for packed, cls in ((tg.ATTENTION_OPTIONS, tg.AttentionOptions), (tg.TREE_OPTIONS, tg.TreeOptions),
                        (tg.ROTARY_OPTIONS, tg.RotaryOptions)):
        n = sum(3 if name.endswith("strides") else 1 for name, _ in cls._fields_)
        given = [i + 1 for i in range(n)]
        o = cls.from_buffer_copy(packed.pack(*given))
        flat = []
        for name, _ in cls._fields_:
            v = getattr(o, name)
            flat += list(v) if name.endswith("strides") else [v]
        assert packed.size == ctypes.sizeof(cls) and flat == given
    header = open(os.path.join(os.path.dirname(__file__), "..", "include", "tl_gemm.h")).read()
    header = re.sub(r"/\*.*?\*/", "", header, flags=re.S)
    for struct, cls in (("tl_attention_options", tg.AttentionOptions), ("tl_tree_options", tg.TreeOptions),
                        ("tl_rotary_options", tg.RotaryOptions)):
        body = header[:header.index("} " + struct + ";")].rsplit("typedef struct {", 1)[1]
        place = [body.index(name) for name, _ in cls._fields_]
        assert place == sorted(place), struct


def test_frequencies():
    base = [10000.0 ** (-2 * i / 64) for i in range(32)]
    f, s = tg.rotary_frequencies(64)
    assert s == 1.0 and np.allclose(f.numpy(), base, rtol=2 ** -23)
    f, s = tg.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert s == 1.0 and np.allclose(f.numpy(), np.array(base) / 4, rtol=2 ** -23)
    # ntk: the fastest pair stays, the slowest is stretched by the factor
    f, s = tg.rotary_frequencies(64, scaling="ntk", factor=8.0)
    assert s == 1.0 and f[0] == 1.0 and np.isclose(f[-1].item(), base[-1] / 8, rtol=1e-6)
    # yarn: pairs that turn more than 32 times over 4096 positions stay, under one turn they are divided
    f, s = tg.rotary_frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    turns = 4096 * np.array(base) / (2 * math.pi)
    ratio = f.numpy() / np.array(base)
    assert np.isclose(s, 0.1 * math.log(8.0) + 1)
    assert np.allclose(ratio[turns > 34 * 1.4], 1, rtol=1e-6) and np.allclose(ratio[turns < 1 / 1.4], 1 / 8, rtol=1e-6)
    assert np.all(np.diff(ratio) <= 1e-6)
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, factor=0.5), dict(rot_dim=64, base=0.0),
                dict(rot_dim=64, scaling="dynamic"), dict(rot_dim=64, scaling="yarn", factor=2.0),
                dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            tg.rotary_frequencies(**bad)
