"""B200-native (sm_100a) fused tensor-core GEMM:  C = epilogue(A . B).

The work runs in libtlgemm.so (hand-written tcgen05 / TMA kernels behind a C
ABI, include/tl_gemm.h).  This package is its Python binding: the raw C-ABI
calls (``tl_gemm``, ``tl_gemm_ex``, ``tl_check_device``, ``tl_gemm_plan`` ...)
on device pointers, and ``gemm``, ``attention``, ``attention_ex``,
``attention_backward``, ``tree_attention``, ``rotary``, ``softmax`` and
``vector_add``, which take torch CUDA tensors and pass their pointers and the
current stream.  PyTorch only provides device memory
and streams; nothing here computes.

Importing the package fails if the library is not built -- there is no CPU
or library fallback.
"""
from __future__ import annotations

from ._binding import (  # noqa: F401
    ATTENTION_OPTIONS, LIB_PATH, ROTARY_OPTIONS, TREE_OPTIONS, AttentionOptions, Options, Plan, RotaryOptions, Status, TLError, TreeOptions, TL_BF16, TL_EPI_BIAS, TL_EPI_BIAS_GELU, TL_EPI_GELU,
    TL_EPI_NONE, TL_EPI_BIAS_GELU_TANH, TL_EPI_GELU_TANH, TL_EPI_WITH_BIAS, TL_F16,
    SIGNATURES, tl_attention_bwd, tl_attention_ex, tl_attention_fwd, tl_rotary, tl_tree_attention, tl_check_device, tl_config_name, tl_gemm, tl_gemm_ex, tl_gemm_noalloc,
    tl_gemm_plan, tl_num_configs, tl_softmax_rows, tl_vector_add,
    tl_status_string, tl_version,
)

__all__ = [
    "gemm", "attention", "attention_ex", "attention_backward", "tree_attention", "rotary", "rotary_frequencies",
    "AttentionOptions", "TreeOptions", "RotaryOptions", "tl_attention_ex", "tl_attention_bwd", "tl_tree_attention",
    "tl_rotary", "softmax", "vector_add", "check_device", "plan", "configs", "tl_attention_fwd",
    "tl_softmax_rows", "tl_vector_add", "Options", "Plan", "Status", "TLError",
    "tl_gemm", "tl_gemm_ex", "tl_gemm_noalloc", "tl_check_device", "tl_gemm_plan", "tl_num_configs", "tl_config_name",
    "tl_status_string", "tl_version", "TL_F16", "TL_BF16", "TL_EPI_NONE", "TL_EPI_BIAS_GELU",
    "TL_EPI_BIAS", "TL_EPI_GELU", "TL_EPI_BIAS_GELU_TANH", "TL_EPI_GELU_TANH",
]


_DTYPE_CODES = {}  # torch's dtypes: filled at the first call, as torch is imported late


def _dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        import torch
        _DTYPE_CODES.update({torch.float16: TL_F16, torch.bfloat16: TL_BF16})
        code = _DTYPE_CODES.get(t.dtype)
        if code is None:
            raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")
    return code


_EPILOGUES = {None: TL_EPI_NONE, "none": TL_EPI_NONE, "bias_gelu": TL_EPI_BIAS_GELU,
              "bias+gelu": TL_EPI_BIAS_GELU, "bias": TL_EPI_BIAS, "gelu": TL_EPI_GELU,
              "bias_gelu_tanh": TL_EPI_BIAS_GELU_TANH, "gelu_tanh": TL_EPI_GELU_TANH}


def _require_device_tensor(name, t, device, dtype=None, shape=None):
    """Raise ValueError unless `t` is a contiguous CUDA tensor on `device` (and
    of `dtype` / `shape` when given): a host or foreign-device pointer must
    never reach a kernel's loads or stores."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _epi_code(epilogue):
    if isinstance(epilogue, int) and TL_EPI_NONE <= epilogue <= TL_EPI_GELU_TANH:
        return epilogue
    if epilogue in _EPILOGUES:
        return _EPILOGUES[epilogue]
    raise ValueError(f"unknown epilogue {epilogue!r}")


def gemm(A, B, bias=None, epilogue=None, out=None, stream=None, config: int = 0, timeout_ns: int = 0,
         no_split: bool = False, b_transposed: bool = False, out_dtype=None, raster_group: int = 0,
         force_split: bool = False):
    """C = epilogue(A @ B) for row-major CUDA tensors A (M x K) and B (K x N),
    or B given as N x K (``b_transposed=True``: C = epilogue(A @ B.T), the
    layout of a linear layer's weight).

    ``epilogue`` is None / "none", "bias_gelu", "bias", "gelu",
    "bias_gelu_tanh" or "gelu_tanh" (``bias`` of length N for the ones that
    name it; default "bias_gelu" when a bias is given).  C has A's dtype, or
    float32 with ``out_dtype=torch.float32`` (or a float32 ``out``): the
    epilogue's fp32 result without rounding to 16 bits.  ``out`` (M x N) is
    written if given, else allocated.  Runs asynchronously on ``stream``
    (default: torch's current stream).  ``config`` = k > 0 forces kernel
    configuration k - 1; ``raster_group`` > 0 sets the output-tile rows per
    rasterisation group.
    """
    import torch
    epi = _epi_code(epilogue if epilogue is not None else ("bias_gelu" if bias is not None else None))
    k_of_b = B.shape[1] if (b_transposed and B.dim() == 2) else (B.shape[0] if B.dim() == 2 else None)
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != k_of_b:
        raise ValueError(f"shapes {tuple(A.shape)} and {tuple(B.shape)} do not chain")
    for name, t in (("A", A), ("B", B)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if B.device != A.device:
        raise ValueError(f"B is on {B.device}, A on {A.device}")
    dt = _dtype_code(A)
    if B.dtype != A.dtype:
        raise TypeError("A and B must have the same dtype")
    M, K = A.shape
    N = B.shape[0] if b_transposed else B.shape[1]
    if epi in TL_EPI_WITH_BIAS:
        if bias is None:
            raise ValueError("this epilogue needs a contiguous CUDA bias of length N in the input dtype")
        _require_device_tensor("bias", bias, A.device, A.dtype, (N,))
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else A.dtype
    if out_dtype not in (A.dtype, torch.float32):
        raise TypeError("C is either A's dtype or float32")
    c_f32 = out_dtype == torch.float32
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    else:
        _require_device_tensor("out", out, A.device, out_dtype, (M, N))
    s = stream if stream is not None else torch.cuda.current_stream(A.device)
    bias_ptr = bias.data_ptr() if bias is not None and epi in TL_EPI_WITH_BIAS else 0
    with torch.cuda.device(A.device):
        if config or timeout_ns or no_split or b_transposed or c_f32 or raster_group or force_split:
            opt = Options(config=config, inject_fault=0, timeout_ns=timeout_ns, no_split=int(no_split),
                          b_layout=int(bool(b_transposed)), c_float32=int(c_f32), raster_group=raster_group,
                          force_split=int(bool(force_split)))
            st = tl_gemm_ex(A.data_ptr(), B.data_ptr(), bias_ptr, out.data_ptr(), M, N, K, dt, epi,
                            s.cuda_stream, opt)
        else:
            st = tl_gemm(A.data_ptr(), B.data_ptr(), bias_ptr, out.data_ptr(), M, N, K, dt, epi, s.cuda_stream)
    if st != 0:
        raise TLError(st, "tl_gemm")
    return out


def attention(q, k, v, causal: bool = False, scale: float = 0.0, out=None, lse=None, stream=None):
    """softmax(scale q k^T [causal]) v for CUDA tensors q (B, H, Sq, D) and
    k, v (B, H, Sk, D), fp16 or bf16, D in {64, 128}; scale 0 = 1/sqrt(D).
    Returns out (B, H, Sq, D); fills `lse` (B, H, Sq) float32 if given."""
    import torch
    if q.dim() != 4 or k.shape != v.shape or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError(f"shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} do not match")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require_device_tensor(name, t, q.device, q.dtype)
    dt = _dtype_code(q)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    # every given tensor is checked before anything is allocated
    if lse is not None:
        _require_device_tensor("lse", lse, q.device, torch.float32, (B, H, Sq))
    if out is None:
        out = torch.empty_like(q)
    else:
        _require_device_tensor("out", out, q.device, q.dtype, q.shape)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device):
        st = tl_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr() if lse is not None else 0, B, H, Sq, Sk, D, dt, causal, scale,
                              s.cuda_stream)
    if st != 0:
        raise TLError(st, "tl_attention_fwd")
    return out


# None of the calls records anything for autograd: outputs carry no graph,
# whatever the inputs ask for.  A training program calls the backward itself, from
# a torch.autograd.Function or its own loop.
#
# The calls below run as often as a model has layers and tokens, so their checks
# are written to cost little: each tensor's strides are read once, the option
# structs are packed in one go, the device is only switched when it has to be.

def _refuse(name, t, device, dtype, shape):
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _new_like(torch, t, stream):
    """An output laid out like `t`, its memory taken for the stream that writes it, and its strides."""
    if stream is None:
        y = torch.empty_like(t)
    else:
        with torch.cuda.stream(stream):
            y = torch.empty_like(t)
    s0, s1, s2, s3 = y.stride()
    if s3 != 1:  # `t`'s rows overlap a value apart, which leaves open what is innermost: as of a contiguous tensor
        n = y.shape
        s0, s1, s2 = n[1] * n[2] * n[3], n[2] * n[3], n[3]
        y = y.as_strided(n, (s0, s1, s2, 1))
    return y, (s0, s1, s2)


def _rows(name, t, device, dtype, shape):
    """The strides of (outer, middle, row) of a 4-D CUDA tensor, for the C ABI;
    ValueError unless it lies on the CUDA device `device`, has `dtype` and `shape`, a contiguous
    last dimension, positive strides in multiples of 8 elements and a 16-byte
    aligned base."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(name, t, device, dtype, shape)
    return _strides(name, t)


def _strides(name, t):
    st = t.stride()
    s0, s1, s2, s3 = st
    if s3 != 1 or s0 <= 0 or s1 <= 0 or s2 <= 0 or (s0 | s1 | s2) & 7:
        # a dimension of one element takes any stride
        n = t.shape
        s0, s1, s2 = (s if n[i] > 1 else n[3] for i, s in enumerate((s0, s1, s2)))
        if s3 != 1 or s0 <= 0 or s1 <= 0 or s2 <= 0 or (s0 | s1 | s2) & 7:
            raise ValueError(f"{name} must have a contiguous last dimension and positive strides in multiples of 8 "
                             f"elements, got strides {tuple(st)}")
    if t.data_ptr() & 15:
        raise ValueError(f"{name} must be 16-byte aligned")
    return s0, s1, s2


def _flat(name, t, device, dtype, shape):
    """ValueError unless `t` is a contiguous CUDA tensor on `device` of `dtype` and `shape`."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(name, t, device, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The smallest and largest positive float32: what the options hold scales and caps in
_F32_MIN, _F32_MAX = 2.0 ** -149, (2.0 - 2.0 ** -23) * 2.0 ** 127


def _score_arguments(scale, score_cap, slopes, heads, device):
    """The softmax scale, cap and bias slopes, checked; returns the slopes' pointer."""
    if (scale != 0.0 and not _F32_MIN <= scale <= _F32_MAX) or (score_cap != 0.0 and not _F32_MIN <= score_cap <= _F32_MAX):
        raise ValueError("scale and score_cap must be 0 or positive numbers that float32 holds")
    if slopes is None:
        return 0
    import torch
    _flat("slopes", slopes, device, torch.float32, (heads,))
    if slopes.requires_grad:
        raise ValueError("slopes are constants: they get no gradient")
    return slopes.data_ptr()


def _launch(torch, device, stream, options, what, call, *args):
    """call(*args, raw stream, options) with `device` current, on `stream` or torch's current one; raises TLError."""
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        st = call(*args, raw, options)
    else:
        with torch.cuda.device(device):
            st = call(*args, raw, options)
    if st != 0:
        raise TLError(st, what)


def _attention_arguments(q, k, v, causal, scale, score_cap, slopes, doc_offsets, prefix, q_offset):
    """Checks what attention_ex and attention_backward share; returns the leading
    option fields, the strides of q, k and v, and the dtype code."""
    import torch
    dims = q.dim()
    if dims != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError(f"shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} do not match")
    B, H, _, D = q.shape
    Bk, Hk, _, Dk = k.shape
    if B != Bk or D != Dk or Hk < 1 or H % Hk:
        raise ValueError(f"shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} do not match")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dt = _dtype_code(q)
    dev, dtype = q.device, q.dtype
    if k.dtype is not dtype or k.device != dev:
        _refuse("k", k, dev, dtype, k.shape)
    if v.dtype is not dtype or v.device != dev:
        _refuse("v", v, dev, dtype, v.shape)
    strides = _strides("q", q) + _strides("k", k) + _strides("v", v)
    slopes_ptr = _score_arguments(scale, score_cap, slopes, H, dev)
    docs = docs_ptr = prefix_ptr = 0
    if doc_offsets is not None:
        if doc_offsets.dim() != 2 or doc_offsets.shape[1] < 2:
            raise ValueError(f"doc_offsets must be (batch, documents + 1), got {tuple(doc_offsets.shape)}")
        docs = doc_offsets.shape[1] - 1
        _flat("doc_offsets", doc_offsets, dev, torch.int32, (B, docs + 1))
        docs_ptr = doc_offsets.data_ptr()
    if prefix is not None:
        if not causal:
            raise ValueError("a prefix needs causal=True (without it every key is seen already)")
        _flat("prefix", prefix, dev, torch.int32, (B, max(docs, 1)))
        prefix_ptr = prefix.data_ptr()
    if q_offset < 0:
        raise ValueError("q_offset must not be negative")
    return (1 if causal else 0, scale, score_cap, 0, slopes_ptr, docs_ptr, docs, prefix_ptr, q_offset, Hk), strides, dt


_DENSE = (0, 0, 0)


def attention_ex(q, k, v, *, causal: bool = False, scale: float = 0.0, score_cap: float = 0.0, slopes=None,
                 doc_offsets=None, prefix=None, q_offset: int = 0, out=None, lse=None, stream=None):
    """Attention forward of language models, for CUDA tensors q (B, H, Sq, D)
    and k, v (B, Hkv, Sk, D), fp16 or bf16, D in {64, 128}, H a multiple of Hkv,
    of any strides in multiples of 8 with a contiguous last dimension.

    Scores are scale q.k (scale 0 = 1/sqrt(D)), capped as
    score_cap * tanh(. / score_cap) when score_cap > 0, less
    slopes[h] * |q_offset + i - j| when ``slopes`` (H floats) is given.  Query i
    stands at key q_offset + i.  ``causal`` hides the keys behind it;
    ``doc_offsets`` (B, docs + 1) int32, ascending, keeps each query inside its
    document (positions outside the first to the last offset see nothing);
    ``prefix`` (B, max(docs, 1)) int32 opens the first keys of each document (of
    the sequence) to causal queries.  Queries that see nothing give 0 and lse
    -inf.  Rows of k and v that no query sees -- a padded end, too -- must be
    finite, and so must their products with the rows of the others: a weight of 0
    times NaN is NaN.  Returns out, shaped and by default laid out like q; fills
    ``lse`` (B, H, Sq) float32 if given.  ``out`` must not overlap an input.

    out carries no autograd graph; its gradients are attention_backward's, from
    out and ``lse``."""
    import torch
    head, strides, dt = _attention_arguments(q, k, v, causal, scale, score_cap, slopes, doc_offsets, prefix, q_offset)
    B, H, Sq, D = q.shape
    dev = q.device
    lse_ptr = 0
    if lse is not None:
        _flat("lse", lse, dev, torch.float32, (B, H, Sq))
        lse_ptr = lse.data_ptr()
    if out is None:
        out, so = _new_like(torch, q, stream)
    else:
        so = _rows("out", out, dev, q.dtype, q.shape)
    opt = ATTENTION_OPTIONS.pack(*head, *strides, *so, *_DENSE, *_DENSE, *_DENSE, *_DENSE)
    _launch(torch, dev, stream, opt, "tl_attention_ex", tl_attention_ex, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            out.data_ptr(), lse_ptr, B, H, Sq, k.shape[2], D, dt)
    return out


def attention_backward(dout, q, k, v, out, lse, *, causal: bool = False, scale: float = 0.0, score_cap: float = 0.0,
                       slopes=None, doc_offsets=None, prefix=None, q_offset: int = 0, dq=None, dk=None, dv=None,
                       stream=None):
    """Gradients (dq, dk, dv) of attention_ex, from its inputs, its ``out`` and
    ``lse`` and the gradient ``dout`` of out; the options are the forward's.
    dk and dv are summed over the heads that share them.  What no query sees, and
    queries that see nothing, do not count but must be finite, as must their
    products with the other rows.  The gradients must overlap neither the inputs nor
    one another.  Results repeat bit for bit.  ``slopes`` are constants (a tensor that requires grad is refused)."""
    import torch
    head, strides, dt = _attention_arguments(q, k, v, causal, scale, score_cap, slopes, doc_offsets, prefix, q_offset)
    B, H, Sq, D = q.shape
    dev, dtype = q.device, q.dtype
    sdo = _rows("dout", dout, dev, dtype, q.shape)
    so = _rows("out", out, dev, dtype, q.shape)
    _flat("lse", lse, dev, torch.float32, (B, H, Sq))
    # every given tensor is checked before anything is allocated
    grads = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        grads.append((g, None if g is None else _rows(name, g, dev, dtype, like.shape), like))
    grads = [(g, sg) if g is not None else _new_like(torch, like, stream) for g, sg, like in grads]
    (dq, sdq), (dk, sdk), (dv, sdv) = grads
    opt = ATTENTION_OPTIONS.pack(*head, *strides, *so, *sdo, *sdq, *sdk, *sdv)
    _launch(torch, dev, stream, opt, "tl_attention_bwd", tl_attention_bwd, dout.data_ptr(), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), out.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Sq,
            k.shape[2], D, dt)
    return dq, dk, dv


def tree_attention(q, k_cache, v_cache, block_table, context_lens, parents=None, *, tree_lens=None,
                   scale: float = 0.0, score_cap: float = 0.0, slopes=None, out=None, lse=None, stream=None):
    """Attention of the new tokens q (B, H, T, D), T up to 64, over paged caches
    k_cache, v_cache (pages, page_size, Hkv, D): one token a request (decoding),
    a drafted chain, or a drafted tree.

    Request b has context_lens[b] keys in the cache and its new tokens' keys
    directly behind them, already written; key n is row n % page_size of page
    block_table[b, n // page_size] ((B, max_pages) int32).  Token t sees the
    context, itself and its ancestors by ``parents`` (B, T) int32 (an earlier
    token, or -1; None: a chain).  ``tree_lens`` (B,) int32 gives shorter trees:
    out and lse of later tokens stay as they were.  Scale, cap and bias as in
    attention_ex, a new token standing at context_lens[b] plus its depth.
    Returns out, like q, without an autograd graph; fills ``lse`` (B, H, T) float32
    if given."""
    import torch
    if q.dim() != 4 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError(f"shapes q{tuple(q.shape)} k_cache{tuple(k_cache.shape)} v_cache{tuple(v_cache.shape)} "
                         "do not match")
    B, H, T, D = q.shape
    pages, page_size, Hk, Dk = k_cache.shape
    if D != Dk or Hk < 1 or H % Hk:
        raise ValueError(f"shapes q{tuple(q.shape)} k_cache{tuple(k_cache.shape)} do not match")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dt = _dtype_code(q)
    dev, dtype, i32 = q.device, q.dtype, torch.int32
    if k_cache.dtype is not dtype or k_cache.device != dev:
        _refuse("k_cache", k_cache, dev, dtype, k_cache.shape)
    if v_cache.dtype is not dtype or v_cache.device != dev:
        _refuse("v_cache", v_cache, dev, dtype, v_cache.shape)
    sq, sk, sv = _strides("q", q), _strides("k_cache", k_cache), _strides("v_cache", v_cache)
    if block_table.dim() != 2 or block_table.shape[1] < 1:
        raise ValueError(f"block_table must be (batch, pages), got {tuple(block_table.shape)}")
    max_pages = block_table.shape[1]
    _flat("block_table", block_table, dev, i32, (B, max_pages))
    _flat("context_lens", context_lens, dev, i32, (B,))
    parents_ptr = lens_ptr = lse_ptr = 0
    if parents is not None:
        _flat("parents", parents, dev, i32, (B, T))
        parents_ptr = parents.data_ptr()
    if tree_lens is not None:
        _flat("tree_lens", tree_lens, dev, i32, (B,))
        lens_ptr = tree_lens.data_ptr()
    slopes_ptr = _score_arguments(scale, score_cap, slopes, H, dev)
    if lse is not None:
        _flat("lse", lse, dev, torch.float32, (B, H, T))
        lse_ptr = lse.data_ptr()
    if out is None:
        out, so = _new_like(torch, q, stream)
    else:
        so = _rows("out", out, dev, dtype, q.shape)
    opt = TREE_OPTIONS.pack(scale, score_cap, slopes_ptr, 0, *sq, *so, *sk, *sv)
    _launch(torch, dev, stream, opt, "tl_tree_attention", tl_tree_attention, q.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), parents_ptr, lens_ptr, out.data_ptr(),
            lse_ptr, B, H, Hk, T, pages, page_size, max_pages, D, dt)
    return out


def _rotary_rows(name, t, device, dtype, shape):
    """The strides of a 4-D tensor for rotary, any positive ones with a contiguous last dimension."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(name, t, device, dtype, shape)
    return _rotary_strides(name, t)


def _rotary_strides(name, t):
    s0, s1, s2, s3 = t.stride()
    if s0 <= 0 or s1 <= 0 or s2 <= 0:  # a dimension of one element takes any stride
        n = t.shape
        s0, s1, s2 = (s if n[i] > 1 else n[3] for i, s in enumerate((s0, s1, s2)))
    if s3 != 1 or s0 <= 0 or s1 <= 0 or s2 <= 0:
        raise ValueError(f"{name} must have a contiguous last dimension and positive strides")
    return s0, s1, s2


def rotary(q, k, positions, inv_freq, *, interleaved: bool = False, scale: float = 1.0, inverse: bool = False,
           out_q=None, out_k=None, stream=None):
    """Rotary positions of q (B, H, S, D) and k (B, Hkv, S, D) (or None), fp16 or
    bf16, any positive strides with a contiguous last dimension; returns
    (out_q, out_k).

    ``positions`` is (B, S) or (S,), int32 or int64; ``inv_freq`` (float32, half
    the rotated values) comes from rotary_frequencies or a model.  The first
    2 * len(inv_freq) values of a head are rotated in pairs (i, i + half), or
    (2 i, 2 i + 1) when ``interleaved``, and multiplied by ``scale``; the rest is
    copied.  ``inverse`` turns back: it is the backward of the same call, on the
    gradients (the outputs carry no autograd graph).  ``out_q`` may be q and
    ``out_k`` may be k."""
    import torch
    if q.dim() != 4 or not q.is_cuda:
        raise ValueError("q must be a 4-D CUDA tensor")
    dt = _dtype_code(q)
    B, H, S, D = q.shape
    dev, dtype = q.device, q.dtype
    sq, sk, sok, Hk = _rotary_strides("q", q), _DENSE, _DENSE, 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be 4-D")
        Hk = k.shape[1]
        sk = _rotary_rows("k", k, dev, dtype, (B, Hk, S, D))
    elif out_k is not None:
        raise ValueError("out_k without k")
    shared = positions.dim() == 1
    if positions.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"positions must be int32 or int64, got {positions.dtype}")
    _flat("positions", positions, dev, positions.dtype, (S,) if shared else (B, S))
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D")
    half = inv_freq.shape[0]
    _flat("inv_freq", inv_freq, dev, torch.float32, (half,))
    if not 2 <= 2 * half <= D:
        raise ValueError(f"inv_freq has {half} frequencies for heads of {D} values")
    if not _F32_MIN <= scale <= _F32_MAX:
        raise ValueError("scale must be a positive number that float32 holds")
    # every given tensor is checked before anything is allocated
    if out_q is not None:
        soq = _rotary_rows("out_q", out_q, dev, dtype, q.shape)
    if out_k is not None:
        sok = _rotary_rows("out_k", out_k, dev, dtype, k.shape)
    if out_q is None:
        out_q, soq = _new_like(torch, q, stream)
    k_ptr = ok_ptr = 0
    if k is not None:
        if out_k is None:
            out_k, sok = _new_like(torch, k, stream)
        k_ptr, ok_ptr = k.data_ptr(), out_k.data_ptr()
    opt = ROTARY_OPTIONS.pack(1 if interleaved else 0, 1 if inverse else 0, scale, positions.dtype == torch.int64, shared,
                              0, *sq, *sk, *soq, *sok)
    _launch(torch, dev, stream, opt, "tl_rotary", tl_rotary, q.data_ptr(), k_ptr, out_q.data_ptr(), ok_ptr,
            positions.data_ptr(), inv_freq.data_ptr(), B, H, Hk, S, D, 2 * half, dt)
    return out_q, out_k


def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq, scale) for rotary: base^(-2 i / rot_dim), i < rot_dim / 2, as
    float32 on ``device``, and the factor of the rotated values.

    ``scaling`` serves contexts ``factor`` times the trained length: "linear"
    divides every frequency by it; "ntk" raises the base by
    factor^(rot_dim / (rot_dim - 2)), so that only the slow pairs stretch;
    "yarn" divides the pairs that turn fewer than ``beta_slow`` times over
    ``original_length`` positions, keeps those that turn more than ``beta_fast``
    times, blends linearly in the pair's index in between (from the whole indices
    around those two, 0 at least and rot_dim - 1 at most, which may lie behind the
    last pair), and returns the scale 0.1 ln(factor) + 1 (else the scale is 1)."""
    import math

    import torch
    if rot_dim < 2 or rot_dim % 2 or not base > 0 or not factor >= 1.0:
        raise ValueError("rot_dim must be even and positive, base positive, factor at least 1")
    half = rot_dim // 2
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim of 4 at least")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    scale = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if original_length < 1 or not beta_fast > beta_slow > 0 or not base > 1:
            raise ValueError("yarn needs original_length, beta_fast > beta_slow > 0 and a base above 1")

        def index(turns):  # the pair that turns so many times over original_length positions
            return rot_dim * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        # the upper end may lie behind the last pair: then no pair is divided whole
        lo = max(math.floor(index(beta_fast)), 0)
        hi = min(math.ceil(index(beta_slow)), rot_dim - 1)
        for i in range(half):
            blend = 1.0 if i >= hi else max((i - lo) / (hi - lo), 0.0) if hi > lo else 0.0  # 0: kept, 1: divided
            freq[i] = freq[i] * (1.0 - blend) + freq[i] / factor * blend
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(freq, dtype=torch.float32, device=device), scale


def softmax(x, out=None, stream=None):
    """Row softmax of a contiguous 2-D fp16/bf16 CUDA tensor (over the last dim)."""
    import torch
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    dt = _dtype_code(x)
    if out is None:
        out = torch.empty_like(x)
    else:
        _require_device_tensor("out", out, x.device, x.dtype, x.shape)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    with torch.cuda.device(x.device):
        st = tl_softmax_rows(x.data_ptr(), out.data_ptr(), x.shape[0], x.shape[1], dt, s.cuda_stream)
    if st != 0:
        raise TLError(st, "tl_softmax_rows")
    return out


def vector_add(a, b, out=None, stream=None):
    """a + b for contiguous float32 CUDA tensors of one shape."""
    import torch
    if not a.is_cuda:
        raise ValueError("a must be a CUDA tensor")
    _require_device_tensor("a", a, a.device, torch.float32)
    _require_device_tensor("b", b, a.device, torch.float32, a.shape)
    if out is None:
        out = torch.empty_like(a)
    else:
        _require_device_tensor("out", out, a.device, torch.float32, a.shape)
    s = stream if stream is not None else torch.cuda.current_stream(a.device)
    with torch.cuda.device(a.device):
        st = tl_vector_add(a.data_ptr(), b.data_ptr(), out.data_ptr(), a.numel(), s.cuda_stream)
    if st != 0:
        raise TLError(st, "tl_vector_add")
    return out


def check_device(stream=None) -> int:
    """Synchronize and return the device error word (0 = no wait ran out)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    st, word = tl_check_device(s.cuda_stream)
    if st not in (0, int(Status.DEVICE_TIMEOUT)):
        raise TLError(st, "tl_check_device")
    return word


def plan(M, N, K, dtype=TL_F16, epilogue=None, num_sms=148, config=0, ptrs=(256, 256, 256, 256),
         b_transposed=False, no_split=False, c_float32=False, force_split=False, raster_group=0) -> dict:
    """The host plan for a call (no GPU needed): config, grid, padding, store path."""
    a, b, bias, c = ptrs
    epi = _epi_code(epilogue)
    opt = Options(config=config, b_layout=int(b_transposed), no_split=int(no_split), c_float32=int(c_float32),
                  force_split=int(force_split), raster_group=raster_group) \
        if (config or b_transposed or no_split or c_float32 or force_split or raster_group) else None
    st, p = tl_gemm_plan(a, b, bias if epi in TL_EPI_WITH_BIAS else 0, c, M, N, K, dtype, epi, num_sms, opt)
    if st != 0:
        raise TLError(st, "tl_gemm_plan")
    d = p.as_dict()
    d["config_name"] = tl_config_name(d["config"])
    return d


def configs() -> list[str]:
    return [tl_config_name(i) for i in range(tl_num_configs())]
