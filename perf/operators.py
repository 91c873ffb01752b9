"""The operators that the attention of a language model needs next to the plain forward, as
cases that can be run two ways: in elementary torch operations (32 bits, rounded once), and
through this package's calls (`own`).

  forward   attention with capped scores, a distance bias, document and prefix masks, grouped heads
  train     the same forward, then its backward: out, lse and the three gradients
  tree      drafted tokens (one, a chain or a tree) against a paged key/value cache
  rotary    rotary positions of q and k in one call, either layout, part of the head; its inverse
            (the backward) too
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a prompt's prefill in a model that caps its scores, grouped heads
        dict(name="prefill_cap", kind="forward", batch=1, heads=16, kv_heads=8, seq_q=4096, seq_k=4096, head_dim=128,
             dtype="bf16", causal=True, cap=50.0, bias=False, docs=0, prefix=False, offset=0, rows_first=True),
        # a packed pretraining batch's forward: ragged documents, a padded end, a distance bias
        dict(name="packed_bias", kind="forward", batch=2, heads=16, kv_heads=16, seq_q=4096, seq_k=4096, head_dim=64,
             dtype="bf16", causal=True, cap=0.0, bias=True, docs=9, prefix=False, offset=0, rows_first=False),
        # one short chunk of a long prompt: few queries at an offset, an odd count
        dict(name="chunk", kind="forward", batch=1, heads=8, kv_heads=2, seq_q=77, seq_k=1101, head_dim=128,
             dtype="fp16", causal=True, cap=30.0, bias=False, docs=0, prefix=False, offset=1024, rows_first=True),
        # a training step's attention on packed documents, grouped heads
        dict(name="train_docs", kind="train", batch=4, heads=16, kv_heads=4, seq_q=4096, seq_k=4096, head_dim=128,
             dtype="bf16", causal=True, cap=0.0, bias=False, docs=6, prefix=False, offset=0, rows_first=True),
        # fine-tuning of a model with capped scores: whole rows, no documents
        dict(name="train_cap", kind="train", batch=2, heads=16, kv_heads=8, seq_q=2048, seq_k=2048, head_dim=128,
             dtype="bf16", causal=True, cap=50.0, bias=False, docs=0, prefix=False, offset=0, rows_first=True),
        # a small prefix-LM batch: each row's prefix is seen from everywhere, a distance bias, odd lengths
        dict(name="train_prefix", kind="train", batch=3, heads=8, kv_heads=8, seq_q=1001, seq_k=1001, head_dim=64,
             dtype="fp16", causal=True, cap=0.0, bias=True, docs=0, prefix=True, offset=0, rows_first=False),
        # one request, one token: nothing but latency
        dict(name="tree_one", kind="tree", batch=1, heads=16, kv_heads=8, tokens=1, context=900, head_dim=128, page=16,
             dtype="bf16", cap=0.0, bias=False, tree=False, ragged=False),
        # a batch of single tokens over ragged contexts: ordinary decoding
        dict(name="tree_batch", kind="tree", batch=32, heads=32, kv_heads=8, tokens=1, context=8192, head_dim=128,
             page=64, dtype="bf16", cap=0.0, bias=False, tree=False, ragged=True),
        # verification of drafted trees, capped scores, some requests with shorter trees
        dict(name="tree_draft", kind="tree", batch=8, heads=16, kv_heads=4, tokens=31, context=4096, head_dim=128,
             page=32, dtype="bf16", cap=30.0, bias=False, tree=True, ragged=True),
        # two very long contexts, a short drafted chain each
        dict(name="tree_long", kind="tree", batch=2, heads=32, kv_heads=8, tokens=4, context=65536, head_dim=128,
             page=64, dtype="fp16", cap=0.0, bias=False, tree=False, ragged=False),
        # positions of a training batch, from packed projections
        dict(name="rotary_batch", kind="rotary", batch=4, seq=4096, heads=16, kv_heads=4, head_dim=128, rot=128,
             dtype="bf16", interleaved=False, inverse=False, start=0, factor=1.0, scale=1.0),
        # positions of a few decoded tokens far into a long context: part of the head, interleaved, scaled
        dict(name="rotary_far", kind="rotary", batch=32, seq=3, heads=32, kv_heads=8, head_dim=128, rot=96,
             dtype="fp16", interleaved=True, inverse=False, start=500000, factor=8.0, scale=1.2),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "train", "tree", "rotary"])
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    if kind in ("forward", "train"):
        heads = kv * rng.choice([1, 2, 3, 4])
        batch = rng.randint(1, 4)
        seq_q = _spread(rng, 1, 4096)
        while batch * heads * seq_q > 4 * 16 * 4096 // 2:
            seq_q = max(1, seq_q // 2)
        offset = rng.choice([0, 0, rng.randint(1, 2000)])
        causal = rng.random() < 0.8
        return dict(kind=kind, batch=batch, heads=heads, kv_heads=kv, seq_q=seq_q, seq_k=seq_q + offset, head_dim=dim,
                    dtype=dtype, causal=causal, cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]), bias=rng.random() < 0.4,
                    docs=rng.choice([0, 0, rng.randint(1, 12)]), prefix=causal and rng.random() < 0.3, offset=offset,
                    rows_first=rng.random() < 0.5)
    if kind == "tree":
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        context = _spread(rng, 1, 65536)
        batch = _spread(rng, 1, 64)
        while batch * kv * context > 2 * 8 * 65536:
            batch = max(1, batch // 2)
            context = context if batch > 1 else context // 2
        return dict(kind=kind, batch=batch, heads=heads, kv_heads=kv, tokens=rng.choice([1, 1, 2, 5, 8, 17, 33, 64]),
                    context=context, head_dim=dim, page=rng.choice([8, 16, 24, 32, 64, 128, 256]), dtype=dtype,
                    cap=rng.choice([0.0, 30.0, 50.0]), bias=rng.random() < 0.3, tree=rng.random() < 0.5,
                    ragged=rng.random() < 0.7)
    heads = kv * rng.choice([1, 2, 4, 8])
    seq = _spread(rng, 1, 8192)
    batch = _spread(rng, 1, 64)
    while batch * seq * heads > 4 * 4096 * 16:
        batch, seq = max(1, batch // 2), max(1, seq // 2)
    return dict(kind=kind, batch=batch, seq=seq, heads=heads, kv_heads=kv, head_dim=dim,
                rot=rng.choice([dim, dim, dim // 2, dim // 4, dim - 6]), dtype=dtype, interleaved=rng.random() < 0.5,
                inverse=rng.random() < 0.4, start=rng.choice([0, 1000, 100000, 1000000]),
                factor=rng.choice([1.0, 4.0, 8.0]), scale=rng.choice([1.0, 1.0, 1.2]))


# ------------------------------------------------------------------ inputs
def _rand(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def _heads(g, batch, heads, seq, dim, dtype, rows_first, scale=1.0):
    """(batch, heads, seq, dim), laid out so or with a token's heads next to one another."""
    if rows_first:
        return _rand(g, (batch, seq, heads, dim), dtype, scale).transpose(1, 2)
    return _rand(g, (batch, heads, seq, dim), dtype, scale)


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _slopes(heads):
    return torch.pow(2.0, -8.0 * torch.arange(1, heads + 1, device="cuda", dtype=torch.float32) / heads)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}
    if c["kind"] in ("forward", "train"):
        B, H, D = c["batch"], c["heads"], c["head_dim"]
        # capped models see large raw scores
        s["q"] = _heads(g, B, H, c["seq_q"], D, c["dtype"], c["rows_first"], 4.0 if c["cap"] else 1.0)
        s["k"] = _heads(g, B, c["kv_heads"], c["seq_k"], D, c["dtype"], c["rows_first"])
        s["v"] = _heads(g, B, c["kv_heads"], c["seq_k"], D, c["dtype"], c["rows_first"])
        s["slopes"] = _slopes(H) if c["bias"] else None
        s["doc_offsets"] = s["prefix"] = None
        if c["docs"]:
            end = c["seq_k"] - _ints(g, 0, c["seq_k"] // 16 + 1, (B, 1))  # a padded end
            cuts = (torch.rand((B, c["docs"] - 1), generator=g, device="cuda") * end).to(torch.int32)
            s["doc_offsets"] = torch.cat([torch.zeros_like(end), cuts.sort(dim=1).values, end], dim=1).contiguous()
        if c["prefix"]:
            s["prefix"] = _ints(g, 0, c["seq_k"] // (2 * max(c["docs"], 1)) + 2, (B, max(c["docs"], 1)))
        if c["kind"] == "train":
            s["dout"] = _heads(g, B, H, c["seq_q"], D, c["dtype"], c["rows_first"])
    elif c["kind"] == "tree":
        B, T, D, page = c["batch"], c["tokens"], c["head_dim"], c["page"]
        per = -(-(c["context"] + T) // page)
        s["q"] = _rand(g, (B, T, c["heads"], D), c["dtype"], 4.0 if c["cap"] else 1.0).transpose(1, 2)
        s["k_cache"] = _rand(g, (B * per, page, c["kv_heads"], D), c["dtype"])
        s["v_cache"] = _rand(g, (B * per, page, c["kv_heads"], D), c["dtype"])
        s["block_table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        full = torch.full((B,), c["context"], device="cuda", dtype=torch.int32)
        s["context"] = _ints(g, c["context"] // 4, c["context"] + 1, (B,)) if c["ragged"] else full
        s["tree_lens"] = _ints(g, T // 2, T + 1, (B,)) if c["tree"] and c["ragged"] else None
        s["parents"] = None
        if c["tree"]:  # token t hangs below an earlier one, or below the context (-1)
            s["parents"] = (torch.rand((B, T), generator=g, device="cuda")
                            * (torch.arange(T, device="cuda") + 1)).to(torch.int32) - 1
        s["slopes"] = _slopes(c["heads"]) if c["bias"] else None
        s["out"] = torch.zeros((B, T, c["heads"], D), device="cuda", dtype=DT[c["dtype"]]).transpose(1, 2)
    else:
        B, S, H, Hk, D = c["batch"], c["seq"], c["heads"], c["kv_heads"], c["head_dim"]
        qkv = _rand(g, (B, S, H + 2 * Hk, D), c["dtype"])  # q, k and v of a token side by side
        s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
        s["positions"] = (_ints(g, 0, 1000, (B, 1)) + c["start"]
                          + torch.arange(S, device="cuda", dtype=torch.int32)).contiguous()
        i = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (torch.pow(10000.0, -i / c["rot"]) / c["factor"]).float()
    return s


# ------------------------------------------------------------------ plain forms
def _mask_and_distance(s):
    """Which keys each query sees, (batch, seq_q, seq_k), and how far each is away."""
    c = s["case"]
    i = torch.arange(c["seq_q"], device="cuda")[:, None] + c["offset"]
    j = torch.arange(c["seq_k"], device="cuda")[None, :]
    B = c["batch"]
    start = torch.zeros((B, 1, 1), device="cuda", dtype=torch.int64)
    first = s["prefix"][:, :1, None] if s["prefix"] is not None else None
    seen = torch.ones((B, c["seq_q"], c["seq_k"]), device="cuda", dtype=torch.bool)
    if s["doc_offsets"] is not None:
        off = s["doc_offsets"].long()
        doc_j = (off[:, None, :-1] <= j.reshape(1, -1, 1)).sum(-1) - 1  # the last document that begins at or before it
        doc_i = (off[:, None, :-1] <= i.reshape(1, -1, 1)).sum(-1) - 1
        inside_i, inside_j = i.reshape(1, -1) < off[:, -1:], j.reshape(1, -1) < off[:, -1:]
        seen = (doc_i[:, :, None] == doc_j[:, None, :]) & inside_i[:, :, None] & inside_j[:, None, :]
        start = torch.gather(off, 1, doc_i)[:, :, None]
        if first is not None:
            first = torch.gather(s["prefix"].long(), 1, doc_i)[:, :, None]
    if c["causal"]:
        past = (j <= i)[None]
        seen = seen & (past | (j[None] < start + first) if first is not None else past)
    return seen, (i - j).abs()


def _attend(q, k, v, seen, scale, cap, bias):
    """out, lse, the weights and the caps' tanh; q (B, Hkv, G, Sq, D), k and v (B, Hkv, Sk, D), seen (B, Sq, Sk)."""
    B, Hk, G, Sq, D = q.shape
    x = (q.reshape(B, Hk, G * Sq, D) @ k.transpose(2, 3)).view(B, Hk, G, Sq, -1) * scale
    t = torch.tanh(x / cap) if cap else None
    x = cap * t if cap else x
    x = x + bias if bias is not None else x
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    out = (w.view(B, Hk, G * Sq, -1) @ v).view(B, Hk, G, Sq, D)
    return out, lse, w, t


def _plain_attention(s):
    c = s["case"]
    B, H, Hk, Sq, D = c["batch"], c["heads"], c["kv_heads"], c["seq_q"], c["head_dim"]
    G, dt, scale = H // Hk, DT[c["dtype"]], 1.0 / math.sqrt(D)
    q, k, v = s["q"].float().reshape(B, Hk, G, Sq, D), s["k"].float(), s["v"].float()
    seen, far = _mask_and_distance(s)
    bias = -s["slopes"].view(1, Hk, G, 1, 1) * far.float() if c["bias"] else None
    out, lse, w, t = _attend(q, k, v, seen, scale, c["cap"], bias)
    res = {"out": out.reshape(B, H, Sq, D).to(dt), "lse": lse.reshape(B, H, Sq)}
    if c["kind"] == "forward":
        return res
    do = s["dout"].float().reshape(B, Hk, G * Sq, D)
    w = w.view(B, Hk, G * Sq, -1)
    dv = w.transpose(2, 3) @ do
    dw = do @ v.transpose(2, 3)
    ds = w * (dw - (w * dw).sum(-1, keepdim=True))
    ds = ds * (1 - t * t).view(ds.shape) if c["cap"] else ds
    dq = ((ds @ k) * scale).reshape(B, H, Sq, D)
    dk = (ds.transpose(2, 3) @ q.reshape(B, Hk, G * Sq, D)) * scale
    res.update(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))
    return res


def _plain_tree(s):
    c = s["case"]
    B, H, Hk, T, D = c["batch"], c["heads"], c["kv_heads"], c["tokens"], c["head_dim"]
    G, dt = H // Hk, DT[c["dtype"]]
    k = s["k_cache"][s["block_table"].long()].reshape(B, -1, Hk, D).transpose(1, 2).float()
    v = s["v_cache"][s["block_table"].long()].reshape(B, -1, Hk, D).transpose(1, 2).float()
    t = torch.arange(T, device="cuda")
    parents = s["parents"].long() if s["parents"] is not None else (t - 1).expand(B, T)
    step = (parents[:, :, None] == t).double() + torch.eye(T, device="cuda", dtype=torch.float64)
    above = torch.linalg.matrix_power(step, T) > 0.5  # itself and what it hangs below
    depth = above.sum(-1) - 1
    valid = t < s["tree_lens"][:, None] if s["tree_lens"] is not None else torch.ones_like(depth, dtype=torch.bool)
    j = torch.arange(k.shape[2], device="cuda")
    at = j[None, :] - s["context"][:, None].long()  # a key's place among the drafted tokens
    drafted = torch.gather(above, 2, at.clamp(0, T - 1)[:, None, :].expand(B, T, -1)) & (at >= 0)[:, None] & (at < T)[:, None]
    seen = (at < 0)[:, None] | drafted
    bias = None
    if c["bias"]:
        pos_j = torch.where(at < 0, j[None, :], s["context"][:, None].long() + torch.gather(depth, 1, at.clamp(0, T - 1)))
        far = (s["context"][:, None].long() + depth)[:, :, None] - pos_j[:, None, :]
        bias = -s["slopes"].view(1, Hk, G, 1, 1) * far.abs().float()[:, None, None]
    q = s["q"].float().reshape(B, Hk, G, T, D)
    out, lse, _, _ = _attend(q, k, v, seen, 1.0 / math.sqrt(D), c["cap"], bias)
    out = out.reshape(B, H, T, D).to(dt)
    return {"out": torch.where(valid[:, None, :, None], out, torch.zeros_like(out))}


def _turn(x, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, x[..., 2 * n:]], dim=-1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"].double()
    cos, sin = (torch.cos(angle) * c["scale"]).float(), (torch.sin(angle) * c["scale"]).float()
    sin = -sin if c["inverse"] else sin
    dt = DT[c["dtype"]]
    return {"q": _turn(s["q"].float(), cos, sin, c["interleaved"]).to(dt),
            "k": _turn(s["k"].float(), cos, sin, c["interleaved"]).to(dt)}


# ------------------------------------------------------------------ the calls
def _own_attention(s):
    import tensor_core_gemm_tl_b200 as tg
    c = s["case"]
    how = dict(causal=c["causal"], score_cap=c["cap"], slopes=s["slopes"], doc_offsets=s["doc_offsets"],
               prefix=s["prefix"], q_offset=c["offset"])
    lse = torch.empty(s["q"].shape[:3], dtype=torch.float32, device="cuda")
    out = tg.attention_ex(s["q"], s["k"], s["v"], lse=lse, **how)
    res = {"out": out, "lse": lse}
    if c["kind"] == "train":
        res["dq"], res["dk"], res["dv"] = tg.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)
    return res


def _own_tree(s):
    import tensor_core_gemm_tl_b200 as tg
    return {"out": tg.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context"], s["parents"],
                                     tree_lens=s["tree_lens"], score_cap=s["case"]["cap"], slopes=s["slopes"],
                                     out=s["out"])}


def _own_rotary(s):
    import tensor_core_gemm_tl_b200 as tg
    c = s["case"]
    q, k = tg.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], scale=c["scale"],
                     inverse=c["inverse"])
    return {"q": q, "k": k}


def run(state):
    kind = state["case"]["kind"]
    if kind == "tree":
        return _own_tree(state) if own else _plain_tree(state)
    if kind == "rotary":
        return _own_rotary(state) if own else _plain_rotary(state)
    return _own_attention(state) if own else _plain_attention(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["kind"] == "rotary":
        n = c["batch"] * c["seq"]
        values = n * (c["heads"] + c["kv_heads"]) * c["head_dim"]
        turned = n * (c["heads"] + c["kv_heads"]) * c["rot"]
        return {"bytes": 4 * values + 4 * n + 2 * c["rot"], "flops": 3 * turned}
    if c["kind"] == "tree":
        keys = c["context"] * (5 / 8 if c["ragged"] else 1) + c["tokens"]  # ragged: uniform from a quarter to all
        rows = c["batch"] * c["tokens"] * c["heads"] * c["head_dim"]
        return {"bytes": int(4 * c["batch"] * keys * c["kv_heads"] * c["head_dim"] + 4 * rows), "flops": int(4 * rows * keys)}
    B, D, n, m = c["batch"], c["head_dim"], c["seq_q"], c["seq_k"]
    pairs = n * c["offset"] + n * (n + 1) / 2 if c["causal"] else n * m
    if c["docs"]:
        # uniform cuts of the keys into d documents: a document's share is Beta(1, d - 1), whose square's mean is
        # 2 / (d (d + 1)), so two places lie in one document with probability 2 / (d + 1)
        pairs *= 2 / (c["docs"] + 1)
    qb, kb = 2 * B * c["heads"] * n * D, 2 * B * c["kv_heads"] * m * D
    fwd = 4 * B * c["heads"] * D * pairs
    rows = 4 * B * c["heads"] * n
    if c["kind"] == "forward":
        return {"bytes": 2 * qb + 2 * kb + rows, "flops": int(fwd)}
    # a training step: the forward, then five products of its size's half; q, k, v, dout, out read, gradients written
    return {"bytes": 6 * qb + 6 * kb + 2 * rows, "flops": int(3.5 * fwd)}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(q, k, v, see, scale, cap, bias, do=None):
    """One key/value head: q (G, n, D), k and v (m, D), see (n, m), bias (G, n, m) or None; all in 64 bits."""
    a = torch.einsum("gnd,md->gnm", q, k) * scale
    u = a
    if cap:
        u = cap * torch.tanh(a / cap)
    x = u if bias is None else u + bias
    x = torch.where(see[None], x, torch.full_like(x, -math.inf))
    top = x.max(dim=-1, keepdim=True).values
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    p = e / torch.where(z == 0, torch.ones_like(z), z)
    o = torch.einsum("gnm,md->gnd", p, v)
    lse = (torch.log(z) + top).squeeze(-1)
    if do is None:
        return o, lse
    dp = torch.einsum("gnd,md->gnm", do, v)
    dx = p * (dp - (do * o).sum(-1, keepdim=True))
    if cap:
        dx = dx * (1 - (u / cap) ** 2)
    return (o, lse, scale * torch.einsum("gnm,md->gnd", dx, k), scale * torch.einsum("gnm,gnd->md", dx, q),
            torch.einsum("gnm,gnd->md", p, do))


def _exact_attention(s):
    c = s["case"]
    B, H, Hk, n, m, D = c["batch"], c["heads"], c["kv_heads"], c["seq_q"], c["seq_k"], c["head_dim"]
    G, train = H // Hk, c["kind"] == "train"
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros((B, H, n, D), **f64), torch.zeros((B, H, n), **f64)
    dq, dk, dv = torch.zeros((B, H, n, D), **f64), torch.zeros((B, Hk, m, D), **f64), torch.zeros((B, Hk, m, D), **f64)
    pos = torch.arange(c["offset"], c["offset"] + n, device="cuda")
    key = torch.arange(m, device="cuda")
    for b in range(B):
        lo = torch.zeros(n, dtype=torch.int64, device="cuda")
        hi = torch.full((n,), m, dtype=torch.int64, device="cuda")
        begin, reach = lo.clone(), torch.zeros_like(lo)
        if s["prefix"] is not None:
            reach = reach + int(s["prefix"][b, 0])
        if s["doc_offsets"] is not None:
            hi = torch.zeros_like(hi)
            cuts = s["doc_offsets"][b].tolist()
            for d in range(len(cuts) - 1):
                mine = (pos >= cuts[d]) & (pos < cuts[d + 1])
                lo[mine], hi[mine], begin[mine] = cuts[d], cuts[d + 1], cuts[d]
                if s["prefix"] is not None:
                    reach[mine] = int(s["prefix"][b, d])
        if c["causal"]:
            hi = torch.minimum(hi, torch.maximum(pos + 1, begin + reach))
        see = (key[None] >= lo[:, None]) & (key[None] < hi[:, None])
        for h in range(Hk):
            r = slice(h * G, (h + 1) * G)
            bias = None
            if c["bias"]:
                bias = -s["slopes"][r].double()[:, None, None] * (pos[:, None] - key[None]).abs().double()
            got = _exact_rows(s["q"][b, r].double(), s["k"][b, h].double(), s["v"][b, h].double(), see,
                              1.0 / math.sqrt(D), c["cap"], bias, s["dout"][b, r].double() if train else None)
            out[b, r], lse[b, r] = got[0], got[1]
            if train:
                dq[b, r], dk[b, h], dv[b, h] = got[2], got[3], got[4]
    res = {"out": out, "lse": lse}
    if train:
        res.update(dq=dq, dk=dk, dv=dv)
    return res


def _exact_tree(s):
    c = s["case"]
    B, H, Hk, T, D = c["batch"], c["heads"], c["kv_heads"], c["tokens"], c["head_dim"]
    G = H // Hk
    out = torch.zeros((B, H, T, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["context"][b])
        live = T if s["tree_lens"] is None else int(s["tree_lens"][b])
        up = list(range(-1, T - 1)) if s["parents"] is None else s["parents"][b].tolist()
        see = torch.zeros((T, n + T), dtype=torch.bool)
        see[:, :n] = True
        depth = [0] * T
        for t in range(T):
            a = t
            while a >= 0:
                see[t, n + a] = True
                a = up[a]
                depth[t] += a >= 0
        see = see.cuda()
        pos = torch.tensor(list(range(n)) + [n + d for d in depth], device="cuda", dtype=torch.float64)
        pages = s["block_table"][b].long()
        for h in range(Hk):
            k = s["k_cache"][pages, :, h].reshape(-1, D)[:n + T].double()
            v = s["v_cache"][pages, :, h].reshape(-1, D)[:n + T].double()
            r = slice(h * G, (h + 1) * G)
            bias = None
            if c["bias"]:
                bias = -s["slopes"][r].double()[:, None, None] * (pos[n:, None] - pos[None]).abs()
            o, _ = _exact_rows(s["q"][b, r].double(), k, v, see, 1.0 / math.sqrt(D), c["cap"], bias)
            out[b, r, :live] = o[:, :live]
    return {"out": out}


def _exact_rotary(s):
    c = s["case"]
    n = c["rot"] // 2
    w = torch.polar(torch.full((), c["scale"], dtype=torch.float64, device="cuda").expand(*s["positions"].shape, n),
                    (-1.0 if c["inverse"] else 1.0) * s["positions"].double()[..., None] * s["inv_freq"].double())
    res = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        a = slice(0, 2 * n, 2) if c["interleaved"] else slice(0, n)
        b = slice(1, 2 * n, 2) if c["interleaved"] else slice(n, 2 * n)
        z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * w[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        res[name] = y
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "rotary": _exact_rotary}.get(case["kind"], _exact_attention)(s)
