"""Plain 64-bit forms of the masked attention, the tree attention and the rotary
positions, written from their definitions with masks built token by token, and
the error bounds that a kernel with 16-bit weights and fp32 sums keeps to.

Bounds.  r = eps / 2 of the 16-bit type (2^-8 bf16, 2^-11 fp16) is one rounding.
A score y is an fp32 sum of D products, scaled, perhaps capped and biased: off by
at most

    delta = 2^-23 (D scale sum_d |q_d k_d| + 4 max |y| + 8) + 2^-20 cap

(a sum of D terms loses at most D 2^-23 of its absolute sum; the scaled score,
the bias and the maximum's subtraction a few 2^-23 of their size; 2^x is good to
2^-22; the capped form to 2^-21 of the cap).  A weight exp(y) / sum exp(y) is then
off by 2 delta relatively, and by r once it is rounded to 16 bits (fp16 weights
under 2^-14 of the row's largest: by 2^-25 of it instead).  2^x is flushed to 0
below 2^-126, so a weight P may lose 2^-126, and with it dX = P g as much times |g|;
a dX of its own below 2^-126, bf16's and fp32's smallest normal number, may go to 0:
2^-126 (1 + |g|) in all, which a far key under a steep bias does lose.
"""
from __future__ import annotations

import math

import torch


def visible(batch, seq_q, seq_k, causal=False, q_offset=0, docs=None, prefix=None):
    """(batch, seq_q, seq_k) bool: which keys each query sees, by the definition."""
    see = torch.zeros((batch, seq_q, seq_k), dtype=torch.bool)
    for b in range(batch):
        for i in range(seq_q):
            p = q_offset + i
            lo, hi, d = 0, seq_k, 0
            if docs is not None:
                own = [n for n in range(len(docs[b]) - 1) if docs[b][n] <= p < docs[b][n + 1]]
                if not own:
                    continue
                d = own[0]
                lo, hi = docs[b][d], docs[b][d + 1]
            if causal:
                reach = lo + prefix[b][d] if prefix is not None else 0
                hi = min(hi, max(p + 1, reach))
            see[b, i, max(lo, 0):max(min(hi, seq_k), 0)] = True
    return see


class Plain:
    """One attention problem in 64 bits.  q (B, H, Sq, D), k and v (B, Hkv, Sk, D);
    see (B, Sq, Sk); pos_q (B, Sq) and pos_k (B, Sk) for the bias."""

    def __init__(self, q, k, v, see, scale, cap=0.0, slopes=None, pos_q=None, pos_k=None):
        self.r = torch.finfo(q.dtype).eps / 2
        self.fp16 = q.dtype == torch.float16
        self.q, self.k, self.v = (t.detach().double().requires_grad_() for t in (q, k, v))
        self.scale, self.cap, self.see = scale, cap, see.to(q.device)
        B, H, Sq, D = q.shape
        G = H // k.shape[1]
        self.G = G
        self.kk = self.k.repeat_interleave(G, dim=1)
        self.vv = self.v.repeat_interleave(G, dim=1)
        y = torch.einsum("bhid,bhjd->bhij", self.q, self.kk) * scale
        raw = y.detach()
        if cap:
            y = cap * torch.tanh(y / cap)
        self.c = 1 - (y.detach() / cap) ** 2 if cap else torch.ones_like(raw)
        if slopes is not None:
            far = (pos_q[:, None, :, None] - pos_k[:, None, None, :]).abs().double()
            y = y - slopes.double()[None, :, None, None] * far
        m = self.see[:, None]
        y = torch.where(m, y, torch.full_like(y, -math.inf))
        top = y.detach().amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        e = torch.exp(y - top)
        z = e.sum(-1, keepdim=True)
        self.w = e / torch.where(z == 0, torch.ones_like(z), z)
        self.out = torch.einsum("bhij,bhjd->bhid", self.w, self.vv)
        self.lse = (torch.log(z.detach()) + top).squeeze(-1)
        absdot = torch.einsum("bhid,bhjd->bhij", self.q.detach().abs(), self.kk.detach().abs()) * scale
        size = torch.where(m, y.detach().abs() + raw.abs(), torch.zeros_like(raw))
        self.delta = (2.0 ** -23 * (D * torch.where(m, absdot, torch.zeros_like(absdot)).amax(-1, keepdim=True)
                                    + 4 * size.amax(-1, keepdim=True) + 8) + 2.0 ** -20 * cap)

    def out_bound(self):
        w, v = self.w.detach(), self.vv.detach().abs()
        b = (self.r + 2 * self.delta) * torch.einsum("bhij,bhjd->bhid", w, v)
        if self.fp16:
            b = b + 2.0 ** -25 * torch.einsum("bhij,bhjd->bhid", self.see[:, None].expand_as(w).double(), v)
        return b * (1 + 2.0 ** -6) + self.r * self.out.detach().abs() + self._floor()

    def _floor(self):
        # a result under the type's normal range is off by half its smallest step
        return 2.0 ** -25 if self.fp16 else 1e-38

    def lse_bound(self):
        lse = torch.where(self.lse == -math.inf, torch.zeros_like(self.lse), self.lse)
        return 2 * self.delta.squeeze(-1) + 2.0 ** -21 * (1 + lse.abs())

    def gradients(self, dout):
        """(dq, dk, dv) by differentiating the forward, and their bounds.

        dX = P (dP - e) c with e = rowsum(P dP); dP and e are fp32 sums (eta), the
        kernel's first e comes from the rounded output (zeta off) and is corrected
        by products of 16-bit values, so a rounding of what it adds (r zeta) stays."""
        do = dout.detach().double()
        dq, dk, dv = torch.autograd.grad((self.out * do).sum(), (self.q, self.k, self.v))
        q, kk, vv, w, r = self.q.detach(), self.kk.detach(), self.vv.detach(), self.w.detach(), self.r
        D = q.shape[-1]
        dp = torch.einsum("bhid,bhjd->bhij", do, vv)
        e = (w * dp).sum(-1, keepdim=True)
        g = (dp - e).abs()
        big = torch.einsum("bhid,bhjd->bhij", do.abs(), vv.abs())
        see = self.see[:, None].double()
        eta = 2.0 ** -23 * D * (big * see).amax(-1, keepdim=True)
        zeta = 2 * r * (torch.einsum("bhij,bhjd->bhid", w, vv.abs()) * do.abs()).sum(-1, keepdim=True)
        kappa = 2 * self.delta * (w * g).sum(-1, keepdim=True) + 4 * eta
        err = (r + 4 * self.delta) * w * g * self.c + w * self.c * kappa + 2.0 ** -19 * w * g
        err_q = err + (2 * r + 4 * self.delta) * w * self.c * zeta
        tiny = 2.0 ** -27 * do.abs().amax() if self.fp16 else 0.0  # fp16's smallest step of the scaled dX
        flushed = 2.0 ** -126 * see
        err, err_q = err + tiny * see + flushed * (1 + g), err_q + tiny * see * (1 + zeta) + flushed * (1 + g + zeta)
        ab_p = (r + 4 * self.delta) * w + (2.0 ** -35 * see if self.fp16 else 0.0) + flushed
        f = 1 + 2.0 ** -6

        def per_kv(t):
            return t.view(t.shape[0], -1, self.G, *t.shape[2:]).sum(2)

        bq = f * self.scale * torch.einsum("bhij,bhjd->bhid", err_q, kk.abs()) + r * dq.abs() + self._floor()
        bk = f * self.scale * per_kv(torch.einsum("bhij,bhid->bhjd", err, q.abs())) + r * dk.abs() + self._floor()
        bv = f * per_kv(torch.einsum("bhij,bhid->bhjd", ab_p, do.abs())) + r * dv.abs() + self._floor()
        return (dq, dk, dv), (bq, bk, bv)


def close(name, got, want, bound):
    """Every element of `got` within `bound` of `want`; infinities and NaN equal."""
    got, want = got.detach().double(), want.detach().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    assert torch.equal(odd, ~torch.isfinite(got)), f"{name}: finite where it should not be, or the other way round"
    assert torch.equal(got[odd], want[odd]), name
    over = torch.where(odd, torch.zeros_like(got), (got - want).abs() - bound)
    assert over.max() <= 0, (f"{name}: {int((over > 0).sum())} of {over.numel()} over the bound, worst "
                             f"{(got - want)[~odd].abs().max():.3e}, over by {over.max():.3e}")


def tree_visible(context, tokens, keys, parents=None, live=None):
    """One request: (tokens, keys) bool and the tokens' depths.  `live` tokens have keys."""
    live = tokens if live is None else live
    see = torch.zeros((tokens, keys), dtype=torch.bool)
    depth = [0] * tokens
    for t in range(tokens):
        see[t, :min(context, keys)] = True
        a = t
        while a >= 0:
            if context + a < min(keys, context + live):
                see[t, context + a] = True
            up = a - 1 if parents is None else int(parents[a])
            if up < 0 or up >= a:
                break
            depth[t] += 1
            a = up
    return see, depth


def rotate(x, positions, inv_freq, interleaved=False, scale=1.0, inverse=False):
    """x (B, H, S, D) in 64 bits, pair by pair; positions (B, S)."""
    x = x.detach().double()
    y = x.clone()
    n = inv_freq.shape[0]
    f = positions.double()[:, None, :, None] * inv_freq.double()
    c, s = scale * torch.cos(f), scale * torch.sin(-f if inverse else f)
    i = torch.arange(n, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y
