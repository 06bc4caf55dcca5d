"""Softmax attention in 64 bits and the bounds the kernels are held to.

Bounds, element by element, from the roundings the kernels make.  With A = sum_j p_j |v_j| (p the
softmax weights):

* out: exp(s - max) is rounded to bf16 before the second product, the result once more.  bf16 holds 8
  significant bits: the spacing above 1 is 2^-7, so rounding to nearest is off by at most 2^-8 relative
  (1 + 2^-8 lies in the middle).  That makes 2^-8 A in the sum and 2^-8 |o| at the end; fp32 scores,
  exponentials and sums add less than 2^-12 A (a score's error is at most D 2^-24 S, S below; with
  S <= 30 that is 2^-12).  |error| <= 2^-8 |o| + (2^-8 + 2^-12) A, all times 1 + 2^-8 for the products
  of roundings.
* lse: the score's error, D 2^-24 S with S = scale max_j sum_d |q_d k_jd| and D <= 128, plus the
  exponential's, logarithm's and sum's, 2^-20 (1 + |lse|).
"""
from __future__ import annotations

import math

import torch


def reference(q, k, v, scale, first=0):
    """One request: q [A,Hq,D], k, v [L,Hkv,D]; query i sees keys 0 .. first + i.  Returns out, lse and
    the two bounds, in fp64."""
    q, k, v = q.double(), k.double(), v.double()
    A, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("ahd,lhd->ahl", q, kk) * scale
    sabs = torch.einsum("ahd,lhd->ahl", q.abs(), kk.abs()) * scale
    seen = torch.arange(L)[None, :] <= first + torch.arange(A)[:, None]
    s = s.masked_fill(~seen[:, None, :], -math.inf)
    S = sabs.masked_fill(~seen[:, None, :], 0.0).amax(-1) if L else torch.zeros(A, Hq, dtype=torch.float64)
    lse = torch.logsumexp(s, -1) if L else torch.full((A, Hq), -math.inf, dtype=torch.float64)
    p = torch.where(seen[:, None, :], torch.exp(s - lse[..., None]), torch.zeros((), dtype=torch.float64))
    out = torch.einsum("ahl,lhd->ahd", p, vv)
    Aabs = torch.einsum("ahl,lhd->ahd", p, vv.abs())
    fin = torch.where(torch.isfinite(lse), lse, torch.zeros((), dtype=torch.float64))
    extra = torch.clamp(S / 30.0, min=1.0)[..., None]   # larger scores, larger errors in the exponent
    tol_o = (2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -12 * extra) * Aabs) * (1 + 2.0 ** -8)
    tol_l = 2.0 ** -17 * S + 2.0 ** -20 * (1 + fin.abs())
    return out, lse, tol_o, tol_l


def check(out, lse, ref):
    """A request's rows against ``reference``'s answer."""
    ro, rl, to, tl = ref
    o = out.double().cpu()
    assert torch.isfinite(o).all(), "non-finite output"
    bad = (o - ro).abs() - to
    assert bad.numel() == 0 or bad.max() <= 0, f"out off its bound by {bad.max():.3e} at {bad.argmax()}"
    if lse is not None:
        l = lse.double().cpu()
        none = rl == -math.inf
        assert torch.equal(l == -math.inf, none)
        off = ((l - rl).abs() - tl)[~none]
        assert off.numel() == 0 or off.max() <= 0, f"lse off its bound by {off.max():.3e}"


def normal(gen, *shape, gain=1.0):
    return (torch.randn(*shape, generator=gen) * gain).to(torch.bfloat16)


class Paged:
    """A cache holding requests of the given (cached, new) lengths in shuffled blocks.  Rows that hold no
    token, blocks that belong to nobody, and table entries past a request's blocks hold ``junk``."""

    def __init__(self, cached, new, Hq, Hkv, D, bs, seed=0, gain=1.0, pad=0, extra_cols=2, junk=math.nan):
        g = torch.Generator().manual_seed(seed)
        self.cached, self.new, self.bs = list(cached), list(new), bs
        total = [max(c + a, 0) for c, a in zip(cached, new)]
        held = [-(-t // bs) for t in total]
        nb = sum(held) + 3
        ids = torch.randperm(nb, generator=g)
        self.table = torch.full((len(total), max(held + [0]) + extra_cols), 0x7ffffff0, dtype=torch.int32)
        self.kc = torch.full((nb, Hkv, bs, D), junk, dtype=torch.bfloat16)
        self.vc = torch.full((nb, Hkv, bs, D), junk, dtype=torch.bfloat16)
        self.ks, self.vs = [], []
        at = 0
        for n, t in enumerate(total):
            k, v = normal(g, t, Hkv, D), normal(g, t, Hkv, D)
            self.ks.append(k)
            self.vs.append(v)
            for j in range(held[n]):
                b = int(ids[at])
                self.table[n, j] = b
                part = slice(j * bs, min((j + 1) * bs, t))
                m = part.stop - part.start
                self.kc[b, :, :m] = k[part].transpose(0, 1)
                self.vc[b, :, :m] = v[part].transpose(0, 1)
                at += 1
        self.cu = [0]
        for a in new:
            self.cu.append(self.cu[-1] + a)
        self.q = normal(g, self.cu[-1] + pad, Hq, D, gain=gain)
        self.lens = torch.tensor(total, dtype=torch.int32)
        self.scale = D ** -0.5

    def run(self, **kw):
        from gated_delta_rule_40_gb300 import kda
        return kda.kda_attn_paged(self.q.cuda(), self.kc.cuda(), self.vc.cuda(), self.table.cuda(), self.lens.cuda(),
                                  torch.tensor(self.cu, dtype=torch.int32, device="cuda"), self.scale, **kw)

    def check(self, out, lse):
        for n, (c, a) in enumerate(zip(self.cached, self.new)):
            rows = slice(self.cu[n], self.cu[n + 1])
            if a:
                ref = reference(self.q[rows], self.ks[n], self.vs[n], self.scale, first=c)
                check(out[rows], None if lse is None else lse[rows], ref)
