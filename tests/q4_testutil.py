"""The 4-bit cache format in 64 bits, and paged caches in it.

Every value of the format has at most 8 significant bits, so a cache's values are held here as bf16 without a
rounding, and attention over them is bound by attn_testutil's limits as it stands."""
from __future__ import annotations

import numpy as np
import torch

import attn_testutil as A


def scale_of(b: int) -> float:
    return 2.0 ** ((b >> 3) - 15) * (1 + (b & 7) / 8)


TABLE = np.array([scale_of(b) for b in range(256)])


def quantise(x):
    """x [..., D] (numpy, fp64) as codes [..., D] and scale bytes [..., D / 32]; NaN counts as 0."""
    x = np.where(np.isnan(x), 0.0, x).reshape(*x.shape[:-1], -1, 32)
    most = np.abs(x).max(-1)
    b = np.minimum(np.searchsorted(7 * TABLE, most), 255)
    s = TABLE[b][..., None]
    n = np.minimum(np.floor(np.minimum(np.abs(x) / s, 100.0) + 0.5), 7)
    codes = np.where(x < 0, 8 - n, 8 + n)
    return codes.reshape(*codes.shape[:-2], -1).astype(np.uint8), b.astype(np.uint8)


def values(codes, b):
    c = codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float64)
    v = (c - 8) * TABLE[b][..., None]
    return v.reshape(*codes.shape)


def pack(codes, b):
    """codes [..., rows, D] and scales [..., rows, D / 32] as cache bytes [..., rows, D / 2 + D / 32]."""
    rows, D = codes.shape[-2:]
    lead = codes.shape[:-2]
    words = np.zeros((*lead, rows, D // 8), dtype=np.uint32)
    for c in range(8):
        words |= codes[..., c::8].astype(np.uint32) << np.uint32(4 * (c // 2) + 16 * (c % 2))
    raw = words.astype("<u4").view(np.uint8).reshape(*lead, rows * D // 2)
    flat = np.concatenate([raw, b.reshape(*lead, rows * (D // 32))], -1)
    return flat.reshape(*lead, rows, D // 2 + D // 32)


def unpack(cache, D):
    """The inverse: codes and scale bytes."""
    rows = cache.shape[-2]
    lead = cache.shape[:-2]
    flat = np.ascontiguousarray(cache).reshape(*lead, -1)
    words = np.ascontiguousarray(flat[..., :rows * D // 2]).view("<u4").reshape(*lead, rows, D // 8)
    codes = np.empty((*lead, rows, D), dtype=np.uint8)
    for c in range(8):
        codes[..., c::8] = (words >> np.uint32(4 * (c // 2) + 16 * (c % 2))) & 15
    return codes, flat[..., rows * D // 2:].reshape(*lead, rows, D // 32)


def bf16_values(x):
    """What the format makes of a bf16 tensor, as bf16 (exact)."""
    v = torch.from_numpy(values(*quantise(x.double().numpy())))
    out = v.to(torch.bfloat16)
    assert torch.equal(out.double(), v)
    return out


def reference(q, k, v, scale, first=0):
    """A.reference, with room for what computing with the codes themselves adds:

    * A block's product of q with codes c = 8 + n, less 8 times q's sum: at most four roundings of 2^-24 (two products of
      16 channels, the sum, the difference) of at most 15 + 8 times sum|q|.  A score is off by e = scale 2^-22 23 sum over
      blocks of s sum|q|, a weight by a factor of 2 e more.  A block's s is at most a sixth of its largest value (its
      largest n is 6 or 7, as scales are 1.125 apart or less), or 2^-15 for a block of zeros.
    * An exponential below 2^-126 of the largest may become 0, which takes at most 2^-126 |v_j| from a sum of which
      the largest term's weight is 1: 2^-126 L max |v| over L keys.  It shows where v is 0 in every key of weight,
      which values rounded to 4 bits often are.  bf16's smallest step is 2^-133."""
    o, l, to, tl = A.reference(q, k, v, scale, first)
    if k.shape[0] == 0:
        return o, l, to, tl
    q, k, v = q.double(), k.double(), v.double()
    G = q.shape[1] // k.shape[1]
    seen = torch.arange(k.shape[0])[None, :] <= first + torch.arange(q.shape[0])[:, None]
    s = torch.einsum("ahd,lhd->ahl", q, k.repeat_interleave(G, 1)) * scale
    p = torch.where(seen[:, None, :], torch.exp(s - torch.where(torch.isfinite(l), l, 0.0)[..., None]), 0.0)
    ks = torch.where(seen[:, :, None, None], (k.unflatten(-1, (-1, 32)).abs().amax(-1) / 6 + 2.0 ** -15)[None], 0.0).amax(1)
    e = scale * 2.0 ** -22 * 23 * (ks.repeat_interleave(G, 1) * q.unflatten(-1, (-1, 32)).abs().sum(-1)).sum(-1)
    sums = torch.einsum("ahl,lhd->ahd", p, v.abs().repeat_interleave(G, 1))
    tiny = 2.0 ** -126 * k.shape[0] * float(v.abs().max()) + 2.0 ** -133
    return o, l, to + torch.expm1(2 * e)[..., None] * sums + tiny, tl + e


class PagedQ4(A.Paged):
    """A.Paged whose cache is held in 4 bits; rows that hold no token, and blocks of nobody, hold arbitrary bytes."""

    def __init__(self, cached, new, Hq, Hkv, D, bs, seed=0, gain=1.0, pad=0, extra_cols=2):
        super().__init__(cached, new, Hq, Hkv, D, bs, seed=seed, gain=gain, pad=pad, extra_cols=extra_cols, junk=0.0)
        rng = np.random.default_rng(seed)
        nb = self.kc.shape[0]
        used = np.zeros((nb, bs), dtype=bool)
        for n, k in enumerate(self.ks):
            for j in range(-(-k.shape[0] // bs)):
                used[int(self.table[n, j]), :min(bs, k.shape[0] - j * bs)] = True
        self.caches = []
        for plain in (self.kc, self.vc):
            codes, b = quantise(plain.double().numpy())
            off = ~used[:, None, :, None]
            codes = np.where(off, rng.integers(0, 16, codes.shape, dtype=np.uint8), codes)
            b = np.where(off, rng.integers(200, 256, b.shape).astype(np.uint8), b)
            self.caches.append(torch.from_numpy(pack(codes, b)))
        self.ks = [bf16_values(k) if k.numel() else k for k in self.ks]
        self.vs = [bf16_values(v) if v.numel() else v for v in self.vs]

    def run(self, **kw):
        from gated_delta_rule_40_gb300 import kda
        kc, vc = (c.cuda() for c in self.caches)
        return kda.kda_attn_paged_q4(self.q.cuda(), kc, vc, self.table.cuda(), self.lens.cuda(),
                                     torch.tensor(self.cu, dtype=torch.int32, device="cuda"), self.scale, **kw)

    def check(self, out, lse):
        for n, (c, a) in enumerate(zip(self.cached, self.new)):
            rows = slice(self.cu[n], self.cu[n + 1])
            if a:
                ref = reference(self.q[rows], self.ks[n], self.vs[n], self.scale, first=c)
                A.check(out[rows], None if lse is None else lse[rows], ref)
