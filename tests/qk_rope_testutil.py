"""Query/key norms with rotation in 64 bits, and bounds for fp32 computations of them (see test_qk_rope_gpu.py)."""
from __future__ import annotations

import math
from fractions import Fraction

import torch

# 1 / (2 pi), to 200 bits, from pi's first 70 digits
_PI = Fraction("3.141592653589793238462643383279502884197169399375105820974944592307816")


def freqs_of(rot, base=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (base ** (-2 * i / max(rot, 1))).float()


def angles(pos, freqs):
    """position x frequency in [-pi, pi], reduced in exact arithmetic: [T, R/2] fp64."""
    out = torch.empty((len(pos), len(freqs)), dtype=torch.float64)
    fr = [Fraction(float(f)) if math.isfinite(f) else None for f in freqs.tolist()]
    big = int(pos.max()) > 4096 if len(pos) else False
    for i, p in enumerate(pos.tolist()):
        for j, f in enumerate(fr):
            if big and f is not None:
                a = p * f
                a -= 2 * _PI * round(a / (2 * _PI))
                out[i, j] = float(a)
            else:
                out[i, j] = p * float(freqs[j])
    return out


def turned(y, ang, pairs, sign=1.0):
    """y [T, H, D] with its first pairs turned by sign x ang, and |a| + |b| of each channel's pair."""
    half = ang.shape[1]
    c, s = torch.cos(ang)[:, None], sign * torch.sin(ang)[:, None]
    size = y.abs().clone()
    out = y.clone()
    ia, ib = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


def normed(x, w, eps, norm):
    x = x.double()
    if not norm:
        return x, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return (x * r if w is None else x * r * w.double()), r


def reference(x, pos, freqs, w, eps, norm, pairs):
    """The forward in 64 bits, and the size that its fp32 error is relative to."""
    y, _ = normed(x, w, eps, norm)
    return turned(y, angles(pos, freqs), pairs)


def gradients(x, pos, freqs, w, eps, norm, pairs, dout):
    """By automatic differentiation of the 64-bit forward: dx, and dw or None."""
    x = x.double().requires_grad_(True)
    wd = None if w is None else w.double().requires_grad_(True)
    if norm:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if wd is not None:
            y = y * wd
    else:
        y = x
    ang = angles(pos, freqs)
    half = ang.shape[1]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if pairs:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        z = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        z = torch.cat([a * c - b * s, a * s + b * c], -1)
    z = torch.cat([z, y[..., 2 * half:]], -1)
    grads = torch.autograd.grad((z * dout.double()).sum(), [x] + ([] if wd is None else [wd]))
    return grads[0], (grads[1] if wd is not None else None)


def grad_bounds(x, pos, freqs, w, eps, norm, pairs, dout):
    g, size = turned(dout.double(), angles(pos, freqs), pairs, -1.0)
    if not norm:
        return 2.0 ** -18 * size, None
    y, r = normed(x, None, eps, True)
    wd = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double().abs()
    first = r * size * wd
    second = r * y.abs() * (size * wd * y.abs()).mean(-1, keepdim=True)
    terms = (size * y.abs()).sum((0, 1))
    n = x.shape[0] * x.shape[1]
    return 2.0 ** -18 * (first + second), terms * (2.0 ** -18 + 2.0 ** -24 * (104 + n / 4096))
