"""Operators around the softmax layers' cache: inputs, plain forms, and what each has to move.

  rope      norms of queries and keys for each head, with the position rotation, before they are stored and used
  rope_bwd  its gradients: queries, keys and both norm weights
  store     keys and values into the paged cache held in 4 bits, and rows of it read back as the values they stand for
  paged     causal attention of new tokens (one or many per request) over the paged cache held in 4 bits

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (angles in 64); with ``own``
true it makes the framework's calls.

The 4-bit cache is [blocks, kv heads, block size, D/2 + D/32] bytes.  A (block, head) holds D/2 bytes of codes for
each row and then D/32 scale bytes for each row.  A scale byte b stands for 2^((b >> 3) - 15) (1 + (b & 7) / 8) and
serves 32 channels; a code c for (c - 8) times the scale.  The 32-bit word of 8 channels has channel 2j in bits
4j .. 4j + 3 and channel 2j + 1 in bits 16 + 4j .. 19 + 4j.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # queries and keys of one decode step, as slices of a fused projection; positions far into long conversations
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "q": 32, "kv": 8, "dim": 128, "rot": 128, "pairs": 0,
         "norm": 2, "fused": 1, "far": 1000000, "one": 1},
        # a packed prompt batch, only a quarter of the channels rotated
        {"name": "rope_prompt_32768", "op": "rope", "tokens": 32768, "q": 32, "kv": 8, "dim": 128, "rot": 32, "pairs": 0,
         "norm": 2, "fused": 1, "far": 4000, "one": 0},
        # an odd number of tokens, small heads, neighbouring channels as pairs, no norm
        {"name": "rope_1001_d64", "op": "rope", "tokens": 1001, "q": 16, "kv": 16, "dim": 64, "rot": 64, "pairs": 1,
         "norm": 0, "fused": 0, "far": 200000, "one": 0},
        # a training step's micro-batch
        {"name": "rope_bwd_16384", "op": "rope_bwd", "tokens": 16384, "q": 32, "kv": 8, "dim": 128, "rot": 128,
         "pairs": 0, "norm": 2, "fused": 1, "far": 10, "one": 0},
        # a short odd sequence, small heads, partial rotation
        {"name": "rope_bwd_777_d64", "op": "rope_bwd", "tokens": 777, "q": 12, "kv": 4, "dim": 64, "rot": 32, "pairs": 1,
         "norm": 2, "fused": 0, "far": 50000, "one": 0},
        # the keys and values of one decode step
        {"name": "store_decode_64", "op": "store", "tokens": 64, "read": 80, "kv": 8, "dim": 128, "block": 64, "fused": 1},
        # the keys and values of a packed prompt batch
        {"name": "store_prompt_32768", "op": "store", "tokens": 32768, "read": 32800, "kv": 8, "dim": 128, "block": 64,
         "fused": 1},
        # interactive decoding of a few requests: latency counts
        {"name": "paged_decode_4", "op": "paged", "requests": 4, "context": 1000, "new": 1, "q": 32, "kv": 8, "dim": 128,
         "block": 64, "mix": 4},
        # a full decode batch with contexts from hundreds to thousands of tokens
        {"name": "paged_decode_256", "op": "paged", "requests": 256, "context": 8192, "new": 1, "q": 32, "kv": 8,
         "dim": 128, "block": 64, "mix": 5},
        # one long conversation, four drafted tokens checked at once: few rows over a long cache
        {"name": "paged_verify_131072", "op": "paged", "requests": 1, "context": 131072, "new": 4, "q": 32, "kv": 8,
         "dim": 128, "block": 64, "mix": 0},
        # chunks of prompts beside single tokens in one call, small blocks, seven query heads a group
        {"name": "paged_mixed_24", "op": "paged", "requests": 24, "context": 8192, "new": 512, "q": 28, "kv": 4,
         "dim": 128, "block": 16, "mix": 6},
        # decoding with small heads
        {"name": "paged_decode_100_d64", "op": "paged", "requests": 100, "context": 8000, "new": 1, "q": 16, "kv": 8,
         "dim": 64, "block": 32, "mix": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "rope_bwd", "store", "paged", "paged", "paged"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    q = kv * group if kv * group <= 32 else kv * 4
    block = rng.choice([16, 32, 64, 128])
    if op in ("rope", "rope_bwd"):
        return {"op": op, "tokens": _log(rng, 1, 32768 if op == "rope" else 16384), "q": q, "kv": kv, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, dim // 4, 24, 0]), "pairs": rng.randrange(2),
                "norm": rng.choice([0, 1, 2, 2]), "fused": rng.randrange(2), "far": _log(rng, 1, 1000000),
                "one": rng.randrange(2)}
    if op == "store":
        tokens = _log(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "read": rng.randrange(1, tokens + 40), "kv": kv, "dim": dim, "block": block,
                "fused": rng.randrange(2)}
    new = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 512)])
    requests = _log(rng, 1, 256)
    context = _log(rng, 16, 131072)
    # what the plain form holds: padded scores, and keys and values of the longest context for each request
    context = max(16, min(context, (1 << 31) // (requests * q * new), (256 * 8192 * 8) // (requests * kv)))
    return {"op": op, "requests": requests, "context": context, "new": new, "q": q, "kv": kv, "dim": dim,
            "block": block, "mix": rng.randrange(1, 1 << 20)}


def _lengths(case):
    """(cached, new) tokens of each request, from the case alone."""
    rng = random.Random(case["mix"])
    n = case["requests"]
    if n == 1:
        return [case["context"] - min(case["new"], case["context"])], [min(case["new"], case["context"])]
    total = [case["context"]] + [_log(rng, max(1, case["context"] // 64), case["context"]) for _ in range(n - 1)]
    if case["new"] <= 8:
        new = [case["new"]] * n
    else:  # a few chunks, single tokens for the rest
        new = [case["new"]] + [rng.randrange(1, case["new"] + 1) if rng.random() < 0.25 else 1 for _ in range(n - 1)]
    new = [min(a, t) for a, t in zip(new, total)]
    return [t - a for a, t in zip(new, total)], new


def _blocks(tokens, block):
    return -(-tokens // block)


# ------------------------------------------------------------------ the 4-bit format, plainly
_ORDER = [0, 2, 4, 6, 1, 3, 5, 7]  # channels of a word's eight codes, from its lowest bits up


def _scales(device):
    b = torch.arange(256, device=device)
    return torch.exp2((b >> 3) - 15.0) * (1.0 + (b & 7) / 8.0)


def _quantise(x):
    """x [..., D] as codes (uint8 [..., D]) and scale bytes (uint8 [..., D/32]): the smallest scale whose sevenfold
    reaches the largest magnitude of 32 channels; codes rounded to nearest, halves away from zero."""
    x = x.float().unflatten(-1, (-1, 32))
    table = _scales(x.device)
    b = torch.searchsorted(table * 7.0, x.abs().amax(-1)).clamp_(max=255)
    n = (x.abs() / table[b][..., None] + 0.5).floor_().clamp_(max=7.0)
    n = torch.where(x < 0, 8.0 - n, 8.0 + n)
    return n.to(torch.uint8).flatten(-2), b.to(torch.uint8)


def _values(codes, scales):
    return ((codes.float() - 8.0).unflatten(-1, (-1, 32)) * _scales(codes.device)[scales.int()][..., None]).flatten(-2)


def _join(codes, scales):
    """codes [..., rows, D] and scales [..., rows, D/32] of (block, head)s as their bytes [..., rows, D/2 + D/32]."""
    rows, d = codes.shape[-2:]
    c = codes.unflatten(-1, (-1, 8))[..., _ORDER]
    c = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-3)
    return torch.cat([c, scales.flatten(-2)], -1).unflatten(-1, (rows, d // 2 + d // 32)).contiguous()


def _split(cache):
    """The inverse of ``_join``."""
    rows, width = cache.shape[-2:]
    d = width * 32 // 17
    flat = cache.flatten(-2)
    c = flat[..., :rows * d // 2].unflatten(-1, (rows, d // 8, 4))
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    back = torch.tensor(_ORDER, device=cache.device).argsort()
    return c[..., back].flatten(-2), flat[..., rows * d // 2:].unflatten(-1, (rows, d // 32))


def _cache(shape, gen):
    """A cache [blocks, heads, rows, D] of normal values, quantised, some channels larger than others."""
    blocks, heads, rows, d = shape
    out = torch.empty((blocks, heads, rows, d // 2 + d // 32), dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.5 * torch.randn((heads, 1, d), generator=gen, device="cuda"))
    step = max(1, (1 << 26) // (heads * rows * d))
    for at in range(0, blocks, step):
        part = out[at:at + step]
        x = torch.randn((part.shape[0], heads, rows, d), generator=gen, device="cuda").mul_(gain)
        part.copy_(_join(*_quantise(x.to(torch.bfloat16))))
    return out


# ------------------------------------------------------------------ inputs
def _normal(shape, gen, gain=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _heads(case, gen, parts):
    """Tensors [tokens, heads, dim] for heads of ``parts``: slices of one projection's output, or tensors by themselves."""
    t, d = case["tokens"], case["dim"]
    if case["fused"]:
        return _normal((t, sum(parts), d), gen).split(parts, 1)
    return [_normal((t, h, d), gen) for h in parts]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"op": op}
    if op in ("rope", "rope_bwd"):
        t, hq, hk, d, rot = case["tokens"], case["q"], case["kv"], case["dim"], case["rot"]
        q, k, _ = _heads(case, gen, [hq, hk, hk])
        if case["one"]:  # single tokens of many requests
            pos = torch.randint(0, case["far"] + 1, (t,), generator=gen, device="cuda")
        else:
            pos = torch.arange(t, device="cuda") + case["far"]
        i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        st.update(q=q, k=k, pos=pos.to(torch.int32), freqs=(500000.0 ** (-2.0 * i / max(rot, 1))).float(), eps=1e-6,
                  norm=case["norm"] > 0, pairs=bool(case["pairs"]), qw=None, kw=None)
        if case["norm"] == 2:
            st["qw"], st["kw"] = (1.0 + 0.3 * torch.randn((2, d), generator=gen, device="cuda")).unbind(0)
        if op == "rope_bwd":
            st.update(dq=_normal((t, hq, d), gen, 0.01), dk=_normal((t, hk, d), gen, 0.02))
        return st
    if op == "store":
        t, hk, bs = case["tokens"], case["kv"], case["block"]
        _, k, v = _heads(case, gen, [hk, hk, hk])
        blocks = _blocks(t, bs) + 40
        order = torch.randperm(blocks, generator=gen, device="cuda")
        at = torch.arange(blocks * bs, device="cuda")
        slots = (order[at // bs] * bs + at % bs).to(torch.int32)
        shape = (blocks, hk, bs, case["dim"])
        # rows read back: written ones and, where there are more, others
        st.update(k=k, v=v, slots=slots[:t].contiguous(), read=slots[:case["read"]].contiguous(),
                  k_cache=_cache(shape, gen), v_cache=_cache(shape, gen))
        return st
    d, hq, hk, bs = case["dim"], case["q"], case["kv"], case["block"]
    cached, new = _lengths(case)
    total = [c + a for c, a in zip(cached, new)]
    held = [_blocks(n, bs) for n in total]
    ids = torch.randperm(sum(held) + 3, generator=gen, device="cuda").to(torch.int32)
    wide = max(held)
    col = torch.arange(wide, device="cuda", dtype=torch.int32)[None]
    table = torch.zeros((len(new), wide), dtype=torch.int32, device="cuda")
    table[col < _ints(held)[:, None]] = ids[:sum(held)]
    shape = (sum(held) + 3, hk, bs, d)
    st.update(q=_normal((sum(new), hq, d), gen, 1.5), k_cache=_cache(shape, gen), v_cache=_cache(shape, gen), table=table,
              lens=_ints(total), cu=_ints(_offsets(new)), most=max(new), scale=1.0 / math.sqrt(d))
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        from gated_delta_rule_40_gb300 import kda
        if op == "rope":
            return kda.kda_qk_norm_rope(st["q"], st["k"], st["pos"], st["freqs"], q_weight=st["qw"], k_weight=st["kw"],
                                        eps=st["eps"], norm=st["norm"], interleaved=st["pairs"])
        if op == "rope_bwd":
            grads = kda.kda_qk_norm_rope_bwd(st["q"], st["k"], st["pos"], st["freqs"], st["dq"], st["dk"],
                                             q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"], norm=st["norm"],
                                             interleaved=st["pairs"])
            return {name: g for name, g in grads.items() if g is not None}  # no weights, no gradients of them
        if op == "store":
            kda.kda_kv_write_q4(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
            return kda.kda_kv_read_q4(st["k_cache"], st["v_cache"], st["read"])
        return kda.kda_attn_paged_q4(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"],
                                     st["scale"])
    return {"rope": _rope, "rope_bwd": _rope_bwd, "store": _store, "paged": _paged}[op](st)


def _turn(x, st, back=False):
    """Rotates the first 2 len(freqs) channels of x [T, H, D] by position times frequency."""
    half = st["freqs"].numel()
    if not half:
        return x
    angle = (st["pos"].double()[:, None] * st["freqs"].double())[:, None]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    if back:
        s = -s
    if st["pairs"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _rope(st):
    out = []
    for name, weight in (("q", st["qw"]), ("k", st["kw"])):
        x = st[name].float()
        if st["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
            if weight is not None:
                x = x * weight
        out.append(_turn(x, st).to(torch.bfloat16))
    return tuple(out)


def _rope_bwd(st):
    out = {}
    for name, weight in (("q", st["qw"]), ("k", st["kw"])):
        x, g = st[name].float(), _turn(st["d" + name].float(), st, back=True)
        if not st["norm"]:
            out["d" + name] = g
            continue
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
        x = x * r
        if weight is not None:
            out["d" + name + "_weight"] = (g * x).sum((0, 1))
            g = g * weight
        out["d" + name] = r * (g - x * (g * x).mean(-1, keepdim=True))
    return out


def _store(st):
    out = []
    for new, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        bs = cache.shape[2]
        codes, scales = _split(cache)
        s = st["slots"].long()
        codes[s // bs, :, s % bs], scales[s // bs, :, s % bs] = _quantise(new)
        cache.copy_(_join(codes, scales))
        r = st["read"].long()
        out.append(_values(codes[r // bs, :, r % bs], scales[r // bs, :, r % bs]).to(torch.bfloat16))
    return tuple(out)


def _softmax(s, v):
    """exp(s - max) v / sum and log of the sum, for scores s (overwritten) whose masked places hold -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v)
    o = torch.where(total > 0, o / total, 0.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _paged(st):
    q, table, lens, cu, most = st["q"], st["table"], st["lens"], st["cu"], st["most"]
    t, hq, d = q.shape
    hk, bs = st["k_cache"].shape[1:3]
    n, g = lens.numel(), hq // hk
    wide = table.shape[1] * bs
    # keys and values of each request side by side, its queries padded to the most of any
    k, v = (_values(*_split(c))[table.long()].transpose(1, 2).reshape(n, hk, wide, d)
            for c in (st["k_cache"], st["v_cache"]))
    a = cu[1:] - cu[:-1]
    at = torch.arange(t, device=q.device)
    r = torch.searchsorted(cu[1:], at, right=True)
    i = at - cu[r]
    qp = torch.zeros((n, most, hq, d), dtype=torch.float32, device=q.device)
    qp[r, i] = q.float()
    qp = qp.reshape(n, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * most, d)
    s = torch.matmul(qp, k.transpose(-1, -2)).mul_(st["scale"]).reshape(n, hk, g, most, wide)
    last = (lens - a)[:, None] + torch.arange(most, device=q.device)  # [n, most]
    hide = torch.arange(wide, device=q.device) > last[..., None]
    s.masked_fill_(hide[:, None, None], -math.inf)
    o, lse = _softmax(s.reshape(n, hk, g * most, wide), v)
    o = o.reshape(n, hk, g, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)[r, i]
    lse = lse.reshape(n, hk, g, most).permute(0, 3, 1, 2).reshape(n, most, hq)[r, i]
    return o.to(torch.bfloat16), lse.contiguous()


# ------------------------------------------------------------------ 64 bits
def _exact_norm(x, case, st):
    """Normalised x [T, H, D] and the reciprocal root, both in 64 bits."""
    if not case["norm"]:
        return x, None
    r = 1.0 / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / case["dim"] + st["eps"])
    return x * r, r


def _exact_pairs(case):
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    return (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)


def _exact_turn(x, case, st, sign):
    """Rotation of pairs as a product of complex numbers."""
    a, b = _exact_pairs(case)
    z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                    sign * st["pos"].double()[:, None] * st["freqs"].double()[None])
    w = torch.complex(x[..., a], x[..., b]) * z[:, None]
    y = x.clone()
    y[..., a], y[..., b] = w.real, w.imag
    return y


def _exact_cache(cache):
    """A cache's values [blocks, heads, rows, D] in 64 bits, code by code from the words' bits."""
    rows, width = cache.shape[2:]
    d = width // 17 * 32
    raw = cache.reshape(cache.shape[0], cache.shape[1], -1).long()
    words = raw[..., :rows * d // 2].reshape(*raw.shape[:2], rows, d // 8, 4)
    words = words[..., 0] + (words[..., 1] << 8) + (words[..., 2] << 16) + (words[..., 3] << 24)
    b = raw[..., rows * d // 2:].reshape(*raw.shape[:2], rows, d // 32)
    scale = (8 + b % 8).double() * torch.pow(2.0, (b // 8 - 18).double())
    out = torch.empty((*raw.shape[:2], rows, d), dtype=torch.float64, device=cache.device)
    for c in range(8):
        code = (words >> (4 * (c // 2) + 16 * (c % 2))) & 15
        out[..., c::8] = (code - 8).double() * scale.repeat_interleave(4, -1)
    return out


def _exact_quantised(x):
    """What the 4-bit format makes of x [T, H, D], in 64 bits."""
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    most = x.abs().amax(-1, keepdim=True)
    scale = torch.full_like(most, 15 * 2.0 ** 13)
    for b in range(254, -1, -1):  # the smallest that will do
        s = (8 + b % 8) * 2.0 ** (b // 8 - 18)
        scale = torch.where(7 * s >= most, s, scale)
    n = torch.clamp(torch.floor(x.abs() / scale + 0.5), max=7)
    return (torch.sign(x) * n * scale).reshape(*x.shape[:-2], -1)


def _exact_rows(q, k, v, scale, first):
    """Attention of q [A, H, D] over k, v [L, K, D] in 64 bits; query i sees keys 0 .. first + i."""
    a, hq, d = q.shape
    n, hk, _ = k.shape
    o = torch.empty((a, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.empty((a, hq), dtype=torch.float64, device=q.device)
    seen = torch.arange(n, device=q.device)[None] <= first + torch.arange(a, device=q.device)[:, None]
    for h in range(hq):
        s = (q[:, h].double() @ k[:, h // (hq // hk)].T) * scale
        s = torch.where(seen, s, -math.inf)
        lse[:, h] = torch.logsumexp(s, -1)
        o[:, h] = torch.exp(s - lse[:, h:h + 1]) @ v[:, h // (hq // hk)]
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        out = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            y, _ = _exact_norm(x.double(), case, st)
            out.append(_exact_turn(y if w is None else y * w.double(), case, st, 1.0))
        return tuple(out)
    if op == "rope_bwd":
        out = {}
        for name in "qk":
            w = st[name + "w"]
            y, r = _exact_norm(st[name].double(), case, st)
            g = _exact_turn(st["d" + name].double(), case, st, -1.0)
            if w is not None:
                out["d" + name + "_weight"] = torch.einsum("thd,thd->d", g, y)
                g = g * w.double()
            if r is not None:
                g = (g - y * torch.einsum("thd,thd->th", g, y)[..., None] / case["dim"]) * r
            out["d" + name] = g
        return out
    if op == "store":
        out = []
        for new, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
            flat = _exact_cache(cache).transpose(1, 2).reshape(-1, case["kv"], case["dim"])  # by slot
            flat.index_copy_(0, st["slots"].long(), _exact_quantised(new))
            out.append(flat[st["read"].long()])
        return tuple(out)
    cached, new = _lengths(case)
    outs, lses, at = [], [], 0
    for n, (c, a) in enumerate(zip(cached, new)):
        ids = st["table"][n, :_blocks(c + a, case["block"])].long()
        k, v = (_exact_cache(x[ids]).transpose(1, 2).reshape(-1, case["kv"], case["dim"])[:c + a]
                for x in (st["k_cache"], st["v_cache"]))
        o, lse = _exact_rows(st["q"][at:at + a], k, v, st["scale"], c)
        outs.append(o)
        lses.append(lse)
        at += a
    return torch.cat(outs), torch.cat(lses)


# ------------------------------------------------------------------ floors
def work(case):
    op, d = case["op"], case["dim"]
    if op in ("rope", "rope_bwd"):
        t, heads = case["tokens"], case["q"] + case["kv"]
        small = 4 * t + 2 * case["rot"] + (8 * d if case["norm"] == 2 else 0)
        per = (3 * d + 4 if case["norm"] else 0) + 3 * case["rot"]
        if op == "rope":
            return {"bytes": 4 * t * heads * d + small, "flops": t * heads * per}
        return {"bytes": 8 * t * heads * d + small + (8 * d if case["norm"] == 2 else 0), "flops": 3 * t * heads * per}
    row = d // 2 + d // 32
    if op == "store":  # new keys and values in, rows of the cache out, values out
        t, r, hk = case["tokens"], case["read"], case["kv"]
        return {"bytes": t * (4 * hk * d + 2 * hk * row + 4) + r * (4 * hk * d + 4), "flops": 6 * t * hk * d + 2 * r * hk * d}
    hq, hk = case["q"], case["kv"]
    cached, new = _lengths(case)
    pairs = sum(c * a + a * (a + 1) // 2 for c, a in zip(cached, new))
    return {"bytes": 2 * row * hk * (sum(cached) + sum(new)) + sum(new) * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
