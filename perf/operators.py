"""The softmax-attention serving operators: inputs, plain forms, and what each has to move.

Four operators of a hybrid model's serving step, next to its linear-attention layers:

  plan    block table, slot map, positions and packed offsets from request lengths
  write   new keys and values into the paged cache
  prompt  causal attention over whole prompts, grouped heads, dense or packed
  paged   causal attention of new tokens (one or many per request) over the paged cache

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with ``own``
true it makes the framework's calls.  The cache is [blocks, kv heads, block size, head dim].
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a mid-sized batch: 64 requests take one token each
        {"name": "plan_decode_64", "op": "plan", "requests": 64, "cached": 4096, "new": 1, "block": 64, "mix": 1},
        # a busy scheduler step: 2000 requests, prompts and chunks among the single tokens, small blocks
        {"name": "plan_mixed_2000", "op": "plan", "requests": 2000, "cached": 8192, "new": 64, "block": 16, "mix": 2},
        # the keys and values of one decode step
        {"name": "write_decode_64", "op": "write", "tokens": 64, "kv": 8, "dim": 128, "block": 64},
        # the keys and values of a packed prompt batch
        {"name": "write_prompt_32768", "op": "write", "tokens": 32768, "kv": 8, "dim": 128, "block": 64},
        # the smallest prompt call: one short question, odd length
        {"name": "prompt_200", "op": "prompt", "batch": 1, "tokens": 200, "packed": 0, "q": 16, "kv": 4, "dim": 128,
         "mix": 0},
        # 20 packed prompts of very different lengths, 16384 tokens together
        {"name": "prompt_packed_16384", "op": "prompt", "batch": 1, "tokens": 16384, "packed": 20, "q": 32, "kv": 8,
         "dim": 128, "mix": 3},
        # one long document
        {"name": "prompt_16384", "op": "prompt", "batch": 1, "tokens": 16384, "packed": 0, "q": 32, "kv": 8,
         "dim": 128, "mix": 0},
        # two ordinary prompts, small heads that are not shared, odd length
        {"name": "prompt_4001_d64", "op": "prompt", "batch": 2, "tokens": 4001, "packed": 0, "q": 16, "kv": 16,
         "dim": 64, "mix": 0},
        # interactive decoding of a few requests: latency counts
        {"name": "paged_decode_4", "op": "paged", "requests": 4, "context": 1000, "new": 1, "q": 32, "kv": 8,
         "dim": 128, "block": 64, "mix": 4},
        # a full decode batch with contexts from tens to thousands of tokens
        {"name": "paged_decode_256", "op": "paged", "requests": 256, "context": 8192, "new": 1, "q": 32, "kv": 8,
         "dim": 128, "block": 64, "mix": 5},
        # one long conversation, four drafted tokens checked at once: few rows over a long cache
        {"name": "paged_verify_131072", "op": "paged", "requests": 1, "context": 131072, "new": 4, "q": 32, "kv": 8,
         "dim": 128, "block": 64, "mix": 0},
        # chunks of prompts beside single tokens in one call, small blocks, seven query heads a group
        {"name": "paged_mixed_24", "op": "paged", "requests": 24, "context": 8192, "new": 512, "q": 28, "kv": 4,
         "dim": 128, "block": 16, "mix": 6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "prompt", "prompt", "paged", "paged"])
    dim = rng.choice([64, 128, 128])
    block = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    mix = rng.randrange(1, 1 << 20)
    if op == "plan":
        return {"op": op, "requests": _log(rng, 1, 2000), "cached": _log(rng, 1, 8192), "new": _log(rng, 1, 64),
                "block": block, "mix": mix}
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 32768), "kv": kv, "dim": dim, "block": block}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "prompt":
        q = kv * group if kv * group <= 32 else kv
        tokens = _log(rng, 16, 16384)
        packed = rng.choice([0, 0, _log(rng, 1, 40)])
        batch = 1
        if not packed:
            most = (16384 * 16384 * 32) // (tokens * tokens * q)
            batch = _log(rng, 1, max(1, min(8, most)))
        return {"op": op, "batch": batch, "tokens": tokens, "packed": packed, "q": q, "kv": kv, "dim": dim, "mix": mix}
    group = rng.choice([1, 2, 4, 5, 7, 8])
    kv = rng.choice([1, 2, 4, 8])
    q = kv * group if kv * group <= 32 else kv * 4
    new = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 512)])
    requests = _log(rng, 1, 256)
    context = _log(rng, 16, 131072)
    # what the plain form holds: padded scores, and keys and values of the longest context for each request
    context = max(16, min(context, (1 << 31) // (requests * q * new), (256 * 8192 * 8) // (requests * kv)))
    return {"op": op, "requests": requests, "context": context, "new": new, "q": q, "kv": kv, "dim": dim,
            "block": block, "mix": mix}


def _lengths(case):
    """Per-request lengths of a case, from the case alone: (cached, new) or the packed prompts' lengths."""
    rng = random.Random(case["mix"])
    op = case["op"]
    if op == "prompt":
        n, total = case["packed"], case["tokens"]
        if not n:
            return [total] * case["batch"]
        share = [math.exp(rng.uniform(0.0, 5.5)) for _ in range(n)]
        share[rng.randrange(n)] = sum(share)  # one prompt holds about half of the tokens
        lens = [int(total * s / sum(share)) for s in share]
        lens[lens.index(max(lens))] += total - sum(lens)
        return lens
    n = case["requests"]
    if op == "plan":
        cached = [_log(rng, 1, case["cached"]) - (1 if rng.random() < 0.1 else 0) for _ in range(n)]
        new = [1 if rng.random() < 0.7 else _log(rng, 1, 8 * case["new"]) if case["new"] > 1 else 1 for _ in range(n)]
        return cached, new
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"op": op}
    if op == "plan":
        cached, new = _lengths(case)
        bs = case["block"]
        wide = max(_blocks(c + a, bs) for c, a in zip(cached, new)) + 2
        held = sum(_blocks(c, bs) for c in cached)
        taken = sum(_blocks(c + a, bs) - _blocks(c, bs) for c, a in zip(cached, new))
        ids = torch.randperm(held + taken + 100, generator=gen, device="cuda").to(torch.int32)
        first = _ints([_blocks(c, bs) for c in cached])[:, None]
        col = torch.arange(wide, device="cuda", dtype=torch.int32)[None]
        table = torch.full((len(new), wide), -1, dtype=torch.int32, device="cuda")
        table[col < first] = ids[:held]
        st.update(cached=_ints(cached), new=_ints(new), table=table, free=ids[held:].contiguous(),
                  start=_ints([7]), tokens=sum(new) + 5, block=bs)  # a few padded tokens, as a captured step has
        return st
    if op == "write":
        t, bs = case["tokens"], case["block"]
        blocks = _blocks(t, bs) + 16
        order = torch.randperm(blocks, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        slots = (order[at // bs] * bs + at % bs).to(torch.int32)
        shape = (blocks, case["kv"], bs, case["dim"])
        st.update(k=_normal((t, case["kv"], case["dim"]), gen), v=_normal((t, case["kv"], case["dim"]), gen),
                  slots=slots, k_cache=_normal(shape, gen), v_cache=_normal(shape, gen))
        return st
    d, hq, hk = case["dim"], case["q"], case["kv"]
    st["scale"] = 1.0 / math.sqrt(d)
    if op == "prompt":
        b, t = case["batch"], case["tokens"]
        st.update(q=_normal((b, t, hq, d), gen, 1.5), k=_normal((b, t, hk, d), gen), v=_normal((b, t, hk, d), gen),
                  cu=_ints(_offsets(_lengths(case))) if case["packed"] else None)
        return st
    cached, new = _lengths(case)
    bs = case["block"]
    total = [c + a for c, a in zip(cached, new)]
    held = [_blocks(n, bs) for n in total]
    ids = torch.randperm(sum(held) + 3, generator=gen, device="cuda").to(torch.int32)
    wide = max(held)
    col = torch.arange(wide, device="cuda", dtype=torch.int32)[None]
    table = torch.zeros((len(new), wide), dtype=torch.int32, device="cuda")
    table[col < _ints(held)[:, None]] = ids[:sum(held)]
    shape = (sum(held) + 3, hk, bs, d)
    st.update(q=_normal((sum(new), hq, d), gen, 1.5), k_cache=_normal(shape, gen), v_cache=_normal(shape, gen),
              table=table, lens=_ints(total), cu=_ints(_offsets(new)), most=max(new))
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        from gated_delta_rule_40_gb300 import kda
        op = st["op"]
        if op == "plan":
            p = kda.kda_page_plan(st["cached"], st["new"], st["free"], st["start"], st["table"], st["block"],
                                  st["tokens"])
            return (p.cu_seqlens, p.seq_lens, p.slots, p.positions, p.free_next, st["table"])
        if op == "write":
            kda.kda_kv_write(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
            return (st["k_cache"], st["v_cache"])
        if op == "prompt":
            return kda.kda_attn_fwd(st["q"], st["k"], st["v"], st["scale"], cu_seqlens=st["cu"])
        return kda.kda_attn_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"],
                                  st["scale"])
    return {"plan": _plan, "write": _write, "prompt": _prompt, "paged": _paged}[st["op"]](st)


def _plan(st):
    c, a, table, bs, t = st["cached"], st["new"], st["table"], st["block"], st["tokens"]
    n = c.numel()
    lens = c + a
    cu = torch.zeros(n + 1, dtype=torch.int32, device=c.device)
    cu[1:] = torch.cumsum(a, 0)
    first = (c + bs - 1) // bs
    want = (lens + bs - 1) // bs - first
    base = st["start"] + torch.cumsum(want, 0) - want
    rel = torch.arange(table.shape[1], device=c.device)[None] - first[:, None]
    fresh = (rel >= 0) & (rel < want[:, None])
    pick = (base[:, None] + rel).clamp_(0, st["free"].numel() - 1)
    table.copy_(torch.where(fresh, st["free"][pick], table))
    at = torch.arange(t, device=c.device)
    held = at < cu[n]
    r = torch.searchsorted(cu[1:], at, right=True).clamp_(max=n - 1)
    pos = c[r] + at - cu[r]
    slot = table[r, (pos // bs).clamp(max=table.shape[1] - 1)].long() * bs + pos % bs
    slots = torch.where(held, slot, -1).to(torch.int32)
    positions = torch.where(held, pos, -1).to(torch.int32)
    return (cu, lens, slots, positions, (st["start"] + want.sum()).to(torch.int32), table)


def _write(st):
    bs = st["k_cache"].shape[2]
    s = st["slots"].long()
    st["k_cache"][s // bs, :, s % bs] = st["k"]
    st["v_cache"][s // bs, :, s % bs] = st["v"]
    return (st["k_cache"], st["v_cache"])


def _softmax(s, v):
    """exp(s - max) v / sum and log of the sum, for scores s (overwritten) whose masked places hold -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v)
    o = torch.where(total > 0, o / total, 0.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _prompt(st):
    q, k, v = (st[x].float().transpose(1, 2) for x in "qkv")  # [B, H, T, D]
    b, hq, t, d = q.shape
    hk = k.shape[1]
    at = torch.arange(t, device=q.device)
    hide = at[None, :] > at[:, None]
    if st["cu"] is not None:
        seq = torch.searchsorted(st["cu"][1:], at, right=True)
        hide = hide | (seq[None, :] != seq[:, None])
    s = torch.matmul(q.reshape(b, hk, hq // hk, t, d), k.transpose(-1, -2)[:, :, None]).mul_(st["scale"])
    s.masked_fill_(hide, -math.inf)
    o, lse = _softmax(s, v[:, :, None])
    o = o.reshape(b, hq, t, d).transpose(1, 2)
    return o.to(torch.bfloat16).contiguous(), lse.reshape(b, hq, t).transpose(1, 2).contiguous()


def _paged(st):
    q, table, lens, cu, most = st["q"], st["table"], st["lens"], st["cu"], st["most"]
    t, hq, d = q.shape
    hk, bs = st["k_cache"].shape[1:3]
    n, g = lens.numel(), hq // hk
    wide = table.shape[1] * bs
    # keys and values of each request side by side, its queries padded to the most of any
    k, v = (c[table.long()].transpose(1, 2).reshape(n, hk, wide, d).float() for c in (st["k_cache"], st["v_cache"]))
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
    v = v.masked_fill(torch.arange(wide, device=q.device)[None, None, :, None] >= lens[:, None, None, None], 0.0)
    o, lse = _softmax(s.reshape(n, hk, g * most, wide), v)
    o = o.reshape(n, hk, g, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)[r, i]
    lse = lse.reshape(n, hk, g, most).permute(0, 3, 1, 2).reshape(n, most, hq)[r, i]
    return o.to(torch.bfloat16), lse.contiguous()


# ------------------------------------------------------------------ 64 bits
def _exact_rows(q, k, v, scale, first):
    """Attention of q [A, H, D] over k, v [L, K, D] in 64 bits; query i sees keys 0 .. first + i."""
    a, hq, d = q.shape
    n, hk, _ = k.shape
    o = torch.empty((a, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.empty((a, hq), dtype=torch.float64, device=q.device)
    limit = first + torch.arange(a, device=q.device)[:, None]
    seen = torch.arange(n, device=q.device)[None] <= limit
    for h in range(hq):
        s = (q[:, h].double() @ k[:, h // (hq // hk)].double().T) * scale
        s = torch.where(seen, s, -math.inf)
        lse[:, h] = torch.logsumexp(s, -1)
        s = torch.exp(s - lse[:, h:h + 1])
        o[:, h] = s @ v[:, h // (hq // hk)].double()
    return o, lse


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers throughout
    st = prepare(case, seed)
    if op == "write":
        bs = case["block"]
        out = []
        for new, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
            flat = cache.double().transpose(1, 2).reshape(-1, case["kv"], case["dim"])  # by slot
            flat = flat.index_copy(0, st["slots"].long(), new.double())
            out.append(flat.reshape(-1, bs, case["kv"], case["dim"]).transpose(1, 2).contiguous())
        return tuple(out)
    if op == "prompt":
        outs, lses = [], []
        for b in range(case["batch"]):
            at = 0
            lens = _lengths(case) if case["packed"] else [case["tokens"]]
            for n in lens:
                part = slice(at, at + n)
                o, lse = _exact_rows(st["q"][b, part], st["k"][b, part], st["v"][b, part], st["scale"], 0)
                outs.append(o)
                lses.append(lse)
                at += n
        shape = (case["batch"], case["tokens"], case["q"])
        return torch.cat(outs).reshape(*shape, case["dim"]), torch.cat(lses).reshape(shape)
    cached, new = _lengths(case)
    outs, lses, at = [], [], 0
    for n, (c, a) in enumerate(zip(cached, new)):
        ids = st["table"][n, :_blocks(c + a, case["block"])].long()
        k, v = (x[ids].transpose(1, 2).reshape(-1, case["kv"], case["dim"])[:c + a]
                for x in (st["k_cache"], st["v_cache"]))
        o, lse = _exact_rows(st["q"][at:at + a], k, v, st["scale"], c)
        outs.append(o)
        lses.append(lse)
        at += a
    return torch.cat(outs), torch.cat(lses)


# ------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case)
        bs = case["block"]
        taken = sum(_blocks(c + a, bs) - _blocks(c, bs) for c, a in zip(cached, new))
        n, t = len(new), sum(new) + 5
        return {"bytes": 4 * (4 * n + 3 + 2 * taken + 2 * t), "flops": 4 * t}
    if op == "write":
        return {"bytes": case["tokens"] * (8 * case["kv"] * case["dim"] + 4), "flops": 0}
    hq, hk, d = case["q"], case["kv"], case["dim"]
    if op == "prompt":
        lens = _lengths(case)
        t = sum(lens)
        return {"bytes": t * (4 * d * (hq + hk) + 4 * hq),
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    cached, new = _lengths(case)
    pairs = sum(c * a + a * (a + 1) // 2 for c, a in zip(cached, new))
    return {"bytes": 4 * d * hk * (sum(cached) + sum(new)) + sum(new) * hq * (4 * d + 4),
            "flops": 4 * d * hq * pairs}
