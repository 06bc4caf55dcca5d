"""A small hybrid decoder served step by step: KDA layers with their recurrent states, softmax-attention
layers with a paged key/value cache.

    python -m gated_delta_rule_40_gb300.hybrid_example

Each step takes any number of new tokens for each request (whole prompts, chunks of them, single tokens).
``kda_page_plan`` lays the step out from lengths that never leave the device; its packed offsets are the
cu_seqlens of both kinds of layers.  A softmax layer stores its keys and values with ``kda_kv_write`` and
attends with ``kda_attn_paged``, or, where a step holds whole prompts only, with ``kda_attn_fwd``.  Random
weights; the check at the end feeds the same tokens in one step and in several and compares what comes out.
"""
from __future__ import annotations

import math

import torch

from gated_delta_rule_40_gb300 import kda

BF = torch.bfloat16


class HybridDecoder:
    """``layers`` KDA layers, every fourth one a softmax layer instead, for up to ``requests`` requests."""

    def __init__(self, layers=4, width=512, heads=8, kv_heads=2, vocab=1000, requests=4, blocks=64, block_size=64,
                 max_blocks=32, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device=device) / math.sqrt(s[0])).to(BF)  # noqa: E731
        self.H, self.Hkv, self.D, self.bs, self.N = heads, kv_heads, 128, block_size, requests
        self.embed, self.head = w(vocab, width) * math.sqrt(vocab), w(width, vocab)
        self.layers = []
        for i in range(layers):
            if i % 4 == 3:
                p = {"kind": "softmax", "qkv": w(width, (heads + 2 * kv_heads) * 128),
                     "k": torch.zeros((blocks, kv_heads, block_size, 128), dtype=BF, device=device),
                     "v": torch.zeros((blocks, kv_heads, block_size, 128), dtype=BF, device=device)}
            else:
                p = {"kind": "kda", "in": w(width, heads * (4 * 128 + 1)),
                     "A": torch.empty(heads, device=device).uniform_(-1, 1, generator=g),
                     "state": torch.zeros((requests, heads, 128, 128), device=device)}
            p["out"] = w(heads * 128, width)
            self.layers.append(p)
        self.table = torch.zeros((requests, max_blocks), dtype=torch.int32, device=device)
        self.free = torch.arange(blocks, dtype=torch.int32, device=device)
        self.free_at = torch.zeros(1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)

    def step(self, tokens: torch.Tensor, new_lens: torch.Tensor, whole_prompts: bool = False) -> torch.Tensor:
        """Logits [T, vocab] of the step's tokens [T] (packed, request by request; new_lens [N] int32)."""
        T = tokens.numel()
        plan = kda.kda_page_plan(self.lens, new_lens, self.free, self.free_at, self.table, self.bs, T)
        x = self.embed[tokens]
        for p in self.layers:
            h = torch.nn.functional.rms_norm(x, x.shape[-1:])
            if p["kind"] == "kda":
                q, k, v, graw, b = (h @ p["in"]).split([self.H * 128] * 4 + [self.H], dim=-1)
                r = lambda t: t.reshape(1, T, self.H, -1).contiguous()  # noqa: E731
                o, p["state"] = kda.kda_fwd(r(q), r(k), r(v), r(graw), b.reshape(1, T, self.H).contiguous(), p["A"],
                                            128 ** -0.5, initial_state=p["state"], cu_seqlens=plan.cu_seqlens)
            else:
                q, k, v = (h @ p["qkv"]).split([self.H * 128, self.Hkv * 128, self.Hkv * 128], dim=-1)
                q, k, v = (t.reshape(T, -1, 128).contiguous() for t in (q, k, v))
                kda.kda_kv_write(k, v, plan.slots, p["k"], p["v"])
                if whole_prompts:
                    o, _ = kda.kda_attn_fwd(q[None], k[None], v[None], 128 ** -0.5, cu_seqlens=plan.cu_seqlens)
                else:
                    o, _ = kda.kda_attn_paged(q, p["k"], p["v"], self.table, plan.seq_lens, plan.cu_seqlens,
                                              128 ** -0.5)
            x = x + o.reshape(T, -1) @ p["out"]
        self.lens, self.free_at = plan.seq_lens, plan.free_next
        return torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head


def main(lens=(300, 1, 77, 130), parts=3, seed=0) -> float:
    """Feeds prompts of these lengths whole, and to a second decoder in ``parts`` chunks and a last single token.
    Returns the relative difference of the last tokens' logits, and prints it with the tokens they choose."""
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(1000, (n,), generator=g) for n in lens]
    whole, stepped = (HybridDecoder(requests=len(lens), seed=seed) for _ in range(2))
    logits = whole.step(torch.cat(prompts).cuda(), ints(lens), whole_prompts=True)
    last = logits[torch.tensor(lens).cumsum(0) - 1].float()
    at = [0] * len(lens)
    for i in range(parts + 1):   # the last step takes what is left: one token of each request
        take = [(n - 1 - a) if i == parts - 1 else min((n - 1) // parts, n - 1 - a) for n, a in zip(lens, at)]
        if i == parts:
            take = [1] * len(lens)
        piece = [p[a:a + t] for p, a, t in zip(prompts, at, take)]
        at = [a + t for a, t in zip(at, take)]
        if sum(take):
            out = stepped.step(torch.cat(piece).cuda(), ints(take))
    out = out.float()
    if kda.kda_get_status() != kda.KDA_OK:
        raise RuntimeError("a call of the steps was refused on the device")
    rel = float((out - last).norm() / last.norm())
    print(f"last tokens' logits, one step against {parts + 1}: relative difference {rel:.2e}; "
          f"next tokens {last.argmax(-1).tolist()} and {out.argmax(-1).tolist()}")
    return rel


if __name__ == "__main__":
    main()
