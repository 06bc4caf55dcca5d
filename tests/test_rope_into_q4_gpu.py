"""GPU tests of the operators before and behind the 4-bit cache in a row, as a softmax layer uses them: a fused
projection's queries and keys normalised and turned at the plan's positions, stored, attended over.

The rows that leave the rotation are held to 64 bits' (bounds: test_qk_rope_gpu.py); the attention to attention in 64 bits
over what the format makes of those rows (bounds: q4_testutil).  Rounding to 4 bits is not continuous, so the second
step starts from the first's own results."""
import pytest
import torch

import attn_testutil as A
import q4_testutil as Q
import qk_rope_testutil as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rotated(x, pos, freqs, w, pairs):
    return R.reference(x, torch.tensor(pos), freqs, w, 1e-6, True, pairs)


@pytest.mark.parametrize("D,rot,pairs", [(128, 128, False), (128, 32, True), (64, 64, True), (64, 24, False)])
def test_projection_to_attention(D, rot, pairs):
    from gated_delta_rule_40_gb300 import kda
    H, Hkv, bs, lens = 8, 2, 16, [150, 40, 70]
    g = torch.Generator().manual_seed(D + rot)
    fused = [torch.randn((n, H + 2 * Hkv, D), generator=g).to(torch.bfloat16) for n in lens]
    w = 1.0 + 0.3 * torch.randn((2, D), generator=g)
    freqs = R.freqs_of(rot)
    dev = (freqs.cuda(), w[0].cuda(), w[1].cuda())
    caches = [torch.zeros((30, Hkv, bs, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    order = torch.randperm(30, generator=g).to(torch.int32).cuda()
    table, at, held = torch.zeros((3, 12), dtype=torch.int32, device="cuda"), _ints([0]), _ints([0] * 3)
    done = [0] * 3
    keys, values = ([torch.zeros((0, Hkv, D), dtype=torch.bfloat16)] * 3 for _ in range(2))
    seen = 0
    # chunks of prompts, drafted and single tokens; the steps are padded
    for step in ([100, 0, 33], [49, 3, 1], [1, 1, 36], [0, 36, 0]):
        T = sum(step) + 5
        part = torch.zeros((T, H + 2 * Hkv, D), dtype=torch.bfloat16)
        part[:sum(step)] = torch.cat([f[d:d + a] for f, d, a in zip(fused, done, step)])
        plan = kda.kda_page_plan(held, _ints(step), order, at, table, bs, T)
        q, k, v = part.cuda().split([H, Hkv, Hkv], 1)
        q, k = kda.kda_qk_norm_rope(q, k, plan.positions, *dev, interleaved=pairs,
                                    q_out=torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                                    k_out=torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda"))
        kda.kda_kv_write_q4(k, v, plan.slots, *caches)
        out, lse = kda.kda_attn_paged_q4(q, *caches, table, plan.seq_lens, plan.cu_seqlens, D ** -0.5)
        assert (q[-5:] == 7).all() and (k[-5:] == 7).all()   # tokens that the plan leaves out
        row = 0
        for n, a in enumerate(step):
            if a == 0:
                continue
            rows, raw = slice(row, row + a), fused[n][done[n]:done[n] + a]
            pos = list(range(done[n], done[n] + a))
            for got, x, weight in ((q, raw[:, :H], w[0]), (k, raw[:, H:H + Hkv], w[1])):
                ref, size = _rotated(x, pos, freqs, weight, pairs)
                assert ((got[rows].double().cpu() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -19 * size)).max() <= 0
            keys[n] = torch.cat([keys[n], Q.bf16_values(k[rows].cpu())])
            values[n] = torch.cat([values[n], Q.bf16_values(raw[:, H + Hkv:].contiguous())])
            A.check(out[rows], lse[rows], Q.reference(q[rows].cpu(), keys[n], values[n], D ** -0.5, first=done[n]))
            # keys turned by other positions than their own (the mistake is the oracle's) are told apart
            if done[n] >= 30:
                raw = fused[n][:done[n] + a, H:H + Hkv]
                for wrong in ([0] * (done[n] + a), list(range(1, done[n] + a + 1))):
                    other = _rotated(raw, wrong, freqs, w[1], pairs)[0].to(torch.bfloat16)
                    ro, rl, to, tl = Q.reference(q[rows].cpu(), Q.bf16_values(other), values[n], D ** -0.5, first=done[n])
                    assert ((out[rows].double().cpu() - ro).abs() - to).max() > 0
                    assert ((lse[rows].double().cpu() - rl).abs() - tl).max() > 0
                    seen += 1
            row += a
            done[n] += a
        held, at = plan.seq_lens, plan.free_next
    assert done == [150, 40, 70] and seen >= 8
