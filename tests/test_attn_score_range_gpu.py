"""GPU tests of attention where the range of scores ends: those that fall below the smallest fp32 number weigh
nothing, and what follows them counts; those past the largest make their rows NaN."""
import math

import pytest
import torch

import q4_testutil as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


# requests of one or two chunks (units whole), of many (units cut among warps and CTAs), and a chunk of a prompt
@pytest.mark.parametrize("N,new,blocks,bs", [(1000, 1, 2, 32), (40, 1, 32, 32), (40, 4, 33, 32), (3, 20, 40, 32), (3, 20, 10, 128),
                                             (2, 200, 32, 128)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_below_the_smallest_number(N, new, blocks, bs, D, sign):
    """Blocks of keys, by turns with scores of -10^40 or less, which fp32 does not hold, and of exactly 0.  (Queries
    are a power of two and keys equal, so that sums are exact.  Chunks have 32 keys, steps of a prompt 64.)"""
    from gated_delta_rule_40_gb300 import kda
    H, Hkv = 16, 4
    g = torch.Generator().manual_seed(N + new)
    k = torch.zeros((2 * bs, Hkv, D), dtype=torch.bfloat16)
    k[:bs] = -12000.0 * sign
    v = torch.randn((2 * bs, Hkv, D), generator=g).to(torch.bfloat16)
    cache = [torch.zeros((2, Hkv, bs, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    kda.kda_kv_write_q4(k.cuda(), v.cuda(), torch.arange(2 * bs, dtype=torch.int32, device="cuda"), *cache)
    q = torch.full((N * new, H, D), 2.0 ** 120, dtype=torch.bfloat16, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = ints([[j % 2 for j in range(blocks)]] * N)
    lens, cu = ints([blocks * bs] * N), ints([new * n for n in range(N + 1)])
    out, lse = kda.kda_attn_paged_q4(q, *cache, table, lens, cu, sign * D ** -0.5)
    values = Q.bf16_values(v).double()[bs:]   # of the keys that weigh something
    for i in range(new):
        last = blocks * bs - new + 1 + i   # keys that token i sees
        count = torch.tensor([sum(1 for j in range(x, last, 2 * bs) if j >= 0) for x in range(bs, 2 * bs)], dtype=torch.float64)
        want = (values * count[:, None, None]).sum(0) / count.sum()
        size = (values.abs() * count[:, None, None]).sum(0) / count.sum()
        rows = out[i::new].double().cpu().unflatten(1, (Hkv, H // Hkv))
        # weights are all alike: two roundings to bf16, of the weight and of the output, and fp32 sums
        assert ((rows - want[:, None]).abs() - 2.0 ** -8 * (want.abs() + 1.02 * size)[:, None]).max() <= 0
        assert (lse[i::new].double().cpu() - math.log(count.sum())).abs().max() <= 2.0 ** -20 * (1 + math.log(count.sum()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("paged", [False, True])
def test_bf16_scores_below_the_smallest_number(paged, D, sign):
    """The same of prompts and pages in bf16: products of q and k in range, their multiples by the scale not.  Keys 0 .. 149
    are of that kind, the others' scores are exactly 0."""
    from gated_delta_rule_40_gb300 import kda
    H, Hkv, T = 4, 2, 500
    g = torch.Generator().manual_seed(D)
    q = torch.full((T, H, D), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    k[:150] = -sign * 2.0 ** 59
    v = torch.randn((T, Hkv, D), generator=g).to(torch.bfloat16)
    scale = sign * 64.0   # D 2^119 64 is 2^131 or more
    if paged:
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pages = [torch.cat([x, x.new_zeros((12, Hkv, D))]).unflatten(0, (32, 16)).transpose(1, 2).contiguous() for x in (k, v.cuda())]
        out, lse = kda.kda_attn_paged(q, *pages, ints([list(range(32))]), ints([T]), ints([0, T]), scale)
    else:
        out, lse = (x[0] for x in kda.kda_attn_fwd(q[None], k[None], v.cuda()[None], scale))
    assert not out[:150].any() and (lse[:150] == -math.inf).all()
    rows = v.double()[150:]
    n = torch.arange(1, 351, dtype=torch.float64)
    want, size = rows.cumsum(0) / n[:, None, None], rows.abs().cumsum(0) / n[:, None, None]
    got = out[150:].double().cpu().unflatten(1, (Hkv, H // Hkv))
    assert ((got - want[:, :, None]).abs() - 2.0 ** -8 * (want.abs() + 1.02 * size)[:, :, None]).max() <= 0
    assert (lse[150:].double().cpu() - n.log()[:, None]).abs().max() <= 2.0 ** -20 * 8


@pytest.mark.parametrize("form", ["decode", "drafted", "chunk", "pages", "prompt"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("at", [0, 5, 70, 290])
def test_scores_above_the_largest_number(at, sign, D, form):
    """One key that scores past fp32's range among others of score 0: NaN for the tokens that see it, not a plain mean or
    nothing.  Rows that do not see it are as they are without it."""
    from gated_delta_rule_40_gb300 import kda
    H, Hkv, L, bs = 8, 2, 300, 16
    new = {"decode": 1, "drafted": 4, "chunk": 250}.get(form, L)
    q4 = form in ("decode", "drafted", "chunk")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(at)
    big = 2.0 ** 120 if q4 else 2.0 ** 60
    q = torch.full((40 * new if form == "decode" else new, H, D), big, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((304, Hkv, D), dtype=torch.bfloat16)
    k[at] = sign * (12000.0 if q4 else 2.0 ** 59)
    v = torch.randn((304, Hkv, D), generator=g).to(torch.bfloat16)
    scale = sign * (D ** -0.5 if q4 else 64.0)
    N = q.shape[0] // new
    lens, cu, table = ints([L] * N), ints([new * n for n in range(N + 1)]), ints([list(range(19))] * N)

    def run(k):
        if form == "prompt":
            return (x[0] for x in kda.kda_attn_fwd(q[None], k[None, :L].cuda(), v[None, :L].cuda(), scale))
        if form == "pages":
            pages = [x.cuda().unflatten(0, (19, bs)).transpose(1, 2).contiguous() for x in (k, v)]
            return kda.kda_attn_paged(q, *pages, table, lens, cu, scale)
        cache = [torch.zeros((19, Hkv, bs, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
        kda.kda_kv_write_q4(k.cuda(), v.cuda(), torch.arange(304, dtype=torch.int32, device="cuda"), *cache)
        return kda.kda_attn_paged_q4(q, *cache, table, lens, cu, scale)

    out, lse = run(k)
    plain, plain_lse = run(torch.zeros_like(k))
    first = L - new   # position of a request's first token
    sees = torch.tensor([first + i >= at for _ in range(N) for i in range(new)])
    assert torch.isnan(out[sees.cuda()]).all()
    l = lse[sees.cuda()]
    assert (torch.isnan(l) | (l == math.inf)).all()
    assert torch.equal(out[~sees.cuda()], plain[~sees.cuda()]) and torch.equal(lse[~sees.cuda()], plain_lse[~sees.cuda()])
    assert torch.isfinite(plain).all()


@pytest.mark.parametrize("new", [1, 4, 30])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** 60, -2.0 ** 60, 2.0 ** 100])
def test_large_queries_under_a_large_scale(scale, D, new):
    """Queries times the scale past fp32's range: scores of exactly 0 stay, lower ones vanish."""
    from gated_delta_rule_40_gb300 import kda
    H, Hkv, L, bs = 8, 2, 200, 16
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(new)
    k = torch.zeros((208, Hkv, D), dtype=torch.bfloat16)
    k[1:120:2] = -1.0 if scale > 0 else 1.0
    v = torch.randn((208, Hkv, D), generator=g).to(torch.bfloat16)
    cache = [torch.zeros((13, Hkv, bs, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    kda.kda_kv_write_q4(k.cuda(), v.cuda(), torch.arange(208, dtype=torch.int32, device="cuda"), *cache)
    q = torch.full((new, H, D), 2.0 ** 110, dtype=torch.bfloat16, device="cuda")
    out, lse = kda.kda_attn_paged_q4(q, *cache, ints([list(range(13))]), ints([L]), ints([0, new]), scale)
    values = Q.bf16_values(v).double()
    for i in range(new):
        rows = torch.cat([values[0:120:2], values[120:L - new + 1 + i]])
        want, size = rows.mean(0), rows.abs().mean(0)
        got = out[i].double().cpu().unflatten(0, (Hkv, H // Hkv))
        assert ((got - want[:, None]).abs() - 2.0 ** -8 * (want.abs() + 1.02 * size)[:, None]).max() <= 0
        assert (lse[i].double().cpu() - math.log(len(rows))).abs().max() <= 2.0 ** -20 * 8
