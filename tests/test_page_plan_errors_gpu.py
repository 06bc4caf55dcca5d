"""GPU tests of what kda_page_plan leaves behind when it cannot lay a step out: no table entry may name a block
that its request does not own, in this step or a later one.  Whole numbers, so every comparison is exact."""
import random

import pytest
import torch

from attn_testutil import check, normal, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


def _kda():
    from gated_delta_rule_40_gb300 import kda
    return kda


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _plan(cached, new, free, start, table, bs, T):
    """cu, lens, slots, positions, next and the table after the call, as lists."""
    tab = _dev(table).reshape(len(cached), -1)
    p = _kda().kda_page_plan(_dev(cached), _dev(new), _dev(free), _dev([start]), tab, bs, T)
    return [x.tolist() for x in (p.cu_seqlens, p.seq_lens, p.slots, p.positions)] + [p.free_next.item(), tab.tolist()]


def _reference(cached, new, free, start, table, bs, T):
    """Token by token and block by block: a new block that cannot be had is entered as -1 unless the entry is negative
    already; blocks of tokens past T are entered like the others."""
    table = [list(r) for r in table]
    width = len(table[0])
    cu, lens, slots, pos, nxt = [0], [], [], [], start
    for n, (c, a) in enumerate(zip(cached, new)):
        held, want = -(-c // bs), min(-(-(c + a) // bs), width)
        for e in range(held, want):
            if nxt < len(free):
                table[n][e] = free[nxt]
            elif table[n][e] >= 0:
                table[n][e] = -1
            nxt += 1
        for p in range(c, c + a):
            e = p // bs
            slots.append(table[n][e] * bs + p % bs if e < width and table[n][e] >= 0 else -1)
            pos.append(p)
        cu.append(cu[-1] + a)
        lens.append(c + a)
    pad = [-1] * (T - len(slots))
    return [cu, lens, slots[:T] + pad, pos[:T] + pad, min(nxt, len(free)), table]


def test_an_exhausted_list_leaves_other_requests_alone():
    """Request 1 gets one of its two blocks.  The next step's token has no place: it must not land in a block of
    request 0, whose id stands in the rest of the zero-initialised table."""
    kda = _kda()
    bs, H, D = 16, 2, 128
    g = torch.Generator().manual_seed(1)
    k0, v0, k1, v1 = normal(g, 16, H, D), normal(g, 16, H, D), normal(g, 21, H, D), normal(g, 21, H, D)
    kc, vc = (torch.zeros((2, H, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    free = _dev([0, 1])
    p1 = kda.kda_page_plan(_dev([0, 0]), _dev([16, 20]), free, _dev([0]), table, bs, 36)
    assert kda.kda_get_status() == kda.KDA_ERR_NO_BLOCKS
    assert table[0, 0].item() == 0 and table[1, 0].item() == 1 and table[1, 1].item() < 0
    assert p1.slots.tolist() == list(range(32)) + [-1] * 4
    kda.kda_kv_write(torch.cat([k0, k1[:20]]).cuda(), torch.cat([v0, v1[:20]]).cuda(), p1.slots, kc, vc)
    p2 = kda.kda_page_plan(p1.seq_lens, _dev([0, 1]), free, p1.free_next, table, bs, 1)
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    assert p2.slots.tolist() == [-1] and p2.seq_lens.tolist() == [16, 21] and p2.free_next.item() == 2
    kda.kda_kv_write(k1[20:].cuda(), v1[20:].cuda(), p2.slots, kc, vc)
    for cache, own in ((kc, k0), (vc, v0)):
        assert torch.equal(cache[0].transpose(0, 1).cpu(), own)
    # request 0 is read as it was; request 1's block that is missing counts as zeros, and is reported
    q = normal(g, 2, 4, D)
    out, lse = kda.kda_attn_paged(q.cuda(), kc, vc, table, p2.seq_lens, _dev([0, 1, 2]), 0.1)
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    k1[16:], v1[16:] = 0, 0
    check(out[:1], lse[:1], reference(q[:1], k0, v0, 0.1, first=15))
    check(out[1:], lse[1:], reference(q[1:], k1, v1, 0.1, first=20))


def test_blocks_of_tokens_past_the_slot_map():
    """More new tokens than T: the blocks are taken and entered all the same, so that table, lengths and free list
    agree in the next step."""
    kda = _kda()
    bs = 16
    cached, new, table = [0, 5, 0], [20, 40, 33], [[0] * 5 for _ in range(3)]
    table[1][0] = 9
    free = [3, 1, 7, 2, 8, 4, 6, 5]
    got = _plan(cached, new, free, 0, table, bs, 24)
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
    assert got == _reference(cached, new, free, 0, table, bs, 24)
    assert got[5] == [[3, 1, 0, 0, 0], [9, 7, 2, 0, 0], [8, 4, 6, 0, 0]] and got[4] == 7
    nxt = _plan(got[1], [1, 1, 1], free, got[4], got[5], bs, 3)
    assert kda.kda_get_status() == 0
    assert nxt[2] == [1 * bs + 4, 2 * bs + 13, 6 * bs + 1]


@pytest.mark.parametrize("N,bs,T,spare", [(3, 16, 40, 2), (40, 16, 500, 30), (1025, 32, 3000, 100), (2500, 16, 20000, 900),
                                          (2500, 64, 70000, 2500), (1, 16, 3000, 100), (1, 16, 100, 5000)])
def test_random_steps_that_do_not_fit(N, bs, T, spare):
    """Free lists that end, slot maps that end, or both, over tables full of old ids: one group of requests and more,
    one thread block and more."""
    rng = random.Random(N * bs + T)
    most = 200 if N > 1 else 20000
    cached = [rng.choice([0, rng.randrange(0, 150)]) for _ in range(N)]
    new = [rng.choice([0, 1, rng.randrange(1, most)]) for _ in range(N)] if N > 1 else [most]
    width = max(-(-(c + a) // bs) for c, a in zip(cached, new)) + 1
    table = [[rng.choice([rng.randrange(5000), -3, 0]) for _ in range(width)] for _ in range(N)]
    for n, c in enumerate(cached):
        for e in range(-(-c // bs)):
            table[n][e] = rng.randrange(5000)
    free = [rng.randrange(5000) for _ in range(spare)]
    got = _plan(cached, new, free, 2, table, bs, T)
    want = _reference(cached, new, free, 2, table, bs, T)
    assert _kda().kda_get_status() != 0
    for name, g, w in zip(("cu", "lens", "slots", "positions", "next", "table"), got, want):
        assert g == w, name
