"""GPU tests of the paged cache's layout and store (kda_page_plan, kda_kv_write): whole numbers and
copies, so every comparison is exact.  The reference is a plain loop over requests and tokens."""
import random

import pytest
import torch

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


def plan_reference(cached, new, free, start, table, bs, T):
    """(cu, lens, slots, positions, next, table) token by token; blocks and slots that cannot be had are -1 or unwritten."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    cu, lens, slots, pos = [0], [], [], []
    nxt = start
    for n, (c, a) in enumerate(zip(cached, new)):
        c, a = max(c, 0), max(a, 0)
        own, want = -(-c // bs), min(-(-(c + a) // bs), width)
        for j in range(own, want):
            if nxt < len(free):
                table[n][j] = free[nxt]
            nxt += 1
        missing = max(0, nxt - len(free)) if want > own else 0   # of this request's last blocks
        for p in range(c, c + a):
            e = p // bs
            ok = e < width and not (e >= own and e >= want - missing)
            slots.append(table[n][e] * bs + p % bs if ok else -1)
            pos.append(p)
        cu.append(cu[-1] + a)
        lens.append(c + a)
    slots, pos = slots[:T] + [-1] * (T - len(slots)), pos[:T] + [-1] * (T - len(pos))
    return cu, lens, slots, pos, min(nxt, len(free)), table


def _run(cached, new, free, start, table, bs, T, **kw):
    kda = _kda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tab = dev(table).reshape(len(cached), -1)
    p = kda.kda_page_plan(dev(cached), dev(new), dev(free), dev([start]), tab, bs, T, **kw)
    torch.cuda.synchronize()
    return ([x.tolist() for x in (p.cu_seqlens, p.seq_lens, p.slots, p.positions)] + [p.free_next.item()] + [tab.tolist()])


def _check(cached, new, bs, T=None, start=0, spare=4, width=None, free=None):
    rng = random.Random(len(cached))
    width = max([-(-(c + a) // bs) for c, a in zip(cached, new)] + [0]) + 1 if width is None else width
    held = sum(min(-(-c // bs), width) for c in cached)
    need = sum(-(-(c + a) // bs) - -(-c // bs) for c, a in zip(cached, new))
    ids = rng.sample(range(held + need + start + spare), held + need + start + spare)
    table, at = [], 0
    for c in cached:
        own = min(-(-c // bs), width)
        table.append(ids[at:at + own] + [-7] * (width - own))
        at += own
    free = ids[at:] if free is None else ids[at:at + free]
    T = sum(new) if T is None else T
    got = _run(cached, new, free, start, table, bs, T)
    want = plan_reference(cached, new, free, start, table, bs, T)
    for name, g, w in zip(("cu", "lens", "slots", "positions", "next", "table"), got, want):
        assert g == w, name


@pytest.mark.parametrize("bs", [16, 64, 128, 1024])
def test_plan_small(bs):
    _check([0], [1], bs)
    _check([bs - 1, bs, bs + 1, 0, 5], [1, 1, 1, 0, 3 * bs], bs, start=3)
    _check([0, 0, 0], [0, 0, 0], bs)
    _check([10, 20], [0, 2], bs, T=40)      # padded
    _check([7], [0], bs, T=0)


@pytest.mark.parametrize("N", [1, 31, 32, 33, 1023, 1024, 1025, 2500])
def test_plan_many_requests(N):
    rng = random.Random(N)
    cached = [rng.randrange(0, 200) for _ in range(N)]
    new = [rng.choice([0, 1, 1, 1, rng.randrange(1, 60)]) for _ in range(N)]
    _check(cached, new, 16, T=sum(new) + 9, start=2)


def test_plan_long_prompts():
    _check([0, 100, 30000], [20000, 1, 5000], 16)
    _check([0], [70001], 64, T=70001)


def test_plan_feeds_attention_layouts():
    """The packed offsets are those that kda_fwd's linear layers take, bit for bit."""
    got = _run([3, 0, 9], [2, 5, 0], list(range(10)), 0, [[9, -1], [-1, -1], [8, -1]], 16, 7)
    assert got[0] == [0, 2, 7, 7] and got[1] == [5, 5, 9]


def test_plan_reports_what_it_cannot_lay_out():
    kda = _kda()
    _check([0, 10, 0], [40, 30, 50], 16, free=4)                # free list ends inside the second request
    assert kda.kda_get_status() == kda.KDA_ERR_NO_BLOCKS
    _check([0, 10], [100, 3], 16, width=3)                      # a request longer than its table row
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
    _check([5, 6], [9, 9], 16, T=12)                            # more new tokens than the slot map holds
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
    got = _run([-4, 3], [2, -5], [4, 5, 6], 0, [[-1], [2]], 16, 2)   # negative lengths count as 0
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
    assert got[0] == [0, 2, 2] and got[1] == [2, 3] and got[2] == [4 * 16, 4 * 16 + 1] and got[4] == 1


def test_plan_steps_follow_each_other():
    """Two steps whose lengths and free list never leave the device equal one step of both's tokens."""
    kda = _kda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    free, bs = dev([9, 3, 5, 1, 7, 2, 8]), 16
    table = torch.full((2, 5), -1, dtype=torch.int32, device="cuda")
    p1 = kda.kda_page_plan(dev([0, 0]), dev([20, 3]), free, dev([0]), table, bs, 23)
    p2 = kda.kda_page_plan(p1.seq_lens, dev([20, 14]), free, p1.free_next, table, bs, 34)
    assert table.tolist() == [[9, 3, 1, -1, -1], [5, 7, -1, -1, -1]]
    assert p2.seq_lens.tolist() == [40, 17] and p2.free_next.item() == 5
    assert p2.slots[:13].tolist() == [3 * 16 + i for i in range(4, 16)] + [16]


# ------------------------------------------------------------------ the store
@pytest.mark.parametrize("T,H,D,bs", [(1, 1, 64, 16), (5, 8, 128, 64), (77, 3, 128, 16), (1000, 2, 64, 128),
                                       (4097, 8, 128, 64), (300, 5, 64, 1024)])
def test_write(T, H, D, bs):
    kda = _kda()
    g = torch.Generator().manual_seed(T)
    nb = -(-T // bs) + 4
    slots = torch.randperm(nb * bs, generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    k, v, kc, vc = (torch.randn(s, generator=g).to(torch.bfloat16) for s in
                    ((T, H, D), (T, H, D), (nb, H, bs, D), (nb, H, bs, D)))
    got_k, got_v = kc.cuda(), vc.cuda()
    kda.kda_kv_write(k.cuda(), v.cuda(), slots.cuda(), got_k, got_v)
    keep = slots >= 0
    s = slots[keep].long()
    kc[s // bs, :, s % bs] = k[keep]
    vc[s // bs, :, s % bs] = v[keep]
    assert torch.equal(got_k.cpu(), kc) and torch.equal(got_v.cpu(), vc)


def test_write_keeps_bits_and_reports_bad_slots():
    """NaN patterns pass unchanged; a slot past the cache is left out and reported."""
    kda = _kda()
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(512, 1, 128)
    kc, vc = (torch.zeros((33, 1, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(512, dtype=torch.int32)
    slots[5] = 33 * 16
    slots[6] = 0x7fffffff
    kda.kda_kv_write(bits.cuda(), bits.cuda(), slots.cuda(), kc, vc)
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    want = torch.zeros(33 * 16, 128, dtype=torch.int16)
    want[:512] = bits.view(torch.int16)[:, 0]
    want[5:7] = 0
    for c in (kc, vc):
        assert torch.equal(c.view(torch.int16).reshape(-1, 128).cpu(), want)
    kda.kda_kv_write(bits[:0].cuda(), bits[:0].cuda(), slots[:0].cuda(), kc, vc)


def test_write_past_32_bit_offsets():
    """A cache of 5.5e9 bytes a tensor: slots whose element offset passes 2^31."""
    kda = _kda()
    nb, H, bs, D = 21000, 8, 128, 128
    kc, vc = (torch.zeros((nb, H, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([nb * bs - 1, 17, nb * bs // 2 + 3], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((3, H, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    kda.kda_kv_write(k, v, slots, kc, vc)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // bs, :, s % bs], k[i]) and torch.equal(vc[s // bs, :, s % bs], v[i])
    # and attention over those blocks
    q = torch.randn((1, 16, D), device="cuda").to(torch.bfloat16)
    table = torch.tensor([[nb - 1]], dtype=torch.int32, device="cuda")
    one = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = kda.kda_attn_paged(q, kc, vc, table, one([bs]), one([0, 1]), 0.1)
    s = 0.1 * (q[0].double() @ torch.zeros(D, dtype=torch.float64, device="cuda"))
    kk = kc[nb - 1].double().repeat_interleave(2, 0)
    vv = vc[nb - 1].double().repeat_interleave(2, 0)
    s = 0.1 * torch.einsum("hd,hld->hl", q[0].double(), kk)
    p = torch.softmax(s, -1)
    want = torch.einsum("hl,hld->hd", p, vv)
    # bf16 rounds to within 2^-8 (attn_testutil): the softmax weights once, the result once
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * torch.einsum("hl,hld->hd", p, vv.abs())
    assert ((out[0].double() - want).abs() <= bound * (1 + 2.0 ** -8)).all()
