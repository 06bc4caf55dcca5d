"""GPU tests of attention over the 4-bit cache against attention in 64 bits over the values that the cache stands
for, element by element (bounds: attn_testutil; the cache's values are bf16 numbers, so the format adds no
rounding)."""
import math

import pytest
import torch

import attn_testutil as A
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


def _kda():
    from gated_delta_rule_40_gb300 import kda
    return kda


def _run(*args, **kw):
    c = Q.PagedQ4(*args, **kw)
    out, lse = c.run()
    torch.cuda.synchronize()
    c.check(out, lse)
    return c, out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (8, 2), (6, 2), (7, 1), (16, 2), (5, 5), (24, 2), (33, 1), (128, 1)])
def test_decode(D, Hq, Hkv):
    _run([0, 1, 15, 16, 17, 40, 63, 64, 127, 200, 700], [1] * 11, Hq, Hkv, D, 16, seed=Hq)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_block_sizes(bs, D):
    _run([bs - 1, bs, bs + 1, 3 * bs + 5, 0], [1, 1, 2, 3, bs + 1 if bs < 100 else 7], 8, 2, D, bs, seed=bs)


@pytest.mark.parametrize("D", [64, 128])
def test_drafted_tokens(D):
    for new in (2, 3, 4, 5, 8):
        _run([300, 0, 31, 1000], [new] * 4, 8, 2, D, 32, seed=new)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (128, 28, 4), (64, 16, 8), (128, 7, 1), (64, 12, 4), (128, 128, 1)])
def test_chunks_beside_single_tokens(D, Hq, Hkv):
    _run([100, 0, 513, 64, 1000, 30, 0], [33, 70, 1, 129, 1, 260, 1], Hq, Hkv, D, 16, seed=Hq + D)


def test_long_contexts_and_many_requests():
    _run([40000], [1], 8, 2, 128, 64)
    _run([20011], [4], 8, 2, 64, 128)
    _run([(37 * i) % 300 for i in range(500)], [1] * 500, 4, 2, 128, 16, seed=3)
    _run([0] * 400 + [50] * 5, [0] * 400 + [1, 0, 3, 1, 0], 4, 4, 64, 16, seed=4)


def test_large_scores():
    """Scores far apart: the reference of a row moves often, and most weights vanish."""
    for gain in (8.0, 30.0):
        _run([500, 64, 1], [1, 5, 40], 8, 2, 128, 16, seed=11, gain=gain)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_values_of_any_size(D, new):
    """Values near the ends of the format's range beside ordinary ones, whole requests of them, and queries with
    channels far apart."""
    for big in (2.0 ** -13, 300.0, 3000.0, 6.0e4, 8.0e5):
        c = Q.PagedQ4([200, 90, 64], [new] * 3, 4, 1, D, 16, seed=21)
        for n, rows in ((0, slice(50, 60)), (2, slice(0, None))):
            import numpy as np
            v = c.vs[n].clone()
            v[rows] = (v[rows].float() * big / 3).to(torch.bfloat16)
            codes, b = Q.quantise(v.double().numpy())
            at_codes, at_b = Q.unpack(c.caches[1].numpy(), D)
            for j in range(v.shape[0]):
                blk = int(c.table[n, j // 16])
                at_codes[blk, :, j % 16], at_b[blk, :, j % 16] = codes[j], b[j]
            c.caches[1] = torch.from_numpy(np.ascontiguousarray(Q.pack(at_codes, at_b)))
            c.vs[n] = Q.bf16_values(v)
        c.q[0, 0, 1] = 40.0
        c.q[0, 0, 2:9] = 0.001
        c.q[0, 1] *= 1e-6
        c.check(*c.run())


def test_infinite_and_nan_queries():
    c = Q.PagedQ4([100, 30], [1, 1], 8, 1, 128, 16)
    c.q[0, 3, 5] = math.inf
    c.q[1, 0, 7] = math.nan
    out, lse = c.run()
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3]) and torch.isnan(out[1, 0]).all()
    assert torch.isfinite(out[0, :3]).all() and torch.isfinite(out[0, 4:]).all() and torch.isfinite(out[1, 1:]).all()


def test_rising_scores():
    """Keys whose scores rise from block to block, and then fall."""
    for sign in (1.0, -1.0):
        c = Q.PagedQ4([600], [3], 4, 1, 128, 16, seed=12)
        import numpy as np
        ramp = torch.linspace(0.0, 6.0, 603)[:, None, None] * sign
        k = (c.q[:1, :1].float() * ramp).to(torch.bfloat16)
        codes, b = Q.quantise(k.double().numpy())
        packed_codes, packed_b = Q.unpack(c.caches[0].numpy(), 128)
        for j in range(603):
            blk = int(c.table[0, j // 16])
            packed_codes[blk, :, j % 16], packed_b[blk, :, j % 16] = codes[j], b[j]
        c.caches[0] = torch.from_numpy(np.ascontiguousarray(Q.pack(packed_codes, packed_b)))
        c.ks[0] = Q.bf16_values(k)
        out, lse = c.run()
        c.check(out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-30, 3.0])
def test_scales(scale):
    c = Q.PagedQ4([77, 200], [1, 20], 8, 2, 128, 16, seed=2, gain=0.5)
    c.scale = scale
    out, lse = c.run()
    for n, (cached, a) in enumerate(zip(c.cached, c.new)):
        rows = slice(c.cu[n], c.cu[n + 1])
        # (attn_testutil takes the scale's size for the scores' bound)
        q = c.q[rows] if scale >= 0 else -c.q[rows]
        A.check(out[rows], lse[rows], Q.reference(q, c.ks[n], c.vs[n], abs(scale), first=cached))


@pytest.mark.parametrize("power", [100, -100])
def test_scales_far_from_one(power):
    c = Q.PagedQ4([77, 200], [1, 20], 8, 2, 128, 16, seed=2)
    c.scale, c.q = 0.09 * 2.0 ** power, c.q * 2.0 ** -power
    c.check(*c.run())


def test_nan_scale():
    c = Q.PagedQ4([20, -2], [1, 3], 2, 1, 64, 16)
    c.scale = math.nan
    out, lse = c.run()
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert not out[1:3].any() and (lse[1:3] == -math.inf).all()   # no key: 0 and -infinity


def test_rows_that_see_nothing():
    c = Q.PagedQ4([-3, 10, -5], [4, 1, 5], 8, 2, 128, 16, seed=5)
    out, lse = c.run()
    assert not out[:3].any() and (lse[:3] == -math.inf).all()
    assert not out[5:].any() and (lse[5:] == -math.inf).all()
    ref = Q.reference(c.q[3:4], c.ks[0], c.vs[0], c.scale, first=0)
    A.check(out[3:4], lse[3:4], ref)


def test_rows_past_the_last_token_stay():
    c = Q.PagedQ4([30, 5], [1, 2], 4, 2, 128, 16, pad=6)
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    got, l = c.run(out=out, lse=lse)
    assert got is out and l is lse
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()
    c.check(out, lse)
    out2, none = c.run(return_lse=False)
    assert none is None and torch.equal(out2[:3], out[:3])


def test_bad_lengths_write_nothing():
    kda = _kda()
    c = Q.PagedQ4([30, 5], [1, 2], 4, 2, 128, 16)
    kc, vc = (x.cuda() for x in c.caches)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, table = c.q.cuda(), c.table.cuda()
    for lens, cu in (([31, 7], [1, 1, 3]), ([31, 7], [0, 2, 1]), ([31, 7], [0, 1, 4]), ([-1, 7], [0, 1, 3]),
                     ([31, 16 * c.table.shape[1] + 1], [0, 1, 3])):
        out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        kda.kda_attn_paged_q4(q, kc, vc, table, dev(lens), dev(cu), c.scale, out=out)
        assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
        assert (out == 7).all()


def test_bad_blocks_count_as_zeros():
    kda = _kda()
    for bs, D, new in ((16, 128, [1, 2]), (32, 64, [1, 40])):
        c = Q.PagedQ4([100, 80], new, 4, 2, D, bs)
        c.table[0, 2] = c.caches[0].shape[0]
        c.table[1, 0] = -1
        for n, e in ((0, 2), (1, 0)):
            c.ks[n][e * bs:(e + 1) * bs] = 0
            c.vs[n][e * bs:(e + 1) * bs] = 0
        out, lse = c.run()
        assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
        c.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("entry", [0, 1, 5, 6])
def test_bad_blocks_of_a_pair(entry, D):
    """Blocks of 16 rows, of which a chunk of 32 keys takes two: the first, the second, one in the last chunk."""
    kda = _kda()
    c = Q.PagedQ4([100, 90], [1, 3], 4, 2, D, 16, seed=entry)
    c.table[0, entry] = -7
    c.ks[0][entry * 16:(entry + 1) * 16] = 0
    c.vs[0][entry * 16:(entry + 1) * 16] = 0
    out, lse = c.run()
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    c.check(out, lse)


def test_nothing_to_do():
    kda = _kda()
    c = Q.PagedQ4([], [], 4, 2, 128, 16, pad=3)
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert (out == 7).all()
    c = Q.PagedQ4([5, 0], [0, 0], 4, 2, 128, 16)
    assert c.run()[0].shape[0] == 0


def test_against_the_bf16_cache():
    """The same values in a bf16 cache give the same answer up to the roundings of both."""
    c = Q.PagedQ4([300, 40], [1, 30], 8, 2, 128, 16, seed=9)
    out, lse = c.run()
    kda = _kda()
    kc, vc = (torch.from_numpy(Q.values(*Q.unpack(x.numpy(), 128))).to(torch.bfloat16).cuda() for x in c.caches)
    o, l = kda.kda_attn_paged(c.q.cuda(), kc, vc, c.table.cuda(), c.lens.cuda(),
                              torch.tensor(c.cu, dtype=torch.int32, device="cuda"), c.scale)
    c.check(out, lse)
    c.check(o, l)


def test_bits_repeat_streams_workspaces_and_graphs():
    kda = _kda()
    c = Q.PagedQ4([700, 40, 0], [1, 30, 5], 8, 2, 128, 16, seed=9)
    out, lse = c.run()
    for _ in range(3):
        o, l = c.run()
        assert torch.equal(o, out) and torch.equal(l, lse)
    ws = torch.empty(kda.kda_attn_q4_workspace_size(128), dtype=torch.uint8, device="cuda")
    o, _ = c.run(workspace=ws)
    assert torch.equal(o, out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, l = c.run(stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    kc, vc = (x.cuda() for x in c.caches)
    q, table, lens = c.q.cuda(), c.table.cuda(), c.lens.cuda()
    cu = torch.tensor(c.cu, dtype=torch.int32, device="cuda")
    graphs = []
    for _ in range(2):   # two graphs, each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, kda.kda_attn_paged_q4(q, kc, vc, table, lens, cu, c.scale)[0]))
    q.copy_(c.q.neg())
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    c.q = c.q.neg()
    for _, o in graphs:
        c.check(o, None)


def test_streams_at_once():
    """Calls that overlap on two streams, eager ones and graphs, have a workspace each."""
    kda = _kda()
    cs = [Q.PagedQ4([3000, 40, 0, 900], [1, 30, 5, 2], 8, 2, 128, 16, seed=s) for s in (1, 2)]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    args = [(c.q.cuda(), *(x.cuda() for x in c.caches), c.table.cuda(), c.lens.cuda(),
             torch.tensor(c.cu, dtype=torch.int32, device="cuda"), c.scale) for c in cs]
    graphs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, kda.kda_attn_paged_q4(*a)))
    torch.cuda.synchronize()
    got = [[kda.kda_attn_paged_q4(*a, stream=s) for a, s in zip(args, streams)] for _ in range(10)]
    for _ in range(10):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for pair in got + [[o for _, o in graphs]]:
        for (o, l), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_past_32_bits_of_bytes(D):
    """A cache of more than 2^32 bytes whose last blocks hold what a small one's do: the same bits."""
    kda = _kda()
    c = Q.PagedQ4([300, 40, 130, 500], [1, 60, 4, 100], 8, 2, D, 64, seed=5)
    out, lse = c.run()
    c.check(out, lse)
    small = [x.cuda() for x in c.caches]
    n = small[0].shape[0]
    blocks = 2 ** 32 // small[0][0].numel() + n + 5
    first = blocks - n
    assert first * small[0][0].numel() >= 2 ** 32
    far = []
    for x in small:
        far.append(torch.full((blocks, *x.shape[1:]), 255, dtype=torch.uint8, device="cuda"))
        far[-1][first:] = x
    o, l = kda.kda_attn_paged_q4(c.q.cuda(), *far, (c.table + first).cuda(), c.lens.cuda(),
                                 torch.tensor(c.cu, dtype=torch.int32, device="cuda"), c.scale)
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_after_the_store():
    """Plan, store, attention, step by step: a prompt in one step or in chunks gives the same cache and answers
    within the bounds."""
    kda = _kda()
    D, H, Hkv, bs, lens = 128, 8, 2, 16, [70, 1, 33]
    g = torch.Generator().manual_seed(3)
    T = sum(lens)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fused = [A.normal(g, n, H + 2 * Hkv, D) for n in lens]
    ref = []
    for f in fused:
        q, k, v = f.split([H, Hkv, Hkv], 1)
        ref.append(Q.reference(q, Q.bf16_values(k.contiguous()), Q.bf16_values(v.contiguous()), D ** -0.5))
    caches = [torch.zeros((20, Hkv, bs, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table, free, at, held = torch.zeros((3, 8), dtype=torch.int32, device="cuda"), dev(list(range(20))), dev([0]), dev([0] * 3)
    done = [0, 0, 0]
    for step in ([30, 0, 33], [39, 0, 0], [1, 1, 0]):
        part = torch.cat([f[d:d + a] for f, d, a in zip(fused, done, step)]).cuda()
        plan = kda.kda_page_plan(held, dev(step), free, at, table, bs, part.shape[0])
        q, k, v = part.split([H, Hkv, Hkv], 1)
        kda.kda_kv_write_q4(k, v, plan.slots, *caches)
        out, lse = kda.kda_attn_paged_q4(q.contiguous(), *caches, table, plan.seq_lens, plan.cu_seqlens, D ** -0.5)
        row = 0
        for n, a in enumerate(step):
            if a:
                A.check(out[row:row + a], lse[row:row + a], [x[done[n]:done[n] + a] for x in ref[n]])
            row += a
            done[n] += a
        held, at = plan.seq_lens, plan.free_next
    assert done == lens
