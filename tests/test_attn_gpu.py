"""GPU tests of softmax attention (kda_attn_fwd, kda_attn_paged) against 64 bits, at the sizes and masks
where such kernels go wrong.  Bounds: attn_testutil."""
import math

import pytest
import torch

from attn_testutil import Paged, check, normal, reference

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


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ whole prompts
@pytest.mark.parametrize("B,T,Hq,Hkv,D", [
    (1, 1, 1, 1, 128), (1, 2, 4, 1, 64), (2, 17, 2, 2, 128), (1, 63, 8, 2, 128), (1, 64, 8, 2, 64), (3, 65, 3, 1, 128),
    (1, 127, 1, 1, 128), (1, 128, 1, 1, 64), (1, 129, 1, 1, 128), (2, 130, 10, 2, 64), (1, 255, 7, 1, 128),
    (1, 256, 2, 2, 128), (1, 257, 2, 1, 128), (1, 300, 12, 1, 64), (1, 385, 4, 4, 128), (1, 513, 5, 1, 128),
    (1, 40, 32, 1, 128), (1, 9, 128, 1, 128), (1, 700, 16, 2, 64), (1, 1111, 6, 2, 128)])
def test_prompt_sizes(B, T, Hq, Hkv, D):
    g = torch.Generator().manual_seed(T + Hq)
    q, k, v = normal(g, B, T, Hq, D, gain=1.5), normal(g, B, T, Hkv, D), normal(g, B, T, Hkv, D)
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), D ** -0.5)
    for b in range(B):
        check(out[b], lse[b], reference(q[b], k[b], v[b], D ** -0.5))


@pytest.mark.parametrize("lens", [[5], [0, 130, 1, 0, 205, 64, 0], [1] * 37, [128, 128, 256], [300, 2, 600, 17]])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (2, 2, 64)])
def test_prompt_packed(lens, Hq, Hkv, D):
    T = sum(lens)
    g = torch.Generator().manual_seed(T)
    q, k, v = normal(g, 1, T, Hq, D), normal(g, 1, T, Hkv, D), normal(g, 1, T, Hkv, D)
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), D ** -0.5, cu_seqlens=_cu(lens))
    at = 0
    for n in lens:
        part = slice(at, at + n)
        if n:
            check(out[0, part], lse[0, part], reference(q[0, part], k[0, part], v[0, part], D ** -0.5))
        at += n


def test_packed_equals_one_by_one_and_many_prompts():
    """1500 prompts in one call (more than one group of any per-CTA scan) equal the same prompts alone."""
    lens = [(i * 7) % 23 for i in range(1500)]
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    q, k, v = normal(g, 1, T, 4, 128), normal(g, 1, T, 2, 128), normal(g, 1, T, 2, 128)
    cu = _cu(lens)
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.09, cu_seqlens=cu)
    for n in (1, 2, 22, 700, 1023, 1024, 1025, 1498):
        part = slice(int(cu[n]), int(cu[n + 1]))
        check(out[0, part], lse[0, part], reference(q[0, part], k[0, part], v[0, part], 0.09))


def test_other_prompts_hold_nan_and_infinity():
    """A packed prompt's neighbours hold NaN and infinity: its own rows are what they are alone."""
    lens, D = [70, 133, 90], 128
    g = torch.Generator().manual_seed(4)
    q, k, v = (normal(g, 1, sum(lens), 2, D) for _ in range(3))
    for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan)):
        x[0, :70] = bad
        x[0, 203:] = -bad
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), D ** -0.5, cu_seqlens=_cu(lens))
    part = slice(70, 203)
    check(out[0, part], lse[0, part], reference(q[0, part], k[0, part], v[0, part], D ** -0.5))


@pytest.mark.parametrize("shape", ["rising", "falling", "spike"])
def test_prompt_scores_of_hundreds(shape):
    """Scores up to +-400 whose maximum moves along the keys: every rescaling of the running softmax."""
    T, D = 700, 128
    g = torch.Generator().manual_seed(5)
    u = torch.randn(D, generator=g)
    u /= u.norm()
    ramp = torch.linspace(-1, 1, T) * 8
    if shape == "falling":
        ramp = -ramp
    if shape == "spike":
        ramp = torch.zeros(T)
        ramp[[3, 200, 450]] = torch.tensor([4.0, 8.0, 6.0])
    k = (ramp[:, None] * u + 0.05 * torch.randn(T, D, generator=g)).to(torch.bfloat16)[None, :, None]
    q = (50 * u + 0.2 * torch.randn(T, D, generator=g)).to(torch.bfloat16)[None, :, None]
    v = normal(g, 1, T, 1, D)
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 1.0)
    check(out[0], lse[0], reference(q[0], k[0], v[0], 1.0))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
def test_prompt_scales(scale):
    """No scale (a plain mean of the values), a negative and a vanishing one."""
    g = torch.Generator().manual_seed(6)
    q, k, v = (normal(g, 1, 200, 1, 64) for _ in range(3))
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale)
    ro, rl, to, tl = reference(q[0], k[0], v[0], scale)
    tl = tl.abs() + 2.0 ** -17 * reference(q[0], k[0], v[0], abs(scale))[3]
    check(out[0], lse[0], (ro, rl, to.abs(), tl))


def test_prompt_long_rows():
    """One prompt of 5000 tokens: sampled rows of sampled heads."""
    T, D = 5000, 128
    g = torch.Generator().manual_seed(7)
    q, k, v = normal(g, 1, T, 8, D, gain=1.5), normal(g, 1, T, 2, D), normal(g, 1, T, 2, D)
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), D ** -0.5)
    for t in (0, 127, 128, 1000, 2048, 4095, 4999):
        check(out[0, t:t + 1], lse[0, t:t + 1], reference(q[0, t:t + 1], k[0, :t + 1], v[0, :t + 1], D ** -0.5, first=t))


def test_prompt_options():
    kda = _kda()
    g = torch.Generator().manual_seed(8)
    q, k, v = (normal(g, 1, 140, 2, 128).cuda() for _ in range(3))
    out, lse = kda.kda_attn_fwd(q, k, v, 0.1)
    o2, none = kda.kda_attn_fwd(q, k, v, 0.1, return_lse=False)
    assert none is None and torch.equal(out, o2)
    mine, mine_lse = torch.zeros_like(out), torch.zeros_like(lse)
    o3, l3 = kda.kda_attn_fwd(q, k, v, 0.1, out=mine, lse=mine_lse)
    assert o3 is mine and l3 is mine_lse and torch.equal(mine, out) and torch.equal(mine_lse, lse)
    o4, l4 = kda.kda_attn_fwd(q[:, :0], k[:, :0], v[:, :0], 0.1)
    assert o4.shape == (1, 0, 2, 128) and l4.shape == (1, 0, 2)
    o5, _ = kda.kda_attn_fwd(q[:, :0], k[:, :0], v[:, :0], 0.1, cu_seqlens=_cu([0, 0]))
    assert o5.numel() == 0


# ------------------------------------------------------------------ over the cache
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (7, 1, 128), (4, 4, 64)])
def test_decode(bs, Hq, Hkv, D):
    """One token a request, contexts at and around block and tile ends, the first token among them."""
    total = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 400, 1000]
    c = Paged([t - 1 for t in total], [1] * len(total), Hq, Hkv, D, bs, seed=bs, gain=1.5)
    c.check(*c.run())


@pytest.mark.parametrize("bs,Hq,Hkv,D", [(16, 8, 2, 128), (64, 5, 1, 128), (128, 2, 2, 64), (32, 12, 1, 64)])
def test_chunks(bs, Hq, Hkv, D):
    """Chunks of prompts, drafted tokens, single tokens and idle requests in one call."""
    cached = [0, 100, 0, 511, 64, 0, 300, 128, 17, 0]
    new = [130, 77, 0, 4, 64, 1, 200, 128, 1, 300]
    c = Paged(cached, new, Hq, Hkv, D, bs, seed=1, gain=1.5)
    c.check(*c.run())


def test_idle_requests_and_padding():
    """Requests without new tokens, without any token, and padded rows of q (left alone)."""
    kda = _kda()
    c = Paged([0, 50, 0, 200], [0, 0, 3, 1], 4, 2, 128, 16, pad=5)
    out = torch.full((9, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 4), 7.0, device="cuda")
    c.run(out=out, lse=lse)
    c.check(out, lse)
    assert (out[4:] == 7.0).all() and (lse[4:] == 7.0).all()
    e = Paged([0, 5], [0, 0], 4, 2, 128, 16)
    o, l = e.run()
    assert o.shape == (0, 4, 128) and kda.kda_get_status() == 0


def test_rows_without_keys():
    """seq_lens below the number of new tokens: the first of them see nothing."""
    c = Paged([-3, -200, -5, 40], [10, 300, 5, 2], 4, 2, 128, 32)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[:3] == 0).all() and (lse[:3] == -math.inf).all()
    assert (out[10:210] == 0).all() and torch.isfinite(lse[210:310]).all()


@pytest.mark.parametrize("N,total,new,Hq,Hkv,D,bs", [(1, 20000, 1, 8, 1, 128, 64), (2, 9001, 4, 8, 2, 128, 16),
                                                      (1, 5000, 130, 4, 1, 64, 128), (3, 2500, 1, 16, 1, 128, 32)])
def test_long_context(N, total, new, Hq, Hkv, D, bs):
    """Few rows over long caches: the work of one request is split and joined."""
    c = Paged([total - new - 100 * i for i in range(N)], [new] * N, Hq, Hkv, D, bs, seed=total, gain=1.5)
    c.check(*c.run())


def test_many_requests_ragged():
    """1300 requests of very different lengths in one call."""
    cached = [(i * i * 13) % 190 for i in range(1300)]
    cached[700] = 6000
    new = [1 if i % 5 else i % 7 for i in range(1300)]
    c = Paged(cached, new, 2, 1, 64, 16, seed=2)
    c.check(*c.run())


def test_split_joins_large_scores():
    """A long request whose maximum lies in its first, a middle or its last part."""
    for at in (5, 3000, 5990):
        c = Paged([5999], [1], 4, 1, 128, 64, seed=at)
        u = c.q[0, 0].float()
        c.ks[0][at, 0] = (u * 3).to(torch.bfloat16)
        b, r = divmod(at, 64)
        c.kc[int(c.table[0, b]), 0, r] = c.ks[0][at, 0]
        c.check(*c.run())


def test_paged_equals_prompt_rows():
    """A prompt through the cache in chunks gives the rows that the whole-prompt call gives, within the bounds'
    two roundings, and each call gives the same bits again."""
    kda = _kda()
    T, bs = 333, 32
    c = Paged([0], [T], 6, 2, 128, bs, seed=9)
    q, k, v = c.q.cuda()[None], c.ks[0].cuda()[None], c.vs[0].cuda()[None]
    whole, lse = kda.kda_attn_fwd(q, k, v, c.scale)
    again, lse2 = kda.kda_attn_fwd(q, k, v, c.scale)
    assert torch.equal(whole, again) and torch.equal(lse, lse2)
    ref = reference(c.q, c.ks[0], c.vs[0], c.scale)
    parts = [0, 1, 100, 101, 229, T]
    for a, b in zip(parts, parts[1:]):
        args = (q[0, a:b], c.kc.cuda(), c.vc.cuda(), c.table.cuda(), torch.tensor([b], dtype=torch.int32, device="cuda"),
                torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), c.scale)
        o, l = kda.kda_attn_paged(*args)
        check(o, l, [x[a:b] for x in ref])
        o2, l2 = kda.kda_attn_paged(*args)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_other_stream_and_graph():
    """On a side stream, and replayed from a CUDA graph on new lengths."""
    kda = _kda()
    c = Paged([700, 40], [1, 1], 8, 2, 128, 16, seed=10)
    t = [c.q.cuda(), c.kc.cuda(), c.vc.cuda(), c.table.cuda(), c.lens.cuda(),
         torch.tensor(c.cu, dtype=torch.int32, device="cuda")]
    want, want_lse = kda.kda_attn_paged(*t, c.scale)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_attn_paged(*t, c.scale, out=out, lse=lse, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kda.kda_attn_paged(*t, c.scale, out=out, lse=lse)
    t[4].copy_(torch.tensor([650, 33], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for n, total in enumerate((650, 33)):
        check(out[n:n + 1], lse[n:n + 1],
              reference(c.q[n:n + 1], c.ks[n][:total], c.vs[n][:total], c.scale, first=total - 1))


# ------------------------------------------------------------------ faults found on the device
def test_bad_lengths_are_reported_and_nothing_is_written():
    kda = _kda()
    c = Paged([30, 20], [2, 2], 2, 1, 64, 16)
    fill = lambda: (torch.full((4, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 2), 3.0, device="cuda"))
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    width = c.table.shape[1] * 16
    for cu, lens in (([0, 3, 2], [32, 22]), ([1, 2, 4], [32, 22]), ([0, 2, 5], [32, 22]), ([0, 2, 4], [32, -1]),
                     ([0, 2, 4], [width + 1, 22])):
        out, lse = fill()
        kda.kda_attn_paged(c.q.cuda(), c.kc.cuda(), c.vc.cuda(), c.table.cuda(), dev(lens), dev(cu), c.scale, out=out,
                           lse=lse)
        assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
        assert (out == 3.0).all() and (lse == 3.0).all()
    q = c.q.cuda()[None]
    k = q[:, :, :1].contiguous()
    for cu in ([0, 3], [0, 5], [1, 4], [0, 5, 4]):
        out, lse = fill()
        kda.kda_attn_fwd(q, k, k, 1.0, cu_seqlens=dev(cu), out=out[None], lse=lse[None])
        assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
        assert (out == 3.0).all()


@pytest.mark.parametrize("bad", [-1, -(1 << 31), 1 << 20, 0x7fffffff])
def test_bad_block_ids_are_reported(bad):
    """A block id outside the cache: reported, its keys and values count as zeros, other requests are right."""
    kda = _kda()
    c = Paged([200, 90], [1, 1], 4, 2, 128, 32, seed=11)
    c.table[0, 2] = bad
    c.ks[0][64:96] = 0
    c.vs[0][64:96] = 0
    out, lse = c.run()
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    c.check(out, lse)
