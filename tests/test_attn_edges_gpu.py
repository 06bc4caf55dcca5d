"""GPU tests of softmax attention around its kernels: what lies in memory beside the operands, alignment,
workspaces, streams and refusals of the binding.  Bounds: attn_testutil."""
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


def _poison(D=128):
    """A call whose operands are all NaN: its tiles stay behind in shared and tensor memory."""
    x = torch.full((1, 2048, 8, D), math.nan, dtype=torch.bfloat16, device="cuda")
    _kda().kda_attn_fwd(x, x, x, 1.0)


@pytest.mark.parametrize("Hq,Hkv,D", [(7, 1, 128), (3, 3, 64), (5, 1, 64)])
def test_what_ran_before_does_not_show(Hq, Hkv, D):
    """Query tiles with rows that stand for nothing, after a call that left NaN everywhere."""
    c = Paged([700, 3, 64], [1, 2, 150], Hq, Hkv, D, 32, seed=1)
    _poison(D)
    out, lse = c.run()
    c.check(out, lse)
    g = torch.Generator().manual_seed(2)
    q, k, v = normal(g, 1, 77, Hq, D), normal(g, 1, 77, Hkv, D), normal(g, 1, 77, Hkv, D)
    _poison(D)
    o, l = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), D ** -0.5)
    check(o[0], l[0], reference(q[0], k[0], v[0], D ** -0.5))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_later_keys_are_never_seen(bad):
    """A NaN or infinity in a later token's key leaves every earlier row as it is."""
    T, at = 300, 201
    g = torch.Generator().manual_seed(3)
    q, k, v = (normal(g, 1, T, 2, 128) for _ in range(3))
    ref = reference(q[0, :at], k[0, :at], v[0, :at], 0.1)
    k[0, at:] = bad
    out, lse = _kda().kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.1)
    check(out[0, :at], lse[0, :at], ref)


@pytest.mark.parametrize("D", [64, 128])
def test_negative_scale_is_negated_keys(D):
    """-scale with -k is scale with k, bit for bit: over prompts whose rows' maxima grow and with later keys of any
    value, and over pages."""
    kda = _kda()
    g = torch.Generator().manual_seed(11)
    T, at = 700, 601
    q, k, v = normal(g, 1, T, 4, D, gain=3), normal(g, 1, T, 2, D), normal(g, 1, T, 2, D)
    k[0, 250] *= 8
    k[0, at:at + 2] = torch.tensor([math.inf, math.nan], dtype=torch.bfloat16)[:, None, None]
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    want, got = kda.kda_attn_fwd(q, k, v, 0.25), kda.kda_attn_fwd(q, -k, v, -0.25)
    for a, b in zip(want, got):
        assert torch.isfinite(a[0, :at].float()).all() and torch.equal(a[0, :at], b[0, :at])
    check(got[0][0, :at], got[1][0, :at], reference(q[0, :at].cpu(), k[0, :at].cpu(), v[0, :at].cpu(), 0.25))
    c = Paged([1500, 40, 0], [1, 130, 3], 6, 2, D, 32, seed=12)
    out, lse = c.run()
    c.check(out, lse)
    c.kc, c.scale = -c.kc, -c.scale
    out2, lse2 = c.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_visible_nan_is_not_hidden():
    """A NaN that a row does see is its answer, in a split unit and in a whole one."""
    for total in (90, 9000):
        c = Paged([total - 1], [1], 4, 2, 128, 64, seed=4)
        b = int(c.table[0, 0])
        c.kc[b, 1, 5] = math.nan
        out, lse = c.run()
        assert torch.isfinite(out[0, :2].float()).all() and torch.isfinite(lse[0, :2]).all()
        assert torch.isnan(out[0, 2:].float()).all() and torch.isnan(lse[0, 2:]).all()


@pytest.mark.parametrize("shift", [8, 16, 24])
def test_out_on_any_16_bytes(shift):
    """An out tensor that starts on 16 but not on 32 bytes; nothing around it is written."""
    kda = _kda()
    g = torch.Generator().manual_seed(5)
    q, k, v = normal(g, 1, 140, 4, 128), normal(g, 1, 140, 2, 128), normal(g, 1, 140, 2, 128)
    n = q.numel()
    buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[shift:shift + n].view(q.shape)
    _, lse = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.1, out=out)
    check(out[0], lse[0], reference(q[0], k[0], v[0], 0.1))
    assert (buf[:shift] == 5.0).all() and (buf[shift + n:] == 5.0).all()


def test_own_workspace_and_pool():
    """A caller's workspace of exactly the stated size, and the library's pool on another stream, give the bits of
    the plain call; a workspace too small is refused."""
    kda = _kda()
    c = Paged([5000, 12], [1, 40], 8, 2, 128, 16, seed=6)
    want, want_lse = c.run()
    size = kda.kda_attn_workspace_size(128)
    guard = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    got, got_lse = c.run(workspace=guard[:size])
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert (guard[size:] == 0x5a).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, got_lse = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    with pytest.raises(kda.KdaError) as e:
        c.run(workspace=guard[:size - 1])
    assert e.value.code == kda.KDA_ERR_WORKSPACE
    assert kda.kda_attn_workspace_size(96) == 0


def test_two_streams_at_once():
    """Calls that overlap on two streams do not meet in a workspace."""
    cs = [Paged([6000 + 50 * i], [3], 8, 2, 128, 64, seed=7 + i) for i in range(2)]
    want = [c.run() for c in cs]
    dev = [[x.cuda() for x in (c.q, c.kc, c.vc, c.table, c.lens, torch.tensor(c.cu, dtype=torch.int32))] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_kda().kda_attn_paged(*dev[i], cs[i].scale))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_one_serving_step_in_a_graph():
    """Plan, store and attention captured once and replayed on other lengths, which only the device knows."""
    kda = _kda()
    N, T, Hq, Hkv, D, bs = 3, 24, 4, 2, 128, 16
    g = torch.Generator().manual_seed(9)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cached, new = ints([0, 0, 0]), ints([8, 8, 8])
    free, start, table = torch.arange(40, dtype=torch.int32, device="cuda"), ints([0]), torch.zeros((N, 8), dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((40, Hkv, bs, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        p = kda.kda_page_plan(cached, new, free, start, table, bs, T)
        kda.kda_kv_write(k, v, p.slots, kc, vc)
        return p, kda.kda_attn_paged(q, kc, vc, table, p.seq_lens, p.cu_seqlens, 0.1)

    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan, (out, lse) = step()
    keys, vals = [[] for _ in range(N)], [[] for _ in range(N)]
    for lens in ([8, 3, 0], [1, 1, 20], [0, 17, 5]):
        qs, ks, vs = normal(g, T, Hq, D), normal(g, T, Hkv, D), normal(g, T, Hkv, D)
        for dst, src in ((q, qs), (k, ks), (v, vs)):
            dst.copy_(src)
        new.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for n, a in enumerate(lens):
            before = sum(x.shape[0] for x in keys[n])
            keys[n].append(ks[at:at + a])
            vals[n].append(vs[at:at + a])
            if a:
                check(out[at:at + a], lse[at:at + a],
                      reference(qs[at:at + a], torch.cat(keys[n]), torch.cat(vals[n]), 0.1, first=before))
            at += a
        cached.copy_(plan.seq_lens)
        start.copy_(plan.free_next)


def test_launches_are_counted_and_named():
    kda = _kda()
    c = Paged([40], [1], 2, 1, 64, 16, seed=8)
    c.run()
    assert kda.kda_last_launch_count() == 2
    kda.kda_set_kernel_timing(True)
    try:
        c.run()
        times = kda.kda_kernel_times()
    finally:
        kda.kda_set_kernel_timing(False)
    assert [n for n, _ in times] == ["attn_kernel"] and times[0][1] > 0


def test_binding_refuses_wrong_shapes_and_layouts():
    kda = _kda()
    g = torch.Generator().manual_seed(10)
    q, k = normal(g, 1, 20, 4, 128).cuda(), normal(g, 1, 20, 2, 128).cuda()
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_attn_fwd(q.transpose(1, 2), k, k, 0.1)
    with pytest.raises(ValueError, match="shape"):
        kda.kda_attn_fwd(q, k, k[:, :10].contiguous(), 0.1)
    with pytest.raises(TypeError):
        kda.kda_attn_fwd(q, k.half(), k, 0.1)
    with pytest.raises(ValueError, match="required"):
        kda.kda_kv_write(k[0], k[0], None, q, q)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(normal(g, 1, 4, 3, 128).cuda(), k[:, :4].contiguous(), k[:, :4].contiguous(), 0.1)
    assert e.value.code == kda.KDA_ERR_INVALID_ARG
    bad = torch.zeros((1, 4, 2, 96), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(bad, bad, bad, 0.1)
    assert e.value.code == kda.KDA_ERR_UNSUPPORTED


def _rows_64(q, k, v, scale, limits):
    """Rows q [A,H,D] in fp64 on the GPU, row i over the first limits[i] of k, v [L,H,D]: out, lse and the out bound."""
    outs, lses, tols = [], [], []
    for i, n in enumerate(limits):
        s = torch.einsum("hd,lhd->hl", q[i].double(), k[:n].double()) * scale
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, None])
        o = torch.einsum("hl,lhd->hd", p, v[:n].double())
        a = torch.einsum("hl,lhd->hd", p, v[:n].double().abs())
        outs.append(o)
        lses.append(lse)
        tols.append((2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -12) * a) * (1 + 2.0 ** -8))
    return torch.stack(outs), torch.stack(lses), torch.stack(tols)


def test_a_million_keys():
    """One token over 2^20 + 3 keys: every CTA holds a piece of the same unit."""
    kda = _kda()
    L, bs, D = (1 << 20) + 3, 128, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    nb = -(-L // bs)
    kc, vc = (torch.randn((nb, 1, bs, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)[None]
    one = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = kda.kda_attn_paged(q, kc, vc, table, one([L]), one([0, 1]), D ** -0.5)
    k, v = (c[table[0].long()].reshape(-1, 1, D) for c in (kc, vc))
    ro, rl, to = _rows_64(q, k, v, D ** -0.5, [L])
    assert ((out.double() - ro).abs() <= to).all()
    assert ((lse.double() - rl).abs() <= 2.0 ** -17 * 30 + 2.0 ** -20 * (1 + rl.abs())).all()


def test_long_prompt_and_short_neighbours():
    """A prompt of 70001 tokens packed behind and before short ones: sampled rows."""
    kda = _kda()
    lens, D = [3, 70001, 130], 64
    T = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = (torch.randn((1, T, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0, 3, 70004, T], dtype=torch.int32, device="cuda")
    out, lse = kda.kda_attn_fwd(q, k, v, D ** -0.5, cu_seqlens=cu)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    at = [0, 1, 127, 128, 4095, 30000, 65535, 65536, 70000]
    ro, rl, to = _rows_64(q[0, [3 + a for a in at]], k[0, 3:], v[0, 3:], D ** -0.5, [a + 1 for a in at])
    got = out[0, [3 + a for a in at]].double()
    assert ((got - ro).abs() <= to).all()
    assert ((lse[0, [3 + a for a in at]].double() - rl).abs() <= 2.0 ** -17 * 30 + 2.0 ** -20 * (1 + rl.abs())).all()


@pytest.mark.parametrize("T", [128, 639, 640, 641, 768, 900])
def test_prompts_around_the_first_cut(T):
    """Short prompts run without a workspace and a second kernel; the first lengths that may need them, packed and not."""
    kda = _kda()
    g = torch.Generator().manual_seed(T)
    q, k, v = normal(g, 1, T, 8, 128, gain=1.5), normal(g, 1, T, 1, 128), normal(g, 1, T, 1, 128)
    ref = reference(q[0], k[0], v[0], 0.1)
    out, lse = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.1)
    check(out[0], lse[0], ref)
    assert kda.kda_last_launch_count() == (1 if T <= 640 else 2)
    cu = torch.tensor([0, 0, T], dtype=torch.int32, device="cuda")
    out2, lse2 = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), 0.1, cu_seqlens=cu)
    check(out2[0], lse2[0], ref)
