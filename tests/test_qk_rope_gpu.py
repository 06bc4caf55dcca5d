"""GPU tests of the query/key norms with rotation, and of their gradients, against 64 bits.

Bounds, element by element.  fp32 quantities: the reciprocal root is off by 2^-21 relative (a sum of D <= 128
squares, 2^-24 each step of a tree of 8 + 4, and the root's 2^-22), cos and sin by 2^-22 absolute, each product by
2^-24.  A turned channel of the pair (a, b) is then off by 2^-19 (|a| + |b|), with room of a factor 2, and rounded
to bf16 once: 2^-8 |out|.  The gradients dx = r (gw - x^ m), m = mean(gw x^), stay fp32: 2^-18 r (|ga| + |gb|) |w| for
the first term, 2^-18 r |x^| mean(|gw x^|) for the second.  A weight's gradient is a sum of n terms |g x^|, in
fp32 over chains of at most 64 + n / 2^12 + 40 additions: 2^-18 + 2^-24 times that, of the sum of magnitudes.
The gradients are those of automatic differentiation of the 64-bit forward, which differences confirm."""
import math

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


from qk_rope_testutil import freqs_of, grad_bounds, gradients, normed, reference  # noqa: E402


def _case(T, H, Hkv, D, seed=0, far=1000, fused=False):
    g = torch.Generator().manual_seed(seed)
    f = torch.randn((T, H + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    if T > 3:
        f[2, 0] = 0.0                                 # a row of zeros
        f[3, H] *= 1e3
    pos = torch.randint(0, far + 1, (T,), generator=g).to(torch.int32)
    w = 1.0 + 0.3 * torch.randn((2, D), generator=g)
    dev = f.cuda()
    q, k = dev[:, :H], dev[:, H:H + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    return f[:, :H].contiguous(), f[:, H:H + Hkv].contiguous(), q, k, pos, w


def _check(out, x, pos, freqs, w, eps, norm, pairs):
    ref, size = reference(x, pos, freqs, w, eps, norm, pairs)
    o = out.double().cpu()
    bad = (o - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -19 * size)
    assert torch.isfinite(o).all() and bad.max() <= 0, f"off its bound by {bad.max():.3e}"


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 32), (128, 24), (128, 8), (128, 0), (64, 64), (64, 16),
                                   (64, 40), (64, 0)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [0, 1, 2])
def test_forward(D, rot, pairs, norm):
    kda = _kda()
    for T, H, Hkv in ((1, 1, 1), (5, 8, 2), (37, 7, 3)):
        q, k, dq, dk, pos, w = _case(T, H, Hkv, D, seed=T, fused=T == 5)
        freqs = freqs_of(rot)
        ws = (w[0], w[1]) if norm == 2 else (None, None)
        qo, ko = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda(), *(None if x is None else x.cuda() for x in ws),
                                      norm=norm > 0, interleaved=pairs)
        assert qo.is_contiguous() and ko.is_contiguous()
        _check(qo, q, pos, freqs, ws[0], 1e-6, norm > 0, pairs)
        _check(ko, k, pos, freqs, ws[1], 1e-6, norm > 0, pairs)


@pytest.mark.parametrize("T,H,Hkv", [(1, 32, 8), (64, 32, 8), (1001, 3, 1), (5000, 16, 2), (1, 1, 100)])
def test_sizes(T, H, Hkv):
    kda = _kda()
    for D in (64, 128):
        q, k, dq, dk, pos, w = _case(T, H, Hkv, D, seed=T, fused=True)
        freqs = freqs_of(D)
        qo, ko = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda(), w[0].cuda(), None)
        _check(qo, q, pos, freqs, w[0], 1e-6, True, False)
        _check(ko, k, pos, freqs, None, 1e-6, True, False)


@pytest.mark.parametrize("far", [1 << 20, 1 << 24, (1 << 31) - 1])
def test_far_positions(far):
    """Angles of millions of radians, against products in exact arithmetic."""
    kda = _kda()
    q, k, dq, dk, pos, _ = _case(50, 2, 1, 128, seed=7, far=far)
    pos[0], pos[1] = far, far - 1
    freqs = freqs_of(128)
    freqs[:6] = torch.tensor([3.0, 6.2831855, 100.25, -0.7, 1e-6, 1e-42])
    qo, _ = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda())
    _check(qo, q, pos, freqs, None, 1e-6, True, False)


def test_wild_frequencies_turn_by_nan_and_leave_the_others():
    kda = _kda()
    q, k, dq, dk, pos, _ = _case(4, 2, 1, 64, seed=7)
    freqs = freqs_of(64)
    freqs[3], freqs[5], freqs[9] = math.nan, math.inf, 2.0 ** 24
    qo, _ = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda())
    wild = torch.tensor([3, 5, 9, 35, 37, 41])
    assert torch.isnan(qo[..., wild]).all()
    rest = torch.tensor([c for c in range(64) if c not in wild.tolist()])
    ref, size = reference(q, pos, torch.where(torch.isin(torch.arange(32), wild), 0.0, freqs), None, 1e-6, True, False)
    bad = ((qo.double().cpu() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -19 * size))[..., rest]
    assert bad.max() <= 0


def test_tokens_left_out_and_in_place():
    kda = _kda()
    q, k, dq, dk, pos, w = _case(9, 4, 2, 128)
    pos[4], pos[8] = -1, -2 ** 31
    freqs = freqs_of(128)
    args = (pos.cuda(), freqs.cuda(), w[0].cuda(), w[1].cuda())
    qo, ko = kda.kda_qk_norm_rope(dq, dk, *args, q_out=torch.full_like(dq, 7.0), k_out=torch.full_like(dk, 7.0))
    for o in (qo, ko):
        assert (o[4] == 7).all() and (o[8] == 7).all()
    keep = [0, 1, 2, 3, 5, 6, 7]
    _check(qo[keep], q[keep], pos[keep], freqs, w[0], 1e-6, True, False)
    qi, ki = kda.kda_qk_norm_rope(dq, dk, *args, q_out=dq, k_out=dk)   # in place
    assert qi is dq and torch.equal(dq[keep], qo[keep]) and torch.equal(dk[keep], ko[keep])
    assert torch.equal(dq[4].cpu(), q[4])


def test_infinite_channels():
    """Without the norm, an infinity outside the turned channels passes through and touches no other channel."""
    kda = _kda()
    q, k, dq, dk, pos, _ = _case(5, 2, 1, 128)
    dq[1, 0, 100] = math.inf
    freqs = freqs_of(64)
    qo, _ = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda(), norm=False)
    assert qo[1, 0, 100] == math.inf and torch.isfinite(qo).sum() == qo.numel() - 1


def test_eps_and_zero_rows():
    kda = _kda()
    q, k, dq, dk, pos, w = _case(6, 2, 2, 64)
    freqs = freqs_of(64)
    for eps in (1e-12, 1e-5, 0.5):
        qo, ko = kda.kda_qk_norm_rope(dq, dk, pos.cuda(), freqs.cuda(), w[0].cuda(), w[1].cuda(), eps=eps)
        assert not qo[2, 0].any()
        _check(qo, q, pos, freqs, w[0], eps, True, False)


def test_no_tokens():
    kda = _kda()
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    f, w = freqs_of(64).cuda(), torch.ones(64, device="cuda")
    qo, ko = kda.kda_qk_norm_rope(e, e, i, f)
    assert qo.shape == (0, 2, 64)
    g = kda.kda_qk_norm_rope_bwd(e, e, i, f, e, e, w, w)
    assert not g["dq_weight"].any() and not g["dk_weight"].any()


# ---------------------------------------------------------------- gradients
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 32), (128, 24), (64, 64), (64, 0)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [0, 1, 2])
def test_backward(D, rot, pairs, norm):
    kda = _kda()
    for T, H, Hkv in ((1, 1, 1), (6, 8, 2), (45, 7, 3)):
        q, k, dq, dk, pos, w = _case(T, H, Hkv, D, seed=T, fused=T == 6)
        if T == 45:
            pos[7] = -1
        freqs = freqs_of(rot)
        ws = (w[0], w[1]) if norm == 2 else (None, None)
        g = torch.Generator().manual_seed(T + 1)
        do = [torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in (q, k)]
        got = kda.kda_qk_norm_rope_bwd(dq, dk, pos.cuda(), freqs.cuda(), do[0].cuda(), do[1].cuda(),
                                       *(None if x is None else x.cuda() for x in ws), norm=norm > 0, interleaved=pairs)
        for name, x, d, weight in (("q", q, do[0], ws[0]), ("k", k, do[1], ws[1])):
            keep = pos >= 0
            dx, dw = gradients(x[keep], pos[keep], freqs, weight, 1e-6, norm > 0, pairs, d[keep])
            tol_x, tol_w = grad_bounds(x[keep], pos[keep], freqs, weight, 1e-6, norm > 0, pairs, d[keep])
            err = (got["d" + name][keep.cuda()].double().cpu() - dx).abs() - tol_x
            assert err.max() <= 0, f"d{name} off its bound by {err.max():.3e}"
            if weight is None:
                assert got[f"d{name}_weight"] is None
            else:
                err = (got[f"d{name}_weight"].double().cpu() - dw).abs() - tol_w
                assert err.max() <= 0, f"d{name}_weight off its bound by {err.max():.3e}"


def test_backward_without_eps():
    """eps = 0: rows beside the last head, which are nobody's, have no say in the weights' gradients."""
    kda = _kda()
    for H, Hkv, D in ((3, 1, 128), (5, 2, 64)):
        q, k, dq, dk, pos, w = _case(3, H, Hkv, D, seed=8)
        freqs = freqs_of(D)
        g = torch.Generator().manual_seed(4)
        do = [torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in (q, k)]
        args = (pos.cuda(), freqs.cuda())
        got = kda.kda_qk_norm_rope_bwd(dq, dk, *args, do[0].cuda(), do[1].cuda(), w[0].cuda(), w[1].cuda(), eps=0.0)
        for name, x, d, weight in (("q", q[:2], do[0][:2], w[0]), ("k", k[:2], do[1][:2], w[1])):
            dx, _ = gradients(x, pos[:2], freqs, weight, 0.0, True, False, d)
            tol, _ = grad_bounds(x, pos[:2], freqs, weight, 0.0, True, False, d)
            assert ((got["d" + name][:2].double().cpu() - dx).abs() - tol).max() <= 0
        assert torch.isfinite(got["dq_weight"]).all() and torch.isfinite(got["dk_weight"]).all()
        qo, _ = kda.kda_qk_norm_rope(dq, dk, *args, w[0].cuda(), w[1].cuda(), eps=0.0)
        assert torch.isfinite(qo).all()


def test_backward_sizes_and_bits():
    kda = _kda()
    for T, H, Hkv, D in ((3000, 8, 2, 128), (2001, 6, 3, 64), (1, 33, 1, 128)):
        q, k, dq, dk, pos, w = _case(T, H, Hkv, D, seed=T, fused=True)
        freqs = freqs_of(D)
        g = torch.Generator().manual_seed(T + 1)
        do = [torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in (q, k)]
        args = (dq, dk, pos.cuda(), freqs.cuda(), do[0].cuda(), do[1].cuda(), w[0].cuda(), w[1].cuda())
        got = kda.kda_qk_norm_rope_bwd(*args)
        for name, x, d, weight in (("q", q, do[0], w[0]), ("k", k, do[1], w[1])):
            dx, dw = gradients(x, pos, freqs, weight, 1e-6, True, False, d)
            tol_x, tol_w = grad_bounds(x, pos, freqs, weight, 1e-6, True, False, d)
            assert ((got["d" + name].double().cpu() - dx).abs() - tol_x).max() <= 0
            assert ((got[f"d{name}_weight"].double().cpu() - dw).abs() - tol_w).max() <= 0
        again = kda.kda_qk_norm_rope_bwd(*args)
        assert all(torch.equal(got[n], again[n]) for n in got)
        one = kda.kda_qk_norm_rope_bwd(*args[:6], None, w[1].cuda())
        assert one["dq_weight"] is None and torch.equal(one["dk_weight"], got["dk_weight"])


def test_streams_and_graphs():
    kda = _kda()
    q, k, dq, dk, pos, w = _case(30, 8, 2, 128)
    freqs, p = freqs_of(128).cuda(), pos.cuda()
    args = (dq, dk, p, freqs)
    ws = (w[0].cuda(), w[1].cuda())
    do = [torch.randn_like(x) for x in (dq, dk)]
    want, wantk = kda.kda_qk_norm_rope(*args, *ws)
    grads = kda.kda_qk_norm_rope_bwd(*args, *do, *ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, _ = kda.kda_qk_norm_rope(*args, *ws, stream=side)
    b = kda.kda_qk_norm_rope_bwd(*args, *do, *ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and all(torch.equal(b[n], grads[n]) for n in b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, ok = kda.kda_qk_norm_rope(*args, *ws)
        b = kda.kda_qk_norm_rope_bwd(*args, *do, *ws)
    p.add_(5)
    g.replay()
    torch.cuda.synchronize()
    _check(o, q, pos + 5, freqs.cpu(), w[0], 1e-6, True, False)
    eager = kda.kda_qk_norm_rope_bwd(*args, *do, *ws)
    assert all(torch.equal(b[n], eager[n]) for n in b)


def test_feeds_store_and_attention():
    """Projection slices through norm and rotation into the cache and attention, at the plan's positions: only the
    differences of positions matter, so the same tokens further on give the same answer within the roundings."""
    kda = _kda()
    D, H, Hkv = 128, 4, 2
    g = torch.Generator().manual_seed(1)
    f = torch.randn((40, H + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for cached in (0, 1600):
        q, k, v = f.split([H, Hkv, Hkv], 1)
        pos = torch.arange(40, dtype=torch.int32, device="cuda") + cached
        q, k = kda.kda_qk_norm_rope(q, k, pos, freqs_of(D).cuda(), torch.full((D,), 0.25, device="cuda"))
        outs.append(kda.kda_attn_fwd(q[None], k[None], v[None].contiguous(), D ** -0.5)[0].double())
    # |q| <= sqrt(D) / 4 and |k| <= sqrt(D), each channel off by 2^-8 at both places: a score is off by
    # 4 2^-8 sqrt(D) / 4 = 2^-8 11.4 at most, the weights by a factor e^(2 x that), the outputs' own rounding is 2 x 2^-8
    bound = (math.exp(2 * 2.0 ** -8 * 11.4) - 1 + 4 * 2.0 ** -8) * f[:, H + Hkv:].double().abs().max()
    assert (outs[0] - outs[1]).abs().max() <= bound


def test_tokens_past_32_bits_of_elements():
    """Rows past 2^31 elements of the inputs and outputs, and stored from there: the same bits as alone."""
    kda = _kda()
    H, Hkv, D = 32, 8, 128
    T = 2 ** 31 // (H * D) + 3000
    x = torch.zeros((T, H + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    n = 2900
    x[-n:] = torch.randn((n, H + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([H, Hkv, Hkv], 1)
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[-n:] = torch.arange(n, dtype=torch.int32, device="cuda") + 7
    freqs, w = torch.rand(32, generator=g, device="cuda"), torch.rand(128, generator=g, device="cuda")
    assert q.stride(0) * (T - n) >= 2 ** 31 and H * D * (T - n) >= 2 ** 31
    oq, ok = kda.kda_qk_norm_rope(q, k, pos, freqs, w, w)
    aq, ak = kda.kda_qk_norm_rope(q[-n:], k[-n:], pos[-n:], freqs, w, w)
    assert torch.equal(oq[-n:], aq) and torch.equal(ok[-n:], ak)
    far = kda.kda_qk_norm_rope_bwd(q, k, pos, freqs, oq, ok, w, w)
    near = kda.kda_qk_norm_rope_bwd(q[-n:], k[-n:], pos[-n:], freqs, aq, ak, w, w)
    assert torch.equal(far["dq"][-n:], near["dq"]) and torch.equal(far["dk"][-n:], near["dk"])
    for name, heads in (("dq_weight", H), ("dk_weight", Hkv)):
        # sums in other orders, each a chain of at most 200 additions of 2^-24, of terms whose absolute values add to at
        # most 128 for each of n heads rows (two rows' norms, sqrt(128) at most)
        assert (far[name] - near[name]).abs().max() <= 2 * 200 * 2.0 ** -24 * 128 * n * heads
    caches = [torch.zeros((64, Hkv, 64, kda.q4_row_bytes(D)), dtype=torch.uint8, device="cuda") for _ in range(4)]
    kda.kda_kv_write_q4(ok, v, pos, *caches[:2])
    kda.kda_kv_write_q4(ak, v[-n:], pos[-n:], *caches[2:])
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3]) and caches[0].any()


def test_streams_at_once():
    kda = _kda()
    g = torch.Generator(device="cuda").manual_seed(1)
    freqs, w = torch.rand(32, generator=g, device="cuda"), torch.rand(128, generator=g, device="cuda")
    args = []
    for T in (3000, 777):
        x = torch.randn((T, 24, 128), generator=g, device="cuda").to(torch.bfloat16)
        q, k, _ = x.split([16, 4, 4], 1)
        args.append((q, k, torch.arange(T, dtype=torch.int32, device="cuda"), freqs, q.contiguous(), k.contiguous(), w, w))
    want = [kda.kda_qk_norm_rope_bwd(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[kda.kda_qk_norm_rope_bwd(*a, stream=s) for a, s in zip(args, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(a[name], b[name]) for name in b)
