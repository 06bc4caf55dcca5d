"""GPU tests of the query/key norms with rotation: the workspace's size, whatever the device's number of SMs, the angles
by themselves, rows whose mean square has no fp32 number, and sums of weights' gradients past 2^31 elements."""
from fractions import Fraction

import pytest
import torch

from qk_rope_testutil import _PI as PI
from qk_rope_testutil import angles, freqs_of, grad_bounds, gradients, normed, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 700, 6000])
def test_the_workspace_holds_what_is_written(T, D):
    """Enough tokens for a CTA on every place of the device: nothing behind the stated size is touched."""
    from gated_delta_rule_40_gb300 import kda
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = kda.kda_qk_norm_rope_bwd_workspace_size(D)
    assert size >= 4 * 2 * D * sms   # a partial sum of both weights for each CTA, one an SM at least
    g = torch.Generator().manual_seed(T)
    q, k, dq, dk = (torch.randn((T, h, D), generator=g).to(torch.bfloat16) for h in (4, 2, 4, 2))
    w, pos, freqs = 1.0 + 0.3 * torch.randn((2, D), generator=g), torch.arange(T, dtype=torch.int32), freqs_of(D)
    ws = torch.full((size + 8192,), 0xab, dtype=torch.uint8, device="cuda")
    args = [x.cuda() for x in (q, k, pos, freqs, dq, dk, w[0], w[1])]
    got = kda.kda_qk_norm_rope_bwd(*args, workspace=ws[:size])
    assert (ws[size:] == 0xab).all()
    pooled = kda.kda_qk_norm_rope_bwd(*args)
    assert all(torch.equal(got[n], pooled[n]) for n in got)
    for name, x, d, weight in (("dq_weight", q, dq, w[0]), ("dk_weight", k, dk, w[1])):
        _, dw = gradients(x, pos, freqs, weight, 1e-6, True, False, d)
        _, tol = grad_bounds(x, pos, freqs, weight, 1e-6, True, False, d)
        assert ((got[name].double().cpu() - dw).abs() - tol).max() <= 0


@pytest.mark.parametrize("far", [1, 4000, 1 << 24, (1 << 31) - 1])
def test_angles(far):
    """cos and sin of the angles themselves: the gradients of (1, 0) pairs, which are fp32.  The fraction of a turn is
    rounded to fp32 once, 2^-26 of a turn at most beside the 2^-33 of its own, and the function is off by 2^-24 (an
    ulp) of at most 1, with room for another."""
    from gated_delta_rule_40_gb300 import kda
    g = torch.Generator().manual_seed(far & 1023)
    pos = torch.randint(0, far + 1, (300,), generator=g).to(torch.int32)
    pos[0] = far
    freqs = freqs_of(128)
    freqs[:6] = torch.tensor([3.0, 6.2831855, 100.25, -0.7, 1e-6, 1e7])
    x = torch.zeros((300, 1, 128), dtype=torch.bfloat16, device="cuda")
    x[..., :64] = 1.0
    got = kda.kda_qk_norm_rope_bwd(x, x, pos.cuda(), freqs.cuda(), x, x, norm=False)["dq"][:, 0].double().cpu()
    turn = 2 * PI
    ang = torch.empty((300, 64), dtype=torch.float64)   # reduced in exact arithmetic, near positions too
    for j, f in enumerate(Fraction(float(f)) for f in freqs):
        for i, p in enumerate(pos.tolist()):
            a = p * f
            ang[i, j] = float(a - turn * round(a / turn))
    bound = 2 * 3.1416 * (2.0 ** -26 + 2.0 ** -33) + 2.0 ** -23
    assert (got[:, :64] - torch.cos(ang)).abs().max() <= bound
    assert (got[:, 64:] + torch.sin(ang)).abs().max() <= bound


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pairs", [False, True])
def test_rows_out_of_the_range_of_their_mean_square(D, pairs):
    """Squares are summed in fp32: rows whose sum is above its range become zeros, with gradients of 0, and without eps a
    row of zeros is 0 / 0.  Other rows are as they are alone."""
    from gated_delta_rule_40_gb300 import kda
    g = torch.Generator().manual_seed(D)
    q, k, dq, dk = (torch.randn((6, h, D), generator=g).to(torch.bfloat16) for h in (4, 2, 4, 2))
    w, pos, freqs = 1.0 + 0.3 * torch.randn((2, D), generator=g), torch.arange(6, dtype=torch.int32) + 50, freqs_of(D)
    args = [x.cuda() for x in (pos, freqs, dq, dk, w[0], w[1])]
    run = lambda q, **kw: (*kda.kda_qk_norm_rope(q, k.cuda(), *args[:2], *args[4:], interleaved=pairs, **kw),  # noqa: E731
                           kda.kda_qk_norm_rope_bwd(q, k.cuda(), *args, interleaved=pairs, **kw))
    keep, keepk, grads = run(q.cuda())
    big = q.clone()
    big[2, 1] *= 2.0 ** 70   # the squares' sum is 2^140 or more
    big[4, 3] *= 2.0 ** 50   # 2^107: within the range
    out, outk, got = run(big.cuda())
    assert not out[2, 1].any() and not got["dq"][2, 1].any()
    same = torch.ones((6, 4), dtype=torch.bool)
    same[2, 1] = same[4, 3] = False
    assert torch.equal(out.cpu()[same], keep.cpu()[same]) and torch.equal(got["dq"].cpu()[same], grads["dq"].cpu()[same])
    assert torch.equal(outk, keepk) and torch.equal(got["dk"], grads["dk"]) and torch.equal(got["dk_weight"], grads["dk_weight"])
    # (eps, 1e-6 of a mean square of 1, is 2^-21 of the root)
    off = (out[4, 3].double() - keep[4, 3].double()).abs().cpu()
    assert (off <= 2.0 ** -8 * 2 * keep[4, 3].double().abs().cpu() + 2.0 ** -18 * 4).all()
    assert torch.isfinite(got["dq_weight"]).all()
    big[2, 1] = 0
    out, _, got = run(big.cuda(), eps=0.0)
    assert torch.isnan(out[2, 1]).all() and torch.isnan(got["dq"][2, 1]).all()
    assert torch.isfinite(out.cpu()[same]).all() and torch.isfinite(got["dq"].cpu()[same]).all()


def test_weight_gradients_past_32_bits_of_elements():
    """The weights' gradients of rows past 2^31 elements against sums in 64 bits; a single token less shows."""
    from gated_delta_rule_40_gb300 import kda
    H, Hkv, D, n = 32, 8, 128, 2900
    T = 2 ** 31 // (H * D) + 3000
    x = torch.zeros((T, H + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    x[-n:] = torch.randn((n, H + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, _ = x.split([H, Hkv, Hkv], 1)
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[-n:] = torch.arange(n, dtype=torch.int32, device="cuda") + 7
    freqs, w = torch.rand(32, generator=g, device="cuda"), torch.rand(128, generator=g, device="cuda")
    dq = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    dk = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
    dq[-n:] = torch.randn((n, H, D), generator=g, device="cuda").to(torch.bfloat16)
    dk[-n:] = torch.randn((n, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    assert H * D * (T - n) >= 2 ** 31
    far = kda.kda_qk_norm_rope_bwd(q, k, pos, freqs, dq, dk, w, w)
    near = kda.kda_qk_norm_rope_bwd(q[-n:], k[-n:], pos[-n:], freqs, dq[-n:], dk[-n:], w, w)
    for name, xs, ds in (("dq_weight", q, dq), ("dk_weight", k, dk)):
        args = [xs[-n:].cpu(), pos[-n:].cpu(), freqs.cpu()]
        d = ds[-n:].cpu()
        back, _ = turned(d.double(), angles(args[1], args[2]), False, -1.0)
        terms = (back * normed(args[0], None, 1e-6, True)[0]).sum(1)   # of each token
        _, tol = grad_bounds(*args, w.cpu(), 1e-6, True, False, d)
        for got in (far, near):
            assert ((got[name].double().cpu() - terms.sum(0)).abs() - tol).max() <= 0
        # any one token left out would show in some channel
        assert ((terms.abs() - 2 * tol).amax(1) > 0).all()
