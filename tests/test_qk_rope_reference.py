"""CPU tests of the 64-bit reference of the query/key norms with rotation: its gradients are those of the formula
and of differences."""
import pytest
import torch

from qk_rope_testutil import angles, freqs_of, gradients, normed, reference, turned


def _case(D, rot):
    g = torch.Generator().manual_seed(D + rot)
    x = torch.randn((5, 3, D), generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(D, generator=g, dtype=torch.float64)
    d = torch.randn((5, 3, D), generator=g, dtype=torch.float64)
    return x, torch.tensor([0, 1, 50, 999, 4000], dtype=torch.int32), freqs_of(rot), w, d


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 24), (128, 0)])
def test_formula(D, rot, pairs):
    x, pos, freqs, w, d = _case(D, rot)
    dx, dw = gradients(x, pos, freqs, w, 1e-6, True, pairs, d)
    g, _ = turned(d, angles(pos, freqs), pairs, -1.0)
    y, r = normed(x, None, 1e-6, True)
    assert torch.allclose(dw, (g * y).sum((0, 1)), rtol=1e-12, atol=1e-12)
    gw = g * w
    assert torch.allclose(dx, r * (gw - y * (gw * y).mean(-1, keepdim=True)), rtol=1e-12, atol=1e-12)


def test_differences():
    x, pos, freqs, w, d = _case(64, 32)
    dx, dw = gradients(x, pos, freqs, w, 1e-6, True, False, d)
    loss = lambda a, b: (reference(a, pos, freqs, b, 1e-6, True, False)[0] * d).sum()  # noqa: E731
    h = 1e-5   # central differences: h^2 times a third derivative of order 1, and 2^-52 / h
    for at in ((0, 0, 0), (3, 2, 17), (4, 1, 63)):
        e = torch.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for c in (0, 20, 63):
        e = torch.zeros_like(w)
        e[c] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-7


def test_reduced_angles_are_the_angles():
    pos, freqs = torch.tensor([4097, 100000], dtype=torch.int32), freqs_of(64)
    a = angles(pos, freqs)
    plain = pos.double()[:, None] * freqs.double()
    assert torch.allclose(torch.cos(a), torch.cos(plain), atol=1e-9) and a.abs().max() <= 3.15
