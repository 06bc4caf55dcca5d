"""GPU tests of the query/key norms with rotation: the workspace's size, whatever the device's number of SMs."""
import pytest
import torch

from qk_rope_testutil import freqs_of, grad_bounds, gradients

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
