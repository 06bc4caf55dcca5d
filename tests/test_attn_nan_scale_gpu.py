"""GPU tests of softmax attention under a scale that is NaN: every row that sees a key is NaN, as the formula gives,
and is not hidden behind finite values; a row without keys is 0 and -infinity whatever the scale."""
import math

import pytest
import torch

from attn_testutil import Paged, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


@pytest.mark.parametrize("scale", [math.nan, -math.nan])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 2, 1, 64), (200, 4, 2, 128), (900, 8, 1, 64), (900, 8, 1, 128)])
def test_prompt(T, Hq, Hkv, D, scale):
    from gated_delta_rule_40_gb300 import kda
    g = torch.Generator().manual_seed(T)
    q, k, v = normal(g, 1, T, Hq, D), normal(g, 1, T, Hkv, D), normal(g, 1, T, Hkv, D)
    out, lse = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale)
    assert torch.isnan(out.float()).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("D", [64, 128])
def test_pages_split_units_and_rows_without_keys(D):
    c = Paged([9000, 40, -3, -200], [1, 2, 10, 300], 4, 2, D, 32, seed=D)
    c.scale = math.nan
    out, lse = c.run()
    none = torch.zeros(c.cu[-1], dtype=torch.bool, device="cuda")
    none[3:6] = True
    none[13:213] = True
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    assert torch.isnan(out[~none].float()).all() and torch.isnan(lse[~none]).all()
