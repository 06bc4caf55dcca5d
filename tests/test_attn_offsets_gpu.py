"""GPU tests of packed offsets that fall by more than 2^31, so that their difference in 32 bits is a length like any
other: reported, and nothing written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
# the last of each looks like a short request that begins before the tensor
OFFSETS = [[0, BIG, -2, 5], [0, BIG, -BIG - 1, 0, 5], [0, 2, BIG, -9, -8, 5], [0] * 400 + [BIG, -3, 4]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


@pytest.mark.parametrize("offsets", OFFSETS, ids=range(len(OFFSETS)))
@pytest.mark.parametrize("D,H,Hkv", [(128, 4, 4), (128, 32, 2), (64, 8, 1), (64, 40, 1)])
@pytest.mark.parametrize("q4", [True, False])
def test_offsets_that_fall_by_more_than_half_the_range(q4, D, H, Hkv, offsets):
    from gated_delta_rule_40_gb300 import kda
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    N, T, bs = len(offsets) - 1, 6, 16
    row, dtype = (kda.q4_row_bytes(D), torch.uint8) if q4 else (D, torch.bfloat16)
    cache = [torch.zeros((4, Hkv, bs, row), dtype=dtype, device="cuda") for _ in range(2)]
    q = torch.ones((T, H, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((T, H), 7.0, device="cuda")
    call = kda.kda_attn_paged_q4 if q4 else kda.kda_attn_paged
    call(q, *cache, ints([[0, 1, 2]] * N), ints([20] * N), ints(offsets), 0.1, out=out, lse=lse)
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_SEQLENS
    assert (out == 7).all() and (lse == 7).all()
