"""GPU tests of a free_start outside the list in kda_page_plan: no block is handed out and the place does not move.
Whole numbers, so every comparison is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LIST = [4, 5, 6, 7]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


def _plan(cached, new, start, table, T, free=LIST):
    from gated_delta_rule_40_gb300 import kda
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tab = dev(table)
    p = kda.kda_page_plan(dev(cached), dev(new), dev(free), dev([start]), tab, 16, T)
    return kda.kda_get_status(), p.cu_seqlens.tolist(), p.slots.tolist(), p.free_next.item(), tab.tolist()


@pytest.mark.parametrize("start", [-1, -(1 << 31), len(LIST) + 1, 0x7fffffff])
def test_a_place_outside_the_list_hands_out_nothing(start):
    from gated_delta_rule_40_gb300 import kda
    # request 0 still has room in its own block; request 1 needs two new ones, over entries of old ids
    status, cu, slots, nxt, table = _plan([14, 0], [2, 20], start, [[9, -1], [3, 2]], 24)
    assert status == kda.KDA_ERR_NO_BLOCKS
    assert cu == [0, 2, 22] and slots == [9 * 16 + 14, 9 * 16 + 15] + [-1] * 22
    assert nxt == start and table == [[9, -1], [-1, -1]]
    # reported when nothing is needed, too
    status, _, slots, nxt, table = _plan([14], [1], start, [[9, 8]], 1)
    assert status == kda.KDA_ERR_NO_BLOCKS and slots == [9 * 16 + 14] and nxt == start and table == [[9, 8]]


def test_the_ends_of_the_list_are_places_in_it():
    from gated_delta_rule_40_gb300 import kda
    assert _plan([14], [1], len(LIST), [[9, 8]], 1)[::3] == (kda.KDA_OK, len(LIST))
    assert _plan([0], [1], len(LIST) - 1, [[9, 8]], 1)[2:] == ([7 * 16], len(LIST), [[7, 8]])
    assert _plan([14], [1], 0, [[9, 8]], 1, free=[])[::3] == (kda.KDA_OK, 0)
    assert _plan([0], [0], 0, [[9, 8]], 0)[::3] == (kda.KDA_OK, 0)
