"""GPU tests of outputs that a call makes for a stream of the caller's: not memory that the current stream still
uses, nor memory that the named stream reuses before the current one has read it."""
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


def _call(stream):
    from gated_delta_rule_40_gb300 import kda
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((1, 3000, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
    torch.cuda.synchronize()
    return lambda: kda.kda_attn_fwd(q, k, v, 0.1, stream=stream)


def test_attention():
    side = torch.cuda.Stream()
    want, want_lse = _call(None)()
    call = _call(side)
    old = torch.empty_like(want), torch.empty_like(want_lse)
    freed = {t.data_ptr() for t in old}
    torch.cuda.synchronize()
    del old                                       # the next allocation of the current stream would take these
    out, lse = call()
    assert not freed & {out.data_ptr(), lse.data_ptr()}
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    torch.cuda._sleep(1 << 28)                    # the current stream is busy when the output is released
    at = out.data_ptr()
    del out
    out, _ = call()
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_page_plan():
    from gated_delta_rule_40_gb300 import kda
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = dev([0, 3]), dev([20, 14]), dev([5, 3, 1, 7]), dev([0])
    tables = [dev([[-1, -1], [9, -1]]) for _ in range(2)]
    want = kda.kda_page_plan(*args, tables[0], 16, 34)
    side = torch.cuda.Stream()
    old = [torch.empty_like(t) for t in want]
    freed = {t.data_ptr() for t in old}
    torch.cuda.synchronize()
    del old
    got = kda.kda_page_plan(*args, tables[1], 16, 34, stream=side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(*tables)
