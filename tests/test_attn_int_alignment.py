"""CPU test that the softmax-attention entries refuse an int32 array that does not start on 4 bytes, which a kernel
could not load.  Pointers are stand-ins: the checks answer before any device call."""
import ctypes

import pytest
import torch

from gated_delta_rule_40_gb300 import kda

if torch.cuda.is_available():
    pytest.skip("stand-in pointers stay off a GPU", allow_module_level=True)

GOOD, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100002)
F = ctypes.c_float(0.1)


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def _plan(lib, **kw):
    p = dict.fromkeys(("cached", "new", "free", "start", "table", "cu", "lens", "slots", "pos", "next"), GOOD)
    p.update(kw)
    return lib.kda_page_plan(p["cached"], p["new"], p["free"], p["start"], p["table"], 1, 4, 4, 16, 4, p["cu"],
                             p["lens"], p["slots"], p["pos"], p["next"], None)


def _paged(lib, **kw):
    p = dict.fromkeys(("table", "lens", "cu"), GOOD)
    p.update(kw)
    return lib.kda_attn_paged(GOOD, GOOD, GOOD, F, p["table"], p["lens"], p["cu"], 1, 4, 2, 1, 128, 4, 16, 4, GOOD, None,
                              None)


def _prompt(lib, cu):
    return lib.kda_attn_fwd(GOOD, GOOD, GOOD, F, cu, 1, 1, 4, 2, 1, 128, GOOD, None, None)


def _write(lib, slots):
    return lib.kda_kv_write(GOOD, GOOD, slots, GOOD, GOOD, 4, 2, 128, 4, 16, None)


@pytest.mark.parametrize("name", ["cached", "new", "free", "start", "table", "cu", "lens", "slots", "pos", "next"])
def test_page_plan(lib, name):
    assert _plan(lib, **{name: ODD}) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["table", "lens", "cu"])
def test_paged(lib, name):
    assert _paged(lib, **{name: ODD}) == kda.KDA_ERR_INVALID_ARG


def test_prompt_and_write(lib):
    assert _prompt(lib, ODD) == kda.KDA_ERR_INVALID_ARG and _write(lib, ODD) == kda.KDA_ERR_INVALID_ARG


def test_aligned_arrays_pass_the_checks(lib):
    """Without a device the launch itself fails, after every check."""
    assert {_plan(lib), _paged(lib), _prompt(lib, GOOD), _write(lib, GOOD)} == {kda.KDA_ERR_CUDA}
