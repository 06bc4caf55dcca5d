"""CPU tests of the softmax-attention operators' refusals: every argument check answers before any device
call.  Data pointers are NULL, or a stand-in address where there is no device (see test_abi.py)."""
import ctypes

import pytest
import torch

from gated_delta_rule_40_gb300 import kda

HAS_GPU = torch.cuda.is_available()
_BUF = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") if HAS_GPU else None
FAKE = ctypes.c_void_p(_BUF.data_ptr() if HAS_GPU else 0x100000)
ODD = ctypes.c_void_p(FAKE.value + 2)
F = ctypes.c_float(0.1)
BAD, UNSUP, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def test_status_strings():
    for code in (kda.KDA_ERR_NO_BLOCKS, kda.KDA_ERR_BAD_PAGES):
        assert kda.status_string(code) != "unknown status"


def test_attn_fwd_refusals(lib):
    def fwd(q=None, cu=None, N=0, B=1, T=4, Hq=2, Hkv=1, D=128, out=None, lse=None):
        return lib.kda_attn_fwd(q, q, q, F, cu, N, B, T, Hq, Hkv, D, out, lse, None)
    assert fwd(D=96) == UNSUP and fwd(D=256) == UNSUP
    assert fwd(Hq=3, Hkv=2) == BAD and fwd(Hq=0) == BAD and fwd(Hkv=0) == BAD and fwd(Hq=129, Hkv=1) == BAD
    assert fwd(T=-1) == BAD and fwd(B=-1) == BAD and fwd(N=-1, cu=FAKE, T=0) == BAD
    assert fwd(B=2, N=1, T=0, cu=FAKE) == BAD
    assert fwd() == BAD                                    # NULL tensors
    assert fwd(B=1 << 20, T=1 << 12) == BAD                # rows past 32 bits
    assert fwd(T=0) == OK and fwd(B=0) == OK
    if not HAS_GPU:
        assert fwd(q=ODD, out=FAKE) == BAD and fwd(q=FAKE, out=ODD) == BAD and fwd(q=FAKE, out=FAKE, lse=ODD) == BAD


def test_attn_paged_refusals(lib):
    def paged(q=None, cache=None, table=None, lens=None, cu=None, N=1, T=4, Hq=2, Hkv=1, D=128, nb=4, bs=16, mb=4,
              out=None):
        return lib.kda_attn_paged(q, cache, cache, F, table, lens, cu, N, T, Hq, Hkv, D, nb, bs, mb, out, None, None)
    for bs in (0, 1, 8, 24, 2048, -16):
        assert paged(bs=bs) == UNSUP
    assert paged(D=80) == UNSUP
    assert paged(Hq=3, Hkv=2) == BAD and paged(Hq=130, Hkv=1) == BAD
    assert paged(N=-1) == BAD and paged(T=-1) == BAD and paged(nb=-1, T=0) == BAD and paged(mb=-1, T=0) == BAD
    assert paged(nb=1 << 28, T=0) == BAD                   # slots past 32 bits
    assert paged() == BAD
    assert paged(T=0) == OK and paged(N=0, T=0) == OK
    if not HAS_GPU:
        full = dict(q=FAKE, cache=FAKE, out=FAKE, table=FAKE, lens=FAKE, cu=FAKE)
        for name in ("q", "cache", "out", "table", "lens", "cu"):
            assert paged(**{**full, name: None}) == BAD, name
        for name in ("q", "cache", "out"):
            assert paged(**{**full, name: ODD}) == BAD, name


def test_page_plan_refusals(lib):
    def plan(N=1, T=4, mb=4, bs=16, nf=4, **kw):
        p = dict.fromkeys(("cached", "new", "free", "start", "table", "cu", "lens", "slots", "pos", "next"), FAKE)
        p.update(kw)
        return lib.kda_page_plan(p["cached"], p["new"], p["free"], p["start"], p["table"], N, T, mb, bs, nf, p["cu"],
                                 p["lens"], p["slots"], p["pos"], p["next"], None)
    assert plan(bs=8) == UNSUP and plan(bs=48) == UNSUP
    for bad in (dict(N=-1), dict(T=-1), dict(mb=-1), dict(nf=-1)):
        assert plan(**bad) == BAD
    for name in ("cached", "new", "free", "start", "table", "cu", "lens", "slots", "pos", "next"):
        assert plan(**{name: None}) == BAD, name


def test_kv_write_refusals(lib):
    def write(p=None, slots=None, cache=None, T=4, H=2, D=128, nb=4, bs=16):
        return lib.kda_kv_write(p, p, slots, cache, cache, T, H, D, nb, bs, None)
    assert write(D=32) == UNSUP and write(bs=20) == UNSUP
    assert write(T=-1) == BAD and write(H=0) == BAD and write(nb=1 << 28) == BAD and write(nb=-1) == BAD
    assert write() == BAD
    assert write(T=0) == OK
    if not HAS_GPU:
        assert write(p=ODD, slots=FAKE, cache=FAKE) == BAD and write(p=FAKE, slots=FAKE, cache=ODD) == BAD


def test_binding_refusals():
    """The binding's own checks (host tensors stand for everything that is not on the device)."""
    bf = torch.bfloat16
    q = torch.zeros((1, 4, 2, 128), dtype=bf)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_attn_fwd(q, q, q, 1.0)
    with pytest.raises(TypeError):
        kda.kda_attn_fwd(q.float(), q, q, 1.0)
    c = torch.zeros((2, 1, 16, 128), dtype=bf)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_attn_paged(q[0], c, c, i[None], i, torch.zeros(2, dtype=torch.int32), 1.0)
    with pytest.raises(TypeError):
        kda.kda_kv_write(q[0].float(), q[0], i, c, c)
    with pytest.raises(TypeError):
        kda.kda_page_plan(i.long(), i, i, i, i[None], 16, 4)
