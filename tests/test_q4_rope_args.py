"""CPU tests of the refusals of the 4-bit cache's calls and of the query/key norms with rotation: every argument
check answers before any device call.  Data pointers are NULL, or a stand-in address where there is no device (see
test_abi.py)."""
import ctypes

import pytest
import torch

from gated_delta_rule_40_gb300 import kda

HAS_GPU = torch.cuda.is_available()
_BUF = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") if HAS_GPU else None
FAKE = ctypes.c_void_p(_BUF.data_ptr() if HAS_GPU else 0x100000)
ODD = ctypes.c_void_p(FAKE.value + 2)
F = ctypes.c_float(0.1)
BAD, UNSUP, OK, WS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK, kda.KDA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def _rope(lib, bwd=False, x=None, stride=None, w=None, eps=1e-6, norm=1, freqs=FAKE, rot=8, pos=FAKE, T=4, Hq=2, Hk=1,
          D=128, out=None, dw=None, **kw):
    p = dict(q=x, k=x, sq=Hq * D if stride is None else stride, sk=Hk * D if stride is None else stride)
    p.update(kw)
    args = [p["q"], p["k"], p["sq"], p["sk"], w, w, ctypes.c_float(eps), norm, freqs, rot, 0, pos, T, Hq, Hk, D]
    if not bwd:
        return lib.kda_qk_norm_rope(*args, out, out, None)
    return lib.kda_qk_norm_rope_bwd_ws(*args, p.get("d", x), p.get("d", x), out, out, dw, dw, p.get("ws"),
                                       p.get("size", 0), None)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(lib, bwd):
    for bad in (dict(D=96), dict(D=256), dict(rot=4), dict(rot=-8), dict(rot=136), dict(rot=72, D=64)):
        assert _rope(lib, bwd, **bad) == UNSUP, bad
    for bad in (dict(T=-1), dict(Hq=0), dict(Hk=0), dict(Hq=-2), dict(Hk=65537), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(norm=0, w=FAKE), dict(w=ODD), dict(freqs=ODD), dict(pos=ODD), dict(pos=None), dict(freqs=None),
                dict(dw=FAKE, norm=0, bwd=True), dict()):
        if bad.get("bwd", bwd) != bwd:
            continue
        assert _rope(lib, **{"bwd": bwd, **bad}) == BAD, bad      # (the last: NULL tensors)
    assert _rope(lib, bwd, T=0) == OK and _rope(lib, bwd, T=0, freqs=None, rot=0, pos=None) == OK
    if not HAS_GPU:
        full = dict(x=FAKE, out=FAKE)
        for bad in (dict(x=ODD), dict(out=ODD), dict(sq=255), dict(sq=248), dict(sk=127), dict(sk=132), dict(q=None),
                    dict(k=None), dict(out=None), dict(sq=-256)):
            assert _rope(lib, bwd, **{**full, **bad}) == BAD, bad
    if bwd and not HAS_GPU:
        assert _rope(lib, True, x=FAKE, out=FAKE, d=None) == BAD and _rope(lib, True, x=FAKE, out=FAKE, d=ODD) == BAD
        assert _rope(lib, True, x=FAKE, out=FAKE, dw=FAKE) == WS
        size = kda.kda_qk_norm_rope_bwd_workspace_size(128)
        assert _rope(lib, True, x=FAKE, out=FAKE, dw=FAKE, ws=FAKE, size=size - 1) == WS
        assert _rope(lib, True, x=FAKE, out=FAKE, dw=FAKE, ws=ctypes.c_void_p(FAKE.value + 128), size=size) == WS
        assert _rope(lib, True, x=FAKE, out=FAKE, dw=ODD, ws=FAKE, size=size) == BAD
    assert kda.kda_qk_norm_rope_bwd_workspace_size(96) == 0


def test_store_and_read_refusals(lib):
    def write(p=None, slots=FAKE, cache=None, T=4, H=2, D=128, nb=4, bs=16, stride=256):
        return lib.kda_kv_write_q4(p, p, stride, stride, slots, cache, cache, T, H, D, nb, bs, None)

    def read(p=None, slots=FAKE, cache=None, T=4, H=2, D=128, nb=4, bs=16):
        return lib.kda_kv_read_q4(cache, cache, slots, p, p, T, H, D, nb, bs, None)
    for call in (write, read):
        for bad in (dict(D=32), dict(D=256), dict(bs=8), dict(bs=20), dict(bs=2048)):
            assert call(**bad) == UNSUP, bad
        for bad in (dict(T=-1), dict(H=0), dict(H=65537), dict(nb=-1), dict(nb=1 << 28), dict(slots=None),
                    dict(), dict(T=2 ** 31 - 1, H=65536)):
            assert call(**bad) == BAD, bad
        assert call(T=0) == OK and call(T=0, slots=None) == OK
        if not HAS_GPU:
            full = dict(p=FAKE, cache=FAKE)
            for bad in (dict(p=ODD), dict(cache=ODD), dict(slots=ODD), dict(p=None), dict(cache=None)):
                assert call(**{**full, **bad}) == BAD, bad
    if not HAS_GPU:
        for stride in (248, 260, -256):
            assert write(p=FAKE, cache=FAKE, stride=stride) == BAD


def test_attn_q4_refusals(lib):
    def paged(q=None, cache=None, table=None, lens=None, cu=None, N=1, T=4, Hq=2, Hkv=1, D=128, nb=4, bs=16, mb=4,
              out=None, lse=None, ws=None, size=None):
        args = (q, cache, cache, F, table, lens, cu, N, T, Hq, Hkv, D, nb, bs, mb, out, lse)
        if size is not None:
            return lib.kda_attn_paged_q4_ws(*args, ws, size, None)
        return lib.kda_attn_paged_q4(*args, None)
    for bs in (0, 1, 8, 24, 2048, -16):
        assert paged(bs=bs) == UNSUP
    assert paged(D=80) == UNSUP and paged(D=256) == UNSUP
    for bad in (dict(Hq=3, Hkv=2), dict(Hq=130), dict(Hq=0), dict(Hkv=0), dict(N=-1), dict(T=-1), dict(nb=-1, T=0),
                dict(mb=-1, T=0), dict(nb=1 << 28, T=0), dict(), dict(T=1 << 30)):
        assert paged(**bad) == BAD, bad
    assert paged(T=0) == OK and paged(N=0, T=0) == OK
    if not HAS_GPU:
        full = dict(q=FAKE, cache=FAKE, out=FAKE, table=FAKE, lens=FAKE, cu=FAKE)
        for name in ("q", "cache", "out", "table", "lens", "cu"):
            assert paged(**{**full, name: None}) == BAD, name
            assert paged(**{**full, name: ODD}) == BAD, name
        assert paged(**full, lse=ODD) == BAD
        assert paged(**full, size=0) == WS and paged(**full, ws=FAKE, size=kda.kda_attn_q4_workspace_size(128) - 1) == WS
        assert paged(**full, ws=ctypes.c_void_p(FAKE.value + 16), size=1 << 30) == WS
    assert kda.kda_attn_q4_workspace_size(96) == 0
    for scale, rc in ((2.0 ** 100, OK), (1.3e30, BAD), (-1.3e30, BAD), (float("inf"), BAD), (float("nan"), OK)):
        assert lib.kda_attn_paged_q4(*[None] * 3, scale, *[None] * 3, 0, 0, 2, 1, 128, 4, 16, 4, None, None, None) == rc, scale


def test_binding_refusals():
    """The binding's own checks (host tensors stand for everything that is not on the device)."""
    bf = torch.bfloat16
    q = torch.zeros((4, 2, 128), dtype=bf)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(64)
    c = torch.zeros((2, 2, 16, 68), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_qk_norm_rope(q, q, i, f)
    with pytest.raises(TypeError):
        kda.kda_qk_norm_rope(q.float(), q, i, f)
    with pytest.raises(TypeError):
        kda.kda_qk_norm_rope_bwd(q.half(), q, i, f, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_kv_write_q4(q, q, i, c, c)
    with pytest.raises(TypeError):
        kda.kda_kv_write_q4(q.float(), q, i, c, c)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_kv_read_q4(c, c, i)
    with pytest.raises(ValueError, match="bytes"):
        kda.kda_kv_read_q4(c[..., :60], c, i)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_attn_paged_q4(q, c, c, i[None], i[:1], i[:2], 1.0)
    assert kda.q4_row_bytes(128) == 68 and kda.q4_row_bytes(64) == 34


def test_rows_of_strided_tensors(monkeypatch):
    """Which layouts of [T, H, D] are taken, and the stride that is passed for each."""
    bf = torch.bfloat16

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0
    monkeypatch.setattr(kda, "_check", lambda *a, **kw: None)
    at = lambda t: t.as_subclass(OnDevice)  # noqa: E731
    fused = torch.zeros((6, 12, 64), dtype=bf)
    rows = lambda t: kda._rows_arg(at(t), "x", tuple(t.shape), 0)[1]  # noqa: E731
    assert rows(fused) == 768 and rows(fused[:, 3:7]) == 768 and rows(fused[:, 3:4]) == 768
    assert rows(fused[2:3, 3:7]) == 256 and rows(fused[::2]) == 1536 and rows(fused[:0]) == 768
    for bad in (fused.transpose(0, 1), fused[..., ::2], fused[:, ::2], fused[:1].expand(6, 12, 64),
                torch.zeros((6, 12 * 64 + 4), dtype=bf)[:, :768].unflatten(1, (12, 64))):
        with pytest.raises(ValueError, match="contiguous heads"):
            rows(bad)
    with pytest.raises(ValueError, match="shape"):
        kda._rows_arg(at(fused), "x", (6, 11, 64), 0)
