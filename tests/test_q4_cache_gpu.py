"""GPU tests of the store into the 4-bit cache and the reading of its rows: whole numbers, so every comparison is
exact."""
import numpy as np
import pytest
import torch

import q4_testutil as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_40_gb300 import kda
    kda.load()
    yield
    assert kda.kda_get_status() == 0


def _kda():
    from gated_delta_rule_40_gb300 import kda
    return kda


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check(k, v, slots, blocks, bs, seed=0, strided=False):
    """Stores k, v at slots of caches of random bytes; all other bytes stay; reads the rows back."""
    kda = _kda()
    T, H, D = k.shape
    rng = np.random.default_rng(seed)
    before = [rng.integers(0, 256, (blocks, H, bs, D // 2 + D // 32)).astype(np.uint8) for _ in range(2)]
    caches = [torch.from_numpy(c).cuda() for c in before]
    if strided:   # heads of a fused projection
        fused = torch.cat([v, k, v], 1).cuda()
        dk, dv = fused[:, H:2 * H], fused[:, 2 * H:]
    else:
        dk, dv = k.cuda(), v.cuda()
    kda.kda_kv_write_q4(dk, dv, _ints(slots), *caches)
    torch.cuda.synchronize()
    for x, old, got in ((k, before[0], caches[0]), (v, before[1], caches[1])):
        codes, b = Q.unpack(old, D)
        nc, nb = Q.quantise(x.double().numpy())
        for t, s in enumerate(slots):
            if 0 <= s < blocks * bs:
                codes[s // bs, :, s % bs], b[s // bs, :, s % bs] = nc[t], nb[t]
        assert np.array_equal(got.cpu().numpy(), Q.pack(codes, b))
    return caches


def _normal(seed, *shape, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * gain).to(torch.bfloat16)


@pytest.mark.parametrize("T,H,D,bs", [(1, 1, 128, 16), (1, 1, 64, 16), (3, 2, 64, 32), (7, 3, 128, 64), (130, 8, 128, 128),
                                      (77, 5, 64, 1024), (513, 1, 128, 16)])
@pytest.mark.parametrize("strided", [False, True])
def test_store_and_read(T, H, D, bs, strided):
    blocks = -(-T // bs) + 2
    rng = np.random.default_rng(T)
    slots = rng.permutation(blocks * bs)[:T].tolist()
    k, v = _normal(T, T, H, D, gain=3.0), _normal(T + 1, T, H, D, gain=0.01)
    caches = _check(k, v, slots, blocks, bs, strided=strided)
    rk, rv = _kda().kda_kv_read_q4(*caches, _ints(slots))
    assert torch.equal(rk.cpu(), Q.bf16_values(k)) and torch.equal(rv.cpu(), Q.bf16_values(v))


def test_values_at_the_borders():
    """Halves between codes, scales that are met exactly or just missed, zeros, the smallest and largest numbers."""
    rows = []
    for b in (0, 1, 7, 8, 100, 120, 127, 248, 254, 255):
        s = Q.TABLE[b]
        x = np.zeros(32)
        x[0] = 7 * s                                              # this scale exactly
        halves = [(n + 0.5) * s for n in range(7)]
        x[1:8], x[8:15] = halves, [-h for h in halves]
        x[15], x[16] = s * 6.9, -s * 0.49
        rows.append(x)
        y = x.copy()
        y[0] = np.nextafter(np.float32(7 * s), np.float32(np.inf))
        rows.append(y)
    rows.append(np.zeros(32))
    rows.append(np.full(32, -0.0))
    rows.append(np.full(32, 1e-40))
    rows.append(np.full(32, 3.3e38))
    rows.append(np.linspace(-3.3e38, 3.3e38, 32))
    x = torch.tensor(np.stack(rows + rows[:(-len(rows)) % 4])).to(torch.bfloat16).reshape(-1, 1, 128)
    T = x.shape[0]
    _check(x, x.flip(-1), list(range(T)), 1, 16 if T <= 16 else 32)


def test_every_bf16_magnitude_beside_every_kind_of_scale():
    """All finite bf16 numbers, 32 of neighbouring magnitude together, and each next to a larger one."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    y = x.clone()
    y[1::2] = y[1::2].neg()
    big = (x.double() * 5.3).clamp(max=3.3e38).to(torch.bfloat16).reshape(-1, 32)[:, :1].expand(-1, 32)
    z = torch.where(torch.arange(32) == 9, big, y.reshape(-1, 32)).reshape(-1)
    pad = (-x.numel()) % 128
    fit = lambda t: torch.cat([t, torch.zeros(pad, dtype=t.dtype)]).reshape(-1, 1, 128)  # noqa: E731
    k, v = fit(y), fit(z)
    _check(k, v, list(range(k.shape[0])), 1, 1024 if k.shape[0] > 128 else 128)


def test_infinities_and_nans():
    inf, nan = float("inf"), float("nan")
    k = _normal(5, 6, 2, 128)
    want = k.clone()
    k[0, 0, 3], want[0, 0, 3] = inf, 3.3e38
    k[1, 1, 64], want[1, 1, 64] = -inf, -3.3e38
    k[2, 0, 5], want[2, 0, 5] = nan, 0.0
    k[3, 1, 32:64], want[3, 1, 32:64] = nan, 0.0
    kda = _kda()
    got = []
    for x in (k, want):
        c = [torch.zeros((1, 2, 16, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
        kda.kda_kv_write_q4(x.cuda(), x.cuda(), _ints(range(6)), *c)
        got.append(c[0].cpu())
    assert torch.equal(*got)


def test_slots_left_out_and_bad():
    kda = _kda()
    k, v = _normal(1, 9, 2, 128), _normal(2, 9, 2, 128)
    slots = [5, -1, 7, -5, 31, 0, -2 ** 31, 20, 21]
    caches = _check(k, v, slots, 2, 16)
    assert kda.kda_get_status() == kda.KDA_OK
    rk, rv = kda.kda_kv_read_q4(*caches, _ints([7, -1, 31, -2 ** 31]))
    assert torch.equal(rk.cpu()[[0, 2]], Q.bf16_values(k)[[2, 4]]) and not rk[[1, 3]].any() and not rv[[1, 3]].any()
    assert kda.kda_get_status() == kda.KDA_OK
    caches = _check(k, v, [5, 32, 7, 2 ** 31 - 1, 31, 0, 1, 20, 21], 2, 16)   # outside: left out, reported
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES
    rk, _ = kda.kda_kv_read_q4(*caches, _ints([32, 7, 2 ** 31 - 1]))
    assert torch.equal(rk.cpu()[1], Q.bf16_values(k)[2]) and not rk[[0, 2]].any()
    assert kda.kda_get_status() == kda.KDA_ERR_BAD_PAGES


def test_no_tokens():
    kda = _kda()
    c = [torch.full((1, 2, 16, 34), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    kda.kda_kv_write_q4(e, e, _ints([]), *c)
    k, v = kda.kda_kv_read_q4(*c, _ints([]))
    assert k.shape == (0, 2, 64) and all((x == 9).all() for x in c)


def test_slots_past_32_bits_of_bytes():
    """A cache of more than 4 GiB: its last rows."""
    kda = _kda()
    blocks, H, bs = 4200, 16, 1024
    c = [torch.zeros((blocks, H, bs, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = _normal(3, 4, H, 128), _normal(4, 4, H, 128)
    slots = _ints([0, blocks * bs - 1, 3855 * 1024 + 17, 17])
    kda.kda_kv_write_q4(k.cuda(), v.cuda(), slots, *c)
    rk, rv = kda.kda_kv_read_q4(*c, slots)
    assert torch.equal(rk.cpu(), Q.bf16_values(k)) and torch.equal(rv.cpu(), Q.bf16_values(v))
    codes, b = Q.unpack(c[0][-1, :, -1:].cpu().numpy().reshape(H, 1, 68) * 0, 128)
    assert int(c[0][1:3000].sum(dtype=torch.int64)) == 0


def test_streams_and_graphs():
    kda = _kda()
    k, v = _normal(7, 40, 4, 64).cuda(), _normal(8, 40, 4, 64).cuda()
    c = [torch.zeros((3, 4, 16, 34), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = _ints(list(range(40)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_kv_write_q4(k, v, slots, *c, stream=side)
    rk, _ = kda.kda_kv_read_q4(*c, slots, stream=side)
    side.synchronize()
    assert torch.equal(rk.cpu(), Q.bf16_values(k.cpu()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_kv_write_q4(k, v, slots, *c)
        gk, gv = kda.kda_kv_read_q4(*c, slots)
    k.copy_(_normal(9, 40, 4, 64))
    slots.copy_(_ints(list(range(39, -1, -1))))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gk.cpu(), Q.bf16_values(k.cpu())) and torch.equal(gv.cpu(), Q.bf16_values(v.cpu()))
