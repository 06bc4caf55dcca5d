"""CPU tests of the 4-bit cache's reference format: its values are bf16 numbers, packing is its own inverse, and the
scale is the smallest that will do."""
import numpy as np
import torch

import q4_testutil as Q


def test_values_are_bf16_numbers():
    v = np.outer(np.arange(-8, 8), Q.TABLE)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
    assert np.all(np.diff(Q.TABLE) > 0) and Q.TABLE[0] == 2.0 ** -15 and Q.TABLE[255] == 1.875 * 2.0 ** 16


def test_pack_and_back():
    rng = np.random.default_rng(0)
    for D in (64, 128):
        codes = rng.integers(0, 16, (3, 2, 16, D), dtype=np.uint8)
        b = rng.integers(0, 256, (3, 2, 16, D // 32)).astype(np.uint8)
        raw = Q.pack(codes, b)
        assert raw.shape == (3, 2, 16, D // 2 + D // 32)
        c2, b2 = Q.unpack(raw, D)
        assert np.array_equal(c2, codes) and np.array_equal(b2, b)


def test_the_scale_is_the_smallest_that_will_do():
    x = np.zeros((40, 32))
    x[:, 5] = np.exp(np.random.default_rng(1).uniform(-8, 12, 40))
    _, b = Q.quantise(x)
    for row, i in zip(x, b[:, 0]):
        assert 7 * Q.TABLE[i] >= row[5] and (i == 0 or 7 * Q.TABLE[i - 1] < row[5])


def test_error_of_normal_values():
    x = np.random.default_rng(2).standard_normal((2000, 128))
    v = Q.values(*Q.quantise(x))
    assert np.abs(v - x).max() <= 0.5 * 7.0 / 7 * 1.0 and np.sqrt(((v - x) ** 2).mean()) < 0.11
