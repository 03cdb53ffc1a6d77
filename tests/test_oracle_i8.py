"""The oracle of the 8-bit rows against whole-number arithmetic (CPU)."""

import numpy as np
import pytest

from oracle import i8


@pytest.mark.parametrize("kind", ["f32", "bf16", "ties", "subnormal", "far"])
def test_quantise_is_the_nearest_integer(kind):
    rng = np.random.default_rng(len(kind))
    for _ in range(20):
        x = rng.normal(size=257).astype(np.float32)
        if kind == "bf16":
            x = i8.to_bf16(x)
        if kind == "ties":  # multiples of half a scale
            x = (rng.integers(-254, 255, size=257) * 0.5 * 2.0 ** int(rng.integers(-20, 20))).astype(np.float32)
            x[0] = np.abs(x).max() and 127.0 * 2.0 ** np.ceil(np.log2(np.abs(x).max() / 127.0))
        if kind == "subnormal":
            x = (x * np.float32(1e-42)).astype(np.float32)
        if kind == "far":
            x = (x * np.float32(5e37)).astype(np.float32)
        q, _ = i8.quantise(x)
        assert np.array_equal(q, i8.quantise_exact(x))
        assert np.abs(q.astype(int)).max() <= 127


def test_quantise_of_rows_without_a_scale():
    for x, nan in (([0.0, -0.0, 0.0], False), ([1.0, np.nan, 2.0], True), ([1.0, -np.inf], True), ([1.401298464324817e-45], False)):
        q, s = i8.quantise(np.array(x, dtype=np.float32))
        assert not q.any() and (np.isnan(s) if nan else s == 0)


def test_product_in_whole_numbers():
    rng = np.random.default_rng(3)
    xq, wq = rng.integers(-128, 128, size=(3, 70)), rng.integers(-128, 128, size=(5, 70))
    ones3, ones5 = np.ones(3, np.float32), np.ones(5, np.float32)
    want = [[sum(int(a) * int(b) for a, b in zip(x, w)) for w in wq] for x in xq]
    assert np.array_equal(i8.product(xq, ones3, wq, ones5), np.array(want, dtype=np.float32))
    y = i8.product(xq, ones3 * np.float32(0.3), wq, ones5 * np.float32(0.7))
    assert y.dtype == np.float32
    assert y[1, 2] == np.float32(np.float32(np.float32(want[1][2]) * np.float32(0.3)) * np.float32(0.7))


def test_bf16_rounding():
    y = np.array([1.0, 1.00390625, 1.01171875, -3.0e38, 3.4e38, np.nan], dtype=np.float32)
    want = np.array([1.0, 1.0, 1.015625, -3.0e38, np.inf], dtype=np.float32)
    got = i8.to_bf16(y)
    assert got[0] == 1.0 and got[1] == 1.0 and got[2] == want[2] and got[4] == np.inf and np.isnan(got[5])
    assert abs(got[3] / -3.0e38 - 1) < 2.0 ** -8
