"""Rows in 8-bit integers with one scale each, and their product.

The pages leave the head that makes the logits to the models' own runtimes, so
these definitions are this project's own.  Pinned by tests/test_oracle_i8.py
against whole-number arithmetic.
"""

from fractions import Fraction

import numpy as np


def quantise(x):
    """(q int8 [H], scale fp32) of one row: scale = max |x| / 127 to the nearest
    fp32, q = x / scale to the nearest integer, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, dtype=np.int8), np.float32(np.nan)
    with np.errstate(under="ignore"):
        scale = np.float32(np.abs(x).max() / 127.0)
    if scale == 0:
        return np.zeros(x.shape, dtype=np.int8), scale
    # the fp64 quotient of two fp32 values never rounds onto the middle of two small integers
    return np.clip(np.rint(x / np.float64(scale)), -127, 127).astype(np.int8), scale


def quantise_exact(x):
    """The same q in whole-number arithmetic (slow)."""
    _, scale = quantise(x)
    if not scale > 0:
        return np.zeros(len(x), dtype=np.int8)
    s = Fraction(float(scale))
    return np.array([max(-127, min(127, round(Fraction(float(v)) / s))) for v in x], dtype=np.int8)


def product(xq, xs, wq, ws):
    """fp32 [R, N]: the exact sums, rounded to fp32, times xs, then times ws, each rounded."""
    acc = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T  # whole numbers below 2^53
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        return acc.astype(np.float32) * np.asarray(xs, dtype=np.float32)[:, None] * np.asarray(ws, dtype=np.float32)[None, :]


def to_bf16(y):
    """fp32 to the nearest bf16, ties to even, as fp32."""
    y = np.asarray(y, dtype=np.float32)
    u = y.view(np.uint32).astype(np.uint64)
    r = (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(y), y, r)
