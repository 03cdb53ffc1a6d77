"""GPU parity of dflash_logprobs with the float64 oracle where the largest logit
over the temperature is some 2^22 to 2^31: near such exponents a whole-number
reference has to be right to 1/2 all the same, or the sums have to be taken from
the differences.  The bars are those of test_gpu_logprobs, which count |t| up to
1/2 for the reference.
"""

import numpy as np
import pytest

from test_gpu_logprobs import _say, check, tokens

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_select_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def rows_of(rng, V, kind, m, k):
    """(z [R, V], T [R]): rows whose largest |z| log2 e / T is about 2^k."""
    T = np.float32(abs(m) * LOG2E / 2.0 ** k)
    z = np.full((3, V), -1e4 * abs(m), np.float32)
    for i in range(3):
        top = np.float32(m * (1 - 1e-3 * i))
        if kind == "one":
            z[i, rng.integers(V)] = top
        elif kind == "ties":
            z[i, rng.integers(V, size=min(V, 40))] = top
        else:  # terms of 2^0 to 2^-40 of the largest one, as fp32 gives them, a tenth of them masked
            n = min(V, 2000)
            at = rng.permutation(V)[:n]
            z[i, at] = (float(top) - float(T) / LOG2E * rng.uniform(0, 40, size=n)).astype(np.float32)
            z[i, at[0]] = top
            z[i, at[1::10]] = -np.inf
    return z, [T] * 3


@pytest.mark.parametrize("k", [21.6, 22.9, 23.6, 23.999, 24.3, 25.5, 27.2, 28.7, 29.6, 29.999, 30.3])
@pytest.mark.parametrize("kind", ["one", "ties", "near"])
@pytest.mark.parametrize("V", [9, 1000, 9001, 140011])
def test_large_scales(V, kind, k):
    rng = np.random.default_rng(int(k * 1000) + V)
    for m in (1.0, 35.0, -130.0):
        z, T = rows_of(rng, V, kind, m, k)
        if m < 0:  # all others far below
            z[z == -1e4 * abs(m)] *= 3
        _say(f"[logprobs] V={V} {kind} m={m} 2^{k}")
        check(z, "f32", tokens(rng, 3, V, 2), 5, T=T)
        if kind != "near" and m > 0:
            check(z, "bf16", tokens(rng, 3, V, 1), 0, T=T)


@pytest.mark.parametrize("k", [23.9, 24.1, 28.5, 29.9])
def test_large_scales_of_many_rows(k):
    # one block a row, the oracle looking at some of them
    rng = np.random.default_rng(int(k * 10))
    z, T = rows_of(rng, 9001, "near", 35.0, k)
    z = np.tile(z, (700, 1))
    check(z, "f32", tokens(rng, 2100, 9001, 1), 3, T=T * 700, rows_=[0, 1, 2, 1000, 2099])


def test_a_row_of_both_signs():
    # the largest logit is small, others' own exponents lie beyond every reference
    rng = np.random.default_rng(6)
    z = rng.normal(size=(4, 30011)).astype(np.float32) * 1e3
    z[z > 0] *= -1
    z[:, 100:110] = (1e-4 * rng.uniform(0.99, 1, size=(4, 10))).astype(np.float32)
    check(z, "f32", tokens(rng, 4, 30011, 2), 12, T=[1e-4, 1e-6, 1e-8, 1e-10])
    check(-np.abs(z), "f32", tokens(rng, 4, 30011, 2), 12, T=[1e-4, 1e-6, 1e-8, 1e-10])
