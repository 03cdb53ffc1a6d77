"""The oracle of log probabilities against closed forms and differences (CPU)."""

import numpy as np
import pytest

from oracle import rows as O


def test_uniform_and_two_tokens():
    r = O.logprobs(np.full(8, 5000.0), [0, 7, 8, -1], N=3)
    assert np.allclose(r["logp"], [-np.log(8), -np.log(8), 0, 0]) and r["norm"][0] == 5000 and np.isclose(r["norm"][1], np.log(8))
    assert np.isclose(r["entropy"], np.log(8)) and list(r["top_idx"]) == [0, 1, 2]
    r = O.logprobs([0.0, np.log(3.0) * 2], [0, 1], T=2.0)
    assert np.allclose(np.exp(r["logp"]), [0.25, 0.75])


def test_masked_empty_nan_and_lowest_rows():
    r = O.logprobs([-np.inf, 1.0, -np.inf], [0, 1], N=2)
    assert list(r["logp"]) == [-np.inf, 0.0] and r["entropy"] == 0 and list(r["top_idx"]) == [1, -1] and r["top_logp"][1] == -np.inf
    r = O.logprobs([-np.inf] * 3, [0, 5], N=1)
    assert list(r["logp"]) == [-np.inf, 0.0] and r["norm"] == (-np.inf, 0.0) and r["entropy"] == 0 and r["top_idx"][0] == -1
    for bad in (np.nan, np.inf):
        r = O.logprobs([1.0, bad, 2.0], [0, 9], N=1)
        assert np.isnan(r["logp"][0]) and r["logp"][1] == 0 and np.isnan(r["entropy"]) and r["top_idx"][0] == -1
    low = -3.4028234663852886e38
    r = O.logprobs([low] * 4, [2], N=4)
    assert np.isclose(r["logp"][0], -np.log(4)) and list(r["top_idx"]) == [0, 1, 2, 3]


@pytest.mark.parametrize("T,want", [(0.0, 1.0), (-1.0, 1.0), (np.nan, 1.0), (0.5, 0.5), (np.inf, 1e30), (1e-40, 1e-30)])
def test_temperature(T, want):
    assert O.temperature(T) == want


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_gradient_against_differences(T):
    rng = np.random.default_rng(2)
    z = rng.normal(size=9)
    z[4] = -np.inf
    tok, g, ge = [2, 2, 7, -1, 99], rng.normal(size=5), 0.3

    def value(y):
        r = O.logprobs(y, tok, T=T)
        return float(np.dot(g, r["logp"])) + ge * r["entropy"]

    r = O.logprobs(z, tok, T=T)
    d = O.logprobs_grad(z, tok, g, ge, r["norm"], r["entropy"], T=T)
    assert d[4] == 0
    for j in range(9):
        if j != 4:
            up, dn = z.copy(), z.copy()
            up[j] += 1e-6
            dn[j] -= 1e-6
            assert abs((value(up) - value(dn)) / 2e-6 - d[j]) < 1e-8
    assert abs(d.sum()) < 1e-12  # the distribution does not change with a shift
