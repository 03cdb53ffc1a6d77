"""Pins of oracle.rows: closed forms, the filters one by one, and differences."""

import numpy as np
import pytest

from oracle import rows as R


def test_order_ties_and_masks():
    z = np.array([1.0, 3.0, -np.inf, 3.0, np.nan, 0.0, -0.0])
    assert R.order(z).tolist() == [1, 3, 0, 5, 6]


def test_closed_form_filters():
    # weights 1, 1/2, 1/4, 1/8 (times ln 2 steps), order 2 0 3 1
    z = np.log([0.5, 0.125, 1.0, 0.25])
    assert R.keep(z)[0].tolist() == [2, 0, 3, 1]
    assert R.keep(z, top_k=2)[0].tolist() == [2, 0]
    # shares 8/15, 4/15, 2/15, 1/15
    assert R.keep(z, top_p=0.5)[0].tolist() == [2]
    assert R.keep(z, top_p=0.6)[0].tolist() == [2, 0]
    assert R.keep(z, top_p=0.81)[0].tolist() == [2, 0, 3]
    # after top_k = 2 the shares are 2/3, 1/3
    assert R.keep(z, top_k=2, top_p=0.6)[0].tolist() == [2]
    assert R.keep(z, min_p=0.3)[0].tolist() == [2, 0]
    assert R.keep(z, min_p=7.0)[0].tolist() == [2]
    assert R.keep(z, top_p=-1.0)[0].tolist() == [2]
    assert R.keep(z, T=0.0)[0].tolist() == [2]
    assert R.keep(z, T=float("nan"))[0].tolist() == [2]
    assert R.keep(np.full(3, -np.inf))[0].size == 0


def test_draw_inverts_the_running_sum():
    z = np.zeros(8)
    for u, want in [(0.0, 0), (0.124, 0), (0.125, 1), (0.5, 4), (0.999, 7), (1.0, 7), (-1.0, 0), (float("nan"), 0)]:
        assert R.sample(z, u) == (want, 0.125, 8)
    assert R.sample(np.full(4, -np.inf), 0.3) == (-1, 0.0, 0)


def test_draw_frequencies():
    rng = np.random.default_rng(3)
    z = rng.normal(size=12) * 2
    p = np.exp(z - z.max())
    p /= p.sum()
    n = 20000
    got = np.bincount([R.sample(z, u)[0] for u in rng.random(n)], minlength=12)
    chi = ((got - n * p) ** 2 / (n * p)).sum()
    assert chi < 31.3  # 99.9% point of chi-square with 11 degrees


@pytest.mark.parametrize("with_lse", [False, True])
def test_distill_equals_kl_and_differences(with_lse):
    rng = np.random.default_rng(5)
    V, K, tau = 23, 5, 1.7
    s, t = rng.normal(size=V), rng.normal(size=V) * 2
    idx = np.argsort(-t)[:K]
    lse_t = R.log_sum_exp(t / tau) if with_lse else None
    r = R.distill(s, idx, t[idx], tau, lse_t)
    # KL of the two distributions over the listed tokens (and the rest as one class)
    q = np.exp(s / tau - R.log_sum_exp(s / tau))
    if with_lse:
        p = np.exp(t / tau - lse_t)
        P, Q = np.append(p[idx], 1 - p[idx].sum()), np.append(q[idx], 1 - q[idx].sum())
    else:
        P = np.exp(t[idx] / tau - R.log_sum_exp(t[idx] / tau))
        Q = q[idx]
    assert abs(r["loss"] - np.sum(P * np.log(P / Q))) < 1e-12
    h = 1e-6
    for j in range(V):
        e = np.zeros(V)
        e[j] = h
        d = (R.distill(s + e, idx, t[idx], tau, lse_t)["loss"] - R.distill(s - e, idx, t[idx], tau, lse_t)["loss"]) / (2 * h)
        assert abs(d - r["grad"][j]) < 1e-8, j
    assert abs(r["grad"].sum()) < 1e-12


def test_distill_padding_duplicates_and_empty_rows():
    rng = np.random.default_rng(6)
    s = rng.normal(size=9)
    a = R.distill(s, np.array([2, -1, 4, 9]), np.array([1.0, 5.0, 0.5, 7.0]))
    b = R.distill(s, np.array([2, 4]), np.array([1.0, 0.5]))
    assert a["loss"] == b["loss"] and np.array_equal(a["grad"], b["grad"])
    # a token listed twice carries both entries' mass
    c = R.distill(s, np.array([2, 2, 4]), np.array([1.0, 1.0, 0.5]))
    d = R.distill(s, np.array([2, 4]), np.array([1.0 + np.log(2.0), 0.5]))
    np.testing.assert_allclose(c["grad"], d["grad"], atol=1e-15)
    for t_idx, t in [(np.array([-1, 9]), np.zeros(2)), (np.array([1, 2]), np.full(2, -np.inf))]:
        e = R.distill(s, t_idx, t)
        assert e["loss"] == 0 and not e["grad"].any()
    f = R.distill(np.full(4, -np.inf), np.array([1]), np.zeros(1))
    assert f["loss"] == 0 and not f["grad"].any()


def test_log_sum_exp_out_of_range():
    # every logit the type's lowest value: nothing unmasked; far above: no result
    assert R.log_sum_exp(np.full(5, -3.4e38)) == -np.inf and np.isnan(R.log_sum_exp(np.array([1.0, 3e38])))
    d = R.distill(np.full(6, -3.4e38), np.array([1, 4]), np.array([0.0, 1.0]))
    assert d["loss"] == 0 and d["lse"] == -np.inf and not d["grad"].any()


def test_distill_infinite_teacher_logit_has_no_result():
    s = np.random.default_rng(7).normal(size=9)
    for t_lse in (None, 4.0):
        for bad in (np.inf, np.nan):
            d = R.distill(s, np.array([2, 4]), np.array([bad, 0.5]), 1.0, t_lse)
            assert np.isnan(d["loss"]) and np.isfinite(d["lse"])
