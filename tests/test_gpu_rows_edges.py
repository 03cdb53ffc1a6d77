"""GPU tests of the operators on logit rows at the ends of what they accept:
uniforms next to 1, temperatures that leave bins without a value, settings of
the smallest tau, and every plan of the launches.  Bars as in test_gpu_rows.
"""

import numpy as np
import pytest

from oracle import rows as O
from test_gpu_rows import _check_distill, _check_sample, _distill_case, _f64, _logits, _run_distill, _say, _tensor

pytestmark = pytest.mark.gpu

LAST = 1.0 - 2.0 ** -53


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_select_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def _type(dt):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[dt]


@pytest.mark.parametrize("dt,R,V", [("f32", 64, 100003), ("f32", 200, 100003), ("f32", 4, 100003), ("f32", 4, 8001),
                                    ("bf16", 4, 100003), ("bf16", 4, 4001)])
def test_draw_of_the_last_token_before_a_gap(dt, R, V):
    # the kept tokens end where their bin ends, and the next bin in use holds
    # nearly all of the row: a draw at u's upper end stays with the last kept one
    _say(f"[rows] gap {dt} {R} x {V}")
    z = np.zeros((R, V), dtype=np.float32)
    z[:, [7, 1000, 2002, V // 2, V - 3]] = 10.0
    st = [dict(top_k=5), dict(min_p=0.5), dict(top_p=0.4), dict(top_k=5, top_p=0.99)]
    u = [1.0, LAST, 7.0, 0.999]
    _check_sample(z, _type(dt), [st[i % 4] for i in range(R)], np.array([u[i // 4 % 4] for i in range(R)]), pad=1)


@pytest.mark.parametrize("V,n", [(100003, 400), (100003, 3000)])
def test_temperature_that_leaves_bins_without_a_value(V, n):
    # T = 1e-7: fp32 values near 8 are 55 bins apart, so the bin of min-p's
    # border holds no value at all; the row's end holds more equal tokens than a
    # segment lists
    R = 64
    rng = np.random.default_rng(n)
    z = np.minimum(_logits(rng, R, V, "flat"), np.float32(7.0))
    z[:, V - 2 * n:V:2] = 8.0
    _say(f"[rows] empty bins {V} {n}")
    _check_sample(z, _type("f32"), [dict(T=1e-7, min_p=[0.5, 0.3, 1e-3][i % 3]) for i in range(R)], rng.random(R), pad=1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [3e-8, 3e-10, 1e-12, 1e-25])
@pytest.mark.parametrize("with_lse", [False, True])
def test_gradient_beside_lowest_values_at_a_small_tau(dt, tau, with_lse):
    import torch
    t = _type(dt)
    rng = np.random.default_rng(71)
    R, V, K = 4, 3001, 6
    s, teacher, idx, tl = _distill_case(rng, R, V, K, False, False, None)
    s, teacher, tl = s * np.float32(tau), teacher * np.float32(tau), tl * np.float32(tau)
    gone = rng.random(size=s.shape) < 0.6
    np.put_along_axis(gone, idx.astype(np.int64), False, 1)
    s[gone] = float(torch.finfo(t).min)
    s[1, gone[1]] = -np.inf
    _say(f"[rows] lowest values at tau {tau} {dt}")
    lse = np.array([O.log_sum_exp(x.astype(np.float64) / tau) for x in teacher]) if with_lse else None
    g = np.full(R, tau, dtype=np.float32)
    _check_distill(s, idx, tl, t, tau, lse, None, g)
    _check_distill(s, idx, tl, t, tau, lse, None, g, pad=1, inplace=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_lse", [False, True])
def test_gradient_whose_factor_leaves_fp32(dt, with_lse):
    # weight times grad_loss over tau lies beyond fp32, the gradients of unlikely tokens within
    t = _type(dt)
    rng = np.random.default_rng(72)
    R, V, K, tau = 3, 2000, 5, 1e-30
    s, teacher, idx, tl = _distill_case(rng, R, V, K, False, False, None)
    s, tl = s * np.float32(tau * 4), tl * np.float32(tau)
    s[:, 700:900] = -1.0
    lse = np.array([O.log_sum_exp(x.astype(np.float64)) for x in teacher]) if with_lse else None
    import torch
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    v, _ = _tensor(s, t)
    w, g = np.full(R, 1e10, dtype=np.float32), np.array([1.0, -1.0, 1e5], dtype=np.float32)
    _, _, _, dS = _run_distill(v, dev(idx), dev(tl), tau, dev(lse), dev(w), dev(g))
    got, zz, some_big = _f64(dS), _f64(v), False
    for i in range(R):
        ref = O.distill(zz[i], idx[i], tl[i], tau, None if lse is None else lse[i])
        want = float(w[i]) * float(g[i]) * ref["grad"]
        off = ref["p"] == 0
        assert not np.isnan(got[i]).any() and not got[i][700:900][off[700:900]].any()
        big = off & (np.abs(want) > 1.01 * float(torch.finfo(t).max))
        small = off & (np.abs(want) < 0.99 * float(torch.finfo(t).max))
        some_big |= bool(big.any())
        assert small.any()
        assert np.array_equal(got[i][big], np.sign(want[big]) * np.inf)
        half = torch.finfo(t).eps / 2
        x = zz[i] / tau
        tt = np.minimum(np.abs(x - ref["lse"]) / np.log(2), 2.0 ** 30)
        assert (np.abs(got[i] - want)[small] <= (np.abs(want) * (half + (tt + 4) * 2.0 ** -23))[small] + 2.0 ** -125).all()
    assert some_big


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinite_and_nan_teacher_logits(dt):
    import torch
    t = _type(dt)
    rng = np.random.default_rng(73)
    for K in (4, 100):
        s, teacher, idx, tl = _distill_case(rng, 4, 700, K, False, False, None)
        tl[1, 2], tl[2, K - 1] = np.inf, np.nan
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        v, _ = _tensor(s, t)
        for lse in (None, dev(np.full(4, 9.0))):
            loss, own, _, dS = _run_distill(v, dev(idx), dev(tl), 1.0, lse, None, None)
            assert torch.isfinite(own).all()
            for i in range(4):
                assert bool(torch.isnan(loss[i])) == (i in (1, 2)), (K, i, float(loss[i]))
                assert bool(torch.isnan(dS[i]).all()) == (i in (1, 2)) == bool(torch.isnan(dS[i]).any()), (K, i)


@pytest.mark.parametrize("dt,R,V", [("bf16", 1, 4096), ("bf16", 1, 4104), ("bf16", 30, 50021), ("f32", 1, 1000), ("f32", 3, 8192),
                                    ("f32", 3, 8200), ("f32", 40, 100003), ("f32", 80, 100003)])
def test_min_p_at_weights_next_to_one(dt, R, V):
    # T = 1e13: weights differ from 1 by 2^-43 and less, which fp64 still tells apart, on every path
    rng = np.random.default_rng(V)
    z = (np.round(rng.normal(size=(R, V)) * 2 * 16) / 16).astype(np.float32)
    z[:, V // 3] = z[:, V // 2] = 16.0
    z[:, V // 5] = 15.9375
    st = [dict(T=1e13, min_p=1.0), dict(T=1e12, min_p=float(np.float32(1.0 - 2.0 ** -24)))]
    _check_sample(z, _type(dt), [st[i % 2] for i in range(R)], rng.random(R))


@pytest.mark.parametrize("dt,R,V", [("bf16", 6, 4001), ("bf16", 6, 50021), ("f32", 6, 1000), ("f32", 6, 50021), ("f32", 66, 100003)])
def test_min_p_whose_border_lies_near_zero(dt, R, V):
    # max 1, T = 1, min_p next to 1/e: the border lies within 1e-7 of zero, where
    # fp32 values are dense; and borders in the tail, far below and at the maximum
    rng = np.random.default_rng(V + 1)
    z = rng.normal(size=(R, V)).astype(np.float32)
    z[:, ::2] *= 10.0 ** rng.uniform(-12, -5, size=z[:, ::2].shape)
    z = np.minimum(z, np.float32(0.9))
    z[:, V // 3] = 1.0
    e = float(np.exp(-1.0))
    st = [dict(min_p=p) for p in (e, float(np.nextafter(np.float32(e), np.float32(1))), float(np.nextafter(np.float32(e), np.float32(0))),
                                  0.03, 1e-44, 0.95)]
    _check_sample(z, _type(dt), [st[i % 6] for i in range(R)], rng.random(R))
