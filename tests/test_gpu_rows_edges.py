"""GPU tests of the operators on logit rows at the ends of what they accept:
uniforms next to 1, temperatures that leave bins without a value, the smallest
tau, min-p next to its ends, and the plans of the launches.  Bars as in
test_gpu_rows.
"""

import numpy as np
import pytest

from oracle import rows as O
from test_gpu_rows import (MIX, _arr, _as_used, _check_distill, _check_sample, _distill_case, _f64, _filters, _logits,
                           _run_distill, _say, _tensor)

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


# ---------------------------------------------------------------- the launches' plans

# one launch; bf16 segments; fp32 with every token listed; fp32 with the largest
# listed, in segments of 2, 4 and 8 slots a thread
PLANS = [("bf16", 14, 3001), ("f32", 14, 8001), ("bf16", 14, 20011), ("f32", 14, 20011), ("f32", 63, 100003), ("f32", 98, 100003),
         ("f32", 168, 100003)]


@pytest.mark.parametrize("dt,R,V", PLANS)
def test_uniforms_at_their_ends_on_every_plan(dt, R, V):
    rng = np.random.default_rng(R + V)
    u = [0.0, -1.0, float("nan"), 1.0, 7.0, LAST, 2.0 ** -60]
    st = [dict(), dict(top_k=5), dict(top_p=0.8), dict(T=0.5, min_p=0.2), dict(top_k=3000, top_p=0.9999), dict(T=0.0), dict(T=8.0, top_p=0.7)]
    _say(f"[rows] u at its ends {dt} {R} x {V}")
    z = _logits(rng, R, V, "peaked")
    _check_sample(z, _type(dt), [st[i // 7 % 7] for i in range(R)], np.array([u[i % 7] for i in range(R)]), pad=1)


def test_uniforms_at_their_ends_where_a_row_is_binned_by_one_block():
    # bf16 rows with their largest logit over the counters
    rng = np.random.default_rng(81)
    u = [0.0, -1.0, float("nan"), 1.0, 7.0, LAST, 2.0 ** -60]
    z = _logits(rng, 7, 20011, "peaked") + np.float32(900.0)
    for st in (dict(), dict(top_k=5), dict(top_p=0.8, T=4.0)):
        _check_sample(z, _type("bf16"), [st] * 7, np.array(u))


@pytest.mark.parametrize("dt,R,V", [("bf16", 8300, 4104), ("f32", 1030, 8200), ("f32", 170, 400007)])
def test_more_rows_than_a_pass_over_the_workspace(dt, R, V):
    # 8192 bf16 segments a pass, 1024 fp32 rows or 4096 fp32 segments
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(R)
    t = _type(dt)
    n = 300 if V < 10000 else 40  # the same rows over and over, every row with its own uniform and settings
    z = _logits(rng, n, V, "peaked")[np.arange(R) % n]
    st = [MIX[i % len(MIX)] for i in range(R)]
    _say(f"[rows] several passes {dt} {R} x {V}")
    u = rng.random(R)
    _check_sample(z, t, st, u, pad=1)
    v, _ = _tensor(z, t)
    r = dfl.rows(v)
    out = torch.empty_like(v)
    kept = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    dfl.dflash_filter(r, v, out, dfl.rows_workspace(r), kept=kept, **_filters(st))
    torch.cuda.synchronize()
    kept = kept.cpu().numpy()
    low = float(torch.finfo(t).min)
    for i in range(0, R, 7 if V < 10000 else 3):
        zz = _f64(v[i])
        assert np.array_equal(_f64(out[i]), O.filtered(zz, low, **_as_used(st[i]))), (i, st[i])
        assert kept[i] == O.keep(zz, **_as_used(st[i]))[0].size, (i, st[i])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_listed_tokens_at_the_types_lowest_value(dt):
    # a student that a finite mask denies every listed token: the loss is about
    # the mask over tau (beyond fp32: inf), the gradient ordinary
    import torch
    t = _type(dt)
    low = float(torch.finfo(t).min)
    rng = np.random.default_rng(82)
    V = 20005
    s = np.full((3, V), low, dtype=np.float32)
    s[0, 100:200] = rng.normal(size=100)
    s[1, 20004] = 0.5
    s[2] = rng.normal(size=V)
    s[2, 19000] = low
    idx = np.tile(np.array([[3, 19000, 7]], dtype=np.int32), (3, 1))
    tl = np.ones((3, 3), dtype=np.float32)
    for with_lse in (False, True):
        _check_distill(s, idx, tl, t, 2.0, np.full(3, 1.8) if with_lse else None, None, None)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        v, _ = _tensor(s, t)
        loss, lse, _, dS = _run_distill(v, dev(idx), dev(tl), 0.25, dev(np.full(3, 5.2)) if with_lse else None, None, None)
        assert torch.isinf(loss).all() and (loss > 0).all() and torch.isfinite(lse).all() and torch.isfinite(dS).all()


def test_gradient_at_small_tau():
    # x = S / tau up to 2^24: beside the bars of test_gpu_rows the exponent is off
    # by the roundings of x, lse and the products in fp64 (6 of 2^-53 |x|), and of
    # the low pieces in fp32: theirs and the high piece's remainder, each below
    # 2^-22 |x|, are rounded to 2^-24 of that in five places
    import torch
    rng = np.random.default_rng(83)
    R, V, K = 4, 5003, 8
    for tau in (1e-3, 1e-6):
        for t in (torch.bfloat16, torch.float32):
            for with_lse in (False, True):
                s, teacher, idx, tl = _distill_case(rng, R, V, K, False, False, None)
                v, _ = _tensor(s, t)
                zz = _f64(v)
                # a bulk within a few nats of the top keeps the exponentials in range
                zz = zz.max(1, keepdims=True) * (1.0 + rng.integers(-4, 1, size=zz.shape) * float(torch.finfo(t).eps))
                v.copy_(torch.from_numpy(zz))
                zz = _f64(v)
                lse_t = np.array([O.log_sum_exp(tl[i].astype(np.float64) / tau) + 0.3 for i in range(R)]) if with_lse else None
                dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
                _, lse, _, dS = _run_distill(v, dev(idx), dev(tl), tau, dev(lse_t), None, None)
                got = _f64(dS)
                for i in range(R):
                    ref = O.distill(zz[i], idx[i], tl[i], tau, None if lse_t is None else lse_t[i])
                    x = zz[i] / tau
                    big = np.abs(x).max()
                    assert big < 2.0 ** 25
                    assert abs(float(lse[i]) - ref["lse"]) <= 2e-11 + big * 2.0 ** -49
                    half = torch.finfo(t).eps / 2
                    size = (ref["A"] * np.exp(x - ref["lse"]) + ref["p"] + (0 if lse_t is None else np.where(
                        ref["p"] > 0, 0.0, ref["p_rest"] * np.exp(np.minimum(x - ref["lse_rest"], 0.0))))) / tau
                    d = np.abs(x - ref["lse"]) / np.log(2)
                    tol = np.abs(ref["grad"]) * half + size * ((np.minimum(d, 126.0) + 4) * 2.0 ** -23 + 1e-10 + big * (
                        6 * 2.0 ** -53 + 5 * 2.0 ** -46)) + 2.0 ** -125 * (1 + 1 / tau)
                    assert (np.abs(got[i] - ref["grad"]) <= tol).all(), (tau, t, i, np.abs(got[i] - ref["grad"]).max())


def test_per_kernel_timers_of_the_four():
    import torch
    import block_draft_select_amd as dfl
    v = torch.randn(5, 20011, device="cuda")
    r = dfl.rows(v)
    ws, out = dfl.rows_workspace(r), torch.empty_like(v)
    u, lse = torch.rand(5, dtype=torch.float64, device="cuda"), torch.empty(5, dtype=torch.float64, device="cuda")
    token, loss = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    idx = torch.arange(20, dtype=torch.int32, device="cuda").view(5, 4)
    tl = torch.randn(5, 4, device="cuda")
    dfl.dflash_profile_enable(True)
    try:
        for n in range(3):
            dfl.dflash_sample(r, v, u, token, ws, top_p=_arr([0.9] * 5, torch.float32))
            dfl.dflash_filter(r, v, out, ws)
            dfl.dflash_distill(r, v, idx, tl, loss, lse, ws)
            dfl.dflash_distill_grad(r, v, idx, tl, lse, out)
        for name in ("sample", "filter", "distill", "distill_grad"):
            calls, ms = dfl.dflash_profile_collect(name)
            assert calls == 3 and 0.0 < ms < 1000.0, (name, calls, ms)
            assert dfl.dflash_profile_collect(name) == (0, 0.0)
    finally:
        dfl.dflash_profile_enable(False)


# ---------------------------------------------------------------- the largest sizes, and rows beside rows

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_most_rows_of_one_call(dt):
    import torch
    import block_draft_select_amd as dfl
    t = _type(dt)
    R, V, group = dfl.ROWS_MAX, 3, 1 << 21
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    z = torch.randn(R, V, device="cuda", generator=gen).to(t)
    u = torch.rand(R, dtype=torch.float64, device="cuda", generator=gen)
    r = dfl.rows(z)
    ws = dfl.rows_workspace(r)
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    kept, T, k = torch.full_like(token, -7), _arr([1.0, 0.5], torch.float32), _arr([0, 2], torch.int32)
    _say(f"[rows] {R} rows {dt}")
    dfl.dflash_sample(r, z, u, token, ws, T=T, top_k=k, group=group, kept=kept)
    val, at = torch.sort(z.double(), dim=1, descending=True, stable=True)
    temp = T.double().repeat_interleave(group)[:, None]
    w = torch.exp((val - val[:, :1]) / temp)
    w[group:, 2] = 0.0
    run = torch.cumsum(w, 1)
    pos = (run <= u[:, None] * run[:, -1:]).sum(1)
    assert torch.equal(token.long(), at.gather(1, pos[:, None])[:, 0])
    assert (kept[:group] == 3).all() and (kept[group:] == 2).all()
    out = torch.empty_like(z)
    dfl.dflash_filter(r, z, out, ws, T=T, top_k=k, group=group)
    want = z.clone()
    want[group:] = want[group:].scatter(1, at[group:, 2:], torch.finfo(t).min)
    assert torch.equal(out, want)
    idx, tl = at[:, 1:2].to(torch.int32).contiguous(), torch.zeros(R, 1, device="cuda")
    loss, lse, _, dS = _run_distill(z, idx, tl, 1.0, None, None, None)
    ref = torch.logsumexp(z.double(), 1)
    assert (lse - ref).abs().max() <= 2e-11 + 2.0 ** -46
    d = ref - val[:, 1]
    assert ((loss.double() - d).abs() <= d.abs() * 2.0 ** -24 + 1e-10 * (1 + ref.abs())).all()
    x = z.double() - ref[:, None]
    g = torch.exp(x).scatter_add(1, at[:, 1:2], torch.full((R, 1), -1.0, dtype=torch.float64, device="cuda"))
    tol = g.abs() * (torch.finfo(t).eps / 2 + (x.abs() / np.log(2) + 4) * 2.0 ** -23) + 1e-10 * (torch.exp(x) + 1)
    assert ((dS.double() - g).abs() <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_longest_rows_and_lists(dt):
    import torch
    import block_draft_select_amd as dfl
    t = _type(dt)
    rng = np.random.default_rng(84)
    V, K = dfl.V_MAX, dfl.DISTILL_K_MAX
    z = _logits(rng, 2, V, "peaked")
    _say(f"[rows] V {V} {dt}")
    v, _ = _tensor(z, t, 1, 1)
    zz = _f64(v)
    st = [dict(top_p=0.9), dict(min_p=1e-4, T=1.5)]
    _check_sample(z, t, st, rng.random(2), pad=1, shift=1)
    out = torch.empty(2, V + 3, dtype=t, device="cuda")[:, :V]
    r = dfl.rows(v)
    dfl.dflash_filter(r, v, out, dfl.rows_workspace(r), **_filters(st))
    got = _f64(out)
    for i in range(2):
        assert np.array_equal(got[i], O.filtered(zz[i], float(torch.finfo(t).min), **_as_used(st[i]))), i
    s, teacher, idx, tl = _distill_case(rng, 2, V, K, True, True, None)
    lse = np.array([O.log_sum_exp(x.astype(np.float64)) for x in teacher])
    _check_distill(s, idx, tl, t, 1.0, lse, None, None, pad=1, shift=1)
    _check_distill(s, idx, tl, t, 1.0, None, None, None, inplace=True)


@pytest.mark.parametrize("dt,R,V", [("bf16", 5, 1000), ("f32", 5, 1000), ("bf16", 5, 30001), ("f32", 5, 30001)])
def test_outputs_in_the_gaps_between_the_rows(dt, R, V):
    # input and output rows alternate in one allocation
    import torch
    import block_draft_select_amd as dfl
    t = _type(dt)
    rng = np.random.default_rng(85)
    both = torch.zeros(R, 2 * V + 1, dtype=t, device="cuda")
    v, out = both[:, :V], both[:, V:2 * V]
    s, _, idx, tl = _distill_case(rng, R, V, 5, False, False, None)
    v.copy_(torch.from_numpy(s))
    zz = _f64(v)
    r = dfl.rows(v)
    st = [dict(top_k=7), dict(top_p=0.5), dict(min_p=0.2), dict(), dict(T=0.0)]
    dfl.dflash_filter(r, v, out, dfl.rows_workspace(r), **_filters(st))
    got = _f64(out)
    for i in range(R):
        assert np.array_equal(got[i], O.filtered(zz[i], float(torch.finfo(t).min), **_as_used(st[i]))), i
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    _, _, _, alone = _run_distill(v.contiguous(), dev(idx), dev(tl), 1.0, None, None, None)
    _run_distill(v, dev(idx), dev(tl), 1.0, None, None, None, out)
    assert torch.equal(out, alone) and np.array_equal(_f64(v), zz) and not both[:, 2 * V].any()


def test_samples_and_filters_on_two_streams_at_once():
    # each call with a workspace of its own
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(86)
    for dt, R, V in (("bf16", 20, 50021), ("f32", 20, 50021), ("f32", 70, 100003)):
        z = torch.from_numpy(_logits(rng, R, V, "peaked")).cuda().to(_type(dt))
        u = torch.rand(R, dtype=torch.float64, device="cuda")
        f = _filters([MIX[i % len(MIX)] for i in range(R)])
        r = dfl.rows(z)
        ws = [dfl.rows_workspace(r) for _ in range(3)]
        token = [torch.full((R,), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
        out = [torch.empty_like(z) for _ in range(3)]
        side = [None, torch.cuda.Stream(), torch.cuda.Stream()]

        def call(i):
            dfl.dflash_sample(r, z, u, token[i], ws[i], stream=side[i], **f)
            dfl.dflash_filter(r, z, out[i], ws[i], stream=side[i], **f)

        call(0)
        torch.cuda.synchronize()
        for _ in range(5):
            call(1)
            call(2)
        torch.cuda.synchronize()
        for i in (1, 2):
            assert torch.equal(token[0], token[i]) and torch.equal(out[0], out[i]), (dt, R, i)
