"""GPU parity of the operators on logit rows (dflash_sample, dflash_filter,
dflash_distill, dflash_distill_grad) with the float64 oracle (oracle.rows).

Bars.  Tokens, kept counts and filtered rows: equal.  prob: half a step of
fp32 (2^-24 relative) plus 2^-40 for the fp64 sums.  lse: the library's
exponential is off by at most 1.4e-11 relative, so a log-sum-exp by 2e-11
absolute, plus 2^-49 of its own size.  loss: half a step of fp32 plus what lse
and 1 - sum p bring in (1e-10 of the terms' size).  Gradients: half a step of
the type, plus (|t| + 4) 2^-23 relative for the fp32 exponent t (|t| <= 126:
smaller ones flush to 0, off by 2^-126 of the factor).
"""

import sys

import numpy as np
import pytest

from oracle import rows as O

pytestmark = pytest.mark.gpu


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_select_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def _tensor(z, dtype, pad=0, shift=0):
    """z [R, V] on the GPU, `pad` elements between rows, `shift` elements after an aligned address; the gaps hold 777."""
    import torch
    R, V = z.shape
    flat = torch.full((R * (V + pad) + shift + 8,), 777.0, dtype=dtype, device="cuda")
    v = flat[shift:shift + R * (V + pad)].view(R, V + pad)[:, :V]
    v.copy_(torch.from_numpy(np.ascontiguousarray(z)).to(dtype))
    return v, flat


def _f64(t):
    return t.double().cpu().numpy()


def _arr(vals, dtype):
    import torch
    return torch.tensor(vals, dtype=dtype, device="cuda")


def _filters(settings):
    import torch
    return dict(T=_arr([s.get("T", 1.0) for s in settings], torch.float32),
                top_k=_arr([s.get("top_k", 0) for s in settings], torch.int32),
                top_p=_arr([s.get("top_p", 1.0) for s in settings], torch.float32),
                min_p=_arr([s.get("min_p", 0.0) for s in settings], torch.float32))


def _as_used(s):
    """The settings as the kernel sees them: rounded to fp32."""
    return {k: (int(v) if k == "top_k" else float(np.float32(v))) for k, v in s.items()}


def _check_sample(z, dtype, settings, u, pad=0, shift=0, group=1):
    import torch
    import block_draft_select_amd as dfl
    v, _ = _tensor(z, dtype, pad, shift)
    R = z.shape[0]
    r = dfl.rows(v)
    ws = torch.randint(0, 255, (dfl.rows_workspace_bytes(r),), dtype=torch.uint8, device="cuda")  # any contents
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    kept = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((R,), float("nan"), dtype=torch.float32, device="cuda")
    dfl.dflash_sample(r, v, _arr(list(u), torch.float64), token, ws, prob=prob, kept=kept, group=group, **_filters(settings))
    torch.cuda.synchronize()
    zz = _f64(v)
    for i in range(R):
        want = O.sample(np.minimum(zz[i], float(torch.finfo(dtype).max)), u[i], **_as_used(settings[i // group]))
        got = (int(token[i]), float(prob[i]), int(kept[i]))
        assert (got[0], got[2]) == (want[0], want[2]), f"row {i} {settings[i // group]} u={u[i]!r}: got {got}, want {want}"
        assert abs(got[1] - want[1]) <= want[1] * (2.0 ** -24 + 2.0 ** -40), (i, got, want)


MIX = [dict(), dict(T=0.6), dict(T=0.0), dict(top_k=1), dict(top_k=50, top_p=0.95), dict(T=0.7, top_k=20, top_p=0.9, min_p=0.05),
       dict(top_p=0.9), dict(top_p=0.5, T=1.5), dict(min_p=0.1), dict(min_p=1e-3, T=2.0), dict(top_k=100000), dict(top_p=0.0),
       dict(min_p=1.0), dict(T=float("nan")), dict(T=1e-30), dict(T=float("inf")), dict(T=50.0, top_p=0.97), dict(top_k=3, min_p=0.5)]


def _logits(rng, R, V, kind):
    z = rng.normal(size=(R, V)) * 2
    if kind == "peaked":
        for i in range(R):
            at = rng.integers(0, V, size=min(V, 24))
            z[i, at] += rng.uniform(4, 14, size=at.size)
    if kind == "ties":
        z = np.round(z)
    if kind == "masked":
        z[rng.random(size=z.shape) < 0.7] = -np.inf
        z[R // 2] = -np.inf
    if kind == "lowest":
        z[rng.random(size=z.shape) < 0.7] = -3.0e38
    if kind == "shifted":
        z += 5000.0
    if kind == "constant":
        z[:] = z[:, :1]
    return z.astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 65, 1000, 4096, 4104])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties", "masked"])
def test_sample_small_rows(dt, V, kind):
    import torch
    rng = np.random.default_rng(V * 31 + len(kind))
    z = _logits(rng, len(MIX), V, kind)
    _say(f"[rows] sample {dt} V={V} {kind}")
    _check_sample(z, dict(bf16=torch.bfloat16, f32=torch.float32)[dt], MIX, rng.random(len(MIX)), pad=V % 3, shift=V % 5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties", "masked", "lowest", "shifted"])
@pytest.mark.parametrize("V", [50021, 151936])
def test_sample_large_rows(dt, kind, V):
    import torch
    rng = np.random.default_rng(V + len(kind))
    z = _logits(rng, len(MIX), V, kind)
    _say(f"[rows] sample {dt} V={V} {kind}")
    _check_sample(z, dict(bf16=torch.bfloat16, f32=torch.float32)[dt], MIX, rng.random(len(MIX)), pad=3 if V % 2 else 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sample_constant_rows_and_dyadic_settings(dt):
    # every running sum is an exact multiple of one weight, so cuts and draws
    # at dyadic settings fall exactly on token borders
    import torch
    _say(f"[rows] constant rows {dt}")
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    st = [dict(top_p=0.5), dict(top_p=0.75, T=0.3), dict(top_k=512, top_p=0.25), dict(min_p=1.0), dict(T=3.0), dict(top_k=7000)]
    for V in (1000, 8192, 40000):
        z = np.repeat(np.array([[0.0], [3.25], [-7.5], [1.0e4], [0.3], [2.0]], dtype=np.float32), V, axis=1)
        _check_sample(z, t, st, np.array([0.0, 0.25, 0.5, 0.75, 0.999999, 1.0 - 2.0 ** -53]))


def test_sample_uniforms_at_their_ends_and_outside():
    import torch
    rng = np.random.default_rng(8)
    u = [0.0, -1.0, float("nan"), 1.0, 7.0, 1.0 - 2.0 ** -53, 2.0 ** -60]
    for st in (dict(), dict(top_k=5), dict(top_p=0.8), dict(T=0.5, min_p=0.2)):
        z = _logits(rng, len(u), 3001, "peaked")
        _check_sample(z, torch.bfloat16, [st] * len(u), np.array(u))


def test_sample_infinite_and_nan_logits():
    import torch
    rng = np.random.default_rng(9)
    z = _logits(rng, 8, 2000, "flat")
    z[0, 5] = z[0, 900] = np.inf
    z[1, ::2] = np.nan
    z[2] = np.nan
    z[3] = -np.inf
    z[4, :] = -np.inf
    z[4, 1999] = -3.0e38
    z[5, 0] = np.inf
    z[6] = np.inf
    z[7, 17] = np.nan
    for st in (dict(), dict(top_k=2), dict(top_p=0.4, T=0.8), dict(min_p=0.1), dict(T=0.0)):
        for t in (torch.bfloat16, torch.float32):
            _check_sample(z, t, [st] * 8, rng.random(8))


def test_sample_tail_and_tiny_min_p():
    # cuts far below the maximum: top-k and min-p between tokens whose weight
    # is under 2^-64 of the largest
    import torch
    rng = np.random.default_rng(10)
    z = rng.uniform(-300.0, -80.0, size=(6, 9001)).astype(np.float32)
    z[:, 4000] = 0.0
    z[:, 20] = -1.0
    st = [dict(top_k=3), dict(top_k=5000), dict(min_p=1e-38), dict(min_p=1e-44, T=2.0), dict(top_k=8000, min_p=1e-40, T=3.0),
          dict(min_p=1e-30, T=1.5)]
    for t in (torch.bfloat16, torch.float32):
        _check_sample(z, t, st, np.array([0.0, 0.5, 0.7, 0.72, 0.9, 0.99]))


def test_sample_group_shares_settings():
    import torch
    rng = np.random.default_rng(11)
    z = _logits(rng, 20, 5000, "peaked")
    _check_sample(z, torch.bfloat16, [dict(top_k=4), dict(top_p=0.5), dict(T=0.0)], rng.random(20), group=9)


def test_sample_many_rows_pass_through_the_workspace_in_batches():
    import torch
    rng = np.random.default_rng(12)
    R = 9001  # more rows than one pass over the workspace takes
    z = _logits(rng, R, 33, "flat")
    st = [MIX[i % len(MIX)] for i in range(R)]
    _check_sample(z, torch.bfloat16, st, rng.random(R), pad=1)


def test_sample_longest_vocabulary():
    import torch
    rng = np.random.default_rng(13)
    z = _logits(rng, 2, 2097152, "flat")
    _check_sample(z, torch.bfloat16, [dict(top_p=0.9), dict()], rng.random(2))
    _check_sample(np.zeros((1, 2097152), dtype=np.float32), torch.float32, [dict(top_p=0.5)], np.array([0.75]))


@pytest.mark.parametrize("kind", ["flat", "peaked", "ties", "masked", "shifted", "lowest", "constant"])
@pytest.mark.parametrize("R,V", [(260, 16003), (420, 16003), (520, 15998), (1030, 5003), (1300, 5003), (345, 40009)])
def test_sample_f32_rows_in_long_segments(kind, R, V):
    # many fp32 rows: segments of 2, 4 and 8 slots a thread list only their
    # largest tokens, and deep cuts ask for more
    import torch
    rng = np.random.default_rng(R + V + len(kind))
    z = _logits(rng, R, V, kind)
    _say(f"[rows] sample f32 R={R} V={V} {kind}")
    _check_sample(z, torch.float32, [MIX[i % len(MIX)] for i in range(R)], rng.random(R), pad=V % 2)


def test_filter_f32_rows_in_long_segments():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(41)
    for R, V, kind in ((420, 16003, "ties"), (1300, 5003, "flat"), (520, 15998, "peaked")):
        z = _logits(rng, R, V, kind)
        st = [MIX[i % len(MIX)] for i in range(R)]
        v, _ = _tensor(z, torch.float32)
        r = dfl.rows(v)
        dfl.dflash_filter(r, v, v, dfl.rows_workspace(r), **_filters(st))
        torch.cuda.synchronize()
        got, zz = _f64(v), z.astype(np.float64)
        for i, s in enumerate(st):
            assert np.array_equal(got[i], O.filtered(zz[i], torch.finfo(torch.float32).min, **_as_used(s))), (R, i, s)


DEEP = [dict(), dict(top_k=5000), dict(top_k=9000, T=0.5), dict(top_p=0.6, T=8.0), dict(min_p=0.9, T=30.0), dict(top_p=0.99, T=50.0),
        dict(min_p=0.999999, T=300.0), dict(top_p=0.5, T=float("inf")), dict(T=1e-3, top_p=0.9)]


@pytest.mark.parametrize("kind", ["zeros", "half zeros", "positive and zeros", "near zero", "near zero, few", "mixed", "over", "under",
                                  "over and masked"])
def test_bf16_values_at_the_ends_of_the_counters(kind):
    # exact zeros of both signs, magnitudes below the counters' range (listed
    # one by one, or too many for that), values over and under it
    import torch
    rng = np.random.default_rng(42 + len(kind))
    R, V = len(DEEP), 12007
    z = (rng.normal(size=(R, V)) * 2).astype(np.float32)
    if kind == "zeros":
        z[:] = 0.0
        z[:, ::3] = -0.0
    if kind == "half zeros":
        z[:, ::2] = 0.0
        z[:, ::6] = -0.0
    if kind == "positive and zeros":
        z = np.maximum(z, 0.0)
        z[:, 5:9] = 1e-7
    if kind == "near zero":
        z *= 1e-7
    if kind == "near zero, few":
        z[:, 100:140] *= 1e-8
        z[:, 11000:11012] *= 1e-12
        z[:, 7000:7300] = 0.0
    if kind == "mixed":
        z[:, ::5] = 0.0
        z[:, 1::700] = 1e-38
        z[:, 2::900] = -1e-30
        z[:, 3::800] = 1e-42  # subnormal
    if kind == "over":
        z += 900.0
    if kind == "under":
        z -= 90000.0
        z[:, 6000:] += 89000.0
    if kind == "over and masked":
        z[:, ::4] = -np.inf
        z[:, 1::4] = np.nan
        z[:, 2::4] *= 1e4
    v, _ = _tensor(z, torch.bfloat16)
    _say(f"[rows] bf16 {kind}")
    for u in (rng.random(R), 1.0 - rng.random(R) * 1e-3):
        _check_sample(z, torch.bfloat16, DEEP, u, pad=1)
    import block_draft_select_amd as dfl
    r = dfl.rows(v)
    zz = _f64(v)
    kept = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    dfl.dflash_filter(r, v, v, dfl.rows_workspace(r), kept=kept, **_filters(DEEP))
    torch.cuda.synchronize()
    got = _f64(v)
    for i, s in enumerate(DEEP):
        assert np.array_equal(got[i], O.filtered(zz[i], torch.finfo(torch.bfloat16).min, **_as_used(s))), (i, s)
        assert int(kept[i]) == O.keep(zz[i], **_as_used(s))[0].size


@pytest.mark.parametrize("dt,reps,V", [("bf16", 80, 150001), ("f32", 80, 150001), ("bf16", 462, 5001)])
def test_sample_does_not_depend_on_the_other_rows(dt, reps, V):
    # the same rows alone and among many, which are split differently and pass
    # through the workspace in batches
    import torch
    import block_draft_select_amd as dfl
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    rng = np.random.default_rng(43)
    n = len(MIX)
    z = torch.from_numpy(_logits(rng, n, V, "peaked")).cuda().to(t)
    u = torch.from_numpy(rng.random(n)).cuda()
    f = _filters(MIX)

    def run(z, u, f):
        R = z.shape[0]
        r = dfl.rows(z)
        token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
        kept, prob = torch.full_like(token, -7), torch.full((R,), -7.0, device="cuda")
        dfl.dflash_sample(r, z, u, token, dfl.rows_workspace(r), prob=prob, kept=kept, **f)
        torch.cuda.synchronize()
        return token, kept, prob

    one = run(z, u, f)
    many = run(z.repeat(reps, 1), u.repeat(reps), {k: v.repeat(reps) for k, v in f.items()})
    assert torch.equal(one[0].repeat(reps), many[0]) and torch.equal(one[1].repeat(reps), many[1])
    assert ((one[2].repeat(reps) - many[2]).abs() <= many[2] * 2.0 ** -23).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind,V,pad,shift,opad,oshift", [
    ("peaked", 1000, 0, 0, 0, 0), ("masked", 1003, 5, 3, 2, 1), ("ties", 50021, 3, 0, 3, 0), ("flat", 7, 1, 1, 0, 2),
    ("lowest", 20000, 0, 0, 8, 4), ("peaked", 1, 0, 0, 0, 0)])
def test_filter(dt, kind, V, pad, shift, opad, oshift):
    import torch
    import block_draft_select_amd as dfl
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    rng = np.random.default_rng(V + 1)
    R = len(MIX)
    v, _ = _tensor(_logits(rng, R, V, kind), t, pad, shift)
    out, flat = _tensor(np.zeros((R, V), dtype=np.float32), t, opad, oshift)
    r = dfl.rows(v)
    ws = dfl.rows_workspace(r)
    kept = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    _say(f"[rows] filter {dt} V={V} {kind}")
    dfl.dflash_filter(r, v, out, ws, fill=-16384.0, kept=kept, **_filters(MIX))
    torch.cuda.synchronize()
    got, zz = _f64(out), _f64(v)
    for i, s in enumerate(MIX):
        want = O.filtered(zz[i], -16384.0, **_as_used(s))
        assert np.array_equal(got[i], want), (i, s, int((got[i] != want).sum()))
        assert int(kept[i]) == O.keep(zz[i], **_as_used(s))[0].size
    # nothing outside the rows is written
    gap = flat.double().cpu().numpy()
    mask = np.ones(gap.size, dtype=bool)
    for i in range(R):
        mask[oshift + i * (V + opad): oshift + i * (V + opad) + V] = False
    assert (gap[mask] == gap[-1]).all()
    # in place, with the default fill
    dfl.dflash_filter(r, v, v, ws, **_filters(MIX))
    torch.cuda.synchronize()
    got = _f64(v)
    for i, s in enumerate(MIX):
        assert np.array_equal(got[i], O.filtered(zz[i], torch.finfo(t).min, **_as_used(s))), i


# ---------------------------------------------------------------- distillation

def _distill_case(rng, R, V, K, dup, pads, dtype, kind="peaked"):
    import torch
    s = _logits(rng, R, V, kind)
    t = (s * 0.5 + rng.normal(size=(R, V))).astype(np.float32)
    t[~np.isfinite(t)] = -50.0
    idx = np.argsort(-t, axis=1, kind="stable")[:, :K].astype(np.int32)
    tl = np.take_along_axis(t, idx.astype(np.int64), 1).astype(np.float32)
    if dup and K > 2:
        idx[:, 2] = idx[:, 0]
    if pads and K > 1:
        idx[::2, K // 2] = -1
        idx[1::2, K - 1] = V + 3
    return s, t, idx, tl


def _run_distill(v, idx, tl, tau, t_lse, weight, g, out=None):
    import torch
    import block_draft_select_amd as dfl
    R = v.shape[0]
    r = dfl.rows(v)
    ws = torch.randint(0, 255, (dfl.rows_workspace_bytes(r),), dtype=torch.uint8, device="cuda")
    loss = torch.full((R,), float("nan"), dtype=torch.float32, device="cuda")
    lse = torch.full((R,), float("nan"), dtype=torch.float64, device="cuda")
    rest = torch.full_like(lse, float("nan")) if t_lse is not None else None
    kw = dict(tau=tau, t_lse=t_lse, weight=weight, lse_rest=rest)
    dfl.dflash_distill(r, v, idx, tl, loss, lse, ws, **kw)
    dS = torch.empty_like(v) if out is None else out
    dfl.dflash_distill_grad(r, v, idx, tl, lse, dS, grad_loss=g, **kw)
    torch.cuda.synchronize()
    return loss, lse, rest, dS


def _grad_tol(ref, x, f, tau, dtype):
    """Element-wise bound on one row's gradient (the module's docstring; the
    two exponentials and p are fp64-accurate to 1e-10, also where they cancel)."""
    import torch
    half = torch.finfo(dtype).eps / 2
    rest = ref["lse_rest"] if ref["lse_rest"] is not None and ref["lse_rest"] > -np.inf else None
    base = ref["lse"] if rest is None else rest
    t = np.minimum(np.where(np.isfinite(x), np.abs(x - base) / np.log(2), 0.0), 126.0)
    parts = ref["A"] * np.exp(x - ref["lse"]) + ref["p"]
    if rest is not None:
        parts = parts + np.where(ref["p"] > 0, 0.0, ref["p_rest"] * np.exp(np.minimum(x - rest, 0.0)))
    return f * (np.abs(ref["grad"]) * (half + (t + 4) * 2.0 ** -23) + 1e-10 * parts / tau) + 2.0 ** -125 * (1 + f * (1 + ref["A"]))


def _check_distill(s, idx, tl, dtype, tau, t_lse_np, weight_np, g_np, pad=0, shift=0, inplace=False, opad=None):
    import torch
    v, _ = _tensor(s, dtype, pad, shift)
    zz = _f64(v)
    R, V = zz.shape
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out, flat = (v, None) if inplace else _tensor(np.zeros((R, V), dtype=np.float32), dtype, pad if opad is None else opad,
                                                  shift if opad is None else 1)
    loss, lse, rest, dS = _run_distill(v, dev(idx), dev(tl), tau, dev(t_lse_np), dev(weight_np), dev(g_np), out)
    got = _f64(dS)
    for i in range(R):
        w = 1.0 if weight_np is None else float(weight_np[i])
        g = 1.0 if g_np is None else float(g_np[i])
        if w == 0:
            assert float(loss[i]) == 0 and float(lse[i]) == 0 and not got[i].any()
            continue
        ref = O.distill(zz[i], idx[i], tl[i], tau, None if t_lse_np is None else t_lse_np[i])

        def near(a, b):
            return a == b or abs(a - b) <= 2e-11 + abs(b) * 2.0 ** -49

        assert near(float(lse[i]), ref["lse"]), (i, float(lse[i]), ref["lse"])
        if rest is not None:
            assert near(float(rest[i]), ref["lse_rest"]), (i, float(rest[i]), ref["lse_rest"])
        want = w * ref["loss"]
        size = abs(w) * (1.0 + abs(ref["lse"]) + np.abs(tl[i][np.abs(tl[i]) < 1e30] / tau).max(initial=0.0))
        assert float(loss[i]) == want or abs(float(loss[i]) - want) <= abs(want) * 2.0 ** -24 + 1e-10 * size + 2.0 ** -149, \
            (i, float(loss[i]), want)
        f = abs(w * g)
        x = zz[i] / tau
        if ref["lse"] == -np.inf or ref["A"] == 0:  # an empty row on either side
            assert not got[i].any()
            continue
        err = np.abs(got[i] - w * g * ref["grad"])
        tol = _grad_tol(ref, x, f, tau, dtype)
        bad = np.flatnonzero(~(err <= tol))
        assert bad.size == 0, (i, bad[:5], got[i][bad[:5]], (w * g * ref["grad"])[bad[:5]], tol[bad[:5]])


SHAPES = [  # R, V, K, pad, shift
    (3, 1, 1, 0, 0), (4, 2, 1, 1, 1), (5, 7, 3, 0, 0), (5, 8, 8, 0, 0), (4, 9, 4, 2, 3), (6, 65, 64, 0, 0), (7, 1000, 16, 0, 0),
    (5, 1003, 33, 5, 3), (3, 50021, 64, 3, 0), (2, 151936, 16, 0, 0), (3, 20000, 1024, 0, 0), (2, 4099, 256, 1, 7)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("R,V,K,pad,shift", SHAPES)
def test_distill_and_gradient(dt, with_lse, R, V, K, pad, shift):
    import torch
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    rng = np.random.default_rng(V * 7 + K + with_lse)
    tau = [1.0, 2.0, 0.7][(V + K) % 3]
    s, teacher, idx, tl = _distill_case(rng, R, V, K, dup=V % 2 == 1, pads=V % 3 == 1, dtype=t)
    lse = np.array([O.log_sum_exp(x.astype(np.float64) / tau) for x in teacher]) if with_lse else None
    w = rng.uniform(0.2, 2.0, size=R).astype(np.float32)
    w[R // 2] = 0.0
    g = rng.normal(size=R).astype(np.float32)
    _say(f"[rows] distill {dt} R={R} V={V} K={K} rest={with_lse}")
    _check_distill(s, idx, tl, t, tau, lse, w, g, pad, shift)
    _check_distill(s, idx, tl, t, tau, lse, None, None, pad, shift, opad=pad + 1)
    _check_distill(s, idx, tl, t, tau, lse, w, g, pad, shift, inplace=True)


@pytest.mark.parametrize("dt,R,V,K", [("bf16", 260, 1000, 16), ("bf16", 260, 4003, 100), ("bf16", 300, 8195, 64), ("bf16", 520, 16411, 16),
                                     ("f32", 300, 4099, 65), ("f32", 520, 8203, 16)])
def test_distill_and_gradient_of_many_rows(dt, R, V, K):
    # one, two, four and eight slots a thread in the gradient
    import torch
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    rng = np.random.default_rng(R + V + K)
    s, teacher, idx, tl = _distill_case(rng, R, V, K, dup=True, pads=True, dtype=t)
    w = rng.uniform(0.2, 2.0, size=R).astype(np.float32)
    w[::7] = 0.0
    _say(f"[rows] distill {dt} R={R} V={V} K={K}")
    for with_lse in (False, True):
        lse = np.array([O.log_sum_exp(x.astype(np.float64)) for x in teacher]) if with_lse else None
        _check_distill(s, idx, tl, t, 1.0, lse, w, None, pad=V % 2, inplace=with_lse)


@pytest.mark.parametrize("with_lse", [False, True])
def test_distill_masked_and_empty_rows(with_lse):
    import torch
    rng = np.random.default_rng(21)
    s, teacher, idx, tl = _distill_case(rng, 8, 900, 12, False, True, None, "masked")
    s[np.arange(8)[:, None], np.clip(idx, 0, 899)] = 0.25  # listed tokens stay possible
    s[4] = -np.inf                                            # an empty student row
    idx[5] = -1                                               # an empty list
    tl[6] = -np.inf
    tl[7, 3] = -np.inf
    lse = np.array([O.log_sum_exp(x.astype(np.float64)) for x in teacher]) if with_lse else None
    if with_lse:
        lse[2], lse[3] = -np.inf, np.inf                      # teacher rows without a normaliser
    for t in (torch.bfloat16, torch.float32):
        _check_distill(s, idx, tl, t, 1.0, lse, None, None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_the_types_lowest_value(dt):
    # a mask of finite lowest values that leaves nothing, some, or only listed
    # tokens; and logits beyond fp64's reach on the other side
    import torch
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dt]
    low = float(torch.finfo(t).min)
    rng = np.random.default_rng(61)
    V = 20005
    s = np.full((6, V), low, dtype=np.float32)
    idx = np.tile(np.array([[3, 19000, 7]], dtype=np.int32), (6, 1))
    tl = np.ones((6, 3), dtype=np.float32)
    s[1, 100:200] = rng.normal(size=100)      # only unlisted tokens remain (the listed ones are unlikely beyond fp32)
    s[2, [3, 19000, 7]] = rng.normal(size=3)  # only listed ones
    s[3] = rng.normal(size=V)
    s[3, ::2] = low
    s[3, [3, 19000, 7]] = rng.normal(size=3)
    s[4, 20004] = 0.5
    _say(f"[rows] lowest values {dt}")
    for with_lse in (False, True):
        lse = np.full(6, 2.5) if with_lse else None
        keep = [0, 2, 3, 5]
        _check_distill(s[keep], idx[keep], tl[keep], t, 0.8, None if lse is None else lse[keep], None, None)
    z = s.copy()
    z[5] = low
    st = [dict(top_p=0.5), dict(), dict(top_k=2), dict(min_p=0.1), dict(), dict(top_k=7, T=0.01)]
    _check_sample(z, t, st, rng.random(6))
    import block_draft_select_amd as dfl
    big = np.full((1, 3000), -1.0, dtype=np.float32)
    big[0, 5] = 3e38
    v, _ = _tensor(big, t)
    lse = torch.zeros(1, dtype=torch.float64, device="cuda")
    r = dfl.rows(v)
    dfl.dflash_distill(r, v, None, None, None, lse, dfl.rows_workspace(r))
    assert torch.isnan(lse).all()


@pytest.mark.parametrize("K", [2, 40, 100])
def test_lists_of_the_lowest_value(K):
    # a teacher's list that a finite mask leaves without mass, and one with some
    import torch
    rng = np.random.default_rng(64)
    s, _, idx, tl = _distill_case(rng, 4, 500, K, False, False, None)
    tl[0] = tl[2] = -3.0e38
    tl[2, 1] = 0.5
    tl[3] = -np.inf
    for t in (torch.bfloat16, torch.float32):
        _check_distill(s, idx, tl, t, 0.7, None, None, None)
        _check_distill(s, idx, tl, t, 0.7, np.full(4, 6.0), None, None)


def test_rows_past_32_bit_offsets():
    # two rows 2^31 elements apart
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(62)
    V, stride = 4999, 2 ** 31 + 3
    flat = torch.empty(stride + V + 8, dtype=torch.bfloat16, device="cuda")
    v = flat.as_strided((2, V), (stride, 1), 1)
    z = _logits(rng, 2, V, "peaked")
    v.copy_(torch.from_numpy(z))
    zz = _f64(v)
    r = dfl.rows(v)
    assert r.stride == stride
    ws = dfl.rows_workspace(r)
    u = torch.rand(2, dtype=torch.float64, device="cuda")
    token = torch.empty(2, dtype=torch.int32, device="cuda")
    p = _arr([0.9, 0.9], torch.float32)
    dfl.dflash_sample(r, v, u, token, ws, top_p=p)
    for i in range(2):
        assert int(token[i]) == O.sample(zz[i], float(u[i]), top_p=float(np.float32(0.9)))[0]
    idx = torch.from_numpy(np.argsort(-zz, axis=1)[:, :8].astype(np.int32)).cuda()
    tl = torch.gather(v.float(), 1, idx.long())
    loss, lse, _, dS = _run_distill(v, idx, tl, 1.0, None, None, None, flat.as_strided((2, V), (stride, 1), 1))
    for i in range(2):
        ref = O.distill(zz[i], idx[i].cpu().numpy(), tl[i].cpu().numpy())
        assert abs(float(lse[i]) - ref["lse"]) <= 2e-11 + 1e-13
        err = np.abs(_f64(dS)[i] - ref["grad"])
        assert (err <= _grad_tol(ref, zz[i], 1.0, 1.0, torch.bfloat16)).all()
    v.copy_(torch.from_numpy(z))
    dfl.dflash_filter(r, v, v, ws, top_p=p)
    got = _f64(v)
    for i in range(2):
        assert np.array_equal(got[i], O.filtered(zz[i], torch.finfo(torch.bfloat16).min, top_p=float(np.float32(0.9))))


def test_settings_and_outputs_left_out():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(63)
    for t in (torch.bfloat16, torch.float32):
        z = _logits(rng, 5, 3000, "peaked")
        v, _ = _tensor(z, t)
        zz, u = _f64(v), rng.random(5)
        r = dfl.rows(v)
        token = torch.empty(5, dtype=torch.int32, device="cuda")
        dfl.dflash_sample(r, v, _arr(list(u), torch.float64), token, dfl.rows_workspace(r))
        assert [int(x) for x in token] == [O.sample(zz[i], u[i])[0] for i in range(5)]
        out = torch.empty_like(v)
        dfl.dflash_filter(r, v, out, dfl.rows_workspace(r))
        assert np.array_equal(_f64(out), zz)


def test_distill_whole_vocabulary_listed():
    # no unlisted token: the rest class is left out
    import torch
    rng = np.random.default_rng(22)
    V = 40
    s = rng.normal(size=(3, V)).astype(np.float32)
    idx = np.tile(np.arange(V, dtype=np.int32), (3, 1))
    tl = rng.normal(size=(3, V)).astype(np.float32)
    lse = np.array([O.log_sum_exp(x.astype(np.float64)) + 0.1 for x in tl])
    for t in (torch.bfloat16, torch.float32):
        _check_distill(s, idx, tl, t, 1.0, lse, None, None)


def test_distill_confident_student_keeps_its_rest():
    # the listed token leads by 60 nats and more: the unlisted share is far
    # below the rounding of the total, and its gradient still comes out
    import torch
    rng = np.random.default_rng(23)
    s = rng.normal(size=(4, 3000)).astype(np.float32)
    idx = np.tile(np.array([[7, 2000]], dtype=np.int32), (4, 1))
    s[:, 7] = [40.0, 60.0, 100.0, 300.0]
    tl = np.tile(np.array([[2.0, 1.0]], dtype=np.float32), (4, 1))
    lse = np.full(4, 2.6)
    for t in (torch.bfloat16, torch.float32):
        _check_distill(s, idx, tl, t, 1.0, lse, None, None)


def test_distill_nan_and_infinite_student():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(24)
    s = rng.normal(size=(5, 5000)).astype(np.float32)
    s[1, 4000], s[2, 3], s[3, 4] = np.nan, np.inf, -np.inf
    idx = np.tile(np.array([[4, 17]], dtype=np.int32), (5, 1))
    tl = np.ones((5, 2), dtype=np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for t_lse in (None, dev(np.full(5, 2.0))):
        for t in (torch.bfloat16, torch.float32):
            v, _ = _tensor(s, t)
            w = torch.ones(5, device="cuda")
            w[2] = 0.0  # not read
            loss, lse, rest, dS = _run_distill(v, dev(idx), dev(tl), 1.0, t_lse, w, None)
            loss, dS = loss.cpu(), dS.float().cpu()
            assert torch.isfinite(loss[[0, 2, 4]]).all() and torch.isnan(loss[1]) and float(loss[3]) == float("inf")
            assert torch.isfinite(dS[[0, 2, 3, 4]]).all() and not dS[2].any() and torch.isnan(dS[1]).any()
    dfl.dflash_profile_enable(0)


def test_lse_alone_is_the_teachers_normaliser():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(25)
    z = _logits(rng, 6, 7777, "peaked")
    for t in (torch.bfloat16, torch.float32):
        v, _ = _tensor(z, t, 1, 1)
        r = dfl.rows(v)
        lse = torch.empty(6, dtype=torch.float64, device="cuda")
        dfl.dflash_distill(r, v, None, None, None, lse, dfl.rows_workspace(r), tau=0.8)
        for i, x in enumerate(_f64(v)):
            assert abs(float(lse[i]) - O.log_sum_exp(x / 0.8)) <= 2e-11 + 1e-14 * abs(float(lse[i]))


def test_gradient_against_differences():
    # central differences of the library's own loss, in fp32 logits: h = 2^-5
    # keeps the third-order term below h^2 / 6 of the largest third derivative
    # (each softmax derivative is at most 1), the loss's rounding below
    # 2^-24 loss / h
    import torch
    rng = np.random.default_rng(26)
    V, K = 300, 6
    s, teacher, idx, tl = _distill_case(rng, 1, V, K, False, False, None)
    h = 2.0 ** -5
    at = np.concatenate([idx[0, :3], rng.choice(V, 5, replace=False).astype(np.int32)])
    many = np.repeat(s, 1 + 2 * len(at), axis=0)
    for n, j in enumerate(at):
        many[1 + 2 * n, j] += np.float32(h)
        many[2 + 2 * n, j] -= np.float32(h)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    R = many.shape[0]
    t_lse = np.full(R, O.log_sum_exp(teacher[0].astype(np.float64)))
    for lse in (None, dev(t_lse)):
        v, _ = _tensor(many, torch.float32)
        loss, _, _, dS = _run_distill(v, dev(np.repeat(idx, R, 0)), dev(np.repeat(tl, R, 0)), 1.0, lse, None, None)
        loss, g = _f64(loss), _f64(dS)[0]
        zz = many.astype(np.float64)
        for n, j in enumerate(at):
            step = zz[1 + 2 * n, j] - zz[2 + 2 * n, j]
            d = (loss[1 + 2 * n] - loss[2 + 2 * n]) / step
            assert abs(d - g[j]) <= h * h / 6 * 2 + 2.0 ** -23 * max(1.0, abs(loss[0])) / h, (j, d, g[j])


# ---------------------------------------------------------------- streams, graphs, the operators together

@pytest.mark.parametrize("dt,V", [("bf16", 50021), ("f32", 50021), ("f32", 400007)])
def test_sample_and_filter_replayed_from_a_graph(dt, V):
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(31)
    z = torch.from_numpy(_logits(rng, 18, V, "peaked")).cuda().to(dict(bf16=torch.bfloat16, f32=torch.float32)[dt])
    st = _filters(MIX)
    u = torch.rand(18, dtype=torch.float64, device="cuda")
    r = dfl.rows(z)
    outs = [dict(token=torch.zeros(18, dtype=torch.int32, device="cuda"), prob=torch.zeros(18, device="cuda"),
                 kept=torch.zeros(18, dtype=torch.int32, device="cuda"), out=torch.zeros_like(z)) for _ in range(3)]
    ws = [dfl.rows_workspace(r) for _ in range(3)]

    def call(k):
        o = outs[k]
        dfl.dflash_sample(r, z, u, o["token"], ws[k], prob=o["prob"], kept=o["kept"], **st)
        dfl.dflash_filter(r, z, o["out"], ws[k], **st)

    call(0)
    torch.cuda.synchronize()
    graphs = []
    for k in (1, 2):  # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(k)
        graphs.append(g)
    for rep in range(4):
        # new inputs in place, other eager work between the replays
        z.copy_(torch.from_numpy(_logits(rng, 18, V, "peaked" if rep % 2 else "ties")).cuda())
        u.copy_(torch.rand(18, dtype=torch.float64, device="cuda"))
        call(0)
        torch.cuda.synchronize()
        for k, g in zip((1, 2), graphs):
            for v in outs[k].values():
                v.fill_(-3)
            g.replay()
        torch.cuda.synchronize()
        for k in (1, 2):
            for name in outs[0]:
                assert torch.equal(outs[0][name], outs[k][name]), (rep, k, name)
        _say(f"[rows] replay {rep}: equal to the eager call")


def test_distill_replayed_from_a_graph_and_on_another_stream():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(32)
    s, teacher, idx, tl = _distill_case(rng, 9, 20011, 16, False, True, None)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    v, idx, tl = dev(s).to(torch.bfloat16), dev(idx), dev(tl)
    t_lse = dev(np.array([O.log_sum_exp(x.astype(np.float64)) for x in teacher]))
    r = dfl.rows(v)

    def new():
        return dict(loss=torch.zeros(9, device="cuda"), lse=torch.zeros(9, dtype=torch.float64, device="cuda"),
                    rest=torch.zeros(9, dtype=torch.float64, device="cuda"), dS=torch.zeros_like(v), ws=dfl.rows_workspace(r))

    def call(o, stream=None):
        dfl.dflash_distill(r, v, idx, tl, o["loss"], o["lse"], o["ws"], t_lse=t_lse, lse_rest=o["rest"], stream=stream)
        dfl.dflash_distill_grad(r, v, idx, tl, o["lse"], o["dS"], t_lse=t_lse, lse_rest=o["rest"], stream=stream)

    eager, graph, side = new(), new(), new()
    call(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(graph)
    st = torch.cuda.Stream()
    for rep in range(3):
        v.copy_(dev(_logits(rng, 9, 20011, "peaked")))
        call(eager)
        torch.cuda.synchronize()
        call(side, st)  # two calls at once, each with its own workspace
        g.replay()
        torch.cuda.synchronize()
        for k in ("loss", "lse", "rest", "dS"):
            assert torch.equal(eager[k], graph[k]), (rep, k)
            assert torch.equal(eager[k], side[k]), (rep, k)


def test_filtered_cycle_follows_the_filtered_target():
    # the operators as a serving engine uses them: the first token from the
    # prompt's last target row, then a cycle whose target rows are filtered.
    # The cycle on the filtered rows equals the cycle on rows that the oracle
    # filtered, and every token it draws is one that the filters keep
    import torch
    import block_draft_select_amd as dfl
    import synth
    from gpu_util import alloc_outputs, device_inputs, dims_of
    inp = synth.make(3, set_id=51, B=6, V=20008, hidden=256)
    B, L, V = inp["B"], inp["L"], inp["V"]
    d, dev = dims_of(inp), device_inputs(inp)
    Z = dev["Z"].view(B, L + 1, V)
    prompt = Z[:, L]  # any target rows: the last of each stream, a strided view
    settings = [dict(top_k=20), dict(top_p=0.3), dict(min_p=0.2), dict(top_k=50, top_p=0.8, min_p=0.01), dict(), dict(T=0.0)]
    f = _filters(settings)
    x0 = torch.empty(B, dtype=torch.int32, device="cuda")
    u = torch.rand(B, dtype=torch.float64, device="cuda")
    rp = dfl.rows(prompt)
    dfl.dflash_sample(rp, prompt, u, x0, dfl.rows_workspace(rp), **f)
    for b in range(B):
        assert int(x0[b]) == O.sample(_f64(prompt)[b], float(u[b]), **_as_used(settings[b]))[0]
    Zf = torch.empty_like(Z)
    r = dfl.rows(Z)
    dfl.dflash_filter(r, Z, Zf, dfl.rows_workspace(r), group=L + 1, **f)
    ref = Z.clone()
    zz = _f64(Z)
    low = float(torch.finfo(torch.bfloat16).min)
    for b in range(B):
        for t in range(L + 1):
            ref[b, t] = torch.from_numpy(O.filtered(zz[b, t], low, **_as_used(settings[b]))).to(torch.bfloat16)
    assert torch.equal(Zf, ref)
    got = []
    for target in (Zf, ref):
        o = alloc_outputs(inp)
        dfl.dflash_cycle(d, dev["U"], target, x0, dev["E"], dev["W"], dev["h"], f["T"], dev["seed"], inp["cycle"],
                         o["accept_len"], o["out_tok"], dfl.workspace(d))
        torch.cuda.synchronize()
        got.append((o["accept_len"].cpu().numpy(), o["out_tok"].cpu().numpy()))
    assert np.array_equal(got[0][0], got[1][0]) and np.array_equal(got[0][1], got[1][1])
    for b in range(B):
        for t in range(int(got[0][0][b]) + 1):
            assert got[0][1][b, t] in O.keep(zz[b, t], **_as_used(settings[b]))[0], (b, t)


def test_training_step_from_the_targets_own_lists():
    # a drafter's step: the target's lists by dflash_topk, its normaliser by
    # dflash_distill with no list, the loss and its gradient; one step down the
    # gradient is the fp64 one
    import torch
    import block_draft_select_amd as dfl
    import synth
    from gpu_util import device_inputs
    inp = synth.make(3, set_id=52, B=2, L=4, V=8192, hidden=64)
    B, L, V, K = inp["B"], inp["L"], inp["V"], inp["K"]
    dev = device_inputs(inp)
    U = dev["U"].view(B * L, V)
    target = dev["Z"].view(B, L + 1, V)[:, :L].contiguous()
    d = dfl.dims(B, L, V, K, inp["r"], inp["hidden"], "bf16", "bf16")
    idx = torch.empty(B * L, K, dtype=torch.int32, device="cuda")
    tl = torch.empty(B * L, K, dtype=torch.float32, device="cuda")
    dfl.dflash_topk(d, target, idx, tl, dfl.workspace(d))
    rt, r = dfl.rows(target), dfl.rows(U)
    t_lse = torch.empty(B * L, dtype=torch.float64, device="cuda")
    ws = dfl.rows_workspace(r)
    dfl.dflash_distill(rt, target, None, None, None, t_lse, ws)
    torch.cuda.synchronize()
    zt = _f64(target).reshape(B * L, V)
    for i in range(B * L):
        assert abs(float(t_lse[i]) - O.log_sum_exp(zt[i])) <= 2e-11 + 1e-14 * 20
    _check_distill(U.float().cpu().numpy(), idx.cpu().numpy(), tl.cpu().numpy(), torch.bfloat16, 1.0, t_lse.cpu().numpy(),
                   None, None)


def test_outputs_on_another_device_or_type_are_refused():
    import torch
    import block_draft_select_amd as dfl
    z = torch.zeros(3, 64, device="cuda")
    r = dfl.rows(z)
    ws = dfl.rows_workspace(r)
    u = torch.zeros(3, dtype=torch.float64, device="cuda")
    token = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(u=u.float()), dict(token=token.long()), dict(T=torch.ones(2, device="cuda")), dict(kept=token[:2]),
                dict(u=u.cpu()), dict(ws=ws.cpu()), dict(top_k=torch.ones(3, device="cuda")), dict(group=0)):
        kw = dict(u=u, token=token, ws=ws)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, dfl.DFlashError)):
            dfl.dflash_sample(r, z, **kw)
    for out in (z[:, :32], z.to(torch.bfloat16), z.cpu(), torch.zeros(4, 64, device="cuda")):
        with pytest.raises((TypeError, ValueError, dfl.DFlashError)):
            dfl.dflash_filter(r, z, out, ws)
