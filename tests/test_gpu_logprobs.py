"""GPU parity of dflash_logprobs and dflash_logprobs_grad with the float64
oracle (oracle.rows).

Bars.  Alternatives' tokens: equal.  With t_i the exponent of two of a term
(log2 of p_i over the largest, plus at most 1/2 for the whole-number reference),
a term is off by t_i's rounding (2^-24 |t_i| ln 2), the constant's (2^-25 |t_i|
ln 2), the exponential's last bit (2^-23) and ten fp32 additions (10 * 2^-24);
l by the terms' mean under p, the entropy by their mean times |log p_i + H| and
the products' additions (11 * 2^-24 of sum p_i |t_i| ln 2).  Each output is
rounded once (2^-24).  Gradients: half a step of the type, plus, for p from an
fp32 exponent, (|log2 p| + 4) 2^-23 of the terms' size; what lies below 2^-126
of the factor may flush to 0.
"""

import sys

import numpy as np
import pytest

from oracle import rows as O

pytestmark = pytest.mark.gpu

LN2 = np.log(2.0)
LOWEST = -3.3895313892515355e38  # of bf16, a value of fp32 too


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


def _type(name):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[name]


def _tensor(z, dtype, pad=0, shift=0):
    """z [R, V] on the GPU, `pad` elements between rows, `shift` elements after an aligned address; the gaps hold 777."""
    import torch
    R, V = z.shape
    flat = torch.full((R * (V + pad) + shift + 8,), 777.0, dtype=dtype, device="cuda")
    v = flat[shift:shift + R * (V + pad)].view(R, V + pad)[:, :V]
    v.copy_(torch.from_numpy(np.ascontiguousarray(z)).to(dtype))
    return v, flat


def _gpu_arr(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)


def _f64(t):
    return t.double().cpu().numpy()


def _bars(logp, H):
    """(what l may be off by, what the entropy may be) of one row"""
    p = np.exp(logp)
    on = p > 0
    p, lp = p[on], logp[on]
    t = (lp.max() - lp) / LN2 + 0.5
    e = t * LN2 * 1.5 * 2.0 ** -24 + 2.0 ** -23 + 10 * 2.0 ** -24
    return float((p * e).sum()), float((p * e * np.abs(lp + H)).sum() + 11 * 2.0 ** -24 * (p * t).sum() * LN2)


def forward(v, tok, N, T=None, group=1, ent=True, stream=None, ws=None):
    import torch
    import block_draft_select_amd as dfl
    r = dfl.rows(v)
    R = r.R
    if ws is None:
        ws = torch.randint(0, 255, (max(dfl.rows_workspace_bytes(r), 16),), dtype=torch.uint8, device="cuda")  # any contents
    M = tok.shape[1]
    out = dict(logp=torch.full((R, M), 7.0, dtype=torch.float32, device="cuda") if M else None,
               norm=torch.full((R, 2), 7.0, dtype=torch.float32, device="cuda"),
               entropy=torch.full((R,), 7.0, dtype=torch.float32, device="cuda") if ent else None,
               top_idx=torch.full((R, N), 7, dtype=torch.int32, device="cuda") if N else None,
               top_logp=torch.full((R, N), 7.0, dtype=torch.float32, device="cuda") if N else None)
    dfl.dflash_logprobs(r, v, tok if M else None, out["logp"], out["norm"], ws, T=T, group=group, entropy=out["entropy"],
                        top_idx=out["top_idx"], top_logp=out["top_logp"], stream=stream)
    return out


def close(got, want, bar, what):
    got, want = float(got), float(want)
    if abs(want) >= 3.4028235677973366e38:  # rounds to an infinity of fp32 (largest value plus half a step)
        want = float(np.copysign(np.inf, want))
    if not np.isfinite(want):
        assert got == want or (np.isnan(got) and np.isnan(want)), (what, got, want)
    else:
        assert abs(got - want) <= bar + abs(want) * 2.0 ** -24, (what, got, want, abs(got - want), bar)


def check(z, dt, tok, N, T=None, group=1, pad=0, shift=0, ent=True, rows_=None):
    import torch
    v, _ = _tensor(z, _type(dt), pad, shift)
    t = None if T is None else _gpu_arr(np.asarray(T, np.float32), torch.float32)
    o = forward(v, _gpu_arr(tok, torch.int32), N, t, group, ent)
    torch.cuda.synchronize()
    zz = _f64(v)
    got = {k: None if x is None else x.cpu().numpy() for k, x in o.items()}
    for i in range(z.shape[0]) if rows_ is None else rows_:
        Ti = 1.0 if T is None else float(np.float32(T[i // group]))
        want = O.logprobs(zz[i], tok[i], N, Ti)
        bl, bh = _bars(O.distribution(zz[i], Ti)[2], want["entropy"]) if np.isfinite(want["norm"][0]) else (0.0, 0.0)
        what = f"row {i} T={Ti}"
        close(got["norm"][i, 0], want["norm"][0], 0.0, what + " m")
        close(got["norm"][i, 1], want["norm"][1], bl, what + " l")
        if ent:
            close(got["entropy"][i], want["entropy"], bh, what + " H")
        for k in range(tok.shape[1]):
            close(got["logp"][i, k], want["logp"][k], bl, what + f" token {tok[i, k]}")
        if N:
            assert np.array_equal(got["top_idx"][i], want["top_idx"]), (what, got["top_idx"][i], want["top_idx"])
            for k in range(N):
                close(got["top_logp"][i, k], want["top_logp"][k], bl, what + f" alternative {k}")
    return v, o


def logits(rng, R, V, kind):
    z = rng.normal(size=(R, V)) * 2
    if kind == "peaked":
        for i in range(R):
            z[i, rng.integers(0, V, size=min(V, 24))] += rng.uniform(4, 14)
    if kind == "ties":
        z = np.round(z)
    if kind == "masked":
        z[rng.random(size=z.shape) < 0.7] = -np.inf
        z[R // 2] = -np.inf
    if kind == "lowest":
        z[rng.random(size=z.shape) < 0.7] = LOWEST
        z[R // 2] = LOWEST
    if kind == "shifted":
        z += 5000.0
    if kind == "negative":
        z -= 300.0
    if kind == "constant":
        z[:] = z[:, :1]
    if kind == "odd":
        z[0, V // 2] = np.nan
        z[R // 2, V - 1] = np.inf
        z[R - 1] = -np.inf
        z[R - 1, 0] = np.nan
    if kind == "down":
        z = np.sort(z, 1)[:, ::-1].copy()
    if kind == "up":
        z = np.sort(z, 1)
    return z.astype(np.float32)


def tokens(rng, R, V, M):
    tok = rng.integers(0, V, size=(R, M))
    if M > 1:
        tok[:, -1] = -1
    if M > 3:
        tok[:, 1] = tok[:, 0]
        tok[:, 2] = V
    return tok


KINDS = ["flat", "peaked", "ties", "masked", "lowest", "shifted", "negative", "constant", "odd", "down", "up"]
TS = [1.0, 0.6, 0.0, 2.5, 0.05]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 65, 1000, 2049, 8193])
@pytest.mark.parametrize("kind", KINDS)
def test_short_rows(dt, V, kind):
    rng = np.random.default_rng(V * 31 + len(kind))
    R = 5
    _say(f"[logprobs] {dt} V={V} {kind}")
    check(logits(rng, R, V, kind), dt, tokens(rng, R, V, 5), 20, T=TS, pad=V % 3, shift=V % 5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,N", [(50021, 32), (151936, 5)])
def test_long_rows(dt, kind, V, N):
    rng = np.random.default_rng(V + len(kind))
    _say(f"[logprobs] {dt} V={V} {kind} N={N}")
    check(logits(rng, 3, V, kind), dt, tokens(rng, 3, V, 2), N, T=[1.0, 0.7, 1.3], pad=3 if V % 2 else 0)


@pytest.mark.parametrize("kind", ["flat", "ties", "constant", "down", "odd", "masked"])
@pytest.mark.parametrize("dt,R,V", [("bf16", 2050, 20000), ("f32", 2050, 9001), ("bf16", 300, 30011), ("f32", 1030, 20000),
                                    ("bf16", 300, 140011), ("f32", 129, 270001), ("bf16", 40, 140011)])
def test_many_rows(dt, R, V, kind):
    # one block a row, and segments of rows; the oracle looks at some of the rows
    rng = np.random.default_rng(R + V)
    z = np.tile(logits(rng, 25, V, kind), (R // 25 + 1, 1))[:R]
    _say(f"[logprobs] {dt} {R} x {V} {kind}")
    check(z, dt, tokens(rng, R, V, 1), 20, rows_=list(range(0, 25)) + [R // 2, R - 1])


@pytest.mark.parametrize("N", [1, 2, 31, 32])
@pytest.mark.parametrize("M", [0, 1, 300, 1024])
def test_counts(N, M):
    rng = np.random.default_rng(N * 7 + M)
    check(logits(rng, 2, 12000, "peaked"), "bf16", tokens(rng, 2, 12000, M), N)
    check(logits(rng, 2, 900, "peaked"), "f32", tokens(rng, 2, 900, M), 0, ent=False)


def test_one_thread_holds_all_alternatives():
    # every large logit lies in the places that one thread loads (a thread's slots
    # come round every 4 x 256 of 16 bytes), more of them than its list of pieces holds
    rng = np.random.default_rng(5)
    for dt, ve in (("bf16", 8), ("f32", 4)):
        V = 120000
        z = rng.normal(size=(2060, V) if dt == "bf16" else (2, V)).astype(np.float32)
        at = np.arange(0, V - ve, 256 * ve)  # slot 0, 256, ... of thread 0
        z[:2, at] = 20 + rng.normal(size=(2, at.size))
        check(z, dt, tokens(rng, z.shape[0], V, 1), 32, rows_=[0, 1])


def test_temperatures_per_group_and_their_ends():
    rng = np.random.default_rng(9)
    z = logits(rng, 9, 4001, "peaked")
    tok = tokens(rng, 9, 4001, 4)
    check(z, "f32", tok, 3, T=[0.5, 1.5, 0.0], group=4)
    check(z[:8], "f32", tok[:8], 3, T=[np.nan, -1.0, np.inf, 1e30, 50.0, 1e-3, 1e-5, 1.0])
    # exponents beyond 2^30: summed again from the differences
    check(np.round(z[:4]), "f32", tok[:4], 3, T=[1e-9, 1e-12, 1e-30, 1e-38])


def test_values_at_the_types_ends():
    rng = np.random.default_rng(10)
    z = rng.normal(size=(5, 3000)).astype(np.float32)
    z[0] *= np.float32(1e30)
    z[1] = LOWEST
    z[2] = -LOWEST
    z[3, ::2], z[3, 1::2] = LOWEST, -LOWEST
    z[4] = 0.0
    z[4, ::3] = -0.0
    for dt in ("bf16", "f32"):
        check(z, dt, tokens(rng, 5, 3000, 2), 8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_the_longest_row(dt):
    rng = np.random.default_rng(11)
    check(logits(rng, 1, 2097152, "flat"), dt, tokens(rng, 1, 2097152, 3), 32)


def test_repeated_calls_and_streams_give_equal_bits():
    import torch
    rng = np.random.default_rng(12)
    v, _ = _tensor(logits(rng, 40, 50021, "ties"), torch.bfloat16)
    tok = _gpu_arr(tokens(rng, 40, 50021, 3), torch.int32)
    first = forward(v, tok, 20)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        again = forward(v, tok, 20, stream=s)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_rows_of_none():
    import torch
    import block_draft_select_amd as dfl
    z = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, 1, device="cuda")
    r = dfl.rows(z)
    ws = dfl.rows_workspace(r)
    dfl.dflash_logprobs(r, z, e.int(), e, torch.empty(0, 2, device="cuda"), ws)
    dfl.dflash_logprobs_grad(r, z, e.int(), e, torch.empty(0, 2, device="cuda"), torch.empty(0, 50, device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------- gradient

EPS = dict(bf16=2.0 ** -8, f32=2.0 ** -24)


def check_grad(z, dt, tok, g, ge=None, T=None, group=1, pad=0, shift=0, in_place=False, rows_=None):
    import torch
    import block_draft_select_amd as dfl
    v, _ = _tensor(z, _type(dt), pad, shift)
    R, V = z.shape
    zz = _f64(v)
    Ts = [1.0 if T is None else float(np.float32(T[i // group])) for i in range(R)]
    norm, H = np.zeros((R, 2), np.float32), np.zeros(R, np.float32)
    with np.errstate(over="ignore"):
        for i in range(R) if rows_ is None else rows_:
            m, l, _, h = O.distribution(zz[i], Ts[i])
            norm[i], H[i] = (m, l), h
    g, r = np.asarray(g, np.float32), dfl.rows(v)
    out, flat = (v, None) if in_place else _tensor(np.full((R, V), 5.0, np.float32), _type(dt), pad + 2, shift)
    gpu = lambda a, t: None if a is None else _gpu_arr(a, t)  # noqa: E731
    f32 = torch.float32
    M = tok.shape[1]
    ge = None if ge is None else np.asarray(ge, np.float32)
    dfl.dflash_logprobs_grad(r, v, gpu(tok, torch.int32) if M else None, gpu(g, f32) if M else None, gpu(norm, f32), out,
                             T=gpu(None if T is None else np.asarray(T, np.float32), f32), group=group,
                             entropy=gpu(None if ge is None else H, f32), grad_entropy=gpu(ge, f32))
    torch.cuda.synchronize()
    got = _f64(out)
    for i in range(R) if rows_ is None else rows_:
        Ti = O.temperature(Ts[i])
        want = O.logprobs_grad(zz[i], tok[i], g[i], 0.0 if ge is None else float(ge[i]), norm[i], float(H[i]), Ts[i])
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(got[i])), i
        if nan.any():
            continue
        with np.errstate(invalid="ignore", over="ignore", under="ignore"):
            lp = (zz[i] - float(norm[i, 0])) / Ti - float(norm[i, 1])
            p = np.exp(lp)
            t = np.abs(np.where(p > 0, lp, 0.0)) / LN2
            on = (tok[i] >= 0) & (tok[i] < V)
            A = abs(float(g[i][on].astype(np.float64).sum()))
            e = 0.0 if ge is None else abs(float(ge[i]))
            size = (A + e * (abs(float(H[i])) + t * LN2)) / Ti
            bar = np.abs(want) * EPS[dt] + p * size * ((t + 4) * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -126 * (size + 1)
            over = np.abs(want) >= 3.4028235677973366e38  # rounds to an infinity of fp32, as close() has it
            bad = np.where(over, got[i] != np.sign(want) * np.inf, np.abs(got[i] - want) > bar)
        assert not bad.any(), (i, int(bad.argmax()), got[i][bad][:3], want[bad][:3], bar[bad][:3])
    if flat is not None and pad + 2:
        full = flat[shift:shift + R * (V + pad + 2)].view(R, V + pad + 2)
        assert bool((full[:, V:] == 777.0).all())  # what lies between rows stays
    return out


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 9, 65, 1000, 8193])
@pytest.mark.parametrize("kind", KINDS)
def test_grad_short_rows(dt, V, kind):
    rng = np.random.default_rng(V * 31 + len(kind))
    R = 5
    g, ge = rng.normal(size=(R, 5)), rng.normal(size=R)
    g[1], ge[1] = 0.0, 0.0
    _say(f"[logprobs] grad {dt} V={V} {kind}")
    check_grad(logits(rng, R, V, kind), dt, tokens(rng, R, V, 5), g, ge, T=TS, pad=V % 3, shift=V % 5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_grad_long_rows(dt, kind, in_place):
    rng = np.random.default_rng(len(kind))
    V = 50021 if in_place else 151936
    check_grad(logits(rng, 3, V, kind), dt, tokens(rng, 3, V, 2), rng.normal(size=(3, 2)), [0.1, 0.0, -0.5], T=[1.0, 0.7, 1.3],
               in_place=in_place)
    check_grad(logits(rng, 3, V, kind), dt, tokens(rng, 3, V, 1), rng.normal(size=(3, 1)), in_place=in_place)


@pytest.mark.parametrize("M", [0, 1, 2, 64, 65, 300, 1024])
def test_grad_counts(M):
    rng = np.random.default_rng(M)
    for dt in ("bf16", "f32"):
        tok = tokens(rng, 3, 3000, M)
        check_grad(logits(rng, 3, 3000, "peaked"), dt, tok, rng.normal(size=(3, M)), rng.normal(size=3))
        if M:  # one token given again and again
            tok[:] = 1234
            check_grad(logits(rng, 3, 3000, "peaked"), dt, tok, rng.normal(size=(3, M)))


@pytest.mark.parametrize("dt,R,V", [("bf16", 700, 30011), ("f32", 300, 30011), ("bf16", 4000, 1000)])
def test_grad_many_rows(dt, R, V):
    rng = np.random.default_rng(R)
    z = np.tile(logits(rng, 25, V, "peaked"), (R // 25 + 1, 1))[:R]
    check_grad(z, dt, tokens(rng, R, V, 1), rng.normal(size=(R, 1)), rng.normal(size=R), rows_=list(range(0, 25)) + [R // 2, R - 1])


def test_grad_small_temperatures_keep_unlikely_tokens():
    rng = np.random.default_rng(21)
    z = rng.normal(size=(3, 500)).astype(np.float32)
    check_grad(z, "f32", tokens(rng, 3, 500, 1), np.array([[1e3], [1.0], [1e30]]), T=[1e-30, 1e-10, 1e-9])


def test_grad_of_an_incoming_nan_is_nan():
    import torch
    import block_draft_select_amd as dfl
    z = torch.randn(2, 100, device="cuda")
    tok = torch.tensor([[3], [5]], dtype=torch.int32, device="cuda")
    o = forward(z, tok, 0)
    d = torch.empty_like(z)
    dfl.dflash_logprobs_grad(dfl.rows(z), z, tok, torch.tensor([[float("nan")], [1.0]], device="cuda"), o["norm"], d)
    assert bool(torch.isnan(d[0]).all()) and bool(torch.isfinite(d[1]).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_grad_against_differences_of_the_forward(dt):
    # of the whole: directional differences of the float64 oracle along random
    # directions, at the rows as stored; the gradient's rounding adds up to at most
    # half a step of each entry
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(31)
    R, V = 4, 3001
    v, _ = _tensor(logits(rng, R, V, "peaked"), _type(dt))
    tok, g, ge = tokens(rng, R, V, 3), rng.normal(size=(R, 3)).astype(np.float32), rng.normal(size=R).astype(np.float32)
    o = forward(v, _gpu_arr(tok, torch.int32), 0)
    d = torch.empty_like(v)
    dfl.dflash_logprobs_grad(dfl.rows(v), v, _gpu_arr(tok, torch.int32), _gpu_arr(g, torch.float32), o["norm"], d,
                             entropy=o["entropy"], grad_entropy=_gpu_arr(ge, torch.float32))
    zz, dd = _f64(v), _f64(d)
    for i in range(R):
        def value(y):
            r = O.logprobs(y, tok[i])
            return float(np.dot(g[i].astype(np.float64), r["logp"])) + float(ge[i]) * r["entropy"]
        for _ in range(4):
            u = rng.normal(size=V)
            # central difference: off by h^2 / 6 times a third derivative of order |u|_inf^3, and 1e-15 / h
            num = (value(zz[i] + 1e-5 * u) - value(zz[i] - 1e-5 * u)) / 2e-5
            bar = float(np.sum(np.abs(dd[i] * u)) * (EPS[dt] + 32 * 2.0 ** -23)) + 1e-6
            assert abs(num - float(np.dot(dd[i], u))) <= bar


# ---------------------------------------------------------------- far rows, streams


@pytest.mark.parametrize("dt,V,R,stride", [("bf16", 5003, 18, (1 << 27) + 3), ("f32", 140011, 18, 1 << 27), ("bf16", 9, 66, 1 << 25)])
def test_rows_beyond_32_bit_offsets(dt, V, R, stride):
    # the last rows begin 2^31 elements and more behind the first
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(V)
    z = logits(rng, R, V, "peaked")
    far = torch.empty((R - 1) * stride + V, dtype=_type(dt), device="cuda").as_strided((R, V), (stride, 1))
    far.copy_(torch.from_numpy(z).to(far.dtype))
    near = far.contiguous()
    tok, g = _gpu_arr(tokens(rng, R, V, 3), torch.int32), _gpu_arr(rng.normal(size=(R, 3)), torch.float32)
    ge = _gpu_arr(rng.normal(size=R), torch.float32)
    _say(f"[logprobs] {R} rows of {V} {dt}, {stride} apart")
    o, p = forward(far, tok, 9), forward(near, tok, 9)
    for n in o:
        assert torch.equal(o[n], p[n]), n
    want = torch.empty_like(near)
    dfl.dflash_logprobs_grad(dfl.rows(near), near, tok, g, p["norm"], want, entropy=p["entropy"], grad_entropy=ge)
    dfl.dflash_logprobs_grad(dfl.rows(far), far, tok, g, o["norm"], far, entropy=o["entropy"], grad_entropy=ge)
    torch.cuda.synchronize()
    assert torch.equal(far, want)


def test_one_row_of_any_stride():
    import torch
    import block_draft_select_amd as dfl
    z = torch.randn(1, 4001, device="cuda").bfloat16()
    tok = torch.tensor([[17]], dtype=torch.int32, device="cuda")
    want = forward(z, tok, 4)
    for stride in (0, -9, 1 << 40):  # 2^40 is the largest that any call takes
        got = forward(z.as_strided((1, 4001), (max(stride, 0), 1)), tok, 4)
        r = dfl.dflash_rows(1, stride, 4001, dfl.BF16)
        norm, logp = torch.empty(1, 2, device="cuda"), torch.empty(1, 1, device="cuda")
        dfl.dflash_logprobs(r, z, tok, logp, norm, dfl.rows_workspace(dfl.rows(z)))
        assert torch.equal(got["norm"], want["norm"]) and torch.equal(norm, want["norm"]) and torch.equal(logp, want["logp"])


def test_calls_on_two_streams_at_once():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(3)
    R, V = 24, 151936
    ins, wants = [], []
    for _ in range(2):
        v, _ = _tensor(logits(rng, R, V, "peaked"), torch.bfloat16)
        tok, g = _gpu_arr(tokens(rng, R, V, 2), torch.int32), _gpu_arr(rng.normal(size=(R, 2)), torch.float32)
        o = forward(v, tok, 20)
        d = torch.empty_like(v)
        dfl.dflash_logprobs_grad(dfl.rows(v), v, tok, g, o["norm"], d)
        ins.append((v, tok, g, torch.empty_like(v), dfl.rows_workspace(dfl.rows(v))))
        wants.append((o, d))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                v, tok, g, d, ws = ins[k]
                got[k] = forward(v, tok, 20, ws=ws)
                dfl.dflash_logprobs_grad(dfl.rows(v), v, tok, g, got[k]["norm"], d)
    torch.cuda.synchronize()
    for k in range(2):
        for n in wants[k][0]:
            assert torch.equal(got[k][n], wants[k][0][n]), (k, n)
        assert torch.equal(ins[k][3], wants[k][1])


# ---------------------------------------------------------------- graphs

def test_captured_calls_replay_as_eager_ones():
    import torch
    import block_draft_select_amd as dfl
    rng = np.random.default_rng(41)
    V, R = 50021, 12
    v, _ = _tensor(logits(rng, R, V, "peaked"), torch.bfloat16, pad=1)
    tok, g, ge = (_gpu_arr(tokens(rng, R, V, 2), torch.int32), _gpu_arr(rng.normal(size=(R, 2)), torch.float32),
                  _gpu_arr(rng.normal(size=R), torch.float32))
    r = dfl.rows(v)
    ws, ws2 = dfl.rows_workspace(r), dfl.rows_workspace(r)
    d = torch.empty_like(v)

    def both(ws):
        o = forward(v, tok, 20, ws=ws)
        dfl.dflash_logprobs_grad(r, v, tok, g, o["norm"], d, entropy=o["entropy"], grad_entropy=ge)
        return o

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = both(ws)
    for k in range(4):
        v.copy_(torch.from_numpy(logits(rng, R, V, "peaked")).to(v.dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in o.items()}
        dg = d.clone()
        want = both(ws2)
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[n]), (k, n)
        assert torch.equal(dg, d)
