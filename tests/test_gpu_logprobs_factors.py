"""GPU parity of dflash_logprobs_grad with the float64 oracle where a row's
factor sum g / T (or that of the entropy's gradient) is beyond 2^100.

Bars.  With p from an fp32 exponent t = log2 p, right to (|t| + 4) 2^-23 of
itself, and the factor's terms to 2^-22: that much of p times the terms' size;
half a step of the type, of the smallest normal number's at least; for a given
token 2^-50 of its terms, which fp64 may cancel.  Nothing grows with the
factor where p is 0: a masked token's gradient is 0.
"""

import numpy as np
import pytest

from oracle import rows as O
from test_gpu_logprobs import EPS, LN2, _f64, _gpu_arr, _say, _tensor, _type, logits, tokens

pytestmark = pytest.mark.gpu

F32_MAX = 3.4028235677973366e38  # and half a step: what rounds to an infinity
LEAST = dict(bf16=2.0 ** -134, f32=2.0 ** -150)  # half a step of a subnormal number


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_select_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def check(z, dt, tok, g, T, ge=None, in_place=False):
    import torch
    import block_draft_select_amd as dfl
    f32 = torch.float32
    v, _ = _tensor(np.asarray(z, np.float32), _type(dt), pad=3, shift=1)
    zz = _f64(v)
    R, V = zz.shape
    tok, g, T = np.asarray(tok), np.asarray(g, np.float32), np.asarray(T, np.float32)
    ge = None if ge is None else np.asarray(ge, np.float32)
    norm, H = np.zeros((R, 2), np.float32), np.zeros(R, np.float32)
    for i in range(R):
        m, l, _, h = O.distribution(zz[i], float(T[i]))
        norm[i], H[i] = (m, l), h
    out = v if in_place else torch.full((R, V), 5.0, dtype=_type(dt), device="cuda")
    dfl.dflash_logprobs_grad(dfl.rows(v), v, _gpu_arr(tok, torch.int32), _gpu_arr(g, f32), _gpu_arr(norm, f32), out, T=_gpu_arr(T, f32),
                             entropy=None if ge is None else _gpu_arr(H, f32), grad_entropy=None if ge is None else _gpu_arr(ge, f32))
    torch.cuda.synchronize()
    got = _f64(out)
    for i in range(R):
        Ti, e = O.temperature(T[i]), 0.0 if ge is None else float(ge[i])
        want = O.logprobs_grad(zz[i], tok[i], g[i], e, norm[i], float(H[i]), float(T[i]))
        assert not np.isnan(want).any()
        on = (tok[i] >= 0) & (tok[i] < V)
        with np.errstate(over="ignore", under="ignore"):
            lp = (zz[i] - float(norm[i, 0])) / Ti - float(norm[i, 1])
            p = np.exp(lp)
        lp = np.where(p > 0, lp, 0.0)
        t = np.abs(lp) / LN2
        size = (abs(float(g[i][on].astype(np.float64).sum())) + abs(e) * (abs(float(H[i])) + np.abs(lp))) / Ti
        bar = np.abs(want) * EPS[dt] + LEAST[dt] + np.where(p > 0, p * size, 0.0) * ((t + 4) * 2.0 ** -23 + 2.0 ** -22)
        bar[tok[i][on]] += 2.0 ** -50 * (np.abs(g[i][on].astype(np.float64)).sum() / Ti + size[tok[i][on]])
        with np.errstate(over="ignore"):
            ok = np.abs(got[i] - want) <= bar
        # an infinity, or a type's largest number, where a value within the bar rounds to it
        ok |= (np.abs(got[i]) >= F32_MAX * (1 - 2 * EPS[dt])) & (np.sign(got[i]) * want + bar >= F32_MAX)
        k = int((~ok).argmax())
        assert ok.all(), (f"row {i} token {k}", got[i][k], want[k], bar[k], int((~ok).sum()))
        masked = np.isneginf(zz[i])
        masked[tok[i][on]] = False
        assert (got[i][masked] == 0).all()
    return got


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_tokens_get_nothing(dt):
    rng = np.random.default_rng(1)
    g = np.array([1e12, 1e30, 1e38, -1e38, 1e20, 3e38])
    T = [1e-30, 1e-10, 1e-30, 1e-30, 1e-20, 1e-30]
    assert (check([[0.0, -np.inf]] * 6, dt, [[0]] * 6, g[:, None], T) == 0).all()
    z = logits(rng, 6, 3001, "flat")
    z[rng.random(size=z.shape) < 0.7] = -np.inf
    tok = np.where(np.isneginf(z), 0.0, 1.0).argmax(1)[:, None]  # an unmasked one
    check(z, dt, tok, g[:, None], T)
    check(z, dt, [[5]] * 6, g[:, None], T)  # masked or not


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("width", [0.5, 3.0, 40.0])
def test_wide_rows(dt, width):
    # at T of about 1 all results fit the type, most tokens' p being anything down to 2^-300
    rng = np.random.default_rng(int(width))
    for V in (500, 9001, 50021):
        z = (rng.normal(size=(6, V)) * width).astype(np.float32)
        z[:, ::17] = -np.inf
        g = rng.normal(size=(6, 4)) * np.array([1e30, 1e32, 1e33, 1e34, 1e35, 1e36])[:, None]
        _say(f"[logprobs] large factors {dt} V={V} width {width}")
        check(z, dt, tokens(rng, 6, V, 4), g, [1.0, 0.6, 0.0, 1.3, 1.0, 0.9])
        check(z, dt, tokens(rng, 6, V, 4), g, [1.0, 0.6, 0.0, 1.3, 1.0, 0.9], ge=rng.normal(size=6) * 1e33, in_place=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_entropies_of_one_token(dt):
    # H = 0 and log p = 0: nothing, whatever the factor, but what a given token brings
    z = np.full((5, 300), -np.inf, np.float32)
    z[:, 7] = [0.0, 5.0, -3.0, 100.0, 1.0]
    ge = np.array([1e10, 1e30, -1e38, 3e38, 1e35])
    T = [1e-30, 1e-20, 1e-10, 1e-30, 1.0]
    check(z, dt, [[-1]] * 5, np.zeros((5, 1)), T, ge=ge)
    check(z, dt, [[8]] * 5, np.full((5, 1), 1e-10), T, ge=ge)
    # beside tokens so unlikely that H rounds to 0 as well
    z[:, 8] = z[:, 7] - 200.0
    check(z, dt, [[-1]] * 5, np.zeros((5, 1)), [1.0, 1.0, 0.9, 0.8, 1.0], ge=ge)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_unlikely_tokens_whose_gradient_fits(dt):
    # p down to 2^-250 beside factors up to 2^226: results between the smallest and the largest number
    rng = np.random.default_rng(4)
    z = np.zeros((4, 700), np.float32)
    T = np.array([1e-30, 1e-25, 1e-20, 1e-12], np.float32)
    for i in range(4):
        z[i] = -rng.uniform(1, 175, size=700) * T[i]
        z[i, 11] = 0.0
    check(z, dt, [[11]] * 4, np.array([[1e38], [1e36], [-1e37], [1e38]]), T)
