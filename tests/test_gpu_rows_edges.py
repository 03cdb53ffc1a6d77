"""GPU tests of the operators on logit rows at the ends of what they accept:
uniforms next to 1, temperatures that leave bins without a value, settings of
the smallest tau, and every plan of the launches.  Bars as in test_gpu_rows.
"""

import numpy as np
import pytest

from test_gpu_rows import _check_sample, _logits, _say

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
