"""GPU tests of the operators on logit rows at the ends of what they accept:
uniforms next to 1, temperatures that leave bins without a value, settings of
the smallest tau, and every plan of the launches.  Bars as in test_gpu_rows.
"""

import numpy as np
import pytest

from test_gpu_rows import _check_sample, _say

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
