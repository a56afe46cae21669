"""The cross entropy's gradients where the factor of all tokens is no finite number, as the
mean's 1 / count is when no token counts: ignored tokens have no part in it."""
import math

import pytest

from gpu_util import device_ready, log
from test_gpu_cross_entropy import IGNORE, inputs, run, run_back

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


# every kind of product: few tokens (d in two halves; in one pass over fp32 weights), the ring's tiles, rows of no whole
# 16 bytes, 256 x 256 tiles apart and in one launch
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, n, V", [(1, 64, 600), (5, 1024, 600), (40, 64, 900), (300, 64, 700), (300, 65, 700),
                                     (512, 1024, 2000), (2003, 264, 4300)])
def test_a_factor_that_is_not_finite(T, n, V, dt):
    import torch
    log(f"cross entropy, infinite factor T={T} n={n} V={V} {dt}")
    X, W, target, _ = inputs(T, n, V, dt, ignored=0.3)
    X, W = X.cuda(), W.cuda()
    none = torch.full((T,), IGNORE).cuda()
    some = target.cuda()
    some[0] = 3
    out = some == IGNORE
    for g in (math.inf, -math.inf, math.nan):
        one = torch.full((1,), g).cuda()
        a = run(X, W, none, one)
        assert not a["loss"].any() and not a["G_X"].any() and not a["G_W"].any()
        gx, _ = run_back(X, W, none, a["lse"], one, need_w=False)
        _, gw = run_back(X, W, none, a["lse"], one, need_x=False)
        assert not gx.any() and not gw.any()
        # tokens that count have no finite gradient, as with a factor of their own
        b, c = run(X, W, some, one), run(X, W, some, one.expand(T).contiguous())
        for r in (b, c):
            assert not r["G_X"][out].any() and not r["G_X"][~out].isfinite().any() and not r["G_W"][3].isfinite().any()
