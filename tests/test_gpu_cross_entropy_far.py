"""The vocabulary's cross entropy on logits far from zero, in every kernel that takes them:
thousands, whose own digits the exponent must keep, and the largest numbers. The logits are
exact sums here, so that the tolerances hold the exponentials alone."""
import math

import pytest

from gpu_util import device_ready, log
from test_gpu_block_ops import HALF, T_, U, close, gen
from test_gpu_cross_entropy import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


# one and two tokens, the ring's tiles, rows of no whole 16 bytes, 256 x 256 tiles (two of them: with columns behind whole rounds)
SIZES = [(1, 64, 600), (5, 64, 600), (300, 64, 700), (300, 65, 700), (2003, 128, 4300), (2048, 64, 8448), (1003, 128, 1009)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("far", [5120.0, -5120.0, 61440.0])
@pytest.mark.parametrize("T, n, V", SIZES)
def test_logits_of_thousands(T, n, V, far, dt):
    """Every logit is `far` + a multiple of 1/4 below 8: the loss is that of the multiples alone."""
    import torch
    log(f"cross entropy, far logits T={T} n={n} V={V} {far} {dt}")
    g = gen(T + n + V)
    X = torch.zeros(T, n, dtype=T_(dt))
    W = torch.zeros(V, n, dtype=T_(dt))
    # far as a product of two numbers of few bits; 1/4, 1/2, 1, 2 and 4 times a choice of column
    X[:, 0], W[:, 0] = 8.0, far / 8
    X[:, 1:6] = torch.tensor([0.25, 0.5, 1.0, 2.0, 4.0]) * torch.randint(0, 2, (T, 5), generator=g)
    W[:, 1:6] = torch.randint(0, 2, (V, 5), generator=g).to(T_(dt))
    assert float((W[0, 0].double() - far / 8).abs()) == 0
    target = torch.randint(0, V, (T,), generator=g)
    one = torch.ones(1)
    X, W, target = X.cuda(), W.cuda(), target.cuda()
    a = run(X, W, target, one.cuda())
    z = X[:, 1:].double() @ W[:, 1:].double().T
    lse = torch.logsumexp(z, 1)
    # 80 u for the exponentials and their sum as in test_gpu_cross_entropy.py
    loss = lse - z.gather(1, target[:, None])[:, 0]
    close("loss", a["loss"], loss.cpu(), (U * loss.abs() + 80 * U).cpu())
    close("lse", a["lse"], (lse + far).cpu(), (U * (lse + far).abs() + 80 * U).cpu())
    # from the lse as it is handed on, fp32: p is off by its 80 u and by the rounding of z - lse
    r = a["lse"].double() - far
    p = torch.exp(z - r[:, None])
    d = p.clone()
    d[torch.arange(T, device="cuda"), target] -= 1
    half = 0.0 if dt != "bf16" else HALF[dt] if T > 64 else 2.0 ** -17
    dp = p * (80 * U + U * (z - r[:, None]).abs())
    ed = dp + (half + 3 * U) * (d.abs() + dp)
    x, w = X.double(), W.double()
    ex = ed @ w.abs() + 2 * (V + 8) * U * ((d.abs() + ed) @ w.abs())
    ew = ed.T @ x.abs() + 2 * (T + 8) * U * ((d.abs() + ed).T @ x.abs())
    tiny = 2.0 ** -125
    ex, ew = ex + tiny * (w.abs().sum(0) + V + 1), ew + tiny * (x.abs().sum(0) + T + 1)
    gx, gw = d @ w, d.T @ x
    close("G_X", a["G_X"], gx.cpu(), (ex + HALF[dt] * (gx.abs() + ex)).cpu())
    close("G_W", a["G_W"], gw.cpu(), (ew + HALF[dt] * (gw.abs() + ew)).cpu())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T, n, V", SIZES)
def test_the_largest_logits(T, n, V, sign, dt):
    """Logits past 2^127: the softmax is the largest's alone, and nothing overflows in front of it."""
    import torch
    log(f"cross entropy, largest logits T={T} n={n} V={V} {sign} {dt}")
    g = gen(T * 3 + V)
    X, W = torch.zeros(T, n, dtype=T_(dt)), torch.zeros(V, n, dtype=T_(dt))
    X[:, 0] = sign * 2.0 ** 64
    W[:, 0] = 2.0 ** 63 * (1.5 + torch.randint(0, 50, (V,), generator=g).double() / 128).to(T_(dt))
    star = V - 3
    W[star, 0] = 2.0 ** 63 * (1.9921875 if sign > 0 else 1.4921875)   # the one largest logit
    target = torch.randint(0, V, (T,), generator=g)
    target[T // 2] = star
    X, W, target = X.cuda(), W.cuda(), target.cuda()
    a = run(X, W, target, torch.ones(1).cuda())
    z = X[:, 0].double()[:, None] * W[:, 0].double()[None]
    assert torch.equal(a["lse"].double(), z[:, star])
    loss = z[:, star] - z.gather(1, target[:, None])[:, 0]
    close("loss", a["loss"], loss.cpu(), (U * loss).cpu())
    d = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    d[:, star] = 1
    d[torch.arange(T, device="cuda"), target] -= 1
    gx, gw = d @ W.double(), d.T @ X.double()
    close("G_X", a["G_X"], gx.cpu(), (HALF[dt] * gx.abs()).cpu())
    # at most T equal terms of 2^64, exact sums
    assert T < 2 ** 24
    close("G_W", a["G_W"], gw.cpu(), (HALF[dt] * gw.abs()).cpu())
    assert math.isfinite(float(a["G_W"].double().abs().max()))
