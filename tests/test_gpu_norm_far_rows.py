"""The layer norm's backward on rows whose mean is many deviations from zero, against 64 bits
on the CPU. Tolerances count roundings as in test_gpu_train_ops.py: h - m is exact there (or
as good), the mean of what is left is taken off again in one rounding, and up to a mean of 16
deviations u may be off by the mean's own rounding, 2^-24 |m| s."""
import pytest

from gpu_util import device_ready, log
from test_gpu_block_ops import HALF, T_, U, close, gen, rand, strided
from test_gpu_train_ops import back_ref, factor, norm_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", [(7, 64), (1100, 64), (1030, 1000), (9, 1365), (5, 2048), (4, 4097), (3, 8200), (3, 20001)])
def test_backward_of_far_rows(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm backward, far rows T={T} dim={dim} {dt}")
    g = gen(T * 53 + dim)
    z, gy, gh = (rand(g, T, dim, dtype=dt, scale=k) for k in (1.0, 0.1, 0.1))
    # means of 0 to 1e5 deviations (bf16 300, where a step of the type is two of them), of either sign
    far = torch.tensor([0.0, 12.0, -40.0, 300.0, -2e3, 1e5, 300.0] if dt == "f32" else [0.0, 12.0, -40.0, 100.0, -300.0, 300.0, 0.0])
    at = far[torch.arange(T) % 7][:, None]
    x = (z.double() + at.double()).to(T_(dt))
    w, b = 1 + 0.2 * rand(g, dim), 0.2 * rand(g, dim)
    f = oec.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=1e-5, save=True)
    m, s, _, _ = norm_ref(x, w, b, 1e-5)
    ratio = m.abs() * s
    for res, p in ((gh, 0.0), (gh, 0.3)):
        mask = factor(T, dim, p, 11, 4)
        dh, mag, sums, gw, gwm, gb, gbm = back_ref(gy, res, x, w, m, s)
        gs, hs = strided(gy, 5, 1), strided(res, 1)
        o = oec.add_layer_norm_backward(gs, x.cuda(), w.cuda(), f.mean, f.rstd, G_H=hs, p=p, seed=11, site=4, G_X=gs,
                                        G_R=hs if p else None)
        # what u is off by besides its own roundings, s by 2 u of itself: the mean's rounding in near rows, its
        # second part's in far ones
        eu = torch.where(ratio <= 16.5, U * ratio, 2 * U * U * ratio)[:, None]
        gwd = (gy.double() * w.double()).abs()
        u = ((x.double() - m[:, None]) * s[:, None]).abs()
        de = s[:, None] * eu * (gwd.mean(1, keepdim=True) * (u + 1) + (gwd * u).mean(1, keepdim=True))
        tol = HALF[dt] * dh.abs() + 14 * U * mag + 70 * U * sums + 2 * de
        close("G_R", o.G_R, dh, tol)
        close("G_X", o.G_X, dh * mask, (tol + 2 * U * dh.abs()) * mask)
        close("g_w", o.g_weight, gw, 9 * U * gwm + (gy.double().abs() * eu).sum(0))
        close("g_b", o.g_bias, gb, 2 * U * gbm)
