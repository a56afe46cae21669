"""The layer norm on rows whose statistics are hard to take: a first value that dropout takes
out or the residual cancels, means far from zero, the longest rows. Against 64 bits on the
CPU; tolerances count roundings as in test_gpu_train_ops.py."""
import math

import pytest

from gpu_util import device_ready, log
from test_gpu_block_ops import HALF, T_, U, close, gen, rand
from test_gpu_train_ops import SEED, back_ref, factor, norm_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


# every variant: one wave a row, four, sixteen, rows no register holds; whole and cut vectors
SIZES = [(40, 64), (1100, 64), (1100, 1001), (40, 1365), (24, 2048), (16, 9000), (12, 40000)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", SIZES)
def test_a_dropped_first_value_leaves_no_trace(T, dim, dt):
    """Whatever a dropped x_0 was, the results are those of x_0 = 0, bit by bit."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm, dropped first value T={T} dim={dim} {dt}")
    g = gen(T * 43 + dim)
    x, r = rand(g, T, dim, dtype=dt), rand(g, T, dim, dtype=dt)
    w, b = (1 + 0.2 * rand(g, dim)).cuda(), (0.2 * rand(g, dim)).cuda()
    gone = factor(T, dim, 0.5, SEED, 5)[:, 0] == 0
    assert 0 < int(gone.sum()) < T
    x[gone, 0] = 0
    kw = dict(eps=1e-5, p=0.5, seed=SEED, site=5)
    for res in (r.cuda(), None):
        for quant in (False, True):
            want = oec.add_layer_norm(x.cuda(), w, b, residual=res, quantize=quant, save=True, **kw)
            m, s, y, mag = norm_ref(want.H.cpu(), w.cpu(), b.cpu(), 1e-5)
            close("rstd", want.rstd, s, 2 * U * s)
            for big in (1e5, 1e6, 1e9, 1e30, -3e38, math.inf, math.nan):
                far = x.clone()
                far[gone, 0] = big
                o = oec.add_layer_norm(far.cuda(), w, b, residual=res, quantize=quant, save=True, **kw)
                close("rstd", o.rstd, s, 2 * U * s)
                close("mean", o.mean, m, U * m.abs() + 1e-15)
                if not quant:
                    tol = HALF[dt] * y.abs() + U * y.abs() + 6 * U * mag + 2.0 ** -46 * (m.abs() * s)[:, None] * w.cpu().abs()
                    close("Y", o.Y, y, tol)
                for a, e in zip(o, want):
                    assert (a is None and e is None) or torch.equal(a, e), big


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", SIZES)
def test_a_first_value_that_the_residual_cancels(T, dim, dt):
    """x_0 kept, and its double (the factor at p = 1/2) taken off again by r_0: h_0 = 0."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm, cancelled first value T={T} dim={dim} {dt}")
    g = gen(T * 47 + dim)
    x, r = rand(g, T, dim, dtype=dt), rand(g, T, dim, dtype=dt)
    w = (1 + 0.2 * rand(g, dim)).cuda()
    kept = factor(T, dim, 0.5, SEED, 5)[:, 0] > 0
    x[kept, 0], r[kept, 0] = 2.0 ** 30, -2.0 ** 31
    o = oec.add_layer_norm(x.cuda(), w, residual=r.cuda(), save=True, eps=1e-5, p=0.5, seed=SEED, site=5)
    assert not o.H[kept.cuda(), 0].any()
    m, s, y, mag = norm_ref(o.H.cpu(), w.cpu(), None, 1e-5)
    close("rstd", o.rstd, s, 2 * U * s)
    close("mean", o.mean, m, U * m.abs() + 1e-15)
    close("Y", o.Y, y, HALF[dt] * y.abs() + U * y.abs() + 6 * U * mag + 2.0 ** -46 * (m.abs() * s)[:, None] * w.cpu().abs())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_of_the_longest_sums(dt):
    """A row of 2^22 columns whose g w is the same everywhere: a sum in one fp32 number would lose what
    its every addition rounds alike."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm backward of 2^22 columns {dt}")
    T, dim = 2, 2 ** 22
    g = gen(5)
    x = rand(g, T, dim, dtype=dt)
    gy = torch.full((T, dim), 0.3, dtype=T_(dt))
    w = torch.ones(dim)
    f = oec.add_layer_norm(x.cuda(), w.cuda(), eps=1e-5, save=True)
    m, s, _, _ = norm_ref(x, w, None, 1e-5)
    # the gradient of a sum: zero but for the roundings of g w - mean(g w) - u mean(g w u), the two means one each
    dh, mag, sums, gw, gwm, gb, gbm = back_ref(gy, None, x, w, m, s)
    o = oec.add_layer_norm_backward(gy.cuda(), x.cuda(), w.cuda(), f.mean, f.rstd)
    u = ((x.double() - m[:, None]) * s[:, None]).abs()
    eu = (U * m.abs() * s)[:, None]
    cb = gy.double().abs() * (6 * U * u + eu)              # a term's, and so the mean's, error
    tol = HALF[dt] * dh.abs() + 9 * U * mag + s[:, None] * (eu * gy.double().abs().mean() + u * cb.mean(1, keepdim=True))
    close("G_X", o.G_X, dh, tol)
    close("g_w", o.g_weight, gw, 9 * U * gwm + (gy.double().abs() * eu).sum(0))
    close("g_b", o.g_bias, gb, 2 * U * gbm)
