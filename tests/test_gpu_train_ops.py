"""Dropout and the layer norm against plain 64-bit implementations on the CPU, element by
element, the masks bit by bit against the published generator.

Tolerances count roundings, as in test_gpu_block_ops.py: u = 2^-24 for one fp32 step, half
a step of the output's type for its rounding, N u times the sum of the magnitudes for a sum
of N fp32 terms."""
import math

import numpy as np
import pytest

from gpu_util import device_ready, log
from philox_ref import factors
from test_gpu_block_ops import HALF, T_, U, close, f64, gen, rand, strided

pytestmark = pytest.mark.gpu

SEED = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def factor(T, dim, p, seed, site):
    import torch
    return torch.from_numpy(factors(T, dim, p, seed, site))


# ------------------------------------------------------------------ dropout
DROP_SIZES = [(1, 1), (1, 7), (3, 8), (5, 9), (2, 64), (7, 513), (1, 2048), (61, 1365), (300, 2056), (3, 20001), (1500, 96)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", DROP_SIZES)
def test_dropout(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"dropout T={T} dim={dim} {dt}")
    g = gen(T * 31 + dim)
    x, r = rand(g, T, dim, dtype=dt) + 4, rand(g, T, dim, dtype=dt)   # hardly an element of x is zero
    for p, seed, site in ((0.1, SEED, 3), (0.5, 1, 2 ** 32 - 1), (0.93, 2 ** 64 - 1, 0)):
        f = factor(T, dim, p, seed, site)
        want = x.double() * f
        y = oec.dropout(x.cuda(), p, seed, site)
        assert torch.equal(f64(y) != 0, want != 0)
        # the factor rounded, the product, the type
        close("y", y, want, (HALF[dt] + 2 * U) * want.abs())
        assert torch.equal(oec.dropout_backward(x.cuda(), p, seed, site), y)
        # strided, with the residual, and into either in place
        both = want + r.double()
        tol = (HALF[dt] + U) * both.abs() + 3 * U * want.abs()
        xs, rs = strided(x, 3, 1), strided(r, 5, 2)
        z = oec.dropout(xs, p, seed, site, residual=rs)
        close("y + r", z, both, tol)
        assert torch.equal(xs.cpu(), x) and torch.equal(rs.cpu(), r)
        assert oec.dropout(xs, p, seed, site, residual=rs, out=rs) is rs and torch.equal(rs, z)
        assert bool((torch.as_strided(rs, (T, 2), (dim + 5, 1), 0) == 7).all())
        assert torch.equal(oec.dropout(xs, p, seed, site, out=xs), y)


def test_dropout_ends_of_p():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x = rand(gen(1), 5, 37).cuda()
    x[1, 3], x[2, 5], x[4, 36] = math.inf, math.nan, -math.inf
    same = lambda a, b: torch.equal(torch.nan_to_num(a, 77.0), torch.nan_to_num(b, 77.0))  # noqa: E731
    assert same(oec.dropout(x, 0.0, 1), x) and same(oec.dropout(x, 2.0 ** -18, 1), x)
    assert not oec.dropout(x, 1.0, 1).any() and not oec.dropout(x, 1 - 2.0 ** -18, 1).any()
    # a dropped infinity or NaN is zero
    y, f = oec.dropout(x, 0.5, 9), factor(5, 37, 0.5, 9, 0).cuda()
    assert not y[f == 0].any() and same(y[f != 0], (x * 2)[f != 0])
    e = torch.empty(0, 8, device="cuda")
    assert oec.dropout(e, 0.5, 1).shape == (0, 8)


def test_dropout_past_4_gib():
    """Elements past 2^32 bytes and 2^31 elements, by their mask at the far end."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    T, dim = 2 ** 21 + 3, 1032
    x = torch.ones(T, dim, dtype=torch.bfloat16, device="cuda")
    y = oec.dropout(x, 0.25, 5, 6, out=x)
    for at in (0, 2 ** 20 + 1, T - 4):
        from philox_ref import philox
        row, col = np.meshgrid(np.arange(at, at + 4), np.arange(dim // 8), indexing="ij")
        w = philox((col, row, np.full_like(row, 6), np.zeros_like(row)), (5, 0))
        h = np.stack([v for c in w for v in (c & np.uint64(0xFFFF), c >> np.uint64(16))], -1).reshape(4, dim)
        assert np.array_equal((y[at:at + 4] != 0).cpu().numpy(), h >= 16384)


def test_dropout_device_seed_in_a_graph():
    """A captured step is replayed with the seed that stands on the device then."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x = torch.ones(64, 264, device="cuda")
    w = torch.ones(264, device="cuda")
    seed = torch.tensor([41], device="cuda")
    oec.dropout(x, 0.3, seed, 2)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            y = oec.dropout(x, 0.3, seed, 2)
            o = oec.add_layer_norm(x, w, residual=x, p=0.3, seed=seed, site=2, save=True)
            b = oec.add_layer_norm_backward(x, o.H, w, o.mean, o.rstd, p=0.3, seed=seed, site=2)
    for k in range(4):
        seed.fill_(1000 + k)
        graph.replay()
        torch.cuda.synchronize()
        f = factor(64, 264, 0.3, 1000 + k, 2)
        assert torch.equal(f64(y) != 0, f != 0)
        assert torch.equal(f64(o.H) != 1, f != 0)
        assert not b.G_X[(f == 0).cuda()].any()
        e = oec.add_layer_norm_backward(x, o.H, w, o.mean, o.rstd, p=0.3, seed=1000 + k, site=2)
        assert all(torch.equal(u, v) for u, v in zip(b, e))


# ------------------------------------------------------------------ layer norm
def norm_ref(h, w, b, eps):
    """m, s and y in 64 bits, and the magnitude that the roundings of y go by."""
    hd = h.double()
    m = hd.mean(1, keepdim=True)
    s = 1 / ((hd - m).square().mean(1, keepdim=True) + eps).sqrt()
    u = (hd - m) * s * w.double()
    y = u if b is None else u + b.double()
    return m[:, 0], s[:, 0], y, u.abs()


# one row and many, around every variant's longest row, and rows no register variant holds
NORM_SIZES = [(1, 1), (3, 7), (5, 63), (2, 64), (4, 65), (1, 2048), (7, 512), (6, 513), (3, 1000), (9, 1024), (4, 1365),
              (130, 2049), (5, 4096), (3, 4097), (2, 8192), (2, 8200), (3, 16385), (2, 20001), (2, 32769), (1030, 65),
              (1100, 1000), (1024, 512)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES)
def test_norm_forward(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm T={T} dim={dim} {dt}")
    g = gen(T * 31 + dim)
    x, r = rand(g, T, dim, dtype=dt), rand(g, T, dim, dtype=dt, scale=3.0)
    w, b = 1 + 0.2 * rand(g, dim), 0.2 * rand(g, dim)
    for p, bias, res in ((0.0, b, r), (0.2, b, r), (0.2, None, None), (0.0, None, None)):
        f = factor(T, dim, p, SEED, 5)
        kw = dict(eps=1e-3, p=p, seed=SEED, site=5)
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        o = oec.add_layer_norm(x.cuda(), w.cuda(), dev(bias), residual=dev(res), save=True, **kw)
        hw = x.double() * f + (0 if res is None else res.double())
        close("H", o.H, hw, (HALF[dt] + U) * hw.abs() + 3 * U * (x.double() * f).abs())
        m, s, y, mag = norm_ref(o.H.cpu(), w, bias, 1e-3)
        # h - m twice rounded, s, its two products and the sum: 5 u of the product, one of y; m as two floats, 2^-48 of it
        tol = HALF[dt] * y.abs() + U * y.abs() + 6 * U * mag + 2.0 ** -46 * (m.abs() * s)[:, None] * w.abs()
        close("Y", o.Y, y, tol)
        close("mean", o.mean, m, U * m.abs() + 1e-15)
        close("rstd", o.rstd, s, 2 * U * s)
        # the same bits strided, and with H in place
        xs, rs = strided(x, 3, 1), None if res is None else strided(res, 5, 2)
        o2 = oec.add_layer_norm(xs, w.cuda(), dev(bias), residual=rs, H=xs if res is None and p else rs, **kw)
        assert torch.equal(o2.Y, o.Y) and torch.equal(o2.H, o.H) and o2.mean is None
        assert (o2.H is rs) if res is not None else (o2.H is xs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES)
def test_norm_int8(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm int8 T={T} dim={dim} {dt}")
    g = gen(T * 37 + dim)
    x, w, b = rand(g, T, dim, dtype=dt) + 1, 1 + 0.2 * rand(g, dim), 0.2 * rand(g, dim)
    for p in (0.0, 0.3):
        o = oec.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=1e-3, p=p, seed=3, quantize=True)
        _, s, y, mag = norm_ref(o.H.cpu(), w, b, 1e-3)
        err = 2 * U * y.abs() + 6 * U * mag + 2.0 ** -46 * s[:, None] * w.abs() * 4
        a = y.abs().amax(1)
        assert bool((a > 0).all())
        close("scale", o.scale, a / 127, err.amax(1) / 127 + 2 * U * a / 127)
        # q = rint(y / scale): half a step, and what y and the factor are off by
        step = f64(o.scale)[:, None]
        close("values", f64(o.Y) * step, y, 0.5 * step + 2 * err + 4 * U * a[:, None])
        assert int(o.Y.abs().max()) == 127 and bool((o.Y.abs().amax(1) == 127).all())


@pytest.mark.parametrize("dim", [64, 1001, 2048, 9000, 40000])
def test_norm_special_rows(dim):
    """Constant rows, rows far from zero, tiny and huge ones, infinities and NaN: only their own rows show it."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm special dim={dim}")
    g = gen(dim)
    x, w, b = rand(g, 9, dim), 1 + 0.2 * rand(g, dim), 0.2 * rand(g, dim)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, dim // 2] = math.inf
    x[5, dim - 1] = math.nan
    x[6] = 12345.678
    x[7] += 1e5
    eps = 1e-5
    m, s, y, mag = norm_ref(x, w, b, eps)
    o = oec.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=eps, save=True)
    keep = [0, 1, 2, 3, 6, 7, 8]
    tol = 2 * U * y.abs() + 6 * U * mag + 2.0 ** -46 * (m.abs() * s)[:, None] * w.abs()
    close("Y", o.Y[keep], y[keep], tol[keep])
    assert torch.isnan(o.Y[5]).all() and torch.isnan(o.Y[4]).any()
    q = oec.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=eps, quantize=True)
    for t in (4, 5):
        assert math.isnan(float(q.scale[t])) and not q.Y[t].any()
    assert bool(torch.isfinite(q.scale[keep]).all())
    # zero rows without a bias are zero, also as INT8
    q = oec.add_layer_norm(x[1:2].cuda(), w.cuda(), eps=eps, quantize=True)
    assert float(q.scale[0]) == 0 and not q.Y.any()


def back_ref(gy, gh, h, w, m, s):
    """dh and its magnitudes, dw, db and theirs, in 64 bits from the given m and s."""
    g, sd, wd = gy.double(), s.double()[:, None], w.double()
    u = (h.double() - m.double()[:, None]) * sd
    n, gw = h.shape[1], g * wd
    ca, cb = gw.mean(1, keepdim=True), (gw * u).mean(1, keepdim=True)
    q = torch_zero(gh, g)
    dh = sd * (gw - ca - u * cb) + q
    mag = sd * (gw.abs() + ca.abs() + (u * cb).abs()) + q.abs()
    sums = sd * (gw.abs().sum(1, keepdim=True) + u.abs() * (gw * u).abs().sum(1, keepdim=True)) / n
    return dh, mag, sums, (g * u).sum(0), (g * u).abs().sum(0), g.sum(0), g.abs().sum(0)


def torch_zero(gh, g):
    return g * 0 if gh is None else gh.double()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES + [(2100, 96)])
def test_norm_backward(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"layer norm backward T={T} dim={dim} {dt}")
    g = gen(T * 41 + dim)
    h, gy, gh = (rand(g, T, dim, dtype=dt, scale=k) for k in (2.0, 0.1, 0.1))
    h = (h.double() + 1).to(T_(dt))
    w = 1 + 0.2 * rand(g, dim)
    md, sd, _, _ = norm_ref(h, w, None, 1e-3)
    m, s = md.float(), sd.float()
    # additions of a sum in a row: at most 32 in a lane (40 in the longest rows), then across lanes and waves
    nsum = 40 + 6 + 16
    for x, p in ((gh, 0.0), (None, 0.2), (gh, 0.2)):
        f = factor(T, dim, p, 11, 4)
        dh, mag, sums, gw, gwm, gb, gbm = back_ref(gy, x, h, w, m, s)
        kw = dict(p=p, seed=11, site=4)
        o = oec.add_layer_norm_backward(gy.cuda(), h.cuda(), w.cuda(), m.cuda(), s.cuda(),
                                        G_H=None if x is None else x.cuda(), **kw)
        tol = HALF[dt] * dh.abs() + 9 * U * mag + nsum * U * sums
        close("G_R", o.G_R, dh, tol)
        close("G_X", o.G_X, dh * f, (tol + 2 * U * dh.abs()) * f)
        assert (o.G_R is o.G_X) == (p == 0)
        # terms: u two roundings, the product one; the sums in 64 bits, parts and result rounded once each
        close("g_w", o.g_weight, gw, 6 * U * gwm)
        close("g_b", o.g_bias, gb, 2 * U * gbm)
        # the same bits strided and in place
        gs, hs = strided(gy, 5, 1), None if x is None else strided(x, 1)
        o2 = oec.add_layer_norm_backward(gs, strided(h, 2, 2), w.cuda(), m.cuda(), s.cuda(), G_H=hs, G_X=gs,
                                         G_R=hs if p else None, **kw)
        assert o2.G_X is gs and all(torch.equal(a, b) for a, b in zip(o2, o))


def test_norm_backward_by_differences():
    """The gradients against central differences of the forward in 64 bits."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    g = gen(3)
    x, r, gy, gh = (rand(g, 3, 24) for _ in range(4))
    w, b = 1 + 0.2 * rand(g, 24), 0.2 * rand(g, 24)
    kw = dict(p=0.3, seed=77, site=1)
    f = factor(3, 24, 0.3, 77, 1)
    o = oec.add_layer_norm(x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), save=True, **kw)
    q = oec.add_layer_norm_backward(gy.cuda(), o.H, w.cuda(), o.mean, o.rstd, G_H=gh.cuda(), **kw)

    def loss(v):
        h = v["x"] * f + v["r"]
        d = h - h.mean(1, keepdim=True)
        y = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * v["w"] + v["b"]
        return float((y * gy.double()).sum() + (h * gh.double()).sum())
    at = dict(x=x.double(), r=r.double(), w=w.double(), b=b.double())
    e = 1e-5
    for name, got in (("x", q.G_X), ("r", q.G_R), ("w", q.g_weight), ("b", q.g_bias)):
        for k in range(0, at[name].numel(), 5):
            d = torch.zeros_like(at[name])
            d.view(-1)[k] = e
            num = (loss({**at, name: at[name] + d}) - loss({**at, name: at[name] - d})) / (2 * e)
            # fp32 gradients of values of a few: a few u off; the differences e^2 and 2^-53 / e
            assert abs(float(got.view(-1)[k]) - num) < 1e-5, (name, k)


def test_norm_no_tokens():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x, w = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    o = oec.add_layer_norm(x, w, residual=x, save=True, p=0.5, seed=1)
    assert o.Y.shape == (0, 40) and o.rstd.shape == (0,)
    q = oec.add_layer_norm_backward(x, o.H, w, o.mean, o.rstd, p=0.5, seed=1)
    assert q.G_X.shape == (0, 40) and not q.g_weight.any() and not q.g_bias.any() and q.g_bias.shape == (40,)


def test_norm_many_rows_gradient():
    """The weight's gradient over 2^19 rows: small terms behind large ones are not lost."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    T, dim = 2 ** 19, 64
    g = torch.full((T, dim), 2.0 ** -8, device="cuda")
    g[0] = 2.0 ** 14
    h = torch.arange(dim, device="cuda", dtype=torch.float32).repeat(T, 1)
    m = torch.full((T,), (dim - 1) / 2, device="cuda")
    s = torch.full((T,), 0.0625, device="cuda")
    q = oec.add_layer_norm_backward(g, h, torch.ones(dim, device="cuda"), m, s)
    u = (torch.arange(dim, dtype=torch.float64) - (dim - 1) / 2) * 0.0625
    total = 2.0 ** 14 + (T - 1) * 2.0 ** -8
    # at most 512 partial sums and the result, each rounded once
    close("g_w", q.g_weight, u * total, 2 * U * u.abs() * total)
    close("g_b", q.g_bias, torch.full((dim,), total, dtype=torch.float64), torch.tensor(2 * U * total, dtype=torch.float64))


def test_streams_and_two_calls_at_once():
    """Calls on two streams share nothing."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    g = gen(8)
    x, w = rand(g, 700, 1000, dtype="bf16").cuda(), (1 + 0.2 * rand(g, 1000)).cuda()
    ref = oec.add_layer_norm(x, w, residual=x, p=0.1, seed=1, save=True)
    back = oec.add_layer_norm_backward(x, ref.H, w, ref.mean, ref.rstd, p=0.1, seed=1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            o = oec.add_layer_norm(x, w, residual=x, p=0.1, seed=1, save=True)
            got.append((o, oec.add_layer_norm_backward(x, o.H, w, o.mean, o.rstd, p=0.1, seed=1)))
    torch.cuda.synchronize()
    for o, b in got:
        assert torch.equal(o.Y, ref.Y) and torch.equal(o.H, ref.H) and all(torch.equal(u, v) for u, v in zip(b, back))
