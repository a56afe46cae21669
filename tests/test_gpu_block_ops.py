"""The operators around the linears against plain 64-bit implementations on the
CPU, element by element.

Tolerances count roundings: u = 2^-24 for one fp32 step (half a unit), half a
step of the output's type for its rounding (bf16 2^-8, fp32 2^-24, relative),
and for a sum of N terms the worst case over its order, N u times the sum of the
magnitudes (twice that for the matrix instructions, whose inner rounding is not
specified)."""
import math

import numpy as np
import pytest

from gpu_util import device_ready, log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def T_(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def rand(gen, *shape, dtype="f32", scale=1.0):
    import torch
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * scale).to(T_(dtype))


def gen(seed):
    import torch
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return t.detach().cpu().double()


def close(name, got, want, tol):
    """Every |got - want| <= tol (tensors of the same shape); NaN and infinities alike."""
    import torch
    got, want = f64(got), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    odd = ~fin & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), name
    d, t = (got - want).abs()[fin], tol.expand_as(want)[fin]
    bad = d > t
    if bad.any():
        i = int(torch.argmax(d / t))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {d[i]:.3e} allowed {t[i]:.3e}")


def strided(t, pad, off=0):
    """The same values on the GPU inside a wider buffer: rows pad further apart, off elements in."""
    import torch
    rows, cols = t.shape
    buf = torch.full((rows, cols + pad), 7.0 if t.is_floating_point() else 7, dtype=t.dtype, device="cuda")
    v = buf[:, off:off + cols]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ norm
def norm_ref(x, r, w, eps, dt):
    """h (in the type, as 64 bits), rstd and y in 64 bits."""
    h = x if r is None else (x.float() + r.float()).to(T_(dt))
    hd = h.double()
    s = 1 / (hd.square().mean(1) + eps).sqrt()
    return h, s, hd * s[:, None] * w.double()


def quant_ref(h, s, w):
    """The INT8 rule in its own fp32 steps: q and scale."""
    import torch
    y = (h.float() * s.float()[:, None]) * w
    a = y.abs().amax(1)
    none, bad = a < 2.0 ** -119, ~torch.isfinite(a)
    # tensor by tensor: a number over a tensor is taken as a reciprocal and a product, two roundings
    inv = torch.where(none | bad, torch.zeros_like(a), torch.full_like(a, 127) / a)
    q = torch.where((none | bad)[:, None], torch.zeros_like(y), torch.round(y * inv[:, None]))
    scale = torch.where(none, torch.zeros_like(a), a / 127)
    scale = torch.where(bad, torch.full_like(a, math.nan), scale)
    return q.to(torch.int8), scale


# one row and many, around every variant's longest row, and rows no register variant holds
NORM_SIZES = [(1, 1), (3, 7), (5, 63), (2, 64), (4, 65), (1, 2048), (7, 512), (6, 513), (3, 1000), (9, 1024),
              (4, 1365), (130, 2049), (5, 4096), (3, 4097), (2, 8200), (3, 16385), (2, 20001),
              (1030, 65), (1100, 1000), (1024, 512)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES)
def test_norm_forward(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"norm T={T} dim={dim} {dt}")
    g = gen(T * 31 + dim)
    x, r = rand(g, T, dim, dtype=dt), rand(g, T, dim, dtype=dt, scale=3.0)
    w = 1 + 0.2 * rand(g, dim)
    h, s, y = norm_ref(x, r, w, 1e-5, dt)
    # s rounded (u), two products (2 u), the sum's own error far below
    tol = (HALF[dt] + 4 * U) * y.abs()
    o = oec.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5, save=True)
    assert torch.equal(o.H.cpu(), h)
    close("Y", o.Y, y, tol)
    close("rstd", o.rstd, s, 2 * U * s)
    # without a residual; strided input; H over the residual in place
    h2, _, y2 = norm_ref(x, None, w, 1e-5, dt)
    xs = strided(x, 3, 1)
    o2 = oec.add_rms_norm(xs, w.cuda(), eps=1e-5)
    assert o2.H is xs and o2.rstd is None and o2.scale is None
    close("Y alone", o2.Y, y2, (HALF[dt] + 4 * U) * y2.abs())
    rs = strided(r, 5, 2)
    o3 = oec.add_rms_norm(xs, w.cuda(), residual=rs, eps=1e-5, H=rs)
    assert o3.H is rs and torch.equal(rs.cpu(), h) and torch.equal(o3.Y, o.Y)
    assert torch.equal(xs.cpu(), x)
    assert bool((rs.storage_offset() == 2) and (torch.as_strided(rs, (T, 2), (dim + 5, 1), 0) == 7).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES)
def test_norm_int8(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"norm int8 T={T} dim={dim} {dt}")
    g = gen(T * 37 + dim)
    x, r, w = rand(g, T, dim, dtype=dt), rand(g, T, dim, dtype=dt), 1 + 0.2 * rand(g, dim)
    for res in (r, None):
        h, s, _ = norm_ref(x, res, w, 1e-6, dt)
        q, scale = quant_ref(h, s, w)
        o = oec.add_rms_norm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), quantize=True)
        assert torch.equal(o.scale.cpu(), scale)
        assert torch.equal(o.Y.cpu(), q)
        assert int(o.Y.abs().max()) == 127
        assert torch.equal(o.H.cpu(), h)


@pytest.mark.parametrize("dim", [64, 1001, 2048, 20000])
def test_norm_special_rows(dim):
    """Zero rows, tiny and huge ones, infinities and NaN: only their own rows show it."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"norm special dim={dim}")
    g = gen(dim)
    x, w = rand(g, 8, dim), 1 + 0.2 * rand(g, dim)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, dim // 2] = math.inf
    x[5, dim - 1] = math.nan
    x[6] = 0
    x[6, 0] = 1e-38
    _, s, y = norm_ref(x, None, w, 1e-6, "f32")
    o = oec.add_rms_norm(x.cuda(), w.cuda(), save=True)
    keep = [0, 1, 2, 3, 6, 7]
    # values below the normal range round by half of 2^-149 at each of three steps
    close("Y", o.Y[keep], y[keep], 5 * U * y[keep].abs() + 2.0 ** -147)
    assert torch.isnan(o.Y[5]).all() and torch.isnan(o.Y[4, dim // 2]) and (o.Y[4, 0] == 0)
    q = oec.add_rms_norm(x.cuda(), w.cuda(), quantize=True)
    qr, sr = quant_ref(x, s, w)
    for t in (4, 5):
        assert math.isnan(float(q.scale[t])) and not q.Y[t].any()
    assert torch.equal(q.Y.cpu()[keep], qr[keep]) and torch.equal(q.scale.cpu()[keep], sr[keep])
    assert float(q.scale[1]) == 0 and not q.Y[1].any()
    # a weight below the rule's range: rows of zeros
    q = oec.add_rms_norm(x.cuda(), (w * 1e-37).cuda(), quantize=True)
    assert float(q.scale[0]) == 0 and not q.Y[0].any()


def back_ref(gy, gh, h, w, s):
    g, hd, sd = gy.double(), h.double(), s.double()[:, None]
    n = hd.shape[1]
    gw = g * w.double()
    c = (gw * hd).sum(1, keepdim=True) / n * sd * sd
    dx = sd * (gw - hd * c) + (0 if gh is None else gh.double())
    mag = (sd * gw).abs() + (sd * hd * c).abs() + (0 if gh is None else gh.double().abs())
    cmag = (gw * hd).abs().sum(1, keepdim=True) / n * sd * sd
    return dx, mag, sd * hd.abs() * cmag, (g * hd * sd).sum(0), (g * hd * sd).abs().sum(0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, dim", NORM_SIZES + [(2100, 96)])
def test_norm_backward(T, dim, dt):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"norm backward T={T} dim={dim} {dt}")
    g = gen(T * 41 + dim)
    h, gy, gh = (rand(g, T, dim, dtype=dt, scale=k) for k in (2.0, 0.1, 0.1))
    w = 1 + 0.2 * rand(g, dim)
    s = (1 / (h.double().square().mean(1) + 1e-6).sqrt()).float()
    # the dot product's additions in a row: at most 64 in a lane (dim / 256 in the long rows), then across lanes
    nsum = max(64, dim // 256 + 1) + 16
    nrow = T // 4 + 8          # rows a partial sum of g_w can have (fewer)
    for x in (gh, None):
        dx, mag, dc, gw, gwm = back_ref(gy, x, h, w, s)
        G_X, g_w = oec.add_rms_norm_backward(gy.cuda(), h.cuda(), w.cuda(), s.cuda(),
                                             G_H=None if x is None else x.cuda())
        close("G_X", G_X, dx, HALF[dt] * dx.abs() + 6 * U * mag + nsum * U * dc)
        close("g_w", g_w, gw, (nrow + 4) * U * gwm)
        # the same bits again, in place and strided
        gs = strided(gy, 5, 1)
        out, g_w2 = oec.add_rms_norm_backward(gs, strided(h, 2, 2), w.cuda(), s.cuda(),
                                              G_H=None if x is None else strided(x, 1), G_X=gs)
        assert out is gs and torch.equal(out, G_X) and torch.equal(g_w2, g_w)


def test_norm_backward_by_differences():
    """The gradients against central differences of the forward in 64 bits."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    g = gen(3)
    x, r, gy, gh = (rand(g, 3, 24) for _ in range(4))
    w = 1 + 0.2 * rand(g, 24)
    o = oec.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), save=True)
    G_X, g_w = oec.add_rms_norm_backward(gy.cuda(), o.H, w.cuda(), o.rstd, G_H=gh.cuda())

    def loss(xd, wd):
        h = xd + r.double()
        y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * wd
        return float((y * gy.double()).sum() + (h * gh.double()).sum())
    e = 1e-5
    # fp32 inputs of the gradient are a few u off; the differences are off by e^2 and 2^-53 / e
    for i in range(3):
        for j in range(0, 24, 5):
            d = torch.zeros(3, 24, dtype=torch.float64)
            d[i, j] = e
            num = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * e)
            assert abs(float(G_X[i, j]) - num) < 1e-5
    for j in range(24):
        d = torch.zeros(24, dtype=torch.float64)
        d[j] = e
        num = (loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)) / (2 * e)
        assert abs(float(g_w[j]) - num) < 1e-5


def test_norm_no_tokens():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x, w = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    o = oec.add_rms_norm(x, w, residual=x, save=True)
    assert o.Y.shape == (0, 40) and o.rstd.shape == (0,)
    G_X, g_w = oec.add_rms_norm_backward(x, o.H, w, o.rstd)
    assert G_X.shape == (0, 40) and not g_w.any() and g_w.shape == (40,)


# ------------------------------------------------------------------ linear
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act_ref(z, act):
    import torch
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def linear_case(seed, T, n, m, dt, parts):
    import torch
    g = gen(seed)
    c = dict(sx=None, sw=None, b=None, mul=None, res=None)
    yt = "f32" if dt == "f32" else "bf16"
    if dt == "int8":
        c["X"] = torch.randint(-127, 128, (T, n), generator=g, dtype=torch.int8)
        c["W"] = torch.randint(-127, 128, (m, n), generator=g, dtype=torch.int8)
        c["sx"], c["sw"] = rand(g, T).abs() * 0.01, rand(g, m).abs() * 0.02 / math.sqrt(n)
    else:
        c["X"], c["W"] = rand(g, T, n, dtype=dt), rand(g, m, n, dtype=dt, scale=1 / math.sqrt(n))
    if "b" in parts:
        c["b"] = rand(g, m)
    if "m" in parts:
        c["mul"] = rand(g, T, m, dtype=yt)
    if "r" in parts:
        c["res"] = rand(g, T, m, dtype=yt)
    return c


def linear_ref(c, act, half):
    """The result in 64 bits and what its elements may be off."""
    X, W = c["X"].double(), c["W"].double()
    n = X.shape[1]
    z, zt = X @ W.T, (X.abs() @ W.abs().T) * ((n + 8) * 2 * U)
    if c["sx"] is not None:
        k = c["sx"].double()[:, None] * c["sw"].double()
        z, zt = z * k, (z * k).abs() * 4 * U      # the sum is exact: its conversion and two products
    if c["b"] is not None:
        z = z + c["b"].double()
        zt = zt + z.abs() * U
    v = act_ref(z, act)
    # slopes up to 1.13; the hardware's exp2 of a product is |z| u off its exponent, its reciprocal 2 u; the
    # cube inside gelu_tanh multiplies its own few u by the exponent's size
    steps = {"none": 0, "relu": 0, "silu": z.abs() + 8, "gelu": 8, "gelu_tanh": 8 * z.abs() + 8 * z.abs() ** 3 + 8}[act]
    vt = 1.2 * zt + 4 * U * steps * v.abs() + 4 * U * z.abs() * (act != "none")
    if c["mul"] is not None:
        v = v * c["mul"].double()
        vt = vt * c["mul"].double().abs() + U * v.abs()
    if c["res"] is not None:
        v = v + c["res"].double()
        vt = vt + U * v.abs()
    # a value near the smallest normal loses its last bits
    return v, vt * (1 + 2.0 ** -7) + half * v.abs() + 2.0 ** -126


def run_linear(c, act, **kw):
    import orthogonal_equivalence_cayley_amd as oec
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    a = dict(bias=dev(c["b"]), act=act, mul=dev(c["mul"]), residual=dev(c["res"]), x_scale=dev(c["sx"]),
             w_scale=dev(c["sw"]))
    a.update(kw)
    X, W = a.pop("X", None), a.pop("W", None)
    return oec.linear(dev(c["X"]) if X is None else X, dev(c["W"]) if W is None else W, **a)


LINEAR_SIZES = [(1, 1, 1), (1, 64, 16), (1, 2048, 300), (1, 77, 129), (2, 1000, 33), (3, 136, 40), (4, 4112, 17),
                (5, 64, 64), (7, 100, 50), (16, 256, 130), (17, 333, 31), (24, 4096, 48), (33, 512, 100),
                (64, 1040, 96), (65, 64, 128), (100, 1, 100), (127, 8, 5), (128, 128, 128), (129, 100, 257),
                (256, 2048, 256), (300, 1005, 200), (513, 320, 256), (1031, 192, 384), (2000, 130, 77),
                (14, 7184, 76), (33, 4112, 100), (9, 5311, 256), (40, 16400, 33), (6, 16384, 40), (70, 6160, 70)]


@pytest.mark.parametrize("dt", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("T, n, m", LINEAR_SIZES)
def test_linear(T, n, m, dt):
    log(f"linear T={T} n={n} m={m} {dt}")
    half = HALF["f32" if dt == "f32" else "bf16"]
    for i, (act, parts) in enumerate([("none", ""), ("silu", "m"), ("none", "r")]):
        c = linear_case(T * 101 + n * 7 + m + i, T, n, m, dt, parts)
        v, tol = linear_ref(c, act, half)
        close(f"{act} {parts}", run_linear(c, act), v, tol)


# grids that take each tile, with whole rows of 128 bytes and with ragged ones; ends inside tiles
@pytest.mark.parametrize("dt", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("T, m", [(30, 2047), (130, 4096), (500, 2040), (1030, 2040), (4090, 2056), (16380, 1032),
                                  (16390, 1032)])
@pytest.mark.parametrize("n", [70, 48, 208, 256])
def test_linear_tiles(T, n, m, dt):
    """Every part of the epilogue, written over the residual; the rows behind stay as they were."""
    import torch
    log(f"linear tiles T={T} n={n} m={m} {dt}")
    c = linear_case(T + n + m, T, n, m, dt, "bmr")
    v, tol = linear_ref(c, "silu", HALF["f32" if dt == "f32" else "bf16"])
    buf = torch.full((T + 300, m + 8), 3.0, dtype=c["res"].dtype, device="cuda")
    res = buf[:T, :m]
    res.copy_(c["res"])
    y = run_linear(c, "silu", residual=res, out=res)
    close("over the residual", y, v, tol)
    assert bool((buf[T:] == 3).all()) and bool((buf[:, m:] == 3).all())
    first = y.clone()
    res.copy_(c["res"])
    assert torch.equal(run_linear(c, "silu", residual=res, out=res), first)   # the same bits again


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("T, n, m", [(1, 80, 70), (20, 96, 70), (150, 72, 131), (600, 256, 260)])
def test_linear_epilogues(T, n, m, dt, act):
    log(f"linear {act} T={T} {dt}")
    half = HALF["f32" if dt == "f32" else "bf16"]
    for parts in ("b", "bmr", "br"):
        c = linear_case(len(parts) * 13 + T, T, n, m, dt, parts)
        v, tol = linear_ref(c, act, half)
        close(parts, run_linear(c, act), v, tol)


@pytest.mark.parametrize("dt", ["bf16", "int8"])
@pytest.mark.parametrize("T, n, m", [(1, 200, 72), (20, 256, 72), (200, 200, 72), (700, 256, 520), (16390, 128, 1032)])
def test_linear_fp32_result(T, n, m, dt):
    import torch
    for act, parts in (("none", "b"), ("relu", "bmr")):
        c = linear_case(T, T, n, m, dt, parts)
        c["mul"], c["res"] = (None if t is None else t.float() for t in (c["mul"], c["res"]))
        v, tol = linear_ref(c, act, HALF["f32"])
        y = run_linear(c, act, out_dtype=torch.float32)
        assert y.dtype == torch.float32
        close("fp32", y, v, tol)


@pytest.mark.parametrize("dt", ["bf16", "f32", "int8"])
@pytest.mark.parametrize("T, n, m", [(1, 65, 30), (3, 128, 64), (18, 200, 40), (90, 130, 66), (400, 256, 512)])
def test_linear_strides_and_in_place(T, n, m, dt):
    """Rows apart, unaligned starts, results over the residual or the gating operand; what lies beside them stays."""
    import torch
    log(f"linear strided T={T} n={n} m={m} {dt}")
    c = linear_case(5 * T, T, n, m, dt, "mr")
    half = HALF["f32" if dt == "f32" else "bf16"]
    v, tol = linear_ref(c, "silu", half)
    plain = run_linear(c, "silu")
    close("plain", plain, v, tol)
    for over in ("res", "mul", None):
        X, W = strided(c["X"], 3, 1), strided(c["W"], 5, 3)
        mul, res = strided(c["mul"], 7, 5), strided(c["res"], 2, 1)
        out = {"res": res, "mul": mul, None: strided(torch.zeros_like(c["res"]), 9, 4)}[over]
        y = run_linear(c, "silu", X=X, W=W, mul=mul, residual=res, out=out)
        assert y is out
        close(f"over {over}", y, v, tol)
        buf = torch.as_strided(out, (T, out.stride(0)) if T > 1 else (1, out.shape[1] + 1),
                               (out.stride(0), 1), 0)
        k = out.storage_offset()
        assert bool((buf[:, :k] == 7).all()) and bool((buf[:, k + m:] == 7).all())
    # no row behind the last is written
    big = torch.full((T + 40, m), 5.0, dtype=plain.dtype, device="cuda")
    run_linear(c, "silu", out=big[:T])
    assert bool((big[T:] == 5).all())
    assert torch.equal(big[:T], plain)


def test_linear_special_values():
    """Infinities and NaN of one token or one weight row stay in its row or column."""
    import torch
    for T in (1, 2, 20, 130, 300):
        c = linear_case(T, T, 256, 256, "bf16", "")
        base = run_linear(c, "none")
        c["X"][T - 1, 3], c["W"][5, 7] = math.nan, math.inf
        y = run_linear(c, "none")
        assert torch.isnan(y[T - 1]).all()
        assert torch.isinf(y[:T - 1, 5]).all()
        keep = [j for j in range(256) if j != 5]
        assert torch.equal(y[:T - 1, keep], base[:T - 1, keep])
    c = linear_case(1, 130, 64, 32, "int8", "")
    c["sx"][7] = math.nan   # the row a norm could not quantise
    y = run_linear(c, "none")
    assert torch.isnan(y[7]).all() and torch.isfinite(y[8]).all()


def test_linear_no_tokens():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    y = oec.linear(torch.empty(0, 16, device="cuda"), torch.ones(8, 16, device="cuda"))
    assert y.shape == (0, 8)


@pytest.mark.parametrize("T", [2, 40, 600])
def test_linear_int8_largest_sum(T):
    """131071 products of 128 * 128, exact below 2^31."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    n = 131071
    X = torch.full((T, n), -128, dtype=torch.int8, device="cuda")
    W = torch.full((3, n), -128, dtype=torch.int8, device="cuda")
    W[1] = 127
    one = lambda k: torch.ones(k, device="cuda")  # noqa: E731
    y = oec.linear(X, W, x_scale=one(T), w_scale=one(3), out_dtype=torch.float32)
    want = torch.tensor([128 * 128 * n, -128 * 127 * n, 128 * 128 * n], dtype=torch.float64).float()
    assert torch.equal(y.cpu(), want.expand(T, 3))


@pytest.mark.parametrize("dt", ["bf16", "int8"])
def test_rows_beyond_32_bits(dt):
    """Rows so far apart that byte offsets pass 2^32, in every operator that takes row strides."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    T, n, m = 70, 128, 48
    ld = (2 ** 32 + 2 ** 20) // 60 // (2 if dt == "bf16" else 1) // 16 * 16
    log(f"far rows {dt}: {T * ld} elements")
    c = linear_case(9, T, n, m, dt, "")
    buf = torch.empty(T, ld, dtype=c["X"].dtype, device="cuda")
    X = buf[:, 32:32 + n]
    X.copy_(c["X"])
    v, tol = linear_ref(c, "none", HALF["bf16"])
    close("linear", run_linear(c, "none", X=X), v, tol)
    W = torch.empty(T, ld, dtype=c["X"].dtype, device="cuda")[:m, :n]
    W.copy_(c["W"])
    close("far weight", run_linear(c, "none", W=W), v, tol)
    if dt == "bf16":
        w = 1 + 0.2 * rand(gen(1), n)
        h, s, y = norm_ref(c["X"], None, w, 1e-6, "bf16")
        o = oec.add_rms_norm(X, w.cuda(), save=True)
        close("norm", o.Y, y, (HALF["bf16"] + 4 * U) * y.abs())
        G = c["X"].flip(1).contiguous().cuda()
        want, gw = oec.add_rms_norm_backward(G, c["X"].cuda(), w.cuda(), o.rstd)
        got, gw2 = oec.add_rms_norm_backward(G, X, w.cuda(), o.rstd)
        assert torch.equal(got, want) and torch.equal(gw, gw2)


def test_linear_activations_of_infinities():
    """+inf of a sum passes every activation; large negative sums end at zero."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    for dt in (torch.bfloat16, torch.float32):
        for T in (1, 40, 300):
            X = torch.zeros(T, 64, dtype=dt, device="cuda")
            X[:, 0] = 1
            W = torch.zeros(24, 64, dtype=dt, device="cuda")
            W[0, 0], W[1, 0], W[2, 0] = math.inf, -1e30, 1e30
            for act in ACTS:
                y = oec.linear(X, W, act=act).double()
                assert bool((y[:, 0] == math.inf).all()), (act, T)
                assert bool((y[:, 2] == float(W[2, 0])).all()) and bool((y[:, 3:] == 0).all())
                assert bool((y[:, 1] == (float(W[1, 0]) if act == "none" else 0)).all())


# ------------------------------------------------------------------ large
def test_norm_past_4_gib():
    """Rows past 2^32 bytes, and more of them than one launch counts."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    for T, dim in ((1100003, 2048), (2 ** 23 + 5, 8)):
        log(f"norm {T} x {dim}")
        g = torch.Generator("cuda").manual_seed(T)
        x = torch.empty(T, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        w = (1 + 0.2 * rand(gen(1), dim))
        rows = torch.tensor([0, 1, T // 2, 2 ** 20 + 1, T - 6, T - 1])
        xc = x[rows.cuda()].cpu()
        h, s, y = norm_ref(xc, xc, w, 1e-6, "bf16")
        o = oec.add_rms_norm(x, w.cuda(), residual=x, save=True, H=x)
        close("h", x[rows.cuda()], h.double(), torch.zeros(1, dtype=torch.float64))
        close("y", o.Y[rows.cuda()], y, (HALF["bf16"] + 4 * U) * y.abs())
        close("rstd", o.rstd[rows.cuda()], s, 2 * U * s)
        G_X, g_w = oec.add_rms_norm_backward(o.Y, x, w.cuda(), o.rstd, G_X=o.Y)
        dx, mag, dc, _, _ = back_ref(y.bfloat16(), None, h, w, s.float())
        # the gradient is y itself, rounded: 2^-8 of it through a linear map of slope s w and s h c
        close("dx", G_X[rows.cuda()], dx, HALF["bf16"] * dx.abs() + 80 * U * (mag + dc) + HALF["bf16"] * 2 * (mag + dc))
        assert torch.isfinite(g_w).all()
        del x, o, G_X


def test_linear_past_4_gib():
    """Activations past 2^32 bytes, and a result of more than 2^32 elements."""
    import torch
    for T, n, m, dt in ((1100003, 2048, 264, "bf16"), (2100001, 2048, 256, "int8"), (1100003, 64, 4096, "bf16"),
                        (1100003, 1001, 40, "bf16")):
        import orthogonal_equivalence_cayley_amd as oec
        log(f"linear {T} x {n} -> {m} {dt}")
        g = torch.Generator("cuda").manual_seed(T)
        kw = {}
        if dt == "int8":
            X = torch.empty(T, n, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
            W = torch.empty(m, n, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
            kw = dict(x_scale=torch.rand(T, device="cuda", generator=g) * 0.01,
                      w_scale=torch.rand(m, device="cuda", generator=g) * 0.001)
        else:
            X = torch.empty(T, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            W = torch.empty(m, n, dtype=torch.bfloat16, device="cuda").normal_(0, n ** -0.5, generator=g)
        y = oec.linear(X, W, **kw)
        rows = torch.tensor([0, 255, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 300, T - 257, T - 256, T - 1]).cuda()
        c = dict(X=X[rows].cpu(), W=W.cpu(), sx=None, sw=None, b=None, mul=None, res=None)
        if dt == "int8":
            c.update(sx=kw["x_scale"][rows].cpu(), sw=kw["w_scale"].cpu())
        v, tol = linear_ref(c, "none", HALF["bf16"])
        close("rows", y[rows], v, tol)
        del X, W, y


def test_clip_past_4_gib():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    for dt, n in ((torch.float32, 2 ** 30 + 12345), (torch.bfloat16, 2 ** 31 + 77)):
        log(f"clip {n} {dt}")
        g = torch.full((n,), 0.5, dtype=dt, device="cuda")
        g[-1] = 1.0
        norm = math.sqrt(0.25 * (n - 1) + 1)
        got = oec.clip_grads([g], 1.0, out=[g])
        assert abs(float(got) - norm) <= 2 * U * norm
        c = torch.tensor(1.0 / (norm + 1e-6), dtype=torch.float64)
        half = HALF["bf16" if dt == torch.bfloat16 else "f32"]
        for i, v in ((0, 0.5), (n // 2, 0.5), (n - 2, 0.5), (n - 1, 1.0)):
            assert abs(float(g[i]) - v * float(c)) <= (half + 2 * U) * v * float(c)
        del g


# ------------------------------------------------------------------ clip
def clip_ref(grads, max_norm):
    import torch
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.double() * c for g in grads], c


def check_clip(grads, max_norm, where):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    norm, want, c = clip_ref(grads, max_norm)
    dev = [g.cuda() for g in grads]
    keep = [g.clone() for g in dev]

    def off(g, w):
        # c and the product rounded, then the type; subnormals by half of their step
        half = HALF["bf16" if g.dtype == torch.bfloat16 else "f32"] if c < 1 else 0.0
        return (half + 2 * U) * w.abs() + 2.0 ** -133
    n = oec.clip_grads(dev, max_norm)
    assert abs(float(n) - norm) <= 2 * U * norm
    assert all(torch.equal(a, b) for a, b in zip(dev, keep))
    outs = [torch.full_like(g, 3.0) for g in dev]
    n2 = oec.clip_grads(dev, max_norm, out=outs)
    assert torch.equal(n, n2) and all(torch.equal(a, b) for a, b in zip(dev, keep))
    for i, (g, o, w) in enumerate(zip(grads, outs, want)):
        close(f"{where} out {i}", o, w, off(g, w))
    n3 = oec.clip_grads(dev, max_norm, out=dev)
    assert torch.equal(n, n3) and all(torch.equal(a, b) for a, b in zip(dev, outs))


@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
def test_clip_sizes(max_norm):
    g = gen(1)
    sizes = [1, 2, 3, 4, 7, 8, 9, 255, 256, 1023, 1025, 8191, 8192, 8193, 100003]
    grads = [rand(g, n, dtype="bf16" if i % 3 == 1 else "f32", scale=0.02) for i, n in enumerate(sizes)]
    log(f"clip sizes max_norm={max_norm}")
    check_clip(grads, max_norm, "sizes")


@pytest.mark.parametrize("count", [1, 119, 120, 121, 500, 1300])
def test_clip_many_tensors(count):
    """Around the tensors of one launch, and more partial sums than a workgroup adds up itself."""
    g = gen(count)
    n = 9000 if count < 600 else 70000
    log(f"clip {count} tensors")
    check_clip([rand(g, 1 + (i * 977) % n, dtype="bf16" if i % 5 == 0 else "f32") for i in range(count)], 1.0,
               f"{count} tensors")


def test_clip_many_partial_sums():
    """800 tensors cut from 288 MB: more than the caches hold, more sums than a workgroup adds up."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    flat = torch.randn(800 * 90000, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    parts = list(torch.split(flat, 90000))
    norm = float(flat.double().square().sum().sqrt())
    n = oec.clip_grads(parts, 2.0, out=parts)
    assert abs(float(n) - norm) <= 2 * U * norm
    assert abs(float(flat.double().square().sum().sqrt()) - 2.0) <= 2e-6


def test_clip_views_at_any_element():
    """Tensors cut out of one buffer at odd places, and empty ones between them."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    for dt in ("bf16", "f32"):
        flat = rand(gen(2), 50001, dtype=dt)
        sizes = [1, 0, 3, 17, 8192, 0, 20000, 5, 21783]
        norm, (want,), c = clip_ref([flat], 1.0)
        d = flat.cuda()
        n = oec.clip_grads(torch.split(d, sizes), 1.0, out=torch.split(d, sizes))
        assert abs(float(n) - norm) <= 2 * U * norm
        close(dt, d, want, (HALF[dt] + 2 * U) * want.abs() + 2.0 ** -133)
    e = torch.empty(0, device="cuda")
    assert float(oec.clip_grads([e], 1.0, out=[e])) == 0.0


def test_clip_range_and_special_values():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    big = torch.full((1000,), 1e30, device="cuda")     # squares past fp32
    n = oec.clip_grads([big], 1.0, out=[big])
    assert abs(float(n) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    close("big", big, torch.full((1000,), 1 / math.sqrt(1000), dtype=torch.float64), torch.tensor(1e-7))
    small = torch.full((1000,), 1e-30, device="cuda")  # squares below it
    assert abs(float(oec.clip_grads([small], 1.0)) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6
    a, b = torch.ones(5, device="cuda"), torch.ones(9, device="cuda")
    b[3] = math.inf
    n = oec.clip_grads([a, b], 1.0, out=[a, b])
    assert math.isinf(float(n)) and not a.any() and math.isnan(float(b[3])) and float(b[2]) == 0
    a, b = torch.ones(5, device="cuda"), torch.ones(9, device="cuda")
    b[3] = math.nan
    n = oec.clip_grads([a, b], 1.0, out=[a, b])
    assert math.isnan(float(n)) and torch.isnan(a).all() and torch.isnan(b).all()


def test_clip_refuses():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    a, b = torch.ones(8, 8, device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: oec.clip_grads([a.T[:, :4]], 1.0), lambda: oec.clip_grads([a.double()], 1.0),
                lambda: oec.clip_grads([a, b], 1.0, out=[a]), lambda: oec.clip_grads([a], 1.0, out=[b[:60]]),
                lambda: oec.clip_grads([a], 1.0, out=[a.bfloat16()])):
        with pytest.raises(ValueError):
            bad()
    from orthogonal_equivalence_cayley_amd.poetx import PoetxError
    for bad in (lambda: oec.clip_grads([a, a], 1.0, out=[a, a]), lambda: oec.clip_grads([b], math.inf),
                lambda: oec.clip_grads([b[:40], b[30:]], 1.0, out=[b[:40], b[30:]])):
        with pytest.raises(PoetxError):
            bad()
    assert float(oec.clip_grads([a, a], 1.0)) == pytest.approx(math.sqrt(128))   # the norm alone may read twice
    assert bool((a == 1).all())


# ------------------------------------------------------------------ streams, graphs, the run of them
def test_other_stream():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    c = linear_case(3, 300, 256, 128, "bf16", "r")
    want = run_linear(c, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_linear(c, "silu")
        grads = [got.float(), got.clone()]
        n = oec.clip_grads(grads, 1.0, out=grads)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    assert abs(float(n) - math.sqrt(2 * float(want.double().square().sum()))) < 1e-4 * float(n)


def test_graphs_share_nothing():
    """Two captured graphs of the same operators, replayed in turn with eager work between."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    g = gen(8)
    T, dim, ff = 37, 256, 512
    w = (1 + 0.1 * rand(g, dim)).cuda()
    Wu = rand(g, ff, dim, dtype="bf16", scale=1 / 16).cuda()
    Wd = rand(g, dim, ff, dtype="bf16", scale=1 / 23).cuda()

    def run(x, r, gy):
        o = oec.add_rms_norm(x, w, residual=r, save=True)
        u = oec.linear(o.Y, Wu, act="silu")
        y = oec.linear(u, Wd, residual=o.H)
        gx, gw = oec.add_rms_norm_backward(gy, o.H, w, o.rstd, G_H=y)
        grads = [gx, gw]
        outs = [torch.empty_like(t) for t in grads]
        n = oec.clip_grads(grads, 1.0, out=outs)
        return [o.Y, y, gx, gw, n] + outs

    ins = [[rand(g, T, dim, dtype="bf16").cuda() for _ in range(3)] for _ in range(2)]
    graphs, outs = [], []
    for x in ins:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(*x)
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run(*x))
        graphs.append(gr)
    for it in range(4):
        for x in ins:
            for t in x:
                t.mul_(1.0 + 0.25 * it)
        want = [[t.clone() for t in run(*x)] for x in ins]
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b)), it


def test_shared_sums_on_two_streams_and_graphs():
    """Products whose n several workgroups share: calls side by side on two streams, and two graphs of them
    replayed side by side, each have sums of their own."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    from orthogonal_equivalence_cayley_amd import poetx as px
    g = gen(12)
    T, n, m = 9, 16384, 72
    assert px.LIB.poetx_linear_workspace(px.LinearDesc(T, m, n, px.POETX_BF16, px.POETX_BF16, 0)) > 0
    W = rand(g, m, n, dtype="bf16", scale=1 / 128).cuda()
    xs = [rand(g, T, n, dtype="bf16").cuda() for _ in range(2)]
    want = [oec.linear(x, W) for x in xs]
    assert not torch.equal(want[0], want[1])
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(oec.linear(x, W))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for x in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append([oec.linear(x, W) for _ in range(3)])
        graphs.append(gr)
    for it in range(4):
        for x in xs:
            x.mul_(1.25)
        want = [oec.linear(x, W) for x in xs]
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert all(torch.equal(y, v) for y in o), it


def test_merged_block():
    """A feed-forward as it is served: norm, gate and up and down with merged POET-X layers, dense and INT8."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    import oracle
    import workloads
    from gpu_util import make_layer
    h, ff = 256, 512
    inps = [workloads.small_case(m, n, (128,) * (m // 128), (128,) * (n // 128), T=4, seed=i, dtype="bf16",
                                 theta_std=0.01) for i, (m, n) in enumerate([(ff, h), (ff, h), (h, ff)])]
    layers = [make_layer(i, 4, "bf16") for i in inps]
    for L in layers:
        L.build()
    dense = [L.merged() for L in layers]
    int8 = [L.merged(weight="int8") for L in layers[:2]]
    g = gen(0)
    for T in (1, 9, 140, 512):
        x, r = rand(g, T, h, dtype="bf16"), rand(g, T, h, dtype="bf16")
        w = 1 + 0.1 * rand(g, h)
        W = [f64(d.W) for d in dense]
        hd, _, y = norm_ref(x, r, w, 1e-6, "bf16")
        want = hd.double() + (act_ref(y @ W[0].T, "silu") * (y @ W[1].T)) @ W[2].T
        o = oec.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
        up = dense[1].forward(o.Y)
        a = dense[0].forward(o.Y, act="silu", mul=up, out=up)
        out = dense[2].forward(a, residual=o.H, out=o.H)
        # bf16 roundings of y, up, a and the result, each 2^-8 relative
        assert oracle.rel_fro(f64(out).numpy(), want.numpy()) < 4 * 2.0 ** -8
        q = oec.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), quantize=True)
        for d, i in zip(dense, int8):
            wq = f64(i.W) * f64(i.w_scale)[:, None]
            # half a step of the INT8 grid of each row
            assert float((wq - f64(d.W)).abs().max()) <= float(i.w_scale.max()) * 0.5 * (1 + 1e-5)
            yq = f64(q.Y) * f64(q.scale)[:, None]
            got = i.forward(q.Y, x_scale=q.scale)
            assert oracle.rel_fro(f64(got).numpy(), (yq @ wq.T).numpy()) < 2.0 ** -8
    # the layer itself: its forward on a token equals the merged product up to the roundings of its stages
    X = rand(g, 16, h, dtype="bf16").cuda()
    y0, y1 = layers[0].forward(X, save=False), dense[0].forward(X)
    assert oracle.rel_fro(f64(y1).numpy(), f64(y0).numpy()) < 2e-2


def test_trained_block_step_clips():
    """The block's step with clip_norm: the parameter gradients of the step without it, clipped as documented."""
    import torch
    import workloads
    from orthogonal_equivalence_cayley_amd.block_step import BlockStep
    inps = []
    for i, (name, m, n) in enumerate([("q", 256, 256), ("gate", 512, 256), ("down", 256, 512)]):
        inp = workloads.small_case(m, n, (128,) * (m // 128), (128,) * (n // 128), T=64, seed=i, dtype="bf16",
                                   theta_std=0.01)
        inp.spec = workloads.LayerSpec(name, m, n, inp.spec.bsz_R, inp.spec.bsz_P)
        inps.append(inp)
    plain, clipped = BlockStep(inps, 4), BlockStep(inps, 4, clip_norm=0.75)
    for b in (plain, clipped):
        b.step()
        b.step()
    torch.cuda.synchronize()
    grads = [t.cpu() for b in plain.bufs for t in b["g"]]
    norm, want, c = clip_ref(grads, 0.75)
    assert c < 1 and abs(float(clipped.grad_norm) - norm) <= 2 * U * norm
    for w, t in zip(want, (t for b in clipped.bufs for t in b["g"])):
        close("clipped", t, w, 4 * U * w.abs() + 2.0 ** -149)
    assert plain.grad_norm is None


def test_norm_and_layer_trained_together():
    """norm -> POET-X layer -> backward of both -> one clip over all their gradients, against differences."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    import oracle
    import workloads
    from gpu_util import make_layer
    inp = workloads.small_case(96, 64, (32, 32, 32), (32, 32), T=12, seed=4, dtype="f32", theta_std=0.05)
    L = make_layer(inp, 3, "f32")
    L.build()
    g = gen(6)
    x, r, w = rand(g, 12, 64), rand(g, 12, 64), 1 + 0.1 * rand(g, 64)
    o = oec.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), save=True)
    Y = L.forward(o.Y)
    G = torch.from_numpy(inp.G_Y).cuda()
    G_N, gR, gP = L.backward(o.Y, G)
    G_X, g_w = oec.add_rms_norm_backward(G_N, o.H, w.cuda(), o.rstd)
    Wm = f64(L.merge())
    hd = x.double() + r.double()

    def loss(h, ww):
        return float(((h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * ww) @ Wm.T * torch.from_numpy(inp.G_Y).double()).sum())
    e = 1e-5
    scale = float(f64(G_X).abs().max())
    for i, j in ((0, 0), (3, 17), (11, 63)):
        d = torch.zeros_like(hd)
        d[i, j] = e
        num = (loss(hd + d, w.double()) - loss(hd - d, w.double())) / (2 * e)
        assert abs(float(G_X[i, j]) - num) < 1e-5 * max(scale, 1.0)
    grads = [gR, gP, g_w]
    norm, want, _ = clip_ref([t.cpu() for t in grads], 0.1)
    n = oec.clip_grads(grads, 0.1, out=grads)
    assert abs(float(n) - norm) <= 2 * U * norm
    for t, v in zip(grads, want):
        close("clipped", t, v, 4 * U * v.abs() + 2.0 ** -149)
