"""Host-only checks of the calls around the linears (norm, merged-weight product,
gradient clipping): every refusal has its documented status and comes before
anything is launched, so fake addresses are safe here."""
import ctypes

import pytest

from orthogonal_equivalence_cayley_amd import poetx as px

L = px.LIB
# far apart: no two of these buffers overlap at the sizes used below
A, B, C, D, E, F, G, H = (0x100000 * (i + 1) for i in range(8))
MAX64 = 2 ** 62


def norm(T=4, dim=64, dtype=px.POETX_BF16, y_dtype=None, ld=(64, 64, 64, 64), eps=1e-6, X=A, R=B, w=C, Hp=D,
         Y=E, scale=None, rstd=F, null=False):
    d = px.NormDesc(T, dim, dtype, dtype if y_dtype is None else y_dtype, *ld, eps)
    return L.poetx_add_rms_norm(None if null else d, X, R, w, Hp, Y, scale, rstd, None)


INV, SHAPE, DTYPE, ALIGN, UNSUP, WS = (px.POETX_ERR_INVALID_ARG, px.POETX_ERR_SHAPE, px.POETX_ERR_DTYPE,
                                      px.POETX_ERR_ALIGNMENT, px.POETX_ERR_UNSUPPORTED, px.POETX_ERR_WORKSPACE)


@pytest.mark.parametrize("kw, status", [
    (dict(T=0), px.POETX_OK),
    (dict(T=0, X=None, Y=None, w=None), px.POETX_OK),
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=2 ** 24 + 1), SHAPE),
    (dict(dtype=px.POETX_INT8), DTYPE), (dict(dtype=7), DTYPE), (dict(y_dtype=px.POETX_FP32), DTYPE),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(X=None), INV), (dict(w=None), INV), (dict(Y=None), INV),
    (dict(scale=G), INV),                              # a scale without INT8 rows
    (dict(y_dtype=px.POETX_INT8), INV),                # INT8 rows without a scale
    (dict(ld=(63, 64, 64, 64)), SHAPE), (dict(ld=(64, 0, 64, 64)), SHAPE), (dict(ld=(64, 64, -64, 64)), SHAPE),
    (dict(ld=(64, 64, 64, MAX64)), SHAPE),
    (dict(X=A + 1), ALIGN), (dict(w=C + 2), ALIGN), (dict(rstd=F + 2), ALIGN),
    (dict(y_dtype=px.POETX_INT8, scale=G + 1), ALIGN),
    (dict(Y=A), INV), (dict(Y=D), INV), (dict(Y=B + 128), INV), (dict(Hp=C), INV), (dict(rstd=E), INV),
    (dict(Hp=A + 2), INV),                             # h a little behind x
    (dict(Hp=A, ld=(64, 64, 128, 64)), INV),           # the start of x, but other rows
    (dict(Y=A + 64, ld=(96, 64, 64, 96)), INV),        # side by side, but the columns meet
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def norm_back(T=4, dim=64, dtype=px.POETX_BF16, ld=(64, 64, 64, 64), g=A, gh=B, h=C, w=D, rstd=E, gx=F, gw=G,
              ws=H, wsb=None, null=False):
    d = px.NormBackwardDesc(T, dim, dtype, *ld)
    wsb = L.poetx_rms_norm_backward_workspace(max(T, 0) % 2 ** 31, max(dim, 1)) if wsb is None else wsb
    return L.poetx_rms_norm_backward(None if null else d, g, gh, h, w, rstd, gx, gw, ws, wsb, None)


@pytest.mark.parametrize("kw, status", [
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(dim=0), SHAPE),
    (dict(dtype=px.POETX_INT8), DTYPE), (dict(gw=None), INV), (dict(gw=G + 1), ALIGN),
    (dict(g=None), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(rstd=None), INV), (dict(gx=None), INV),
    (dict(ld=(63, 64, 64, 64)), SHAPE), (dict(ld=(64, 64, 64, 1)), SHAPE),
    (dict(g=A + 1), ALIGN), (dict(gx=F + 1), ALIGN), (dict(ws=H + 8), ALIGN),
    (dict(ws=None), WS), (dict(wsb=0), WS), (dict(wsb=100), WS),
    (dict(gx=C), INV),                                 # in place over h: it is read again
    (dict(gx=A + 2), INV), (dict(gw=D), INV), (dict(gw=F), INV), (dict(ws=A), INV),
    (dict(gx=A, ld=(64, 64, 64, 128)), INV),
])
def test_norm_backward_refusals(kw, status):
    assert norm_back(**kw) == status


def test_norm_backward_workspace():
    f = L.poetx_rms_norm_backward_workspace
    assert f(-1, 8) == 0 and f(2 ** 31, 8) == 0 and f(4, 0) == 0 and f(4, 2 ** 24 + 1) == 0
    assert f(0, 8) > 0
    assert f(1000, 64) >= 4 * 64 * (1000 // 4)
    # rows longer than any register variant keep one more value each
    assert f(100000, 20000) >= 4 * 100000 + 4 * 20000


def linear(T=4, m=32, n=64, dtype=px.POETX_BF16, y_dtype=px.POETX_BF16, act=0, ld=(64, 64, 32, 32, 32), X=A, W=B,
           sx=None, sw=None, bias=C, mul=D, res=E, Y=F, null=False, ws=None, wsb=0):
    d = px.LinearDesc(T, m, n, dtype, y_dtype, act, *ld)
    return L.poetx_linear(None if null else d, X, W, sx, sw, bias, mul, res, Y, ws, wsb, None)


Q = dict(dtype=px.POETX_INT8, sx=G, sw=H)
LONG = dict(T=8, n=16384, ld=(16384, 16384, 32, 32, 32))


@pytest.mark.parametrize("kw, status", [
    (dict(T=0), px.POETX_OK), (dict(T=0, X=None, Y=None), px.POETX_OK),
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(m=0), SHAPE), (dict(n=0), SHAPE),
    (dict(m=2 ** 24 + 1), SHAPE),
    (dict(dtype=3), DTYPE), (dict(y_dtype=px.POETX_INT8), DTYPE), (dict(dtype=px.POETX_FP32), DTYPE),
    (dict(act=-1), INV), (dict(act=5), INV),
    (dict(Q, n=131072, ld=(131072, 131072, 32, 32, 32)), UNSUP),
    (dict(X=None), INV), (dict(W=None), INV), (dict(Y=None), INV),
    (dict(sx=G), INV), (dict(sw=H), INV), (dict(Q, sx=None), INV), (dict(Q, sw=None), INV),
    (dict(ld=(63, 64, 32, 32, 32)), SHAPE), (dict(ld=(64, 63, 32, 32, 32)), SHAPE),
    (dict(ld=(64, 64, 31, 32, 32)), SHAPE), (dict(ld=(64, 64, 32, 31, 32)), SHAPE),
    (dict(ld=(64, 64, 32, 32, 31)), SHAPE), (dict(ld=(MAX64, 64, 32, 32, 32)), SHAPE),
    (dict(X=A + 1), ALIGN), (dict(W=B + 1), ALIGN), (dict(Y=F + 1), ALIGN), (dict(bias=C + 2), ALIGN),
    (dict(Q, sx=G + 2), ALIGN), (dict(mul=D + 1), ALIGN), (dict(res=E + 1), ALIGN),
    (dict(Y=A), INV), (dict(Y=B), INV), (dict(Y=C), INV), (dict(Y=D + 2), INV), (dict(Y=E + 64), INV),
    (dict(Q, Y=G), INV), (dict(Y=D, ld=(64, 64, 64, 32, 32)), INV),
    # a long n, shared by workgroups whose sums need room
    (dict(LONG), WS), (dict(LONG, ws=H), WS), (dict(LONG, ws=H + 8, wsb=1 << 20), ALIGN),
    (dict(LONG, ws=A, wsb=1 << 20), INV), (dict(LONG, ws=F, wsb=1 << 20), INV),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace():
    f = L.poetx_linear_workspace
    d = lambda T, m, n, dt=px.POETX_BF16: px.LinearDesc(T, m, n, dt, px.POETX_FP32, 0)  # noqa: E731
    assert f(None) == 0 and f(d(0, 32, 16384)) == 0 and f(d(8, 0, 16384)) == 0
    assert f(d(1, 32, 65536)) == 0 and f(d(8, 32, 256)) == 0 and f(d(16384, 4096, 4096)) == 0
    assert f(d(8, 31, 16384)) % (8 * 32 * 4) == 0 and f(d(8, 31, 16384)) >= 2 * 8 * 32 * 4


def clip(grads=(A, B), ns=(10, 20), dtypes=(0, 1), outs=(C, D), max_norm=1.0, norm=E, ws=H, wsb=None, count=None):
    n = len(grads) if count is None else count
    arr = lambda t, v: (t * max(1, len(v)))(*v)  # noqa: E731
    g, o = arr(ctypes.c_void_p, grads), None if outs is None else arr(ctypes.c_void_p, outs)
    wsb = L.poetx_clip_grads_workspace(max(n, 0)) if wsb is None else wsb
    return L.poetx_clip_grads(n, g, arr(ctypes.c_int64, ns), arr(ctypes.c_int32, dtypes), o, max_norm, norm, ws,
                              wsb, None)


@pytest.mark.parametrize("kw, status", [
    (dict(count=-1), INV), (dict(count=2 ** 20 + 1, wsb=2 ** 40), SHAPE),
    (dict(max_norm=-1.0), INV), (dict(max_norm=float("nan")), INV), (dict(max_norm=float("inf")), INV),
    (dict(ns=(10, -1)), INV), (dict(ns=(10, 2 ** 41)), SHAPE), (dict(dtypes=(0, 2)), DTYPE),
    (dict(grads=(A, None)), INV), (dict(outs=(C, None)), INV),
    (dict(grads=(A + 2, B)), ALIGN), (dict(grads=(A, B + 1)), ALIGN), (dict(outs=(C + 1, D)), ALIGN),
    (dict(norm=E + 2), ALIGN), (dict(ws=H + 8), ALIGN), (dict(ws=None), WS), (dict(wsb=64), WS),
    (dict(outs=(C, C)), INV),                          # two outputs in one place
    (dict(grads=(A, A), dtypes=(0, 0), ns=(10, 10), outs=(A, A)), INV),   # one tensor clipped twice
    (dict(grads=(A, A + 36), dtypes=(0, 0), ns=(10, 10), outs=(A, A + 36)), INV),
    (dict(outs=(B, D)), INV),                          # an output over another gradient
    (dict(outs=(A + 4, D)), INV),                      # a little behind its own gradient
    (dict(norm=A + 8), INV), (dict(norm=C), INV), (dict(ws=B), INV),
])
def test_clip_refusals(kw, status):
    assert clip(**kw) == status


def test_clip_workspace():
    f = L.poetx_clip_grads_workspace
    assert f(-1) == 0 and f(2 ** 20 + 1) == 0
    assert 0 < f(0) <= f(1) <= f(1000) and f(1) % 8 == 0


def test_python_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    import orthogonal_equivalence_cayley_amd as oec
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: oec.add_rms_norm(x, w), lambda: oec.add_rms_norm(x[0], w),
                 lambda: oec.add_rms_norm_backward(x, x, w, torch.ones(2)),
                 lambda: oec.linear(x, x), lambda: oec.clip_grads([], 1.0), lambda: oec.clip_grads([w], 1.0),
                 lambda: oec.MergedLinear(x, w_scale=w), lambda: oec.MergedLinear(x.to(torch.int8))):
        with pytest.raises(ValueError):
            call()
