"""Host-only checks of the calls that train around the linears (dropout, layer norm):
every refusal has its documented status and comes before anything is launched, so fake
addresses are safe here."""
import pytest

from orthogonal_equivalence_cayley_amd import poetx as px

L = px.LIB
# far apart: no two of these buffers overlap at the sizes used below
A, B, C, D, E, F, G, H, I, J, K = (0x100000 * (i + 1) for i in range(11))
MAX64 = 2 ** 62
INV, SHAPE, DTYPE, ALIGN, WS = (px.POETX_ERR_INVALID_ARG, px.POETX_ERR_SHAPE, px.POETX_ERR_DTYPE,
                               px.POETX_ERR_ALIGNMENT, px.POETX_ERR_WORKSPACE)
NAN, INF = float("nan"), float("inf")
RULE = (0.1, 1, None, 0)


def drop(T=4, dim=64, dtype=px.POETX_BF16, ld=(64, 64, 64), rule=RULE, X=A, R=B, Y=C, null=False):
    d = px.DropoutDesc(T, dim, dtype, *ld, px.DropoutRule(*rule))
    return L.poetx_dropout(None if null else d, X, R, Y, None)


@pytest.mark.parametrize("kw, status", [
    (dict(T=0), px.POETX_OK), (dict(T=0, X=None, Y=None), px.POETX_OK),
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=2 ** 24 + 1), SHAPE), (dict(dtype=px.POETX_INT8), DTYPE),
    (dict(rule=(-0.1, 1, None, 0)), INV), (dict(rule=(1.01, 1, None, 0)), INV), (dict(rule=(NAN, 1, None, 0)), INV),
    (dict(rule=(0.1, 1, D + 4, 0)), ALIGN), (dict(rule=(0.1, 1, C + 8, 0)), INV),
    (dict(X=None), INV), (dict(Y=None), INV),
    (dict(ld=(63, 64, 64)), SHAPE), (dict(ld=(64, 63, 64)), SHAPE), (dict(ld=(64, 64, 63)), SHAPE),
    (dict(ld=(64, 64, MAX64)), SHAPE),
    (dict(X=A + 1), ALIGN), (dict(R=B + 1), ALIGN), (dict(Y=C + 1), ALIGN),
    (dict(Y=A + 2), INV), (dict(Y=B + 128), INV), (dict(Y=A, ld=(64, 64, 128)), INV),
])
def test_dropout_refusals(kw, status):
    assert drop(**kw) == status


def norm(T=4, dim=64, dtype=px.POETX_BF16, y_dtype=None, ld=(64, 64, 64, 64), eps=1e-5, rule=RULE, X=A, R=B, w=C, b=D,
         Hp=E, Y=F, scale=None, mean=G, rstd=H, null=False):
    d = px.LayerNormDesc(T, dim, dtype, dtype if y_dtype is None else y_dtype, *ld, eps, px.DropoutRule(*rule))
    return L.poetx_add_layer_norm(None if null else d, X, R, w, b, Hp, Y, scale, mean, rstd, None)


@pytest.mark.parametrize("kw, status", [
    (dict(T=0), px.POETX_OK), (dict(T=0, X=None, Y=None, w=None), px.POETX_OK),
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(dim=0), SHAPE), (dict(dim=2 ** 24 + 1), SHAPE),
    (dict(dtype=px.POETX_INT8), DTYPE), (dict(y_dtype=px.POETX_FP32), DTYPE),
    (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(rule=(2.0, 1, None, 0)), INV),
    (dict(X=None), INV), (dict(w=None), INV), (dict(Y=None), INV),
    (dict(scale=I), INV), (dict(y_dtype=px.POETX_INT8), INV),
    (dict(ld=(63, 64, 64, 64)), SHAPE), (dict(ld=(64, 0, 64, 64)), SHAPE), (dict(ld=(64, 64, -64, 64)), SHAPE),
    (dict(ld=(64, 64, 64, MAX64)), SHAPE),
    (dict(X=A + 1), ALIGN), (dict(w=C + 2), ALIGN), (dict(b=D + 2), ALIGN), (dict(mean=G + 2), ALIGN),
    (dict(rstd=H + 2), ALIGN), (dict(y_dtype=px.POETX_INT8, scale=I + 1), ALIGN), (dict(rule=(0.1, 1, I + 4, 0)), ALIGN),
    (dict(Y=A), INV), (dict(Y=E), INV), (dict(Y=B + 128), INV), (dict(Hp=C), INV), (dict(Hp=D), INV), (dict(rstd=F), INV),
    (dict(mean=H), INV), (dict(Hp=A + 2), INV), (dict(Hp=A, ld=(64, 64, 128, 64)), INV), (dict(rule=(0.1, 1, F, 0)), INV),
])
def test_layer_norm_refusals(kw, status):
    assert norm(**kw) == status


def norm_back(T=4, dim=64, dtype=px.POETX_BF16, ld=(64, 64, 64, 64, 64), rule=RULE, g=A, gh=B, h=C, w=D, mean=E, rstd=F,
              gx=G, gr=H, gw=I, gb=J, ws=K, wsb=None, null=False):
    d = px.LayerNormBackwardDesc(T, dim, dtype, *ld, px.DropoutRule(*rule))
    wsb = L.poetx_layer_norm_backward_workspace(max(T, 0) % 2 ** 31, max(dim, 1)) if wsb is None else wsb
    return L.poetx_layer_norm_backward(None if null else d, g, gh, h, w, mean, rstd, gx, gr, gw, gb, ws, wsb, None)


@pytest.mark.parametrize("kw, status", [
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 31), SHAPE), (dict(dim=0), SHAPE),
    (dict(dtype=px.POETX_INT8), DTYPE), (dict(rule=(-1.0, 0, None, 0)), INV),
    (dict(rule=(0.0, 0, None, 0)), INV), (dict(rule=(1e-9, 0, None, 0)), INV),     # a second gradient without dropout
    (dict(gw=None), INV), (dict(gb=None), INV), (dict(gw=I + 1), ALIGN), (dict(gb=J + 2), ALIGN), (dict(gb=I + 16), INV),
    (dict(g=None), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(gx=None), INV),
    (dict(ld=(63, 64, 64, 64, 64)), SHAPE), (dict(ld=(64, 64, 64, 1, 64)), SHAPE), (dict(ld=(64, 64, 64, 64, 3)), SHAPE),
    (dict(g=A + 1), ALIGN), (dict(gx=G + 1), ALIGN), (dict(gr=H + 1), ALIGN), (dict(mean=E + 1), ALIGN),
    (dict(ws=K + 8), ALIGN), (dict(ws=None), WS), (dict(wsb=0), WS), (dict(wsb=100), WS),
    (dict(gx=C), INV), (dict(gr=C), INV), (dict(gx=A + 2), INV), (dict(gw=D), INV), (dict(gw=G), INV), (dict(ws=A), INV),
    (dict(gr=G), INV), (dict(gx=A, gr=A), INV), (dict(gx=A, ld=(64, 64, 64, 128, 64)), INV),
])
def test_layer_norm_backward_refusals(kw, status):
    assert norm_back(**kw) == status


def test_layer_norm_backward_workspace():
    f = L.poetx_layer_norm_backward_workspace
    assert f(-1, 8) == 0 and f(2 ** 31, 8) == 0 and f(4, 0) == 0 and f(4, 2 ** 24 + 1) == 0
    assert f(0, 8) > 0 and f(1000, 64) >= 500 * 2 * 64 * 4
    # rows longer than any register variant keep two more values each
    assert f(100000, 20000) >= 512 * 2 * 4 * 20000 + 8 * 100000


def test_python_refusals():
    torch = pytest.importorskip("torch")
    import orthogonal_equivalence_cayley_amd as oec
    x, w, r = torch.zeros(2, 8), torch.ones(8), torch.ones(2)
    for call in (lambda: oec.dropout(x, 0.1, 1), lambda: oec.dropout_backward(x, 0.1, 1), lambda: oec.add_layer_norm(x, w),
                 lambda: oec.add_layer_norm_backward(x, x, w, r, r), lambda: oec.add_layer_norm(x[0], w)):
        with pytest.raises(ValueError):
            call()


def loss(T=4, V=32, n=64, dtype=px.POETX_BF16, ld=(64, 64), X=A, W=B, target=C, out=D, lse=E, ws=F, wsb=None, null=False):
    d = px.CrossEntropyDesc(T, V, n, dtype, *ld, 64, 64, 1, -100)
    wsb = L.poetx_linear_cross_entropy_workspace(d) if wsb is None else wsb
    return L.poetx_linear_cross_entropy(None if null else d, X, W, target, out, lse, ws, wsb, None)


SIZES = [
    (dict(null=True), INV), (dict(T=-1), INV), (dict(T=2 ** 24 + 1), SHAPE), (dict(V=0), SHAPE), (dict(V=2 ** 24 + 1), SHAPE),
    (dict(n=0), SHAPE), (dict(n=2 ** 16 + 1), SHAPE), (dict(dtype=px.POETX_INT8), DTYPE),
    (dict(X=None), INV), (dict(W=None), INV), (dict(target=None), INV), (dict(lse=None), INV),
    (dict(X=A + 1), ALIGN), (dict(W=B + 1), ALIGN), (dict(target=C + 4), ALIGN), (dict(lse=E + 2), ALIGN),
]


@pytest.mark.parametrize("kw, status", SIZES + [
    (dict(T=0), px.POETX_OK), (dict(T=0, X=None, ws=None), px.POETX_OK),
    (dict(ld=(63, 64)), SHAPE), (dict(ld=(64, 63)), SHAPE), (dict(ld=(MAX64, 64)), SHAPE),
    (dict(out=None), INV), (dict(out=D + 1), ALIGN), (dict(ws=F + 8), ALIGN), (dict(ws=None), WS), (dict(wsb=0), WS),
    (dict(out=A), INV), (dict(out=C), INV), (dict(lse=D), INV), (dict(ws=B), INV), (dict(ws=D), INV), (dict(lse=B + 64), INV),
])
def test_cross_entropy_refusals(kw, status):
    assert loss(**kw) == status


def loss_back(T=4, V=32, n=64, dtype=px.POETX_BF16, ld=(64, 64, 64, 64), count=1, g=D, X=A, W=B, target=C, lse=E, gx=F, gw=G,
              ws=H, wsb=None, null=False):
    d = px.CrossEntropyDesc(T, V, n, dtype, *ld, count, -100)
    wsb = L.poetx_linear_cross_entropy_backward_workspace(d, gx is not None, gw is not None) if wsb is None else wsb
    return L.poetx_linear_cross_entropy_backward(None if null else d, g, X, W, target, lse, gx, gw, ws, wsb, None)


@pytest.mark.parametrize("kw, status", SIZES + [
    (dict(T=0, gw=None), px.POETX_OK), (dict(gx=None, gw=None), INV), (dict(count=2), SHAPE), (dict(count=0), SHAPE),
    (dict(ld=(63, 64, 64, 64)), SHAPE), (dict(ld=(64, 63, 64, 64)), SHAPE), (dict(ld=(64, 64, 63, 64)), SHAPE),
    (dict(ld=(64, 64, 64, 63)), SHAPE), (dict(g=None), INV), (dict(g=D + 2), ALIGN), (dict(gx=F + 1), ALIGN),
    (dict(gw=G + 1), ALIGN), (dict(ws=H + 8), ALIGN), (dict(ws=None), WS), (dict(wsb=0), WS),
    (dict(gx=A), INV), (dict(gw=B), INV), (dict(gx=G), INV), (dict(gw=C), INV), (dict(gx=E), INV), (dict(gw=D), INV),
    (dict(ws=A), INV), (dict(ws=F), INV), (dict(gx=A + 2), INV),
])
def test_cross_entropy_backward_refusals(kw, status):
    assert loss_back(**kw) == status


def test_cross_entropy_workspaces():
    f, b = L.poetx_linear_cross_entropy_workspace, L.poetx_linear_cross_entropy_backward_workspace
    d = lambda T, V, n, dt=px.POETX_BF16: px.CrossEntropyDesc(T, V, n, dt, n, n, n, n, 1, -100)  # noqa: E731
    assert f(None) == 0 and f(d(0, 9, 9)) == 0 and f(d(9, 0, 9)) == 0 and b(None, 1, 1) == 0 and b(d(9, 9, 0), 1, 1) == 0
    assert f(d(1, 32000, 2048)) >= 8 * 32000 // 256
    # far below the logits of a batch, whichever gradients are wanted
    assert f(d(16384, 32000, 2048)) < 2 * 16384 * 32000 / 8
    big = b(d(16384, 32000, 2048), 1, 1)
    assert b(d(16384, 32000, 2048), 0, 1) <= big and b(d(16384, 32000, 2048), 1, 0) <= big < 2 * 16384 * 32000 * 0.6
