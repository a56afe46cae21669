"""The operators that train around the linears in a row, as a model's step has them, and at
sizes past 4 GiB."""
import math

import pytest

from gpu_util import device_ready, log, make_layer
from philox_ref import factors
from test_gpu_block_ops import HALF, U, close, gen, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def test_a_step_against_autograd():
    """norm(drop(x) + r) -> trained linear -> norm(drop + residual) -> loss over a vocabulary, and back: every gradient
    against 64-bit autograd of the same formulas, the linear by its merged weight. All gradients clipped at the end."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    import workloads
    n, T, V, p, seed = 256, 90, 700, 0.2, 12345
    inp = workloads.small_case(n, n, (64, 64, 64, 64), (64, 64, 64, 64), T=T, seed=5, dtype="f32", theta_std=0.02)
    layer = make_layer(inp, 4, "f32")
    layer.build()
    Wm = layer.merged().W.double().cpu()
    g = gen(11)
    x, r = rand(g, T, n), rand(g, T, n)
    w1, b1, w2, b2 = 1 + 0.2 * rand(g, n), 0.2 * rand(g, n), 1 + 0.2 * rand(g, n), 0.2 * rand(g, n)
    W = rand(g, V, n, scale=1.5 / math.sqrt(n))
    target = torch.randint(0, V, (T,), generator=g)
    target[::7] = -100
    count = int((target != -100).sum())
    dev = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    X, R, W1, B1, W2, B2, WV, tgt = dev(x, r, w1, b1, w2, b2, W, target)
    one = torch.full((1,), 1.0 / count, device="cuda")
    o1 = oec.add_layer_norm(X, W1, B1, residual=R, p=p, seed=seed, site=1, save=True)
    f = layer.forward(o1.Y, save=True)
    o2 = oec.add_layer_norm(f, W2, B2, residual=o1.H, p=p, seed=seed, site=2, save=True)
    ce = oec.linear_cross_entropy(o2.Y, WV, tgt)
    gy2, gw = oec.linear_cross_entropy_backward(one, o2.Y, WV, tgt, ce.lse)
    k2 = oec.add_layer_norm_backward(gy2, o2.H, W2, o2.mean, o2.rstd, p=p, seed=seed, site=2)
    gy1, gR, gP = layer.backward(o1.Y, k2.G_X)
    k1 = oec.add_layer_norm_backward(gy1, o1.H, W1, o1.mean, o1.rstd, G_H=k2.G_R, p=p, seed=seed, site=1)

    # the same in 64 bits
    leaf = lambda t: t.double().clone().requires_grad_()  # noqa: E731
    vx, vr, v1, c1, v2, c2, vw = map(leaf, (x, r, w1, b1, w2, b2, W))
    m1, m2 = (torch.from_numpy(factors(T, n, p, seed, s)) for s in (1, 2))
    norm = lambda h, w, b: torch.nn.functional.layer_norm(h, (n,), w, b, 1e-5)  # noqa: E731
    h1 = vx * m1 + vr
    h2 = (norm(h1, v1, c1) @ Wm.T) * m2 + h1
    z = norm(h2, v2, c2) @ vw.T
    loss = torch.nn.functional.cross_entropy(z, target, ignore_index=-100)
    loss.backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    want = float(loss.detach())
    assert abs(float(ce.loss.double().sum()) / count - want) < 1e-5 * want
    # fp32 throughout; products of 256 and 700 terms, the linear's series itself within 1e-5
    for name, got, want in (("x", k1.G_X, vx), ("r", k1.G_R, vr), ("w1", k1.g_weight, v1), ("b1", k1.g_bias, c1),
                            ("w2", k2.g_weight, v2), ("b2", k2.g_bias, c2), ("W", gw, vw)):
        e = rel(got, want.grad)
        log(f"  {name}: {e:.2e}")
        assert e < 2e-5, (name, e)
    grads = [k1.g_weight, k1.g_bias, k2.g_weight, k2.g_bias, gw, gR, gP]
    before = [t.clone() for t in grads]
    total = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    got = oec.clip_grads(grads, total / 3, out=grads)
    assert abs(float(got) - total) < 1e-6 * total
    for a, b in zip(grads, before):
        assert float((a.double() - b.double() / 3).norm()) <= 1e-6 * float(b.double().norm() + 1e-30)


def test_dropout_alone_in_front_of_the_other_norm():
    """drop(x) + r in one call, then the norm without a mean: the same h as by hand."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    g = gen(2)
    x, r, w = rand(g, 300, 640, dtype="bf16").cuda(), rand(g, 300, 640, dtype="bf16").cuda(), torch.ones(640).cuda()
    h = oec.dropout(x, 0.1, 3, 4, residual=r)
    o = oec.add_layer_norm(x, w, residual=r, p=0.1, seed=3, site=4)
    assert torch.equal(o.H, h)
    y = oec.add_rms_norm(h, w)
    assert torch.equal(y.Y, oec.add_rms_norm(o.H, w).Y)
    # the gradient through dropout alone is the mask's
    gy = rand(g, 300, 640, dtype="bf16").cuda()
    assert torch.equal(oec.dropout_backward(gy, 0.1, 3, 4) != 0, (gy != 0) & (torch.from_numpy(factors(300, 640, 0.1, 3, 4)).cuda() != 0))


def chunked(X, W, target, g):
    """lse, loss, G_X in 64 bits, and dL/dz of a slice of the vocabulary on demand."""
    import torch
    T, V = X.shape[0], W.shape[0]
    lse, zt = [], []
    for a in range(0, V, 1 << 17):
        z = X.double() @ W[a:a + (1 << 17)].double().T
        lse.append(torch.logsumexp(z, 1))
        here = (target >= a) & (target < a + (1 << 17))
        zt.append(torch.where(here, z.gather(1, (target - a).clamp(0, z.shape[1] - 1)[:, None])[:, 0], 0.0))
    lse = torch.logsumexp(torch.stack(lse), 0)

    def share(a, b):
        d = torch.exp(X.double() @ W[a:b].double().T - lse[:, None])
        here = (target >= a) & (target < b)
        d[torch.arange(T, device="cuda")[here], target[here] - a] -= 1
        return d * g.double()[:, None]
    gx = sum(share(a, min(V, a + (1 << 17))) @ W[a:a + (1 << 17)].double() for a in range(0, V, 1 << 17))
    return lse, lse - sum(zt), gx, share


@pytest.mark.parametrize("T", [2, 40, 300])
def test_weight_past_4_gib(T):
    """1.1 M rows of 2048 (4.5 GB), targets at both ends."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"cross entropy, a weight past 4 GiB, T={T}")
    V, n = 1_100_003, 2048
    g = torch.Generator(device="cuda").manual_seed(T)
    W = torch.empty(V, n, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 1 << 17):
        W[a:a + (1 << 17)] = torch.randn(W[a:a + (1 << 17)].shape, generator=g, device="cuda") * (2 / math.sqrt(n))
    X = torch.randn(T, n, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[0], target[1] = V - 1, 0
    each = torch.rand(T, generator=g, device="cuda") + 0.5
    o = oec.linear_cross_entropy(X, W, target)
    G_X, G_W = oec.linear_cross_entropy_backward(each, X, W, target, o.lse)
    lse, loss, gx, share = chunked(X, W, target, each)
    # z is off by 2 n u sum |x w| at most (some 2 n u 2 sqrt(n) there), lse by as much and a few u
    ez = 2 * n * U * float((X.double().abs() @ W[:4096].double().abs().T).max()) * 1.5
    close("lse", o.lse, lse.cpu(), torch.tensor(ez + 100 * U + U * 20))
    close("loss", o.loss, loss.cpu(), torch.tensor(2 * ez + 200 * U + U * 40))
    # by 2-norms: d is off by half a step of bf16 and 2 ez, all of them apart, and the result by half a step
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    bound = 2 * HALF["bf16"] + 2 * ez
    assert rel(G_X, gx) < bound
    for a, b in ((0, 3000), (V // 2, V // 2 + 3000), (V - 3000, V)):
        assert rel(G_W[a:b], share(a, b).T @ X.double()) < bound, a


def test_tokens_past_4_gib():
    """1.1 M tokens of 2048 (4.5 GB) and their gradient."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    T, n, V = 1_100_003, 2048, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    for a in range(0, T, 1 << 17):
        X[a:a + (1 << 17)] = torch.randn(X[a:a + (1 << 17)].shape, generator=g, device="cuda")
    W = (torch.randn(V, n, generator=g, device="cuda") * (2 / math.sqrt(n))).bfloat16()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[5::9] = -100
    one = torch.full((1,), 0.5, device="cuda")
    o = oec.linear_cross_entropy(X, W, target)
    G_X, G_W = oec.linear_cross_entropy_backward(one, X, W, target, o.lse)
    gw = torch.zeros(V, n, dtype=torch.float64, device="cuda")
    ez = 2 * n * U * 2 * n ** 0.5 * 1.5
    for a in range(0, T, 1 << 17):
        x, t = X[a:a + (1 << 17)].double(), target[a:a + (1 << 17)]
        z = x @ W.double().T
        lse = torch.logsumexp(z, 1)
        want = torch.where(t < 0, 0.0, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0])
        assert float((o.loss[a:a + (1 << 17)].double() - want).abs().max()) < 2 * ez + 100 * U
        d = torch.exp(z - lse[:, None])
        d[torch.arange(len(t), device="cuda"), t.clamp(min=0)] -= 1
        d *= 0.5 * (t >= 0)[:, None]
        gx = d @ W.double()
        assert float((G_X[a:a + (1 << 17)].double() - gx).norm() / gx.norm()) < 2 * HALF["bf16"] + 2 * ez
        gw += d.T @ x
    assert float((G_W.double() - gw).norm() / gw.norm()) < 2 * HALF["bf16"] + 2 * ez
    # the norms over the same rows, in place, at both ends
    w = torch.ones(n, device="cuda")
    s = oec.add_layer_norm(X[-3:], w, residual=G_X[-3:], eps=1e-3)
    y = oec.add_layer_norm(X, w, residual=G_X, H=G_X, eps=1e-3).Y
    assert torch.equal(y[-3:], s.Y) and torch.equal(G_X[-3:], s.H)
