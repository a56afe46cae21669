"""The cross entropy of a vocabulary's product and its gradients against plain 64-bit
implementations on the CPU, element by element.

Tolerances count roundings, as in test_gpu_block_ops.py (u = 2^-24, half a step of the
type, N u times the sum of the magnitudes for a sum of N terms, twice that for the matrix
instructions). With z off by ez: lse and a target's logit are off by ez at most; the sum of
exponentials adds u for each of the at most 64 additions in a row and a few u for exp; p =
exp(z - lse) is off by p (2 ez + u (|lse| + |z - lse|) + 80 u), d = p - 1 likewise, and by
half a step of its type; the products' sums go as above."""
import math

import pytest

from gpu_util import device_ready, log
from test_gpu_block_ops import HALF, T_, U, close, gen, rand, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


IGNORE = -100


def inputs(T, n, V, dt, seed=0, spread=2.0, ignored=0.2):
    import torch
    g = gen(seed * 7919 + T * 31 + n * 7 + V)
    X, W = rand(g, T, n, dtype=dt), rand(g, V, n, dtype=dt, scale=spread / math.sqrt(n))
    target = torch.randint(0, V, (T,), generator=g)
    target[torch.rand(T, generator=g) < ignored] = IGNORE
    return X, W, target, g


def reference(X, W, target, g, dt):
    """Values and what they may be off by: loss, lse, G_X, G_W. g: [T] or one value."""
    import torch
    x, w = X.double(), W.double()
    T, n = x.shape
    V = w.shape[0]
    z = x @ w.T
    ez = 2 * n * U * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(z, 1)
    e = ez.amax(1) + 80 * U
    counts = target != IGNORE
    t = target.clamp(min=0)
    loss = torch.where(counts, lse - z.gather(1, t[:, None])[:, 0], torch.zeros_like(lse))
    out = dict(lse=(lse, e + U * lse.abs()), loss=(loss, torch.where(counts, 2 * e + U * loss.abs(), 0 * e)))
    if g is None:
        return out
    p = torch.exp(z - lse[:, None])
    dp = p * (2 * ez.amax(1, keepdim=True) + U * (lse[:, None].abs() + (z - lse[:, None]).abs()) + 80 * U)
    d = p.clone()
    d[torch.arange(T, device=d.device), t] -= 1
    d, dp = d * counts[:, None], dp * counts[:, None]
    # up to 64 tokens what d loses in rounding is multiplied as well
    half = 0.0 if dt != "bf16" else HALF[dt] if T > 64 else 2.0 ** -17
    ed = dp + (half + 3 * U) * (d.abs() + dp)
    gd = g.double().expand(T)[:, None]
    gx, gw = (d * gd) @ w, (d * gd).T @ x
    a = (d.abs() + ed) * gd.abs()
    ex = (ed * gd.abs()) @ w.abs() + 2 * (V + 8) * U * (a @ w.abs()) + 2 * U * gx.abs()
    ew = (ed * gd.abs()).T @ x.abs() + 2 * (T + 8) * U * (a.T @ x.abs()) + 2 * U * gw.abs()
    # below the normal range a value is off by a step of 2^-149 (bf16 2^-133) or is taken as zero, up to 2^-126: the p of a
    # row, d, each of its products, and the result
    tiny = 2.0 ** -125
    ex, ew = ex + tiny * (w.abs().sum(0) + V + 1), ew + tiny * (x.abs().sum(0) + T + 1)
    out.update(G_X=(gx, ex + HALF[dt] * (gx.abs() + ex)), G_W=(gw, ew + HALF[dt] * (gw.abs() + ew)))
    return out


def run(X, W, target, g, **kw):
    import orthogonal_equivalence_cayley_amd as oec
    o = oec.linear_cross_entropy(X, W, target, ignore_index=IGNORE)
    out = dict(loss=o.loss, lse=o.lse)
    if g is not None:
        out["G_X"], out["G_W"] = oec.linear_cross_entropy_backward(g, X, W, target, o.lse, ignore_index=IGNORE, **kw)
    return out


def compare(got, want):
    for k, (v, tol) in want.items():
        close(k, got[k], v, tol)


# tokens, width, vocabulary: single ones, each tile's edges, ragged rows, several pieces
SIZES = [(1, 1, 1), (1, 7, 2), (3, 5, 63), (1, 64, 1000), (2, 100, 257), (4, 1001, 333), (5, 64, 5003), (33, 40, 130),
         (64, 256, 512), (65, 129, 129), (130, 72, 1000), (200, 1000, 700), (257, 64, 4099), (600, 130, 2049),
         (1031, 96, 300), (300, 512, 2600), (1, 1030, 900), (2, 1024, 65), (4, 2049, 500), (7, 1100, 1000), (8, 3001, 300),
         (9, 1024, 200)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T, n, V", SIZES)
def test_loss_and_gradients(T, n, V, dt):
    import torch
    log(f"cross entropy T={T} n={n} V={V} {dt}")
    X, W, target, g = inputs(T, n, V, dt)
    each, one = torch.rand(T, generator=g) + 0.1, torch.tensor([0.37])
    Xc, Wc, tc = X.cuda(), W.cuda(), target.cuda()
    for k in (one, each):
        a = run(Xc, Wc, tc, k.cuda())
        compare(a, reference(X, W, target, k, dt))
        b = run(Xc, Wc, tc, k.cuda())
        assert all(torch.equal(a[q], b[q]) for q in a)
    # each gradient alone, strided operands, results into strided places
    gx, none = run_back(Xc, Wc, tc, a["lse"], each, need_w=False)
    assert none is None and torch.equal(gx, a["G_X"])
    none, gw = run_back(Xc, Wc, tc, a["lse"], each, need_x=False)
    assert none is None and torch.equal(gw, a["G_W"])
    Xs, Ws = strided(X, 3, 1), strided(W, 5, 2)
    px, pw = strided(torch.zeros_like(X), 7, 3), strided(torch.zeros_like(W), 1, 1)
    s = run(Xs, Ws, tc, each.cuda(), G_X=px, G_W=pw)
    assert s["G_X"] is px and s["G_W"] is pw
    compare(s, reference(X, W, target, each, dt))
    assert bool((torch.as_strided(px, (T, 3), (n + 7, 1), 0) == 7).all() and
                (torch.as_strided(pw, (V, 1), (n + 1, 1), 0) == 7).all())
    assert torch.equal(Xs.cpu(), X) and torch.equal(Ws.cpu(), W)


# the large tiles of bf16: every product of them alone and together, ends moved back in both directions, pieces of the
# vocabulary with an end that is no multiple of 64, an odd width
BIG = [(2003, 128, 4300), (8300, 1032, 700), (301, 1091, 8403), (4200, 2112, 4299), (70000, 256, 4301)]


@pytest.mark.parametrize("T, n, V", BIG)
def test_many_tokens(T, n, V):
    import torch
    log(f"cross entropy T={T} n={n} V={V} bf16")
    X, W, target, g = inputs(T, n, V, "bf16")
    each = torch.rand(T, generator=g) + 0.1
    Xc, Wc, tc = X.cuda(), W.cuda(), target.cuda()
    a = run(Xc, Wc, tc, each.cuda())
    want = {k: (v.cpu(), e.cpu()) for k, (v, e) in reference(Xc, Wc, tc, each.cuda(), "bf16").items()}
    compare(a, want)
    # rows further apart, results into strided places, each gradient alone
    px, pw = strided(torch.zeros_like(X), 8, 0), strided(torch.zeros_like(W), 3, 1)
    s = run(strided(X, 8, 0), strided(W, 16, 8), tc, each.cuda(), G_X=px, G_W=pw)
    compare(s, want)
    assert bool((torch.as_strided(px, (T, 8), (n + 8, 1), n) == 7).all() and
                (torch.as_strided(pw, (V, 1), (n + 3, 1), 0) == 7).all())
    gx, _ = run_back(Xc, Wc, tc, a["lse"], each, need_w=False)
    _, gw = run_back(Xc, Wc, tc, a["lse"], each, need_x=False)
    assert torch.equal(gx, a["G_X"]) and torch.equal(gw, a["G_W"])
    del s, px, pw, gx, gw
    one = torch.tensor([0.37])
    b = run(Xc, Wc, tc, one.cuda())
    compare(b, {k: (v.cpu(), e.cpu()) for k, (v, e) in reference(Xc, Wc, tc, one.cuda(), "bf16").items()})


# few tiles of 256 x 256, whose two gradients are one launch: each axis's edges, sums shared by few and by many
@pytest.mark.parametrize("T, n, V", [(256, 256, 256), (257, 264, 300), (512, 1024, 2000), (300, 512, 5000),
                                     (1003, 1000, 1009), (1031, 520, 4160)])
def test_both_gradients_of_few_tiles(T, n, V):
    import torch
    log(f"cross entropy, both gradients of few tiles T={T} n={n} V={V}")
    X, W, target, g = inputs(T, n, V, "bf16", seed=3)
    each = torch.rand(T, generator=g) + 0.1
    # what a padded token holds is nobody's business
    pad = target == IGNORE
    junk = X.clone()
    junk[pad] = float("nan")
    Xc, Wc, tc, gc = X.cuda(), strided(W, 8), target.cuda(), each.cuda()
    a = run(Xc, Wc, tc, gc)
    compare(a, reference(X, W, target, each, "bf16"))
    b = run(junk.cuda(), Wc, tc, gc)
    for k in ("G_X", "G_W"):
        assert torch.equal(a[k], b[k])
    # into places with rows a stride apart, whose gaps stay as they were
    gx, gw = torch.full((T, n + 8), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((V, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    run(Xc, Wc, tc, gc, G_X=gx[:, :n], G_W=gw[:, :n])
    assert torch.equal(gx[:, :n], a["G_X"]) and torch.equal(gw[:, :n], a["G_W"])
    assert (gx[:, n:] == 7).all() and (gw[:, n:] == 7).all()


# a little more than whole rounds of 256 tiles: the last columns are a launch of their own, with targets at the seam
@pytest.mark.parametrize("T, n, V, seam", [(2048, 64, 8448, 8192), (2500, 72, 6700, 6400), (4099, 128, 4400, 3840),
                                           (2048, 256, 8300, 8192)])
def test_columns_behind_whole_rounds(T, n, V, seam):
    import torch
    log(f"cross entropy, columns behind whole rounds T={T} n={n} V={V}")
    X, W, target, g = inputs(T, n, V, "bf16", seed=5)
    target[:8] = torch.tensor([0, seam - 1, seam, seam + 1, V - 1, IGNORE, seam - 257, seam + 63])
    each = (torch.rand(T, generator=g) + 0.1).cuda()
    Xc, Wc, tc = X.cuda(), W.cuda(), target.cuda()
    a = run(Xc, Wc, tc, each)
    compare(a, {k: (v.cpu(), e.cpu()) for k, (v, e) in reference(Xc, Wc, tc, each, "bf16").items()})
    tc[3], tc[4] = V, -1   # outside: a loss of their own, and the gradients that they reach
    b = run(Xc, Wc, tc, each)
    assert b["loss"][3:5].isnan().all() and not b["loss"][5:].isnan().any()
    assert torch.equal(b["lse"], a["lse"]) and torch.equal(b["loss"][5:], a["loss"][5:])
    assert b["G_X"][3:5].isnan().all() and b["G_W"].isnan().all() and torch.equal(b["G_X"][5:], a["G_X"][5:])


def run_back(X, W, target, lse, g, **kw):
    import orthogonal_equivalence_cayley_amd as oec
    return oec.linear_cross_entropy_backward(g.cuda(), X, W, target, lse, ignore_index=IGNORE, **kw)


WHOLE = [(1, 64, 1000), (40, 72, 999), (70, 65, 2001), (300, 264, 1500), (513, 512, 3000), (1000, 256, 260),
         (700, 384, 10007)]


@pytest.mark.parametrize("T, n, V, dt", [(*c, dt) for c in WHOLE for dt in ("bf16", "f32")] +
                         [(*c, "bf16") for c in BIG])
def test_nothing_is_lost(T, n, V, dt):
    """Sums of whole numbers under a uniform softmax, in which a lost or repeated term shows: equal in bf16, whose d is
    then a power of two times 8 bits, and in fp32 but for the roundings of the sum."""
    import torch
    log(f"cross entropy exact T={T} n={n} V={V} {dt}")
    q = torch.tensor(1.0 / V, dtype=torch.float64).to(torch.bfloat16).double()
    few = dt == "bf16" and T <= 64      # what d loses in rounding is multiplied as well
    # exp(-lse) is off by 2^-20 of itself at most: no border of bf16 that near
    for k in (1 - 2.0 ** -19, 1 + 2.0 ** -19):
        assert torch.tensor(k / V, dtype=torch.float64).float().to(torch.bfloat16).double() == q
    if dt == "f32" or few:
        q = torch.tensor(1.0 / V, dtype=torch.float64)
    g = gen(T + n + V)
    whole = torch.randint(1, 5, (max(T, V), n), generator=g).to(T_(dt))
    star = V // 2
    target = torch.full((T,), star)
    one = torch.ones(1).cuda()
    # all logits zero by W: dW of every other row is the sum of all tokens over V
    X, W = whole[:T], torch.zeros(V, n, dtype=T_(dt))
    a = run(X.cuda(), W.cuda(), target.cuda(), one)
    others = torch.arange(V) != star
    want = (X.double().sum(0) * q).expand(V, n)[others]
    # by X: dX is the sum of the vocabulary's rows over V, the target's row being zero
    X2, W2 = torch.zeros(T, n, dtype=T_(dt)), whole[:V].clone()
    W2[star] = 0
    b = run(X2.cuda(), W2.cuda(), target.cuda(), one)
    want2 = (W2.double().sum(0) * q).expand(T, n)
    if few:
        # d to half a step of its second half, 2^-17, and exp as in fp32
        tol = HALF[dt] + 2.0 ** -17 + (2 * math.log(V) + 100 + 2 * max(T, V)) * U
        close("G_W", a["G_W"].cpu()[others], want, tol * want)
        close("G_X", b["G_X"], want2, tol * want2)
    elif dt == "bf16":
        # 8 bits times at most 4, in sums of less than 2^24 of their last place
        assert V * 4 * 255 < 2 ** 24
        assert torch.equal(b["G_X"].cpu(), want2.float().to(torch.bfloat16))
        if T * 4 * 255 < 2 ** 24:
            assert torch.equal(a["G_W"].cpu()[others], want.float().to(torch.bfloat16))
        else:
            close("G_W", a["G_W"].cpu()[others], want, (HALF[dt] + 2 * T * U) * want)
    else:
        lse = math.log(V)
        close("G_W", a["G_W"].cpu()[others], want, (2 * T + 2 * lse + 100) * U * want)
        close("G_X", b["G_X"], want2, (2 * V + 2 * lse + 100) * U * want2)
    for o in (a, b):
        close("lse", o["lse"], torch.full((T,), math.log(V), dtype=torch.float64), torch.tensor(100 * U + U * math.log(V)))
    assert not a["G_X"].any() and not b["G_W"].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 300])
def test_special_values(T, dt):
    """Ignored tokens whatever they hold, targets outside the vocabulary, infinite and NaN logits, far ones."""
    import torch
    X, W, target, g = inputs(T, 64, 600, dt, ignored=0.0)
    W[7] = 0
    W[7, 0] = -math.inf                     # this row's logit is -inf for x_0 > 0
    X[:, 0] = X[:, 0].abs() + 0.5
    target[target == 7] = 8
    X[1], target[1] = math.nan, IGNORE      # padding may hold anything
    X[2], target[2] = math.inf, IGNORE
    keep = torch.arange(T) != -1
    keep[1] = keep[2] = False
    each = torch.rand(T, generator=g)
    a = run(X.cuda(), W.cuda(), target.cuda(), each.cuda())
    Xr, Wr = X.clone(), W.clone()
    Xr[1] = Xr[2] = 0
    Wr[7] = 0
    # the reference without row 7, which has no share of any token
    rows = torch.arange(600) != 7
    renum = torch.cumsum(rows, 0) - 1
    tr = torch.where(target == IGNORE, target, renum[target.clamp(min=0)])
    want = reference(Xr, Wr[rows], tr, each, dt)
    for k in ("loss", "lse"):
        close(k, a[k].cpu()[keep], want[k][0][keep], want[k][1][keep])
    assert not a["loss"][1:3].any()
    close("G_W", a["G_W"].cpu()[rows], *want["G_W"])
    assert not a["G_W"][7].any()
    # 0 times the infinite weight is NaN in the column that holds it, and only there
    gx = a["G_X"].cpu()
    close("G_X", gx[:, 1:][keep], want["G_X"][0][:, 1:][keep], want["G_X"][1][:, 1:][keep])
    # targets outside the vocabulary: NaN, the others as before
    t2 = target.clone()
    t2[0], t2[4] = 600, -1
    b = run(X.cuda(), W.cuda(), t2.cuda(), each.cuda())
    assert torch.isnan(b["loss"][[0, 4]]).all() and torch.equal(b["loss"][5:], a["loss"][5:]) and b["loss"][3] == a["loss"][3]
    assert torch.isnan(b["G_X"][[0, 4]]).all() and torch.equal(b["G_X"][3, 1:], a["G_X"][3, 1:])
    assert torch.isnan(b["G_W"]).all()
    # a NaN token that counts: its own row
    X3 = X.clone()
    X3[0] = math.nan
    c = run(X3.cuda(), W.cuda(), target.cuda(), None)
    assert torch.isnan(c["loss"][0]) and torch.equal(c["loss"][1:], a["loss"][1:])


@pytest.mark.parametrize("T", [3, 400])
def test_far_logits(T):
    """Logits of hundreds: the softmax is that of the largest alone, nothing overflows."""
    import torch
    X, W, target, g = inputs(T, 64, 700, "f32", spread=200.0, ignored=0.0)
    a = run(X.cuda(), W.cuda(), target.cuda(), torch.ones(1).cuda())
    want = reference(X, W, target, torch.ones(1), "f32")
    compare(a, want)
    assert float(a["loss"].max()) > 200


def test_no_tokens_and_all_ignored():
    import torch
    X, W, target, _ = inputs(70, 40, 300, "bf16")
    target[:] = IGNORE
    a = run(X.cuda(), W.cuda(), target.cuda(), torch.ones(1).cuda())
    assert not a["loss"].any() and not a["G_X"].any() and not a["G_W"].any() and torch.isfinite(a["lse"]).all()
    e = run(X[:0].cuda(), W.cuda(), target[:0].cuda(), torch.ones(1).cuda())
    assert e["loss"].shape == (0,) and e["G_X"].shape == (0, 40) and not e["G_W"].any()
    # a vocabulary of one: no loss, no gradient
    one = run(X.cuda(), W[:1].cuda(), torch.zeros(70, dtype=torch.int64).cuda(), torch.ones(1).cuda())
    assert float(one["loss"].abs().max()) < 1e-5 and float(one["G_X"].float().abs().max()) < 1e-5


def test_gradients_by_differences():
    import torch
    X, W, target, g = inputs(6, 20, 50, "f32")
    each = torch.rand(6, generator=g)
    a = run(X.cuda(), W.cuda(), target.cuda(), each.cuda())

    def loss(x, w):
        z = x @ w.T
        v = torch.logsumexp(z, 1) - z.gather(1, target.clamp(min=0)[:, None])[:, 0]
        return float((v * each.double() * (target != IGNORE)).sum())
    e, x, w = 1e-5, X.double(), W.double()
    for name, base in (("G_X", x), ("G_W", w)):
        for k in range(0, base.numel(), 7):
            d = torch.zeros_like(base)
            d.view(-1)[k] = e
            up, down = ((x + d, w), (x - d, w)) if name == "G_X" else ((x, w + d), (x, w - d))
            num = (loss(*up) - loss(*down)) / (2 * e)
            assert abs(float(a[name].view(-1)[k]) - num) < 1e-5, (name, k)


@pytest.mark.parametrize("T, n, V", [(130, 96, 1000), (600, 128, 2048)])
def test_streams_and_graphs(T, n, V):
    """Calls on two streams share nothing; a captured step is replayed on new inputs."""
    import torch
    X, W, target, g = inputs(T, n, V, "bf16")
    X, W, target, one = X.cuda(), W.cuda(), target.cuda(), torch.full((1,), 0.25).cuda()
    ref = run(X, W, target, one)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(run(X, W, target, one))
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], ref[k]) for o in got for k in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        with torch.cuda.graph(graph, stream=streams[0]):
            o = run(X, W, target, one)
    for k in range(4):
        X.copy_(rand(g, T, n, dtype="bf16"))
        want = run(X, W, target, one)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[q], want[q]) for q in want)


def test_python_refusals():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    X, W, target, _ = inputs(4, 16, 30, "bf16")
    X, W, target, lse = X.cuda(), W.cuda(), target.cuda(), torch.zeros(4, device="cuda")
    one = torch.ones(1, device="cuda")
    back = oec.linear_cross_entropy_backward
    for call in (lambda: oec.linear_cross_entropy(X, W.float(), target), lambda: oec.linear_cross_entropy(X, W[:, :8], target),
                 lambda: oec.linear_cross_entropy(X, W, target[:3]), lambda: oec.linear_cross_entropy(X, W, target.int()),
                 lambda: oec.linear_cross_entropy(X, W, target.cpu()), lambda: oec.linear_cross_entropy(X.half(), W.half(), target),
                 lambda: back(one.repeat(3), X, W, target, lse), lambda: back(one.double(), X, W, target, lse),
                 lambda: back(one, X, W, target, lse[:2]), lambda: back(one, X, W, target, lse, need_x=False, need_w=False),
                 lambda: back(one, X, W, target, lse, need_x=False, G_X=X.clone()),
                 lambda: back(one, X, W, target, lse, G_W=W.float())):
        with pytest.raises(ValueError):
            call()
    for bad in (lambda: back(one, X, W, target, lse, G_X=X), lambda: back(one, X, W, target, lse, G_W=W)):
        with pytest.raises(oec.poetx.PoetxError):
            bad()
