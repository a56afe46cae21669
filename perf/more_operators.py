"""Cases of the operators that train a block and the model's end around the linears: dropout into the residual stream,
the residual and layer norm behind it, and the cross entropy of a vocabulary's product without its logits.

Plain forms are elementary torch operations in 32 bits (64 where a sum or a decision needs them); with `own` set, `run`
calls the package. Sizes are those of the framework's blocks (hidden 2048 and 4096, feed-forward 5632, 16384 tokens) with
vocabularies of usual sizes, and ragged ones beside them.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_IGNORE = -100


# ------------------------------------------------------------------ cases
def _norm(name, T, dim, dtype="bf16", p=0.0, residual=True, out="same"):
    return dict(name=name, op="norm", T=T, dim=dim, dtype=dtype, p=p, residual=residual, out=out)


def _norm_train(name, T, dim, dtype, both, p=0.0, gh=True):
    return dict(name=name, op="norm_train", T=T, dim=dim, dtype=dtype, both=both, p=p, gh=gh)


def _drop(name, T, dim, dtype, p, residual, train=False):
    return dict(name=name, op="drop", T=T, dim=dim, dtype=dtype, p=p, residual=residual, train=train)


def _loss(name, T, n, V, dtype="bf16", train=False, ignored=0.0, weighted=False):
    return dict(name=name, op="loss", T=T, n=n, V=V, dtype=dtype, train=train, ignored=ignored, weighted=weighted)


def listed():
    return [
        # one token being generated, between two linears of a hidden-2048 block: latency
        _norm("norm_token", 1, 2048),
        # the training batch of the hidden-2048 block: a sublayer's dropout, the residual and the norm in one
        _norm("norm_batch_dropout", 16384, 2048, p=0.1),
        # its backward, with the gradient that arrives through the residual stream
        _norm_train("norm_backward", 16384, 2048, "bf16", both=False, p=0.1),
        # a ragged fp32 layer trained without dropout: forward and backward
        _norm_train("norm_train_odd_f32", 1003, 1365, "f32", both=True),
        # a sublayer's output dropped into the residual stream, in front of a norm of another kind
        _drop("dropout_residual", 16384, 2048, "bf16", 0.1, True),
        # dropout inside the feed-forward, forward and backward
        _drop("dropout_train_wide", 16384, 5632, "bf16", 0.2, False, train=True),
        # a small ragged fp32 one: latency
        _drop("dropout_odd_f32", 61, 1365, "f32", 0.5, True),
        # the likelihood of one token: bound by the weight's bytes
        _loss("loss_token", 1, 2048, 32000),
        # scoring a document's tokens, a vocabulary of odd size, hidden 4096
        _loss("loss_score", 2048, 4096, 50021),
        # the training batch of the hidden-2048 block: loss and both gradients
        _loss("loss_train", 16384, 2048, 32000, train=True),
        # a ragged batch with padding, each token with a weight of its own, sizes of no round number
        _loss("loss_train_odd", 1003, 1000, 10007, train=True, ignored=0.3, weighted=True),
        # a small model in fp32
        _loss("loss_train_f32", 512, 512, 8000, "f32", train=True, ignored=0.05),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width of a kind in use: a multiple of 256, of 16, or any."""
    step = rng.choice([256, 256, 16, 1])
    return min(hi, max(1, _spread(rng, lo, hi) // step) * step)


def draw(rng):
    op = rng.choice(["norm", "norm_train", "drop", "loss", "loss"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    p = rng.choice([0.0, 0.05, 0.1, 0.3, round(rng.uniform(0.01, 0.9), 3)])
    if op == "norm":
        c = _norm("", _spread(rng, 1, 16384), _width(rng, 64, 8192), dtype, p, rng.random() < 0.75,
                  rng.choice(["same", "same", "int8"]))
    elif op == "norm_train":
        c = _norm_train("", _spread(rng, 1, 16384), _width(rng, 64, 8192), dtype, rng.random() < 0.5, p, rng.random() < 0.7)
    elif op == "drop":
        c = _drop("", _spread(rng, 1, 16384), _width(rng, 64, 8192), dtype, p or 0.15, rng.random() < 0.5, rng.random() < 0.5)
    else:
        n, V = _width(rng, 64, 4096), _width(rng, 100, 64000)
        most = 16384 if dtype == "bf16" else 2048
        T = _spread(rng, 1, max(2, min(most, int(16384 * 2048 * 32000 * (1 if dtype == "bf16" else 1 / 16) / (n * V)))))
        c = _loss("", T, n, V, dtype, rng.random() < 0.6, rng.choice([0.0, 0.05, 0.4]), rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    dt, T = _TYPES[case["dtype"]], case["T"]
    # what a training program counts on for its generator: a seed of the run, and the number of the place in the model
    s = dict(case=case, seed=(seed * 0x9E3779B97F4A7C15 + 1) % 2 ** 64, site=seed % 97)
    if case["op"] in ("norm", "norm_train"):
        d = case["dim"]
        # a residual stream has a few channels far larger than the rest, a mean of its own, and tokens of different sizes
        channel = torch.exp(0.5 * rand(d)) * torch.exp(0.3 * rand(T, 1))
        s.update(X=(rand(T, d) * 0.3).to(dt), R=((rand(T, d) + 0.3) * channel).to(dt), w=1 + 0.1 * rand(d), b=0.1 * rand(d),
                 eps=1e-5)
        if case["op"] == "norm":
            s["values"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda") if case["out"] == "int8" else None
            if not case["residual"]:
                s["X"], s["R"] = s["R"], None
        else:
            s.update(G=(rand(T, d) * 1e-2).to(dt), GH=(rand(T, d) * 1e-2).to(dt) if case["gh"] else None)
            if not case["both"]:
                # what the forward kept
                H = s["R"].double()
                mean = H.mean(1)
                s["H"], s["mean"] = s["R"], mean.float()
                s["rstd"] = ((H - mean[:, None]).square().mean(1) + s["eps"]).rsqrt().float()
    elif case["op"] == "drop":
        s.update(X=rand(T, case["dim"]).to(dt), R=rand(T, case["dim"]).to(dt) if case["residual"] else None,
                 G=(rand(T, case["dim"]) * 1e-2).to(dt) if case["train"] else None)
    else:
        n, V = case["n"], case["V"]
        # logits of a standard deviation of 2; the target's raised by up to 8, as a model in training has it; targets as skewed as words are
        W = rand(V, n) * (2 / math.sqrt(n))
        target = torch.exp(uniform(T) * math.log(V)).long().clamp(1, V) - 1
        X = rand(T, n) + 2 * uniform(T, 1) * W[target]
        target[(uniform(T) < case["ignored"]) & (torch.arange(T, device="cuda") > 0)] = _IGNORE
        s.update(X=X.to(dt), W=W.to(dt), target=target)
        # the mean over the tokens that count, or a weight for each
        valid = (target != _IGNORE).sum().clamp(min=1)
        s["g"] = (uniform(T) + 0.5) / valid if case["weighted"] else (1.0 / valid).reshape(1)
    return s


# ------------------------------------------------------------------ plain forms
def _threshold(p):
    """Elements whose 16 bits lie below it are dropped; the others are scaled by 65536 / (65536 - threshold)."""
    return int(round(p * 65536))


def _plain_keep(T, dim, p, seed, site):
    """Philox 4x32-10 of the counter (column / 8, row, site, 0) under the seed: 128 bits for 8 columns, 16 for each."""
    row = torch.arange(T, device="cuda")[:, None]
    col = torch.arange((dim + 7) // 8, device="cuda")[None, :]
    zero = torch.zeros(T, (dim + 7) // 8, dtype=torch.int64, device="cuda")
    c0, c1, c2, c3 = zero + col, zero + row, zero + site, zero
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # 64 bits that wrap: both halves are right
        c0, c1, c2, c3 = (b >> 32) & 0xFFFFFFFF ^ c1 ^ k0, b & 0xFFFFFFFF, (a >> 32) & 0xFFFFFFFF ^ c3 ^ k1, a & 0xFFFFFFFF
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    bits = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return bits.reshape(T, -1)[:, :dim] >= _threshold(p)


def _plain_drop(x, s):
    p = s["case"]["p"]
    if p == 0:
        return x
    keep = _plain_keep(x.shape[0], x.shape[1], p, s["seed"], s["site"])
    return torch.where(keep, x * (65536 / (65536 - _threshold(p))), torch.zeros_like(x))


def _plain_norm(s):
    """h in the type, mean and 1 / deviation in 32 bits from sums in 64, the normalised row in 32 bits."""
    X, R = s["X"], s["R"]
    H = _plain_drop(X.float(), s)
    H = (H if R is None else H + R.float()).to(X.dtype)
    hf = H.float()
    mean = hf.double().mean(1)
    d = hf.double() - mean[:, None]
    rstd = (1 / torch.sqrt((d * d).mean(1) + s["eps"])).float()
    return H, mean.float(), rstd, (d.float() * rstd[:, None]) * s["w"] + s["b"]


def _plain_back(s, H, mean, rstd):
    g, u = s["G"].float(), (H.float() - mean[:, None]) * rstd[:, None]
    gw = g * s["w"]
    dh = rstd[:, None] * (gw - gw.mean(1, keepdim=True) - u * (gw * u).mean(1, keepdim=True))
    if s["GH"] is not None:
        dh = dh + s["GH"].float()
    dx = _plain_drop(dh, s)
    return dx.to(H.dtype), dh.to(H.dtype), (g * u).sum(0, dtype=torch.float64).float(), g.sum(0, dtype=torch.float64).float()


def _plain_loss(s):
    X, W, target = s["X"], s["W"], s["target"]
    x, w = X.float(), W.float()
    z = x @ w.T
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, dtype=torch.float64)
    lse = (m[:, 0].double() + torch.log(total))
    counts = target != _IGNORE
    t = torch.where(counts, target, torch.zeros_like(target))
    loss = torch.where(counts, lse - z.gather(1, t[:, None])[:, 0].double(), torch.zeros_like(lse)).float()
    if not s["case"]["train"]:
        return dict(loss=loss, lse=lse.float())
    p = torch.div(e, total.float()[:, None], out=e)
    p.scatter_add_(1, t[:, None], torch.full_like(p[:, :1], -1.0))
    p *= torch.where(counts, s["g"].expand(len(t)), torch.zeros_like(lse, dtype=torch.float32))[:, None]
    return dict(loss=loss, G_X=(p @ w).to(X.dtype), G_W=(p.T @ x).to(W.dtype))


def _plain(s):
    case = s["case"]
    if case["op"] == "loss":
        return _plain_loss(s)
    if case["op"] == "drop":
        y = _plain_drop(s["X"].float(), s)
        out = dict(Y=(y if s["R"] is None else y + s["R"].float()).to(s["X"].dtype))
        if case["train"]:
            out["G_X"] = _plain_drop(s["G"].float(), s).to(s["X"].dtype)
        return out
    if case["op"] == "norm":
        H, _, _, y = _plain_norm(s)
        if case["out"] == "same":
            return dict(Y=y.to(H.dtype), H=H)
        a = y.abs().amax(1, keepdim=True)
        none = a < 2.0 ** -119
        inv = torch.where(none, torch.zeros_like(a), 127 / a)
        scale = torch.where(none, torch.zeros_like(a), a / 127)
        return dict(Y=(torch.round(y * inv) * scale).to(torch.bfloat16), scale=scale[:, 0], H=H)
    out = {}
    H, mean, rstd = s.get("H"), s.get("mean"), s.get("rstd")
    if case["both"]:
        H, mean, rstd, y = _plain_norm(s)
        out = dict(Y=y.to(H.dtype), H=H)
    out["G_X"], out["G_R"], out["g_w"], out["g_b"] = _plain_back(s, H, mean, rstd)
    return out


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import orthogonal_equivalence_cayley_amd as oec
    case = s["case"]
    if case["op"] == "loss":
        o = oec.linear_cross_entropy(s["X"], s["W"], s["target"], ignore_index=_IGNORE)
        if not case["train"]:
            return dict(loss=o.loss, lse=o.lse)
        G_X, G_W = oec.linear_cross_entropy_backward(s["g"], s["X"], s["W"], s["target"], o.lse, ignore_index=_IGNORE)
        return dict(loss=o.loss, G_X=G_X, G_W=G_W)
    drop = dict(p=case["p"], seed=s["seed"], site=s["site"])
    if case["op"] == "drop":
        out = dict(Y=oec.dropout(s["X"], residual=s["R"], **drop))
        if case["train"]:
            out["G_X"] = oec.dropout_backward(s["G"], **drop)
        return out
    if case["op"] == "norm":
        o = oec.add_layer_norm(s["X"], s["w"], s["b"], residual=s["R"], eps=s["eps"], quantize=case["out"] == "int8", **drop)
        if case["out"] == "same":
            return dict(Y=o.Y, H=o.H)
        return dict(Y=torch.mul(o.Y, o.scale[:, None], out=s["values"]), scale=o.scale, H=o.H)
    out = {}
    H, mean, rstd = s.get("H"), s.get("mean"), s.get("rstd")
    if case["both"]:
        o = oec.add_layer_norm(s["X"], s["w"], s["b"], residual=s["R"], eps=s["eps"], save=True, **drop)
        H, mean, rstd = o.H, o.mean, o.rstd
        out = dict(Y=o.Y, H=H)
    out["G_X"], out["G_R"], out["g_w"], out["g_b"] = oec.add_layer_norm_backward(s["G"], H, s["w"], mean, rstd, G_H=s["GH"], **drop)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    T = case["T"]
    if case["op"] == "loss":
        n, V = case["n"], case["V"]
        once = e * n * (T + V)      # X and W, or their gradients
        return dict(bytes=once * (2 if case["train"] else 1) + 16 * T, flops=(6 if case["train"] else 2) * T * n * V)
    n = T * case["dim"]
    if case["op"] == "drop":
        return dict(bytes=n * e * (2 + case["residual"] + 2 * case["train"]), flops=2 * n * (1 + case["train"]))
    if case["op"] == "norm":
        # reads x (and r), writes y (and h where it is not x itself)
        kept = case["residual"] or case["p"] > 0
        return dict(bytes=n * (e * (1 + case["residual"] + kept) + (e if case["out"] == "same" else 1)) + 8 * case["dim"],
                    flops=9 * n)
    # g, gh, h and the gradient of r, with dropout that of x beside it
    back = e * (3 + case["gh"] + (case["p"] > 0))
    return dict(bytes=n * ((4 * e if case["both"] else 0) + back) + 16 * case["dim"], flops=(24 if case["both"] else 15) * n)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_factor(case, s):
    """The factor of each element, 0 where it is dropped: the generator in NumPy's unsigned integers."""
    T, dim, p = case["T"], case["dim"], case["p"]
    if p == 0:
        return torch.ones(1, 1, dtype=torch.float64, device="cuda")
    blocks = -(-dim // 8)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = np.zeros((4, T * blocks), dtype=np.uint64)
    x[0], x[1], x[2] = np.tile(np.arange(blocks), T), np.repeat(np.arange(T), blocks), s["site"]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for _ in range(10):
        u, v = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = np.stack([(v >> half) ^ x[1] ^ np.uint64(key[0]), v & low, (u >> half) ^ x[3] ^ np.uint64(key[1]), u & low])
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    halves = np.ascontiguousarray(x.T.astype("<u4")).view("<u2").reshape(T, -1)[:, :dim].astype(np.int32)
    limit = int(np.rint(p * 65536))
    return torch.from_numpy(np.where(halves >= limit, 65536.0 / (65536 - limit), 0.0)).cuda()


def _exact_norm(s, factor):
    h = s["X"].double() * factor
    h = (h if s["R"] is None else h + s["R"].double()).to(s["X"].dtype).double()
    var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
    return h, mean, (var + s["eps"]) ** -0.5


def _exact_loss(case, s):
    X, W, target = s["X"].double(), s["W"].double(), s["target"]
    loss, lses, gx = [], [], []
    gw = torch.zeros_like(W) if case["train"] else None
    g = s["g"].double().expand(case["T"])
    for at in range(0, case["T"], 2048):
        x, t = X[at:at + 2048], target[at:at + 2048]
        z = torch.mm(W, x.T.contiguous()).T
        lse = torch.logsumexp(z, 1)
        lses.append(lse)
        loss.append(torch.nn.functional.cross_entropy(z, t, ignore_index=_IGNORE, reduction="none"))
        if case["train"]:
            share = torch.softmax(z, 1) - torch.nn.functional.one_hot(t.clamp(min=0), case["V"])
            share = share * (g[at:at + 2048] * (t != _IGNORE))[:, None]
            gx.append(torch.mm(share, W))
            gw += torch.mm(share.T.contiguous(), x)
    if not case["train"]:
        return dict(loss=torch.hstack(loss), lse=torch.hstack(lses))
    return dict(loss=torch.hstack(loss), G_X=torch.vstack(gx), G_W=gw)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "loss":
        return _exact_loss(case, s)
    factor = _exact_factor(case, s)
    if case["op"] == "drop":
        y = s["X"].double() * factor
        out = dict(Y=y if s["R"] is None else y + s["R"].double())
        if case["train"]:
            out["G_X"] = s["G"].double() * factor
        return out
    w, b = s["w"].double(), s["b"].double()
    if case["op"] == "norm":
        h, mean, r = _exact_norm(s, factor)
        y = torch.addcmul(b, (h - mean) * r, w)
        if case["out"] == "same":
            return dict(Y=y, H=h)
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127
        return dict(Y=torch.round(y / step[:, None]) * step[:, None], scale=step, H=h)
    out = {}
    if case["both"]:
        h, mean, r = _exact_norm(s, factor)
        out = dict(Y=torch.addcmul(b, (h - mean) * r, w), H=h)
    else:
        h, mean, r = s["H"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    u = (h - mean) * r                               # the row before its weight
    gu = s["G"].double() * w                         # the gradient that reaches it
    along = torch.linalg.vecdot(gu, u)[:, None] / u.shape[1]
    dh = (gu - gu.mean(1, keepdim=True) - u * along) * r
    if s["GH"] is not None:
        dh += s["GH"].double()
    out.update(G_X=dh * factor, G_R=dh, g_w=torch.linalg.vecdot(s["G"].double(), u, dim=0),
               g_b=torch.einsum("td->d", s["G"].double()))
    return out
