"""Cases of the operators around a block's linears: the residual and root-mean-square norm, the product with a merged
weight and its epilogue, and the clipping of all gradients by their global norm.

Plain forms are elementary torch operations in 32 bits (64 where a sum or a decision needs them); with `own` set, `run`
calls the package. Sizes are those of the framework's blocks (hidden 2048 and 4096, feed-forward 5632 and 11008, 16384
tokens), and ragged ones beside them.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _norm(name, T, dim, dtype="bf16", residual=True, out="same"):
    return dict(name=name, op="norm", T=T, dim=dim, dtype=dtype, residual=residual, out=out)


def _norm_train(name, T, dim, dtype, both, gh=True):
    return dict(name=name, op="norm_train", T=T, dim=dim, dtype=dtype, both=both, gh=gh)


def _linear(name, T, n, m, dtype, act="none", bias=False, mul=False, residual=False):
    return dict(name=name, op="linear", T=T, n=n, m=m, dtype=dtype, act=act, bias=bias, mul=mul, residual=residual)


def _clip(name, hidden, ff, block, layers, norms, dense, clipped=True):
    return dict(name=name, op="clip", hidden=hidden, ff=ff, block=block, layers=layers, norms=norms, dense=dense,
                clipped=clipped)


def listed():
    return [
        # one token being generated, between two linears of a hidden-2048 block: latency
        _norm("norm_token", 1, 2048),
        # a prompt in front of INT8 linears, hidden 4096: the output as INT8 rows with scales
        _norm("norm_prompt_int8", 16384, 4096, out="int8"),
        # the training batch of the hidden-2048 block
        _norm("norm_batch", 16384, 2048),
        # its backward, with the gradient that arrives through the residual stream
        _norm_train("norm_backward", 16384, 2048, "bf16", both=False),
        # a ragged fp32 layer trained: forward and backward
        _norm_train("norm_train_odd_f32", 1003, 1365, "f32", both=True),
        # one token through the merged gate projection of the hidden-2048 block: bound by the weight's bytes
        _linear("linear_token", 1, 2048, 5632, "bf16", act="silu"),
        # requests decoded together, hidden 4096, INT8 weight and activation
        _linear("linear_batch_int8", 24, 4096, 11008, "int8", act="silu"),
        # the gated feed-forward of a prompt: silu(X Wg^T) times the up projection
        _linear("linear_prompt", 16384, 2048, 5632, "bf16", act="silu", mul=True),
        # the down projection of a long prompt in INT8, added to the residual stream
        _linear("linear_prompt_int8", 16384, 11008, 4096, "int8", residual=True),
        # a ragged fp32 layer with every part of the epilogue
        _linear("linear_odd_f32", 1531, 1005, 707, "f32", act="gelu", bias=True, mul=True, residual=True),
        # all packed gradients of the hidden-2048 block: 14 sides and two norm weights, 20 MB
        _clip("clip_block", 2048, 5632, 256, 1, 2, 0),
        # 12 blocks at hidden 4096 and blocks of 512, each with a dense weight trained in bf16: 204 tensors, 1.4 GB
        _clip("clip_model", 4096, 11264, 512, 12, 2, 1),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width of a kind in use: a multiple of 256, of 16, or any."""
    step = rng.choice([256, 256, 16, 1])
    return min(hi, max(1, _spread(rng, lo, hi) // step) * step)


def draw(rng):
    op = rng.choice(["norm", "norm_train", "linear", "linear", "clip"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = _norm("", _spread(rng, 1, 16384), _width(rng, 64, 4096), dtype, rng.random() < 0.75,
                  rng.choice(["same", "int8"]))
    elif op == "norm_train":
        c = _norm_train("", _spread(rng, 1, 16384), _width(rng, 64, 4096), rng.choice(["bf16", "bf16", "f32"]),
                        rng.random() < 0.5, rng.random() < 0.7)
    elif op == "linear":
        dtype = rng.choice(["bf16", "bf16", "int8", "int8", "f32"])
        T = _spread(rng, 1, 16384 if dtype != "f32" else 2048)
        c = _linear("", T, _width(rng, 64, 8192), _width(rng, 64, 5632), dtype,
                    rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rng.random() < 0.5, rng.random() < 0.4,
                    rng.random() < 0.5)
    else:
        block = rng.choice([32, 64, 128, 256, 512])
        c = _clip("", block * rng.randint(1, 8), block * rng.randint(2, 22), block, rng.randint(1, 8),
                  rng.randint(0, 3), rng.randint(0, 1), rng.random() < 0.8)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _shapes(case):
    """Element counts and types of the gradients of `clip`, by block: both sides of the seven linears (packed skew
    parameters), `norms` weights as wide as the block, `dense` square weights in bf16."""
    tri = case["block"] * (case["block"] - 1) // 2
    h, f = case["hidden"] // case["block"] * tri, case["ff"] // case["block"] * tri
    f32 = [h] * 8 + [f, h, f, h, h, f] + [case["hidden"]] * case["norms"]
    return ([(k, "f32") for k in f32] + [(case["hidden"] ** 2, "bf16")] * case["dense"]) * case["layers"]


def _draw_int8(shape, g):
    """INT8 rows and scales as quantising a normal row gives them: the largest of a row at 127."""
    v = torch.randn(shape, generator=g, device="cuda")
    a = v.abs().amax(1, keepdim=True)
    return torch.round(v * (127 / a)).to(torch.int8), (a[:, 0] / 127).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] in ("norm", "norm_train"):
        T, d, dt = case["T"], case["dim"], _TYPES[case["dtype"]]
        # a residual stream has a few channels far larger than the rest, and tokens of different sizes
        channel = torch.exp(0.5 * rand(d)) * torch.exp(0.3 * rand(T, 1))
        s.update(X=(rand(T, d) * 0.3).to(dt), R=(rand(T, d) * channel).to(dt), w=1 + 0.1 * rand(d), eps=1e-6)
        if case["op"] == "norm":
            s["values"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda") if case["out"] == "int8" else None
            if not case["residual"]:
                s["X"], s["R"] = s["R"], None
        else:
            s.update(G=(rand(T, d) * 1e-2).to(dt), GH=(rand(T, d) * 1e-2).to(dt) if case["gh"] else None)
            if not case["both"]:
                # what the forward kept
                H = s["R"].double()
                s["H"], s["rstd"] = s["R"], (H.square().mean(1) + s["eps"]).rsqrt().float()
    elif case["op"] == "linear":
        T, n, m = case["T"], case["n"], case["m"]
        dt = torch.bfloat16 if case["dtype"] == "int8" else _TYPES[case["dtype"]]
        if case["dtype"] == "int8":
            s["X"], s["sx"] = _draw_int8((T, n), g)
            s["W"], s["sw"] = _draw_int8((m, n), g)
            s["sw"] = s["sw"] / math.sqrt(n)
        else:
            s.update(X=rand(T, n).to(dt), W=(rand(m, n) / math.sqrt(n)).to(dt), sx=None, sw=None)
        s["b"] = 0.1 * rand(m) if case["bias"] else None
        s["mul"] = rand(T, m).to(dt) if case["mul"] else None
        s["res"] = rand(T, m).to(dt) if case["residual"] else None
        s["dt"] = dt
    else:
        shapes = _shapes(case)
        grads = [(rand(k) * 1e-3).to(_TYPES[t]) for k, t in shapes]
        # the clipped gradients go to one buffer of each type, one tensor behind the other
        s["flat"] = {t: torch.empty(sum(k for k, u in shapes if u == t), dtype=_TYPES[t], device="cuda")
                     for t in ("f32", "bf16")}
        parts = {t: list(torch.split(f, [k for k, u in shapes if u == t])) for t, f in s["flat"].items()}
        # the norm is about 1e-3 sqrt(parameters): the limit lies below it, or above
        s.update(grads=grads, outs=[parts[t].pop(0) for _, t in shapes],
                 limit=1e-3 * math.sqrt(sum(k for k, _ in shapes)) * (0.3 if case["clipped"] else 3.0))
    return s


# ------------------------------------------------------------------ plain forms
def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_norm(X, R, w, eps):
    """h in the type, 1 / rms in 32 bits from sums in 64, the normalised row in 32 bits."""
    H = X if R is None else (X.float() + R.float()).to(X.dtype)
    hf = H.float()
    rstd = (1 / torch.sqrt((hf.double() * hf.double()).mean(1) + eps)).float()
    return H, rstd, hf * rstd[:, None] * w


def _plain_back(G, GH, H, w, rstd):
    g, h, s = G.float(), H.float(), rstd[:, None]
    c = (g * w * h).mean(1, keepdim=True) * s * s
    dx = s * (g * w - h * c)
    if GH is not None:
        dx = dx + GH.float()
    return dx.to(G.dtype), (g * h * s).sum(0, dtype=torch.float64).float()


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        H, _, y = _plain_norm(s["X"], s["R"], s["w"], s["eps"])
        if case["out"] == "same":
            return dict(Y=y.to(H.dtype), H=H)
        a = y.abs().amax(1, keepdim=True)
        none = a < 2.0 ** -119
        inv = torch.where(none, torch.zeros_like(a), 127 / a)
        scale = torch.where(none, torch.zeros_like(a), a / 127)
        return dict(Y=(torch.round(y * inv) * scale).to(torch.bfloat16), scale=scale[:, 0], H=H)
    if case["op"] == "norm_train":
        out = {}
        H, rstd = s.get("H"), s.get("rstd")
        if case["both"]:
            H, rstd, y = _plain_norm(s["X"], s["R"], s["w"], s["eps"])
            out = dict(Y=y.to(H.dtype), H=H)
        out["G_X"], out["g_w"] = _plain_back(s["G"], s["GH"], H, s["w"], rstd)
        return out
    if case["op"] == "linear":
        z = s["X"].float() @ s["W"].float().T
        if s["sx"] is not None:
            z = z * s["sx"][:, None] * s["sw"]
        if s["b"] is not None:
            z = z + s["b"]
        z = _plain_act(z, case["act"])
        if s["mul"] is not None:
            z = z * s["mul"].float()
        if s["res"] is not None:
            z = z + s["res"].float()
        return z.to(s["dt"])
    flat = {t: torch.cat([x for x in s["grads"] if x.dtype == _TYPES[t]] or [f]).float() for t, f in s["flat"].items()}
    total = (flat["f32"].double() * flat["f32"].double()).sum() + (flat["bf16"].double() * flat["bf16"].double()).sum()
    norm = torch.sqrt(total)
    c = torch.clamp(s["limit"] / (norm + 1e-6), max=1.0).float()
    return dict(norm=norm.float(), grads={t: (f * c).to(_TYPES[t]) for t, f in flat.items()})


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import orthogonal_equivalence_cayley_amd as oec
    case = s["case"]
    if case["op"] == "norm":
        o = oec.add_rms_norm(s["X"], s["w"], residual=s["R"], eps=s["eps"], quantize=case["out"] == "int8")
        if case["out"] == "same":
            return dict(Y=o.Y, H=o.H)
        return dict(Y=torch.mul(o.Y, o.scale[:, None], out=s["values"]), scale=o.scale, H=o.H)
    if case["op"] == "norm_train":
        out = {}
        H, rstd = s.get("H"), s.get("rstd")
        if case["both"]:
            o = oec.add_rms_norm(s["X"], s["w"], residual=s["R"], eps=s["eps"], save=True)
            H, rstd = o.H, o.rstd
            out = dict(Y=o.Y, H=H)
        out["G_X"], out["g_w"] = oec.add_rms_norm_backward(s["G"], H, s["w"], rstd, G_H=s["GH"])
        return out
    if case["op"] == "linear":
        return oec.linear(s["X"], s["W"], bias=s["b"], act=case["act"], mul=s["mul"], residual=s["res"],
                          x_scale=s["sx"], w_scale=s["sw"])
    norm = oec.clip_grads(s["grads"], s["limit"], out=s["outs"])
    return dict(norm=norm, grads=s["flat"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors
def work(case):
    if case["op"] in ("norm", "norm_train"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * case["dim"]
        if case["op"] == "norm":
            # reads x (and r), writes y (and h)
            return dict(bytes=n * (e + (2 * e if case["residual"] else 0) + (e if case["out"] == "same" else 1)) +
                        4 * case["dim"], flops=6 * n)
        back = 3 * e + (e if case["gh"] else 0)
        return dict(bytes=n * ((4 * e if case["both"] else 0) + back) + 8 * case["dim"],
                    flops=(16 if case["both"] else 10) * n)
    if case["op"] == "linear":
        T, n, m = case["T"], case["n"], case["m"]
        e = {"bf16": 2, "f32": 4, "int8": 1}[case["dtype"]]
        o = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=e * (T * n + m * n) + o * T * m * (1 + case["mul"] + case["residual"]),
                    flops=2 * T * n * m)
    shapes = _shapes(case)
    return dict(bytes=sum(2 * k * (4 if t == "f32" else 2) for k, t in shapes), flops=3 * sum(k for k, _ in shapes))


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(X, R, w, eps):
    h = X.double() if R is None else (X.double() + R.double()).to(X.dtype).double()
    mean = torch.linalg.vecdot(h, h) / h.shape[1]
    return h, (mean + eps) ** -0.5


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, r = _exact_norm(s["X"], s["R"], s["w"], s["eps"])
        y = torch.einsum("td,t,d->td", h, r, s["w"].double())
        if case["out"] == "same":
            return dict(Y=y, H=h)
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127
        return dict(Y=torch.round(y / step[:, None]) * step[:, None], scale=step, H=h)
    if case["op"] == "norm_train":
        out = {}
        if case["both"]:
            h, r = _exact_norm(s["X"], s["R"], s["w"], s["eps"])
            out = dict(Y=torch.einsum("td,t,d->td", h, r, s["w"].double()), H=h)
        else:
            h, r = s["H"].double(), s["rstd"].double()
        u = h * r[:, None]                           # the row before its weight
        gu = s["G"].double() * s["w"].double()       # the gradient that reaches it
        along = torch.linalg.vecdot(gu, u) / u.shape[1]
        out["G_X"] = (gu - u * along[:, None]) * r[:, None]
        if s["GH"] is not None:
            out["G_X"] += s["GH"].double()
        out["g_w"] = torch.linalg.vecdot(s["G"].double(), u, dim=0)
        return out
    if case["op"] == "linear":
        X, W = s["X"].double(), s["W"].double()
        if s["sx"] is not None:
            X, W = X * s["sx"].double()[:, None], W * s["sw"].double()[:, None]
        z = torch.mm(W, X.T.contiguous()).T
        if s["b"] is not None:
            z = z + s["b"].double()
        if case["act"] == "relu":
            z = z.clamp(min=0)
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "gelu_tanh":
            # (1 + tanh(u)) / 2 is the logistic function of 2 u
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        if s["mul"] is not None:
            z = z * s["mul"].double()
        return z if s["res"] is None else z + s["res"].double()
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(x.double()) for x in s["grads"]]))
    c = min(1.0, s["limit"] / (norm.item() + 1e-6))
    return dict(norm=norm, grads={t: torch.hstack([x.double() * c for x in s["grads"] if x.dtype == _TYPES[t]] or [f.double()])
                                  for t, f in s["flat"].items()})
