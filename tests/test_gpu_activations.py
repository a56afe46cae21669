"""The activations of the merged-weight product at chosen arguments: one weight
column holds them and one activation is 1, so the sum is the argument itself,
exactly, and only the activation's own error is left."""
import math

import pytest

from gpu_util import device_ready, log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def at_arguments(z, act, T, n, dtype, out_dtype):
    """act(z) through the product: T equal tokens, n columns of which the first counts."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    X = torch.zeros(T, n, dtype=dtype, device="cuda")
    X[:, 0] = 1
    W = torch.zeros(z.numel(), n, dtype=dtype, device="cuda")
    W[:, 0] = z.to(dtype)
    y = oec.linear(X, W, act=act, out_dtype=out_dtype)
    same = torch.where(torch.isnan(y), torch.zeros_like(y), y)   # NaN of every token: compared as one value
    assert torch.equal(same, same[:1].expand_as(same)) and torch.equal(torch.isnan(y), torch.isnan(y[:1]).expand_as(y))
    return y[0].cpu().double()


def gelu_exact(z):
    import torch
    z = z.double()
    return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))


# by rows, in register-filled tiles, in the ring, in the 256 x 256 tiles
@pytest.mark.parametrize("T, n, dt", [(1, 1, "f32"), (5, 1, "f32"), (300, 4, "f32"), (1, 8, "bf16"), (40, 3, "bf16"),
                                      (16390, 64, "bf16")])
def test_gelu_of_negative_arguments_fp32(T, n, dt):
    """fp32 results relative to their own size, far into the tail, and the limits at the ends."""
    import torch
    log(f"gelu fp32 T={T} n={n} {dt}")
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[dt]
    z = torch.linspace(-13, 6, 1032).to(dtype)
    z[-3:] = torch.tensor([-math.inf, math.inf, math.nan]).to(dtype)
    y = at_arguments(z, "gelu", T, n, dtype, torch.float32)
    assert y[-3] == 0 and y[-2] == math.inf and math.isnan(y[-1])
    z, y = z[:-3].double(), y[:-3]
    v = gelu_exact(z)
    # units of 2^-24: t 3 (its sum, the hardware's reciprocal), 1 - 2 t and the polynomial 3.5, its fit 0.2, t P 1, the
    # hardware's exponential 2 and what it is given 1, two products 2, the difference 1
    tol = 14 * U * v.abs()
    bad = (y - v).abs() > tol
    assert not bad.any(), [(float(a), float(b), float(c)) for a, b, c in zip(z[bad][:5], y[bad][:5], v[bad][:5])]


@pytest.mark.parametrize("T, n", [(1, 8), (40, 3), (300, 8), (16390, 64)])
def test_gelu_of_negative_arguments_bf16(T, n):
    """bf16 results by half a step of their own, far into the tail, and the limits at the ends."""
    import torch
    log(f"gelu bf16 T={T} n={n}")
    z = torch.linspace(-13, 6, 1032).bfloat16()
    z[-3:] = torch.tensor([-math.inf, math.inf, math.nan]).bfloat16()
    y = at_arguments(z, "gelu", T, n, torch.bfloat16, torch.bfloat16)
    assert y[-3] == 0 and y[-2] == math.inf and math.isnan(y[-1])
    z, y = z[:-3].double(), y[:-3]
    v = gelu_exact(z)
    # the steps above with a fit of 10.5 units; the exponential's argument z^2 / 2 is off by three of its roundings,
    # (3 / 2) z^2 units; half a step
    tol = ((25 + 2 * z ** 2) * U + 2.0 ** -8) * v.abs()
    bad = (y - v).abs() > tol
    assert not bad.any(), [(float(a), float(b), float(c)) for a, b, c in zip(z[bad][:5], y[bad][:5], v[bad][:5])]


@pytest.mark.parametrize("dt, out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T, n", [(1, 8), (40, 3), (300, 8), (16390, 64)])
def test_limits(T, n, dt, out):
    """Infinite, largest and NaN sums, as the header states them."""
    import torch
    if dt == "f32" and T > 300:
        T = 300
    log(f"limits T={T} n={n} {dt} to {out}")
    t = {"f32": torch.float32, "bf16": torch.bfloat16}
    big = torch.finfo(t[dt]).max
    z = torch.tensor([math.inf, big, -big, -math.inf, math.nan] + [0.0] * 1027)
    at_end = {"none": -math.inf, "relu": 0.0, "gelu": 0.0, "silu": math.nan, "gelu_tanh": math.nan}
    for act, end in at_end.items():
        y = at_arguments(z, act, T, n, t[dt], t[out])
        assert y[0] == math.inf and y[1] == big, act
        assert y[2] == (-big if act == "none" else 0.0), act
        assert y[3] == end or (math.isnan(end) and math.isnan(y[3])), act
        assert math.isnan(y[4]) and not y[5:].any(), act
