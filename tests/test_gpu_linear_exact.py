"""The merged-weight product on small whole numbers: every order of summation is
exact as long as sums of magnitudes stay below 2^24, so results are compared for
equality and one lost or doubled piece of n shows."""
import pytest

from gpu_util import device_ready, log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def test_narrow_result_of_very_many_rows():
    """2^28 rows of a result of two columns, more than one launch of 32-column tiles counts."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    T, n, m = 2 ** 28 + 5, 3, 2
    log(f"narrow {T} x {n} -> {m}")
    X = torch.arange(T * n, device="cuda", dtype=torch.int32).remainder_(1021).float().view(T, n)
    W = torch.tensor([[1.0, -2.0, 3.0], [2.0, 5.0, -7.0]], device="cuda")
    y = oec.linear(X, W)
    for c in range(m):
        want = X[:, 0] * W[c, 0]
        for k in range(1, n):
            want += X[:, k] * W[c, k]
        assert torch.equal(y[:, c], want)


def whole(gen, rows, cols, dtype, pad):
    """Whole numbers from -3 to 3 without 0 in rows `pad` elements apart; beside them lies what would show in a sum."""
    import torch
    other = 77 if dtype == torch.int8 else float("nan")
    buf = torch.full((rows, cols + pad), other, dtype=dtype, device="cuda")
    v = torch.randint(1, 7, (rows, cols), generator=gen, device="cuda", dtype=torch.int32)
    buf[:, :cols] = torch.where(v > 3, 3 - v, v).to(dtype)
    return buf[:, :cols]


def check(T, n, m, dt, pad=0):
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"exact T={T} n={n} m={m} {dt} pad={pad}")
    t = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}[dt]
    g = torch.Generator("cuda").manual_seed(T * 7 + n * 3 + m)
    X, W = whole(g, T, n, t, pad), whole(g, m, n, t, pad)
    kw = {}
    if dt == "int8":
        kw = dict(x_scale=torch.ones(T, device="cuda"), w_scale=torch.ones(m, device="cuda"))
    y = oec.linear(X, W, out_dtype=torch.float32, **kw)
    want = torch.mm(X.double(), W.double().T.contiguous())
    assert torch.equal(y.double(), want), (T, n, m, dt, pad, int((y.double() != want).sum()))


TYPES = pytest.mark.parametrize("dt", ["bf16", "f32", "int8"])


@TYPES
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8])
def test_few_tokens(T, dt):
    """Every length of a row's end, alone and behind whole pieces of it."""
    for n in [*range(1, 36), *range(1010, 1030), 4096, 4097, 4111, 5632, 16385]:
        check(T, n, 37, dt)
    for pad in (1, 16):
        check(T, 1021, 37, dt, pad)
        check(T, 4096, 37, dt, pad)


# grids of every tile; n of whole stages, cut stages, whole 16 bytes of one type and not of another, and odd
@TYPES
@pytest.mark.parametrize("T, m", [(20, 70), (30, 2047), (130, 4096), (500, 2040), (1030, 2040), (4090, 2056),
                                  (16390, 1032)])
def test_every_tile(T, m, dt):
    for n in (1, 5, 16, 40, 48, 64, 70, 112, 129, 135, 192, 208, 256, 333, 512, 1000, 1003, 1024, 1040):
        check(T, n, m, dt)
    for pad in (1, 16):
        check(T, 208, m, dt, pad)
        check(T, 256, m, dt, pad)


@TYPES
@pytest.mark.parametrize("T, n, m", [(40, 16400, 33), (6, 16384, 40), (9, 5311, 256), (14, 7184, 76), (70, 6160, 70),
                                     (33, 4112, 100), (5, 65536, 8), (6, 32000, 40)])
def test_shared_sums(T, n, m, dt):
    """Several workgroups to a tile: pieces of n that end anywhere, down to shares with nothing left."""
    for k in (0, 1, 2, 3, 4, 8, 15, 16, 32, 48, 64, 100, 128, 1000):
        check(T, n - k, m, dt)
    check(T, n, m, dt, 16)
    check(T, n, m, dt, 3)
