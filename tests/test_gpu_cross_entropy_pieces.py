"""The cross entropy's backward over several pieces of the vocabulary, the last one shorter:
the sums of dX across them in every kind of kernel, element by element against 64 bits on the
device, with the tolerances of test_gpu_cross_entropy.py."""
import pytest

from gpu_util import device_ready, log
from test_gpu_cross_entropy import IGNORE, inputs, reference, run, run_back

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def near(name, got, want, tol):
    """close() on the device: these are large."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((d / tol).max()))


# A piece's dL/dz takes 256 MB at most, and 2^19 columns: many tokens in fp32 and in rows of no whole 16 bytes, then few
# tokens with more columns than that (with shared sums of dX, with d in two halves, one pass over the fewest fp32 tokens)
@pytest.mark.parametrize("T, n, V, dt", [
    (40000, 64, 2003, "f32"), (40000, 65, 2003, "f32"), (70000, 65, 2003, "bf16"), (70000, 264, 2003, "bf16"),
    (20, 65, 2 ** 19 + 777, "bf16"), (70, 65, 2 ** 19 + 777, "bf16"), (70, 64, 2 ** 19 + 777, "bf16"),
    (70, 65, 2 ** 19 + 777, "f32"), (70, 64, 2 ** 19 + 777, "f32"),
    (300, 264, 2 ** 19 + 777, "bf16"), (1, 1024, 2 ** 19 + 777, "f32"), (4, 1025, 2 ** 19 + 300, "f32"), (7, 1024, 2 ** 19 + 5, "f32"),
])
def test_several_pieces(T, n, V, dt):
    import torch
    log(f"cross entropy, several pieces T={T} n={n} V={V} {dt}")
    X, W, target, g = inputs(T, n, V, dt, seed=9, ignored=0.1 if T > 1 else 0.0)
    if T > 1:
        target[0], target[-1] = V - 1, 0
    each = (torch.rand(T, generator=g) + 0.1).cuda()
    X, W, target = X.cuda(), W.cuda(), target.cuda()
    assert bool((target != IGNORE).any())
    a = run(X, W, target, each)
    gx, none = run_back(X, W, target, a["lse"], each, need_w=False)
    assert none is None and torch.equal(gx, a["G_X"])
    none, gw = run_back(X, W, target, a["lse"], each, need_x=False)
    assert none is None and torch.equal(gw, a["G_W"])
    del gx, gw
    for k, (v, tol) in reference(X, W, target, each, dt).items():
        near(k, a[k], v, tol.expand_as(v))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tokens_in_several_launches(dt):
    """The forward of more tokens than the parts of their rows have room for (256 MB), the last launch of
    fewer than a tile: losses and statistics of all, and of every token as alone."""
    import torch
    T, n, V = 1100, 16, 2 ** 20 + 5
    log(f"cross entropy, several launches {dt}")
    X, W, target, _ = inputs(T, n, V, dt, seed=4)
    target[0], target[-1] = V - 1, V - 1
    X, W, target = X.cuda(), W.cuda(), target.cuda()
    a = run(X, W, target, None)
    for k, (v, tol) in reference(X, W, target, None, dt).items():
        near(k, a[k], v, tol)
