"""The weight's gradient of the RMS norm, a sum over all rows, where there are
many of them or a few outweigh the rest."""
import pytest

from gpu_util import device_ready, log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


# around each variant's rows: one wave, four waves, none that holds them
@pytest.mark.parametrize("dt, dim", [("bf16", 65), ("bf16", 512), ("bf16", 1000), ("bf16", 2048), ("bf16", 4001),
                                     ("bf16", 8192), ("bf16", 8200), ("f32", 64), ("f32", 333), ("f32", 512),
                                     ("f32", 1024), ("f32", 2047), ("f32", 4096), ("f32", 4100)])
def test_small_terms_behind_large_ones(dt, dim):
    """2048 rows with terms of 2^24, then 2^17 with terms of 1, which a sum held in fp32 would drop."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"small terms behind large ones, dim={dim} {dt}")
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    large, small = 2048, 2 ** 17
    x = torch.ones(large + small, dim, dtype=t, device="cuda")
    x[:large] = 4096
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    _, g_w = oec.add_rms_norm_backward(x, x, one(dim), one(large + small))
    want = large * 2.0 ** 24 + small
    # every term is exact; the partial sums, all positive, are rounded once and their sum once more
    off = (g_w.double() - want).abs().max()
    assert float(off) <= 2 * U * want, float(off) / want / U


@pytest.mark.parametrize("T, dim", [(1100003, 2048), (2 ** 23 + 5, 8)])
def test_rows_past_4_gib(T, dim):
    """Every row counts once: the sum against a 64-bit one, taken in pieces."""
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    log(f"weight gradient of {T} x {dim}")
    g = torch.Generator("cuda").manual_seed(T)
    G, H = (torch.empty(T, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    s = torch.rand(T, device="cuda", generator=g) + 0.5
    w = torch.ones(dim, device="cuda")
    _, g_w = oec.add_rms_norm_backward(G, H, w, s)
    want = torch.zeros(dim, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for a in range(0, T, 2 ** 17):
        t = G[a:a + 2 ** 17].double() * H[a:a + 2 ** 17].double() * s[a:a + 2 ** 17, None].double()
        want += t.sum(0)
        mag += t.abs().sum(0)
    # two roundings a term, one a partial sum, one at the end
    off = (g_w.double() - want).abs()
    assert bool((off <= 4 * U * mag).all()), float((off / mag).max()) / U
