"""The numbers of a dropout's rule that the Python binding takes and refuses (no GPU)."""
import math

import pytest

torch = pytest.importorskip("torch")
from orthogonal_equivalence_cayley_amd import block_ops  # noqa: E402

DEV = 0


@pytest.mark.parametrize("p, seed, site", [
    (-1e-9, 1, 0), (1 + 1e-9, 1, 0), (math.nan, 1, 0), (math.inf, 1, 0), (-math.inf, 1, 0),
    (0.1, -1, 0), (0.1, 2 ** 64, 0), (0.1, 1, -1), (0.1, 1, 2 ** 32),
    # a seed in memory: one int64 value on the device of the matrices
    (0.1, torch.tensor([1]), 0), (0.1, torch.tensor([1], dtype=torch.int32), 0), (0.1, torch.tensor([1.0]), 0),
    (0.1, torch.tensor([1, 2]), 0), (0.1, torch.tensor([], dtype=torch.int64), 0),
])
def test_refused(p, seed, site):
    with pytest.raises(ValueError):
        block_ops._drop_rule(p, seed, site, DEV)


@pytest.mark.parametrize("p, seed, site", [(0.5, 0, 0), (1.0, 2 ** 64 - 1, 2 ** 32 - 1), (2.0 ** -30, 7, 3), (1, 7, 3)])
def test_taken(p, seed, site):
    r = block_ops._drop_rule(p, seed, site, DEV)
    assert (r.p, r.seed, r.seed_dev, r.site) == (p, seed, None, site)


def test_nothing_dropped_needs_no_seed():
    r = block_ops._drop_rule(0.0, None, -5, DEV)
    assert (r.p, r.seed, r.seed_dev, r.site) == (0.0, 0, None, 0)
