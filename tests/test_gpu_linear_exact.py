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
