"""The tests' generator against the published algorithm's known answers, and the mask's
statistics (no GPU)."""
import numpy as np
import pytest

from philox_ref import factors, philox


@pytest.mark.parametrize("counter, key, want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, want):
    assert tuple(int(x) for x in philox(counter, key)) == want


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_share_and_independence(p):
    """Shares of kept elements within 5 standard deviations, whole, by column and between sites."""
    n, (T, dim) = 512 * 400, (512, 400)
    a, b = factors(T, dim, p, 7, 1) > 0, factors(T, dim, p, 7, 2) > 0
    s = (p * (1 - p)) ** 0.5
    assert abs(a.mean() - (1 - p)) < 5 * s / n ** 0.5 + 2.0 ** -16
    assert np.abs(a.mean(0) - (1 - p)).max() < 5 * s / T ** 0.5
    assert abs((a == b).mean() - ((1 - p) ** 2 + p ** 2)) < 5 * 0.5 / n ** 0.5 + 2.0 ** -15
    assert abs(factors(T, dim, p, 7, 1).mean() - 1) < 5 * s / (1 - p) / n ** 0.5
