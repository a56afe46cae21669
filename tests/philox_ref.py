"""Philox 4x32-10 in NumPy's unsigned integers, as the published algorithm has it, and the
mask of dropout made from it: the reference of the dropout tests."""
import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """counter: uint64 array [4, ...] of 32-bit words; key: two 32-bit numbers. The four words of each result."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c0, c1, c2, c3 = (np.asarray(c, dtype=np.uint64) for c in counter)
    k0, k1 = key
    for _ in range(10):
        a, b = c0 * np.uint64(M0), c2 * np.uint64(M1)
        c0, c1, c2, c3 = (b >> half) ^ c1 ^ np.uint64(k0), b & low, (a >> half) ^ c3 ^ np.uint64(k1), a & low
        k0, k1 = (k0 + W0) % 2 ** 32, (k1 + W1) % 2 ** 32
    return c0, c1, c2, c3


def factors(T, dim, p, seed, site):
    """Of each element of [T, dim]: 0 where it is dropped, else 65536 / (65536 - rint(65536 p))."""
    q = int(np.rint(p * 65536))
    if q == 0:
        return np.ones((T, dim))
    blocks = (dim + 7) // 8
    row, col = np.meshgrid(np.arange(T), np.arange(blocks), indexing="ij")
    w = philox((col, row, np.full_like(row, site), np.zeros_like(row)), (seed % 2 ** 32, seed // 2 ** 32))
    halves = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=-1)
    keep = halves.reshape(T, blocks * 8)[:, :dim] >= np.uint64(q)
    return np.where(keep, 65536.0 / (65536 - q) if q < 65536 else 0.0, 0.0)
