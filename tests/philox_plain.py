"""Philox 4x32-10 in Python integers, from its published definition, and the
dropout mask that the library derives from it."""
import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Four words; the counter's four and the key's two words as Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = M0 * c[0], M1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + W0) & 0xffffffff, (k[1] + W1) & 0xffffffff]
    return c


def draws(n, seed, site):
    """The 16 bits of elements 0 .. n - 1."""
    out = []
    for i in range((n + 7) // 8):
        for w in philox((i & 0xffffffff, i >> 32, site & 0xffffffff, site >> 32), (seed & 0xffffffff, seed >> 32)):
            out += [w & 0xffff, w >> 16]
    return np.array(out[:n], dtype=np.int64)


def mask(shape, p, seed, site):
    """0 or the multiplier of each element, float64."""
    n = int(np.prod(shape))
    step = round(p * 65536)
    kept = draws(n, seed % 2 ** 64, site % 2 ** 64) >= step
    return (kept * (65536 / (65536 - step) if step < 65536 else 0.0)).reshape(shape)
