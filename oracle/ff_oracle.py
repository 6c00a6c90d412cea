"""Plain float64 oracles of the feed-forward operators: gated blocks and
products of groups of rows, the sum over a token's experts, dropout.

TEST INFRASTRUCTURE ONLY; the library never calls it and shares no code with
it. Gated block: Shazeer, "GLU Variants Improve Transformer". Dropout's words:
Philox4x32-10 of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
easy as 1, 2, 3", in Python's whole numbers or numpy's 64-bit ones.
"""
import math

import numpy as np


def act(g, kind):
    """(value, slope) of silu or gelu (the exact one, by erf)."""
    g = np.asarray(g, np.float64)
    if kind == "silu":
        s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * np.vectorize(math.erfc, otypes=[float])(-g / math.sqrt(2))
    return g * cdf, cdf + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def spans(offsets, slots):
    """(group, first, end) of the groups that have slots."""
    if offsets is None:
        offsets = [0, slots]
    for g in range(len(offsets) - 1):
        lo, hi = max(0, int(offsets[g])), min(slots, int(offsets[g + 1]))
        if hi > lo:
            yield g, lo, hi


def product(x, w, offsets, slots, source=None, back=False):
    """(y, magnitudes, written) in slot order: y[s] = x[source[s]] w_g^T (back: x[source[s]] w_g), zeros where source is
    negative or past x; magnitudes: the sum of the terms' absolute values; written: the slots that have a group."""
    cols = w.shape[2] if back else w.shape[1]
    y, mag, written = np.zeros((slots, cols)), np.zeros((slots, cols)), np.zeros(slots, bool)
    source = np.arange(slots) if source is None else np.asarray(source)
    for g, lo, hi in spans(offsets, slots):
        m = w[g] if back else w[g].T
        at = source[lo:hi]
        ok = (at >= 0) & (at < len(x))
        rows = np.where(ok[:, None], x[np.where(ok, at, 0)], 0.0) if len(x) else np.zeros((hi - lo, x.shape[1]))
        y[lo:hi], mag[lo:hi], written[lo:hi] = rows @ m, np.abs(rows) @ np.abs(m), True
    return y, mag, written


def philox(counter, key):
    """The four words of a block: counter and key as lists of 4 and 2 words, or 4 arrays and 2 words."""
    c = [np.asarray(v, np.uint64) for v in counter]
    low = np.uint64(0xFFFFFFFF)
    for i in range(10):
        k0, k1 = np.uint64((key[0] + i * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + i * 0xBB67AE85) % 2 ** 32)
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k0, b & low, (a >> np.uint64(32)) ^ c[3] ^ k1, a & low]
    return c


def kept(first, count, p, seed, offset):
    """Which of the elements first .. first + count - 1 dropout keeps."""
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    lo, hi = first // 4, (first + count + 3) // 4
    block = lo + np.arange(hi - lo, dtype=np.uint64)
    low, by = np.uint64(0xFFFFFFFF), np.uint64(32)
    fill = lambda v: np.full_like(block, v)  # noqa: E731
    words = philox([block & low, block >> by, fill(offset & 0xFFFFFFFF), fill(offset >> 32)], [seed & 0xFFFFFFFF, seed >> 32])
    words = np.stack(words, 1).reshape(-1)[first - 4 * lo:][:count]
    return words >= np.uint64(int(float(np.float32(p)) * 2 ** 32))


def dropped(shape, p, seed=0, offset=0):
    """0 or 1 / (1 - p) for each element of a matrix, row by row."""
    if p == 0:
        return np.ones(shape)
    return kept(0, shape[0] * shape[1], p, seed, offset).reshape(shape) / (1 - float(np.float32(p)))
