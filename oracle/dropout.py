"""Dropout oracle: the generator word by word on Python integers' arithmetic in
numpy, and the masked, scaled sum in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The generator is Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", SC 2011): the counter's four
words x0 .. x3 become (hi(B x2) ^ x1 ^ k0, lo(B x2), hi(A x0) ^ x3 ^ k1, lo(A x0))
in every round, and the key's words grow by the golden ratio and sqrt(3) - 1.
"""
import math

import numpy as np

A, B = 0xD2511F53, 0xCD9E8D57
STEP0, STEP1 = 0x9E3779B9, 0xBB67AE85
WORD = 0xFFFFFFFF


def philox(counter, key):
    """Four words of 32 bits for one counter (four words) and key (two)."""
    x, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(10):
        p, q = A * x[0], B * x[2]
        x = [(q >> 32) ^ x[1] ^ k[0], q & WORD, (p >> 32) ^ x[3] ^ k[1], p & WORD]
        k = [(k[0] + STEP0) & WORD, (k[1] + STEP1) & WORD]
    return x


def bits(first: int, n: int, seed: int, offset: int) -> np.ndarray:
    """The 16-bit numbers of elements first .. first + n - 1."""
    b0, b1 = first // 8, -(-(first + n) // 8)
    b = np.arange(b0, b1, dtype=np.uint64)
    x = [b & np.uint64(WORD), b >> np.uint64(32)]
    x += [np.full_like(b, offset & WORD), np.full_like(b, offset >> 32 & WORD)]
    k = [seed & WORD, seed >> 32 & WORD]
    for _ in range(10):
        p, q = np.uint64(A) * x[0], np.uint64(B) * x[2]  # 32 x 32 bits fit 64
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), q & np.uint64(WORD),
             (p >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), p & np.uint64(WORD)]
        k = [(k[0] + STEP0) & WORD, (k[1] + STEP1) & WORD]
    halves = [h for w in x for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))]
    return np.stack(halves, 1).reshape(-1)[first - 8 * b0:][:n].astype(np.int64)


def threshold(p: float) -> int:
    return math.floor(p * 65536 + 0.5)


def dropout(x: np.ndarray, p: float, seed: int, offset: int, residual=None, first: int = 0) -> np.ndarray:
    """residual + dropout(x) of an array seen as its elements first, first + 1, ..."""
    x = np.asarray(x, np.float64)
    t = threshold(p)
    kept = bits(first, x.size, seed, offset).reshape(x.shape) >= t
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    y = np.zeros(x.shape)
    np.multiply(x, scale, out=y, where=kept)
    return y if residual is None else y + np.asarray(residual, np.float64)
