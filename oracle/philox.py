"""Dropout mask of a counter-based generator (oracle; test only).

Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011): ten rounds of two 32 x 32 -> 64 bit products over a 128-bit counter, the 64-bit key
raised by two odd constants between rounds. Value i of a tensor takes half i % 8 (low halves
first) of the four words for the counter (i // 8, offset) and the key `seed`, and is dropped
where those 16 bits are below round(65536 p).
"""
from __future__ import annotations

import numpy as np

_LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key):
    """counter uint32 [n, 4], key (k0, k1) -> uint32 [n, 4]."""
    c = [np.asarray(counter)[:, i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & _LOW, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def dropout_bits(n: int, seed: int, offset: int, first: int = 0):
    """The 16 random bits of values first .. first + n - 1 (first % 8 == 0)."""
    b = np.arange(first // 8, first // 8 + (n + 7) // 8, dtype=np.uint64)
    off = offset & 0xFFFFFFFFFFFFFFFF
    ctr = np.stack([b & _LOW, b >> np.uint64(32), np.full_like(b, off & 0xFFFFFFFF), np.full_like(b, off >> 32)], 1)
    w = philox4x32(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    return np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]


def dropout_threshold(p: float) -> int:
    return round(p * 65536)


def dropout_keep(shape, p: float, seed: int, offset: int = 0):
    """Truth values: which values stay."""
    return (dropout_bits(int(np.prod(shape)), seed, offset) >= dropout_threshold(p)).reshape(shape)


def dropout_scale(p: float) -> float:
    t = dropout_threshold(p)
    return 65536 / (65536 - t) if t < 65536 else 0.0
