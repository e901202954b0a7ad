"""Decode over part of a paged cache, restated from its definition in fp64 (oracle).

Bounds: of a block's keys (64 rows of one KV head) the largest and the smallest per feature, in 8 bits: with a =
max |k|, scale 2^e for the least e in [-32, 16] with a <= 127 * 2^e (16 where there is none), upper = ceil(max / 2^e),
lower = floor(min / 2^e), within [-127, 127]. A NaN counts as the infinity of its sign.

Scores: a query head in 8 bits the same way (nearest, ties to even), q = c 2^f; a block's score is the largest over the
KV head's six query heads of 2^(e + f) sum max(c upper, c lower). Whole numbers and powers of two: exact.

Choice: the first `sink` and the last `recent` blocks, then the largest scores (the lower index first), `budget` in all,
ascending.

Test infrastructure only: nothing in the CUDA library or its binding imports this.
"""
from __future__ import annotations

import math

import numpy as np

from . import bf16

BLOCK = 64
PAGE = 128


def values(bits: np.ndarray) -> np.ndarray:
    """fp64 values of bf16 bits, a NaN as the infinity of its sign."""
    x = bf16.to_f64(bits)
    return np.where(np.isnan(x), np.where(bits & 0x8000, -np.inf, np.inf), x)


def exponent(a: float) -> int:
    for e in range(-32, 16):
        if a <= 127.0 * 2.0 ** e:
            return e
    return 16


def bounds(bits: np.ndarray) -> tuple[np.ndarray, float]:
    """Codes int8 [2, 128] (upper, lower) and scale of one head's rows of a block, bf16 bits [rows, 128]."""
    x = values(bits)
    hi, lo = x.max(0), x.min(0)
    two = 2.0 ** exponent(float(np.abs(x).max()))
    return np.stack((np.clip(np.ceil(hi / two), -127, 127), np.clip(np.floor(lo / two), -127, 127))).astype(np.int8), two


def query(bits: np.ndarray) -> tuple[np.ndarray, float]:
    """Codes [128] and scale of a query head's bf16 bits [128]."""
    x = values(bits)
    two = 2.0 ** exponent(float(np.abs(x).max()))
    return np.clip(np.rint(x / two), -127, 127), two


def scores(q_bits: np.ndarray, codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Scores [n] of blocks with codes [n, 2, 128] and scale [n], for one KV head's queries bf16 bits [6, 128]."""
    best = np.full(len(codes), -np.inf)
    for bits in q_bits:
        c, two = query(bits)
        s = np.maximum(c * codes[:, 0].astype(np.float64), c * codes[:, 1].astype(np.float64)).sum(1) * two
        best = np.maximum(best, s)
    return best * scale


def choose(score: np.ndarray, budget: int, sink: int, recent: int) -> list[int]:
    n = len(score)
    must = [i for i in range(n) if i < sink or i >= n - recent]
    rest = sorted((i for i in range(n) if i not in must), key=lambda i: (-score[i], i))
    return sorted(must + rest[:max(0, budget - len(must))])


def attend(q: np.ndarray, K: np.ndarray, V: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """q [n, 128] over K, V [L, 128] (fp64): outputs, and sum of weights x |v| (what a relative error of weights meets)."""
    c = 30.0 * np.tanh(q @ K.T / math.sqrt(128.0) / 30.0)
    w = np.exp(c - c.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return w @ V, w @ np.abs(V)


def rows_of(entries, n_rows: int) -> np.ndarray:
    """Rows of the listed blocks below n_rows, a block listed twice twice."""
    out = [np.arange(i * BLOCK, min((i + 1) * BLOCK, n_rows)) for i in entries if i >= 0]
    return np.concatenate(out) if out else np.zeros(0, np.int64)


def at(table_row: np.ndarray, rows: np.ndarray) -> np.ndarray:
    """Rows of the pool [n_pages * 128] that hold a sequence's rows."""
    return table_row[rows // PAGE].astype(np.int64) * PAGE + rows % PAGE
