"""The 8-bit KV cache, restated from its definition in fp64 (oracle).

A block is 64 rows of one KV head, keys or values. With a = max |x| over its rows so far and Q = 127
(int8) or 448 (e4m3): scale = RN32(a / Q), code = round(RN32(x RN32(1 / scale))), to a whole number or to an
e4m3 value, ties to even; a < 2^-100 gives scale 0 and codes 0, a block with a NaN or an infinity scale NaN
and codes 0. A sequence's cache is a function of its rows alone: row r lies in block r // 64.

Attention: code-reading guide ch. 4 §4.5.2-§4.5.4 over code * scale. The weight of a block is the softmax
weight of its keys summed over the six query heads of the KV head.

Eviction: of nc full blocks the first `sink` and the last `recent` stay, then the largest weights (the lower
index first, NaN last) up to `keep`; the row becomes kept, open, evicted, rest.

Test infrastructure only: nothing in the CUDA library or its binding imports this.
"""
from __future__ import annotations

import math

import numpy as np

from . import bf16

BLOCK = 64
TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_value(code: int) -> float:
    """The number an e4m3 byte stands for (bias 7, no infinities, 0x7f and 0xff NaN)."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


_E4M3 = np.array([e4m3_value(c) for c in range(127)])


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """Bytes of the e4m3 values nearest to y (|y| <= 448 or a little more), ties to the even byte."""
    a = np.abs(y).astype(np.float64)
    mid = (_E4M3[1:] + _E4M3[:-1]) / 2
    up = np.searchsorted(mid, a, side="left")     # a <= mid[up]: at a tie the lower one
    tie = (up < len(mid)) & (a == mid[np.minimum(up, len(mid) - 1)]) & (up % 2 == 1)
    return ((up + tie) | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def quantise(x: np.ndarray, kind: str) -> tuple[np.ndarray, np.float32]:
    """Codes (uint8 bits) and scale of one block's rows x [r, 128]."""
    a = np.abs(x).max() if x.size else 0.0
    if not np.isfinite(a):
        return np.zeros(x.shape, np.uint8), np.float32(np.nan)
    if a < 2.0 ** -100:
        return np.zeros(x.shape, np.uint8), np.float32(0)
    scale = np.float32(a / TOP[kind])
    inv = np.float32(1.0 / np.float64(scale))
    y = (x.astype(np.float64) * np.float64(inv)).astype(np.float32)
    return (np.rint(y).astype(np.int8).view(np.uint8) if kind == "int8" else e4m3_codes(y)), scale


def code_values(codes: np.ndarray, kind: str) -> np.ndarray:
    if kind == "int8":
        return codes.view(np.int8).astype(np.float64)
    return np.array([e4m3_value(c) for c in range(256)])[codes]


def blocks(rows_bits: np.ndarray, kind: str) -> list[tuple[np.ndarray, np.float32]]:
    """The blocks of one head's bf16 rows [L, 128]: codes [r, 128] and scale each."""
    x = bf16.to_f64(rows_bits)
    return [quantise(x[i:i + BLOCK], kind) for i in range(0, len(x), BLOCK)]


def held(rows_bits: np.ndarray, kind: str) -> np.ndarray:
    """What the cache holds of one head's rows [L, 128], in fp64."""
    return np.concatenate([code_values(c, kind) * np.float64(s) for c, s in blocks(rows_bits, kind)])


def attend(q: np.ndarray, K: np.ndarray, V: np.ndarray, last: np.ndarray | None = None):
    """q [n, 128] over K, V [L, 128] (fp64), query i seeing keys <= last[i]; output and weights."""
    c = 30.0 * np.tanh(q @ K.T / math.sqrt(128.0) / 30.0)
    if last is not None:
        c = np.where(np.arange(len(K))[None, :] <= last[:, None], c, -np.inf)
    w = np.exp(c - c.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return w @ V, w


def block_weights(w: np.ndarray, n: int) -> np.ndarray:
    """Weights [6, L] of a KV head's query heads summed per block, padded to n blocks."""
    out = np.zeros(n)
    for j, x in enumerate(w.sum(0)):
        out[j // BLOCK] += x
    return out


def evict(table, weight, length: int, keep: int, sink: int, recent: int):
    """One head's row: new table, new weights, new length."""
    nc = length // BLOCK
    if nc <= keep:
        return list(table), list(weight), length
    must = [i for i in range(nc) if i < sink or i >= nc - recent]
    rest = [i for i in range(nc) if i not in must]
    rest.sort(key=lambda i: (-(-np.inf if np.isnan(weight[i]) else weight[i]), i))
    kept = sorted(must + rest[:keep - len(must)])
    gone = [i for i in range(nc) if i not in kept]
    order = kept + [i for i in (nc,) if i < len(table)] + gone + list(range(nc + 1, len(table)))
    return ([table[i] for i in order], [0.0 if i in gone else weight[i] for i in order],
            keep * BLOCK + length % BLOCK)
