"""Relative errors of single softmax weights, over the whole range of capped logits.

A head's keys are multiples of its query, so logits are what the test says (their fp32 sums are exact: a product of two bf16
numbers has 16 bits, 128 equal ones 23). Feature d of the values is zero but for keys 2 d and 2 d + 1, where it is +-1 / w, rounded
to bf16: the two contributions all but cancel, so the output's own rounding is small and an output shows the difference of two
weights' errors. With weights off by e at most, |out - want| <= e * (mean of |v| + |want|) under the weights, and half a
step of bf16, 2^-8 of the output at most.

e is what include/grok_attn.h says: 3e-5 over blocks (1.1e-5 of fp32 in the exponent, 4e-6 of the special functions, 2^-16 of two
bf16 halves), 4e-4 over prefixes (30 times the 8e-6 of tanh.approx, 2^-16, 1e-5 of the rest).
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import bf16
from tests.test_gpu_sparse import Paged, expected, grouped, run_shared, run_sparse

pytestmark = pytest.mark.gpu


def rounded(x):
    return bf16.to_f64(bf16.from_f64(np.asarray(x, np.float64)))


def fill(paged, seqs, rows, low, high, seed):
    """Keys and values of the first `rows` rows (of the first sequence's pages); the queries [seqs, 48, 128]."""
    rng = np.random.default_rng(abs(seed))
    q = np.zeros((48, 128))
    K, V = np.zeros((rows, 8, 128)), np.zeros((rows, 8, 128))
    for g in range(8):
        sign, size = rng.choice([-1.0, 1.0], 128), rounded(1.0 + rng.random())
        q[6 * g:6 * g + 6] = sign * size
        logit = rng.uniform(low, high, rows)
        a = rounded(30 * np.arctanh(logit / 30) / (size * np.sqrt(128.0)))
        K[:, g] = a[:, None] * sign
        c = 30 * np.tanh(a * size * np.sqrt(128.0) / 30)
        each = rounded(np.exp(c.min() - c))  # the least weight over the key's own
        for d in range(128):
            V[2 * d, g, d], V[2 * d + 1, g, d] = each[2 * d], -each[2 * d + 1]
    for j in range(rows):
        page, at = paged.table[0, j // 128], j % 128
        paged.k[page, at] = W.from_bits(bf16.from_f64(K[j]))
        paged.v[page, at] = W.from_bits(bf16.from_f64(V[j]))
    return W.from_bits(bf16.from_f64(np.broadcast_to(q, (seqs, 48, 128)).copy()))


def compare(out, want, spread, e):
    got = out.float().cpu().double().numpy()
    tol = e * (spread + np.abs(want)) + 2.0 ** -8 * np.maximum(np.abs(want), np.abs(got))
    worst = float((np.abs(got - want) / tol).max())
    assert np.isfinite(got).all() and worst <= 1, worst


RANGES = [(12.0, 29.0), (-29.0, 29.0), (25.0, 29.9), (-29.9, -12.0), (-3.0, 3.0)]


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("blocks", [1, 4])
def test_weights_over_blocks(low, high, blocks):
    """All four blocks in one list (a cluster's CTAs take parts of it), and among many sequences (equal shares)."""
    seqs = 1 if blocks == 4 else 40
    paged = Paged([256] * seqs, seed=50)
    paged.table[:] = paged.table[0]
    q = fill(paged, seqs, 256, low, high, seed=int(high * 7) + blocks)
    out, st = run_sparse(paged, q, np.broadcast_to(np.arange(4, dtype=np.int32), (seqs, 8, 4)).copy())
    assert st == 0
    want, spread = expected(paged, q[:1], lambda b, g: np.arange(256))
    compare(out, np.broadcast_to(want, (seqs, 48, 128)), np.broadcast_to(spread, (seqs, 48, 128)), 3e-5)


@pytest.mark.parametrize("low,high", RANGES)
def test_weights_over_prefixes(low, high):
    paged, starts = grouped([3], [2], lambda i: 0, seed=51)
    q = fill(paged, 3, 256, low, high, seed=int(high * 5))
    out, st = run_shared(paged, q, starts, [2])
    assert st == 0
    compare(out, *expected(paged, q, lambda b, g: np.arange(256)), 4e-4)
