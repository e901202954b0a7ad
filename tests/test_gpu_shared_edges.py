"""Decode behind shared prefixes where little or nothing is shared. Tolerances as in test_gpu_sparse.py."""
import numpy as np
import pytest

import grok_gqa_attention_gb300 as G
from tests.test_gpu_sparse import check, expected, grouped, queries, run_shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,pages,rows,usable", [
    ([1], [0], lambda i: 1, True), ([1], [0], lambda i: 5000, True), ([32], [0], lambda i: 1 + 37 * i % 300, True),
    ([1] * 40, [2] * 40, lambda i: 257 + 11 * i, True), ([30], [0], lambda i: 700 - 13 * i, True),
    ([3, 0, 2], [0, 4, 0], lambda i: 90 + i, False), ([3, 0, 2], [0, 1, 0], lambda i: 90 + i, True), ([16], [-1], lambda i: 200 + i, False), ([60], [0], lambda i: 400 + i, True)],
    ids=["one row", "one sequence", "short ones", "groups of one", "around one block per CTA", "an empty group of pages that no table has",
         "an empty group between", "unusable", "many blocks"])
def test_nothing_is_shared(sizes, pages, rows, usable):
    """No group has a page in common: every CTA takes blocks of the sequences' own."""
    paged, starts = grouped(sizes, [0] * len(sizes), rows, seed=41)
    B = len(paged.lens)
    q = queries(B, 70)
    out, st = run_shared(paged, q, starts, pages)
    assert st == (0 if usable else G.DEV_BAD_GROUP)
    some = sorted({0, 1, B // 2, B - 2, B - 1} & set(range(B)))
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -12)


def test_a_group_of_one_shares_nothing():
    """Its sequence may be shorter than the pages given for the group; a sequence of a larger group may not."""
    lens = [200, 300, 100, 300, 1]
    paged, starts = grouped([1, 3, 1], [0, 0, 0], lambda i: lens[i], seed=42)
    q = queries(5, 71)
    out, st = run_shared(paged, q, starts, [3, 0, 2])
    assert st == 0
    check(out, *expected(paged, q, lambda b, g: np.arange(lens[b])), 2.0 ** -12)
    paged, starts = grouped([1, 3], [0, 2], lambda i: [200, 40, 50, 60][i], seed=43)
    q = queries(4, 72)
    out, st = run_shared(paged, q, starts, [3, 2], lens=[200, 296, 255, 316])
    assert st == G.DEV_BAD_KV_LEN and (out[2] == 5).all()
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]))
    check(out[[0, 1, 3]], want[[0, 1, 3]], spread[[0, 1, 3]], 2.0 ** -10)
