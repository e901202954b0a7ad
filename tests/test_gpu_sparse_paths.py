"""Attention over lists of blocks: each way that a call is launched, at its limits, and what decides between them.

A call runs as one kernel, in clusters of 8, 4, 2 or 1 CTAs to a (sequence, KV head), or as two: equal shares of all blocks, and
the join of their parts. Which, the number of sequences and the budget alone decide. Tolerances as in test_gpu_sparse.py.
"""
import ctypes

import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
from oracle import sparse
from tests.test_gpu_sparse import DEV, Paged, check, expected, ints, lists, queries, run_sparse, status

pytestmark = pytest.mark.gpu


def kernels(call):
    """Grids of the kernels that call(stream) launches, from a capture that is not run."""
    cu = ctypes.CDLL("libcuda.so.1")

    def do(name, *args):
        assert getattr(cu, name)(*args) == 0, name

    s = torch.cuda.Stream()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t(0)
    do("cuStreamBeginCapture_v2", ctypes.c_void_p(s.cuda_stream), 2)
    try:
        call(s)
    finally:
        do("cuStreamEndCapture", ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph))
    do("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    do("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    grids = []
    for node in nodes:
        kind, params = ctypes.c_int(-1), (ctypes.c_uint32 * 64)()  # (function, grid x, y, z, ...)
        do("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        assert kind.value == 0  # (a kernel)
        do("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), params)
        grids.append(tuple(params[2:5]))
    do("cuGraphDestroy", graph)
    return sorted(grids)


def launched(B, budget):
    """What a call should launch: clusters of as many CTAs, 8 at most, as two on an SM allow for all pairs, where none of them
    gets more than 8 blocks."""
    places = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pairs, ctas = 8 * B, 8
    while ctas and pairs * ctas > places:
        ctas //= 2
    if ctas and -(-budget // ctas) <= 8:
        return [(pairs * ctas, 1, 1)]
    return sorted([(places, 1, 1), (8, B, 1)])


def launches(paged, q, sel, out):
    k, v, table = paged.dev()
    args = (q.to(DEV), k, v, table, ints(paged.lens), ints(sel), G.alloc_decode_sparse_workspace(q.shape[0], sel.shape[2]), out)
    return kernels(lambda s: G.decode_sparse_paged(*args, stream=s))


LIMITS = [(B, budget) for B, top in ((1, 64), (4, 64), (5, 32), (9, 32), (10, 16), (19, 16), (20, 8), (37, 8))
          for budget in (1, top - 1, top, top + 1)] + [(8, 128), (12, 48), (20, 64), (32, 32), (37, 37), (38, 8), (38, 40)]


@pytest.mark.parametrize("B,budget", LIMITS, ids=str)
def test_every_way_of_launching(B, budget):
    """Unequal lengths in a table far wider than they need, gaps, a block behind a sequence's last, a bad length."""
    rng = np.random.default_rng(B * 1000 + budget)
    most = budget * 64 * 5 // 4 + 64
    lens = [int(x) for x in rng.integers(1, most, B)]
    lens[0] = most
    if B > 3:
        lens[2] = 1
    paged, q = Paged(lens, seed=B + budget, max_pages=3 * (-(-most // 128))), queries(B, 60)
    sel = lists(lens, budget, seed=budget, holes=0.2)
    want_status, skip = 0, []
    run_lens = list(lens)
    sel[0, 3, 0] = 2 * paged.max_pages  # (behind the last block; the first entry always counts)
    want_status |= G.DEV_BAD_BLOCK
    if B > 3:
        run_lens[B // 2], skip = 128 * paged.max_pages + 1, [B // 2]
        want_status |= G.DEV_BAD_KV_LEN
    out, st = run_sparse(paged, q, sel, lens=run_lens)
    assert st == want_status
    some = [b for b in sorted({0, 1, 2, B // 3, B - 2, B - 1}) if 0 <= b < B and b not in skip]

    def rows(b, g):
        if b not in some:
            return []
        n = -(-lens[b] // 64)
        return sparse.rows_of([i for i in sel[b, g, :min(budget, n)] if i < n], lens[b])

    want, spread = expected(paged, q, rows)
    check(out[some], want[some], spread[some], 2.0 ** -12)
    for b in skip:
        assert (out[b] == 5).all()
    assert torch.isfinite(out.float()).all()
    assert launches(paged, q, sel, torch.zeros_like(out)) == launched(B, budget)


@pytest.mark.parametrize("B,budget", [(1, 16), (8, 24), (20, 40), (32, 32), (37, 8)], ids=str)
def test_the_tables_width_does_not_matter(B, budget):
    """The same launches and the same bits, whatever the block table has room for."""
    lens = [(budget * 64 if b % 3 == 0 else 100) + b for b in range(B)]
    q, sel = queries(B, 61), lists(lens, budget, seed=3)
    results = []
    for width in (-(-max(lens) // 128), 512):
        paged = Paged(lens, seed=5, max_pages=width)
        out, st = run_sparse(paged, q, sel)
        assert st == 0
        results.append((out, launches(paged, q, sel, torch.zeros_like(out))))
    assert torch.equal(results[0][0], results[1][0])
    assert results[0][1] == results[1][1] == launched(B, budget)


def test_lists_that_are_all_empty_in_every_way_of_launching():
    """Zeros, and no NaN of a part that was not written."""
    for B, budget in ((1, 16), (6, 32), (12, 16), (30, 8), (30, 40)):
        lens = [budget * 64] * B
        paged, q = Paged(lens, seed=B), queries(B, 62)
        out, st = run_sparse(paged, q, np.full((B, 8, budget), -1, np.int32))
        assert st == 0 and (out == 0).all()


def test_status_may_be_left_out():
    """Calls without a status word skip what they cannot read all the same."""
    for B, budget in ((5, 8), (30, 40)):
        lens = [300] * B
        paged, q = Paged(lens, seed=7, max_pages=4), queries(B, 63)
        sel = lists(lens, budget, seed=1)
        k, v, table = paged.dev()
        run_lens = [300] * (B - 1) + [0]
        outs = []
        for st in (status(), None):
            out = torch.full((B, 48, 128), 5.0, dtype=torch.bfloat16, device=DEV)
            G.decode_sparse_paged(q.to(DEV), k, v, table, ints(run_lens), ints(sel), G.alloc_decode_sparse_workspace(B, budget),
                                  out, st)
            outs.append(out)
        assert torch.equal(*outs) and (outs[0][B - 1] == 5).all()
