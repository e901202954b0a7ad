"""Decode over part of a paged cache on the GPU: bounds, choice of blocks, attention over lists, shared prefixes.

Bounds, scores and choices are exact. Attention is held to fp64 with a tolerance made of its roundings: the output's
(bf16, half a step, 2^-8 of the value at most), and a relative error d of the weights, which moves an output by at most
2 d times the mean of |v| under the weights. d: 2^-12 over blocks and over prefixes 2^-10. (Weights are kept to 2^-16 by
two bf16 halves and to about 1e-5 by the special functions, over prefixes to 4e-4 by tanh.approx, 43.3 ln 2 times
its 8e-6, and 3e-5 by the rest; logits are 128-term fp32 sums of products, off by 2^-24 * 12 of the sum of |q k| /
sqrt(128) or less in practice, 2e-5 here.)
"""
import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
import workloads as W
from oracle import bf16, sparse

pytestmark = pytest.mark.gpu

DEV = "cuda"
B64, PG = sparse.BLOCK, sparse.PAGE


def ints(x):
    return torch.tensor(np.asarray(x, np.int32)).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


class Paged:
    """A pool of keys and values with a shuffled table; pages that no sequence owns hold NaN, table entries -1."""

    def __init__(self, lens, seed, common=(), group=None, max_pages=None, scale=1.5):
        rng = np.random.default_rng(seed)
        B = len(lens)
        need = [-(-n // PG) for n in lens]
        self.max_pages = max_pages or max(max(need), 1)
        total = sum(common) + sum(max(0, n - (common[group[b]] if group else 0)) for b, n in enumerate(need)) + 3
        order = list(rng.permutation(total))
        take = lambda m: [order.pop() for _ in range(m)]  # noqa: E731
        shared = [take(m) for m in common]
        self.table = np.full((B, self.max_pages), -1, np.int32)
        for b, n in enumerate(need):
            head = shared[group[b]][:n] if group and group[b] >= 0 else []
            self.table[b, :n] = head + take(n - len(head))
        size = scale * (0.5 + rng.random((1, 1, 8, 1)))
        self.k = (torch.randn(total, PG, 8, 128, generator=torch.Generator().manual_seed(seed)) *
                  torch.tensor(size, dtype=torch.float32)).bfloat16()
        self.v = torch.randn(total, PG, 8, 128, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
        self.spare = order
        for p in order:
            self.k[p] = self.v[p] = float("nan")
        # behind each sequence's last row: NaN
        for b, n in enumerate(lens):
            if n % PG:
                self.k[self.table[b, n // PG], n % PG:] = float("nan")
                self.v[self.table[b, n // PG], n % PG:] = float("nan")
        self.lens = list(lens)

    def dev(self):
        return self.k.to(DEV), self.v.to(DEV), torch.tensor(self.table).to(DEV)

    def rows(self, b, g, rows):
        """fp64 keys and values of these rows of the sequence."""
        flat = sparse.at(self.table[b], rows)
        return tuple(bf16.to_f64(W.bits(x.view(-1, 8, 128)[flat, g])) for x in (self.k, self.v))


def queries(B, seed, scale=1.5):
    return (torch.randn(B, 48, 128, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()


def check(got, want, spread, d, what=""):
    got = got.float().cpu().double().numpy()
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    tol = np.maximum(np.abs(want), np.abs(got)) * 2.0 ** -8 + 2 * d * spread + 1e-30
    assert (err <= tol).all(), (what, float((err / tol).max()))


def expected(paged, q, lists):
    """fp64 outputs over rows lists(b, g) and the mean |v|."""
    B = q.shape[0]
    qb = bf16.to_f64(W.bits(q))
    out, spread = np.zeros((B, 48, 128)), np.zeros((B, 48, 128))
    for b in range(B):
        for g in range(8):
            rows = lists(b, g)
            if len(rows):
                K, V = paged.rows(b, g, rows)
                out[b, 6 * g:6 * g + 6], spread[b, 6 * g:6 * g + 6] = sparse.attend(qb[b, 6 * g:6 * g + 6], K, V)
    return out, spread


# ------------------------------------------------------------------------------------------------------- bounds
def run_bounds(paged, start, valid, T, codes=None, scale=None):
    k, _, table = paged.dev()
    if codes is None:
        codes, scale = G.alloc_kv_bounds(k.shape[0], DEV)
        codes += 77
        scale += 77
    st = status()
    G.kv_bounds_paged(k, table, ints(start), None if valid is None else ints(valid), T, codes, scale, st)
    return codes, scale, int(st.item())


def check_bounds(paged, codes, scale, touched):
    """touched: {(b, block): rows of it}; everything else is as it was (77)."""
    codes, scale = codes.cpu().numpy(), scale.cpu().numpy()
    want_c, want_s = np.full_like(codes, 77), np.full_like(scale, 77)
    for (b, blk), rows in touched.items():
        pg, half = paged.table[b, blk // 2], blk % 2
        bits = W.bits(paged.k[pg, half * 64:half * 64 + rows])
        for g in range(8):
            want_c[pg, half, g], want_s[pg, half, g] = sparse.bounds(bits[:, g])
    assert np.array_equal(codes, want_c)
    assert np.array_equal(scale, want_s)


@pytest.mark.parametrize("start,valid,T", [
    ([0], None, 1), ([63, 64, 65], None, 1), ([0, 5, 127], None, 64), ([0, 100, 1], [300, 1, 129], 300),
    ([130, 0, 383], None, 129)], ids=str)
def test_bounds(start, valid, T):
    ends = [s + (T if valid is None else valid[b]) for b, s in enumerate(start)]
    paged = Paged(ends, seed=len(start) + T, max_pages=-(-(max(start) + T) // PG))
    codes, scale, st = run_bounds(paged, start, valid, T)
    assert st == 0
    check_bounds(paged, codes, scale, {(b, i): min(64, ends[b] - 64 * i) for b, s in enumerate(start)
                                       for i in range(s // 64, -(-ends[b] // 64))})


@pytest.mark.parametrize("kind", ["zero", "small", "large", "mixed", "not finite", "negative"])
def test_bounds_of_unusual_keys(kind):
    paged = Paged([100], seed=4)
    k = paged.k[paged.table[0, 0]]
    if kind == "zero":
        k[:] = 0
        k[:, 1] = -0.0
    elif kind == "small":
        k[:] = (k.nan_to_num(1.0).float() * 2.0 ** -120).bfloat16()
    elif kind == "large":
        k[:] = (k.nan_to_num(1.0).float() * 2.0 ** 100).bfloat16()
    elif kind == "mixed":
        k[3, :, 5], k[4, :, 6] = 3.0e38, 2.0 ** -133
    elif kind == "negative":
        k[:] = -k.nan_to_num(1.0).abs() - 1
    else:
        for i, bits in enumerate((0x7F80, 0xFF80, 0x7FC0, 0xFFC1)):
            k[7 + i, i, 3] = W.from_bits(np.array([bits], np.uint16))[0]
    codes, scale, st = run_bounds(paged, [0], None, 100)
    assert st == 0
    check_bounds(paged, codes, scale, {(0, 0): 64, (0, 1): 36})


def test_bounds_refusals_on_the_device():
    paged = Paged([200, 200, 200, 200, 200], seed=9)
    table = paged.table.copy()
    paged.table[4, 1] = 99
    codes, scale, st = run_bounds(paged, [-1, 190, 0, 0, 100], [50, 50, 0, 51, 50], 50)
    assert st == G.DEV_BAD_START | G.DEV_BAD_VALID | G.DEV_BAD_PAGE
    paged.table = table
    check_bounds(paged, codes, scale, {(1, 2): 64, (1, 3): 48, (4, 1): 64})


def test_bounds_after_rows_were_dropped():
    """Appended, dropped and appended again: the bounds are those of the rows that are there now."""
    paged = Paged([128], seed=10)
    codes, scale, _ = run_bounds(paged, [0], None, 128)
    paged.k[paged.table[0, 0], 70:128] = 0.25
    codes, scale, _ = run_bounds(paged, [70], None, 10, codes, scale)
    got = codes.cpu().numpy()[paged.table[0, 0], 1, 2]
    want, two = sparse.bounds(W.bits(paged.k[paged.table[0, 0], 64:80, 2]))
    assert np.array_equal(got, want) and scale[paged.table[0, 0], 1, 2].item() == two


# ------------------------------------------------------------------------------------------------------- choice
def check_select(paged, q, codes, scale, budget, sink, recent, skip=()):
    B = q.shape[0]
    st = status()
    score = torch.full((B, 8, 2 * paged.max_pages), 7.0, device=DEV)
    sel = torch.full((B, 8, budget), 99, dtype=torch.int32, device=DEV)
    lens = list(paged.lens)
    G.select_blocks_paged(q.to(DEV), codes, scale, torch.tensor(paged.table).to(DEV), ints(lens), sink, recent, score, sel,
                          st)
    score, sel = score.cpu().numpy(), sel.cpu().numpy()
    hc, hs, qb = codes.cpu().numpy(), scale.cpu().numpy(), W.bits(q)
    for b in range(B):
        if b in skip:
            assert (score[b] == 7).all() and (sel[b] == 99).all()
            continue
        n = -(-lens[b] // 64)
        blk = np.arange(n)
        pages = paged.table[b, blk // 2]
        for g in range(8):
            want = sparse.scores(qb[b, 6 * g:6 * g + 6], hc[pages, blk % 2, g], hs[pages, blk % 2, g].astype(np.float64))
            assert np.array_equal(score[b, g, :n].astype(np.float64), want)
            assert (score[b, g, n:] == 7).all()
            took = sparse.choose(want, budget, sink, recent)
            assert sel[b, g].tolist() == took + [-1] * (budget - len(took))
    return int(st.item()), sel


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([1], 1, 0, 0), ([64, 65, 1000], 3, 1, 1), ([1000, 999, 500, 3000], 8, 1, 2), ([3000, 17], 47, 0, 0),
    ([3000], 46, 4, 8), ([2500], 5, 5, 0), ([2500], 5, 0, 5), ([2500, 100], 64, 1, 1), ([8192], 1, 0, 0),
    ([8192], 129, 1, 1), ([65536], 1024, 0, 0), ([65536, 40000], 100, 2, 3)], ids=str)
def test_choice(lens, budget, sink, recent):
    paged = Paged(lens, seed=sum(lens) % 997)
    codes, scale, st = run_bounds(paged, [0] * len(lens), lens, max(lens))
    assert st == 0
    st, _ = check_select(paged, queries(len(lens), 5), codes, scale, budget, sink, recent)
    assert st == 0


@pytest.mark.parametrize("kind", ["zero query", "equal blocks", "two values", "negative", "not finite"])
def test_choice_among_equal_scores(kind):
    """The lower index first."""
    lens = [3000, 2000]
    paged = Paged(lens, seed=3)
    codes, scale, _ = run_bounds(paged, [0, 0], lens, 3000)
    q = queries(2, 6)
    if kind == "zero query":
        q[:] = 0
    elif kind == "not finite":
        q[0, 3, 5], q[0, 9, 6], q[1, 20, 7], q[1, 21, 8] = float("inf"), -float("inf"), float("nan"), -float("nan")
    elif kind == "negative":  # all scores below zero
        codes[..., 0, :], codes[..., 1, :] = -3, -5
        q = q.abs()
    else:
        codes[:] = codes[0, 0, 0]
        scale[:] = scale[0, 0, 0]
        if kind == "two values":
            scale[::3] *= 2
    for budget, sink, recent in ((1, 0, 0), (13, 1, 2), (31, 0, 1)):
        st, _ = check_select(paged, q, codes, scale, budget, sink, recent)
        assert st == 0


def test_choice_refusals_on_the_device():
    paged = Paged([300, 300, 300, 300], seed=8)
    codes, scale, _ = run_bounds(paged, [0] * 4, None, 300)
    paged.lens = [0, 300, 385, -5]
    st, _ = check_select(paged, queries(4, 1), codes, scale, 4, 1, 1, skip=(0, 2, 3))
    assert st == G.DEV_BAD_KV_LEN


# ------------------------------------------------------------------------------------------------------- lists
def run_sparse(paged, q, sel, lens=None, ws=None):
    k, v, table = paged.dev()
    B, budget = q.shape[0], sel.shape[2]
    out = torch.full((B, 48, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    st = status()
    ws = G.alloc_decode_sparse_workspace(B, budget) if ws is None else ws
    ws.fill_(255)  # (NaN in every partial result that a call does not write)
    G.decode_sparse_paged(q.to(DEV), k, v, table, ints(paged.lens if lens is None else lens), ints(sel), ws, out, st)
    return out, int(st.item())


def lists(lens, budget, seed, holes=0.0):
    rng = np.random.default_rng(seed)
    sel = np.full((len(lens), 8, budget), -1, np.int32)
    for b, n in enumerate(lens):
        blocks = -(-n // 64)
        for g in range(8):
            pick = np.sort(rng.permutation(blocks)[:budget])
            sel[b, g, :len(pick)] = np.where(rng.random(len(pick)) < holes, -1, pick)
    return sel


@pytest.mark.parametrize("lens,budget,holes", [
    ([1], 1, 0), ([63, 64, 65], 2, 0), ([1000, 1, 500], 4, 0), ([3000, 128, 2999, 70], 16, 0), ([3000, 2000], 47, 0.5),
    ([8192], 16, 0), ([8192], 128, 0), ([700] * 20, 7, 0.3), ([65536], 3, 0), ([130] * 70, 3, 0)], ids=str)
def test_lists(lens, budget, holes):
    paged, q = Paged(lens, seed=budget + len(lens)), queries(len(lens), 7)
    sel = lists(lens, budget, seed=1, holes=holes)
    out, st = run_sparse(paged, q, sel)
    assert st == 0
    want, spread = expected(paged, q, lambda b, g: sparse.rows_of(sel[b, g], lens[b]))
    check(out, want, spread, 2.0 ** -12)


def test_lists_in_any_order_with_repeats_and_nothing():
    lens = [1000, 1000, 300]
    paged, q = Paged(lens, seed=2), queries(3, 8)
    sel = lists(lens, 6, seed=2)
    sel[0, 0] = [15, 3, 3, -1, 0, 3]   # out of order, a block three times, a gap
    sel[0, 1] = -1                     # nothing
    sel[1] = -1
    sel[1, 7, 5] = 15                  # the last block alone, behind gaps
    sel[2, 0, :5] = [-7, -1, 4, -2, -1]  # (five blocks: five entries count)
    out, st = run_sparse(paged, q, sel)
    assert st == 0
    want, spread = expected(paged, q, lambda b, g: sparse.rows_of(sel[b, g, :5] if b == 2 else sel[b, g], lens[b]))
    check(out, want, spread, 2.0 ** -12)
    assert (out[0, 6:12] == 0).all() and (out[1, :42] == 0).all()


def test_lists_of_large_logits():
    """Logits far beyond the cap, equal weights; a head whose logits are all at the lower cap."""
    lens = [500]
    paged = Paged(lens, seed=5)
    q = queries(1, 9)
    paged.k[:, :, 0] = 4.0
    q[0, :6] = 50.0
    paged.k[:, :, 1] = -4.0
    q[0, 6:12] = 50.0
    sel = lists(lens, 8, seed=3)
    out, st = run_sparse(paged, q, sel)
    want, spread = expected(paged, q, lambda b, g: sparse.rows_of(sel[b, g], 500))
    check(out, want, spread, 2.0 ** -12)


def test_lists_refusals_on_the_device():
    lens = [300, 300, 300, 300]
    paged, q = Paged(lens, seed=6), queries(4, 10)
    sel = lists(lens, 5, seed=4)
    sel[1, 2, 1] = 5  # behind the last block
    out, st = run_sparse(paged, q, sel, lens=[0, 300, 385, 300])
    assert st == G.DEV_BAD_KV_LEN | G.DEV_BAD_BLOCK
    assert (out[0] == 5).all() and (out[2] == 5).all()
    want, spread = expected(paged, q, lambda b, g: sparse.rows_of([i for i in sel[b, g] if i < 5], 300))
    check(out[[1, 3]], want[[1, 3]], spread[[1, 3]], 2.0 ** -12)
    paged.table[3, 1] = 10 ** 6
    out, st = run_sparse(paged, q, lists(lens, 5, seed=4))
    assert st == G.DEV_BAD_PAGE
    check(out[:3], *(x[:3] for x in expected(paged, q, lambda b, g: np.arange(300 if b < 3 else 0))), 2.0 ** -12)


def test_every_block_listed_is_the_whole_decode():
    lens = [4096, 100, 2333]
    paged, q = Paged(lens, seed=7), queries(3, 11)
    out, st = run_sparse(paged, q, lists(lens, 64, seed=5))
    k, v, table = paged.dev()
    ws = G.alloc_decode_workspace(3, 32 * PG, DEV)
    full = torch.empty_like(out)
    G.decode_paged(q.to(DEV), k, v, table, ints(lens), ws)
    G.combine(ws, ints(lens), full, 32 * PG)
    assert st == 0
    want, spread = expected(paged, q, lambda b, g: np.arange(lens[b]))
    check(out, want, spread, 2.0 ** -12)
    check(full, want, spread, 2.0 ** -12)


def test_many_sequences():
    """More sequences than the plan's table has entries."""
    rng = np.random.default_rng(0)
    B = 1500
    lens = [int(x) for x in rng.integers(1, 130, B)]
    paged, q = Paged(lens, seed=11), queries(B, 12)
    sel = lists(lens, 2, seed=6)
    out, st = run_sparse(paged, q, sel)
    assert st == 0
    some = [0, 1, 2, 3, 700, 701, 1498, 1499]
    want, spread = expected(paged, q, lambda b, g: sparse.rows_of(sel[b, g], lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -12)


# ------------------------------------------------------------------------------------------------------- prefixes
def run_shared(paged, q, starts, pages, lens=None, ws=None):
    k, v, table = paged.dev()
    B = q.shape[0]
    out = torch.full((B, 48, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    st = status()
    ws = G.alloc_decode_shared_workspace(B, paged.max_pages, len(pages)) if ws is None else ws
    ws.fill_(255)
    G.decode_shared_paged(q.to(DEV), k, v, table, ints(paged.lens if lens is None else lens), ints(starts), ints(pages), ws,
                          out, st)
    return out, int(st.item())


def grouped(sizes, pages, mine, seed, alone_before=0, alone_after=0, **kw):
    """Groups of these sizes and common pages; mine(i): rows of sequence i behind them."""
    group = [-1] * alone_before + [i for i, n in enumerate(sizes) for _ in range(n)] + [-1] * alone_after
    starts = [alone_before]
    for n in sizes:
        starts.append(starts[-1] + n)
    lens = [(pages[g] * PG if g >= 0 else 0) + mine(i) for i, g in enumerate(group)]
    common = [p for p in pages]
    return Paged(lens, seed, common=common + [0], group=[g if g >= 0 else len(common) for g in group], **kw), starts


@pytest.mark.parametrize("sizes,pages,mine", [
    ([2], [1], lambda i: i), ([1], [2], lambda i: 5), ([21], [3], lambda i: 7 * i), ([22], [2], lambda i: 64),
    ([43], [1], lambda i: 130 - i), ([4], [16], lambda i: 0), ([3, 5, 1, 30], [2, 0, 1, 4], lambda i: 1 + 13 * i % 200),
    ([2, 2, 2], [40, 1, 7], lambda i: 65), ([64], [9], lambda i: 0 if i % 3 else 300), ([2] * 40, [1] * 40, lambda i: i % 5)],
    ids=["one own row", "a group of one", "a whole tile", "a tile and one", "three tiles", "no own rows", "unequal groups",
         "unequal prefixes", "many", "many groups"])
def test_prefixes(sizes, pages, mine):
    paged, starts = grouped(sizes, pages, mine, seed=sum(sizes))
    q = queries(len(paged.lens), 13)
    out, st = run_shared(paged, q, starts, pages)
    assert st == 0
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]))
    check(out, want, spread, 2.0 ** -10)


def test_sequences_outside_the_groups():
    paged, starts = grouped([3, 4], [2, 3], lambda i: 50 + i, seed=1, alone_before=2, alone_after=3)
    q = queries(12, 14)
    out, st = run_shared(paged, q, starts, [2, 3])
    assert st == 0
    check(out, *expected(paged, q, lambda b, g: np.arange(paged.lens[b])), 2.0 ** -10)


@pytest.mark.parametrize("starts,pages", [([0, 6, 4, 9], [1, 1, 1]), ([-1, 4, 6, 9], [1, 1, 1]), ([0, 3, 6, 10], [1, 1, 1]),
                                          ([0, 3, 6, 9], [1, -1, 1]), ([0, 3, 6, 9], [1, 1, 5])], ids=str)
def test_groups_that_are_not_usable_are_decoded_singly(starts, pages):
    paged, _ = grouped([9], [1], lambda i: 40 * i, seed=2)
    q = queries(9, 15)
    out, st = run_shared(paged, q, starts, pages)
    assert st == G.DEV_BAD_GROUP
    check(out, *expected(paged, q, lambda b, g: np.arange(paged.lens[b])), 2.0 ** -12)


def test_prefix_refusals_on_the_device():
    paged, starts = grouped([6], [2], lambda i: 30, seed=3)
    q = queries(6, 16)
    out, st = run_shared(paged, q, starts, [2], lens=[286, 255, 0, 286, 385, 286])
    assert st == G.DEV_BAD_KV_LEN
    assert all((out[b] == 5).all() for b in (1, 2, 4))
    want, spread = expected(paged, q, lambda b, g: np.arange(286))
    ok = [0, 3, 5]
    check(out[ok], want[ok], spread[ok], 2.0 ** -10)
    paged.table[4, 1] = paged.table[4, 0]  # not the group's second page
    out, st = run_shared(paged, q, starts, [2])
    assert st == G.DEV_BAD_GROUP
    paged.table[:, 1] = 10 ** 6
    out, st = run_shared(paged, q, starts, [2])
    assert st == G.DEV_BAD_PAGE


def test_prefix_of_large_logits():
    paged, starts = grouped([5], [3], lambda i: 10, seed=4)
    q = queries(5, 17)
    paged.k[:, :, 0] = 4.0
    paged.k[:, :, 1] = -4.0
    q[:, :12] = 50.0
    out, st = run_shared(paged, q, starts, [3])
    assert st == 0
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]))
    check(out, want, spread, 2.0 ** -10)


def test_a_not_finite_key_shows():
    """A NaN among the visible keys of a prefix or of a sequence's own rows reaches the outputs of those who see it."""
    paged, starts = grouped([4], [2], lambda i: 20, seed=5)
    for key in range(8):  # (every place of a pair of columns and of its two forms)
        paged.k[paged.table[0, 0], 40 + key, key] = float("nan")
    paged.k[paged.table[2, 2], 3, 7] = float("nan")
    out, st = run_shared(paged, queries(4, 18), starts, [2])
    assert st == 0
    assert torch.isnan(out).all()


def test_a_batch_as_long_as_it_gets():
    """65536 rows, most of them common; compared with the whole decode of the paged cache."""
    paged, starts = grouped([24], [500], lambda i: 1536 - 64 * i, seed=6)
    q = queries(24, 19)
    out, st = run_shared(paged, q, starts, [500])
    assert st == 0
    k, v, table = paged.dev()
    ws = G.alloc_decode_workspace(24, 65536, DEV)
    full = torch.empty_like(out)
    G.decode_paged(q.to(DEV), k, v, table, ints(paged.lens), ws)
    G.combine(ws, ints(paged.lens), full, 65536)
    some = [0, 23]
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -10)
    a, z = out.float(), full.float()
    # two bf16 roundings, and weights off by 2^-10
    most = float(paged.v.nan_to_num(0.0).abs().max())
    assert ((a - z).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), z.abs()) + 2.0 ** -9 * most).all()


def test_long_own_rows():
    """More blocks of the sequences' own than half of the CTAs are given; compared with the whole decode."""
    paged, starts = grouped([7, 3], [3, 1], lambda i: 6000 - 517 * i, seed=7)
    q = queries(10, 22)
    out, st = run_shared(paged, q, starts, [3, 1])
    assert st == 0
    some = [0, 6, 7]
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -10)
    k, v, table = paged.dev()
    ws, full = G.alloc_decode_workspace(10, paged.max_pages * PG, DEV), torch.empty_like(out)
    G.decode_paged(q.to(DEV), k, v, table, ints(paged.lens), ws)
    G.combine(ws, ints(paged.lens), full, paged.max_pages * PG)
    a, z = out.float(), full.float()
    most = float(paged.v.nan_to_num(0.0).abs().max())
    assert ((a - z).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), z.abs()) + 2.0 ** -9 * most).all()


def test_many_sequences_in_many_groups():
    """More sequences than the plan's table has entries, as many groups as there may be, some of one sequence, some
    sequences in none."""
    rng = np.random.default_rng(5)
    sizes = [int(x) for x in rng.integers(1, 5, 256)]
    pages = [int(x) for x in rng.integers(0, 3, 256)]
    paged, starts = grouped(sizes, pages, lambda i: 1 + i * 37 % 150, seed=8, alone_before=3, alone_after=4)
    B = len(paged.lens)
    assert B > 512
    q = queries(B, 23)
    out, st = run_shared(paged, q, starts, pages)
    assert st == 0
    some = [0, 1, 2, 3, 4, 5, 6, 300, 301, 302, B - 6, B - 5, B - 4, B - 1]
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -10)


def test_results_do_not_change_from_call_to_call():
    paged, starts = grouped([25, 13], [9, 4], lambda i: 31 * i, seed=9)
    q = queries(38, 24)
    first, _ = run_shared(paged, q, starts, [9, 4])
    sel = lists(paged.lens, 11, seed=10)
    first_sparse, _ = run_sparse(paged, q, sel)
    for _ in range(4):
        assert torch.equal(run_shared(paged, q, starts, [9, 4])[0], first)
        assert torch.equal(run_sparse(paged, q, sel)[0], first_sparse)


# ------------------------------------------------------------------------------------------------------- together
def append_rows(paged_k, paged_v, table, k, v, q, start):
    q_rot = torch.empty_like(q)
    G.rope_kv_append_paged(q, k, v, start, q_rot, paged_k, paged_v, table)
    return q_rot


def test_decode_steps_captured_in_a_graph():
    """Append, bounds, choice and attention over the chosen blocks for some steps, captured once and replayed; another
    call shares the prefix of the same batch."""
    rng = np.random.default_rng(1)
    B, first, steps, budget = 3, [250, 383, 127], 4, 3
    paged = Paged([f + steps for f in first], seed=21)
    k, v, table = paged.dev()
    k.nan_to_num_(1.0)
    v.nan_to_num_(1.0)
    codes, scale = G.alloc_kv_bounds(k.shape[0], DEV)
    G.kv_bounds_paged(k, table, ints([0] * B), ints(first), max(first), codes, scale)
    new = [(torch.tensor(rng.standard_normal((B, 1, h, 128)) * 1.5).bfloat16().to(DEV)) for h in (48, 8, 8)]
    start, length = ints(first), ints([f + 1 for f in first])
    q_rot = torch.zeros(B, 1, 48, 128, dtype=torch.bfloat16, device=DEV)
    score = torch.zeros(B, 8, 2 * paged.max_pages, device=DEV)
    sel = torch.zeros(B, 8, budget, dtype=torch.int32, device=DEV)
    out = torch.zeros(B, 48, 128, dtype=torch.bfloat16, device=DEV)
    ws, st = G.alloc_decode_sparse_workspace(B, budget), status()

    def step():
        G.rope_kv_append_paged(*new, start, q_rot, k, v, table, st)
        G.kv_bounds_paged(k, table, start, None, 1, codes, scale, st)
        G.select_blocks_paged(q_rot.view(B, 48, 128), codes, scale, table, length, 1, 1, score, sel, st)
        G.decode_sparse_paged(q_rot.view(B, 48, 128), k, v, table, length, sel, ws, out, st)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # (warm-up: attributes and lazy loading; the graph's first replay writes the same rows again)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for x in new:
            x.copy_(torch.tensor(rng.standard_normal(tuple(x.shape)) * 1.5).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        paged.k, paged.v = k.cpu(), v.cpu()
        lens = [f + 1 + i for f in first]
        paged.lens = lens
        got = sel.cpu().numpy()
        qb = W.bits(q_rot[:, 0].cpu())
        for b in range(B):
            n = -(-lens[b] // 64)
            for g in range(8):
                blocks = [sparse.bounds(W.bits(paged.k.view(-1, 8, 128)[sparse.at(
                    paged.table[b], np.arange(j * 64, min(j * 64 + 64, lens[b])))][:, g])) for j in range(n)]
                want = sparse.scores(qb[b, 6 * g:6 * g + 6], np.stack([c for c, _ in blocks]),
                                     np.array([s for _, s in blocks]))
                took = sparse.choose(want, budget, 1, 1)
                assert got[b, g].tolist() == took + [-1] * (budget - len(took))
        check(out, *expected(paged, q_rot[:, 0].cpu(), lambda b, g: sparse.rows_of(got[b, g], lens[b])), 2.0 ** -12)
        start += 1
        length += 1


def test_calls_on_two_streams_and_repeated():
    """Two calls of each kind at once, each with its own workspace, give the bits of the calls alone."""
    lens = [2000, 300, 1200]
    paged, q = Paged(lens, seed=22), queries(3, 20)
    sel = lists(lens, 9, seed=7)
    alone, _ = run_sparse(paged, q, sel)
    many, starts = grouped([30], [6], lambda i: 20 * i, seed=23)
    q2 = queries(30, 21)
    alone2, _ = run_shared(many, q2, starts, [6])
    k, v, table = paged.dev()
    k2, v2, table2 = many.dev()
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(ints(lens), ints(sel), G.alloc_decode_sparse_workspace(3, 9), torch.zeros_like(alone), ints(many.lens),
             ints(starts), ints([6]), G.alloc_decode_shared_workspace(30, many.max_pages, 1), torch.zeros_like(alone2))
            for _ in streams]
    qd, qd2 = q.to(DEV), q2.to(DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (n, l, ws, out, n2, g, p, ws2, out2) in zip(streams, args):
            G.decode_sparse_paged(qd, k, v, table, n, l, ws, out, stream=s)
            G.decode_shared_paged(qd2, k2, v2, table2, n2, g, p, ws2, out2, stream=s)
    torch.cuda.synchronize()
    for a in args:
        assert torch.equal(a[3], alone) and torch.equal(a[8], alone2)


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream, they do not disturb each other."""
    paged, starts = grouped([7], [3], lambda i: 9 * i, seed=24)
    k, v, table = paged.dev()
    lens, g, p = ints(paged.lens), ints(starts), ints([3])
    ws = G.alloc_decode_shared_workspace(7, paged.max_pages, 1)
    qs = [queries(7, 30 + i) for i in range(2)]
    dev = [x.to(DEV) for x in qs]
    outs = [torch.zeros(7, 48, 128, dtype=torch.bfloat16, device=DEV) for _ in qs]
    run_shared(paged, qs[0], starts, [3])  # (warm-up)
    graphs = []
    for x, o in zip(dev, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            G.decode_shared_paged(x, k, v, table, lens, g, p, ws, o)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for x, o in zip(qs, outs):
        check(o, *expected(paged, x, lambda b, g: np.arange(paged.lens[b])), 2.0 ** -10)


def test_out_may_be_the_queries():
    paged, starts = grouped([5], [2], lambda i: 70, seed=25)
    q = queries(5, 40)
    want, _ = run_shared(paged, q, starts, [2])
    k, v, table = paged.dev()
    x = q.to(DEV)
    G.decode_shared_paged(x, k, v, table, ints(paged.lens), ints(starts), ints([2]),
                          G.alloc_decode_shared_workspace(5, paged.max_pages, 1), x)
    assert torch.equal(x, want)
    sel = lists(paged.lens, 3, seed=8)
    want, _ = run_sparse(paged, q, sel)
    x = q.to(DEV)
    G.decode_sparse_paged(x, k, v, table, ints(paged.lens), ints(sel), G.alloc_decode_sparse_workspace(5, 3), x)
    assert torch.equal(x, want)


def test_short_workspaces_and_wrong_shapes_are_refused():
    paged, q = Paged([200], seed=26), queries(1, 41).to(DEV)
    k, v, table = paged.dev()
    out, sel = torch.zeros_like(q), ints(lists([200], 2, seed=9))
    ws = G.alloc_decode_sparse_workspace(1, 2)
    with pytest.raises(G.GrokError, match="workspace"):
        G.decode_sparse_paged(q, k, v, table, ints([200]), sel, ws[:ws.numel() - 256], out)
    ws = G.alloc_decode_shared_workspace(1, 2, 1)
    with pytest.raises(G.GrokError, match="workspace"):
        G.decode_shared_paged(q, k, v, table, ints([200]), ints([0, 1]), ints([1]), ws[:ws.numel() - 256], out)
    with pytest.raises(ValueError):
        G.decode_shared_paged(q, k, v, table, ints([200]), ints([0]), ints([1]), ws, out)
    with pytest.raises(ValueError):
        G.decode_sparse_paged(q, k, v, table, ints([200]), sel[:, :4], ws, out)
    with pytest.raises(TypeError):
        G.select_blocks_paged(q, *G.alloc_kv_bounds(k.shape[0], DEV), table, ints([200]), 0, 0,
                              torch.zeros(1, 8, 4, device=DEV, dtype=torch.float64), sel)


@pytest.mark.parametrize("given", [False, True])
def test_both_ways_through_the_binding(monkeypatch, given):
    """The checks in Python, which the extension falls back on, lead to the same calls; with and without a stream."""
    from grok_gqa_attention_gb300 import sparse as binding

    class Back:  # (an extension that hands everything back)
        def __getattr__(self, name):
            return lambda *a: None

    paged, starts = grouped([4], [2], lambda i: 90 * i, seed=31)
    q, sel = queries(4, 50).to(DEV), ints(lists(paged.lens, 3, seed=11))
    k, v, table = paged.dev()
    k.nan_to_num_(0.5)
    lens, zero = ints(paged.lens), ints([0] * 4)
    results = []
    for through in (None, Back()):
        if through is not None:
            monkeypatch.setattr(binding, "_checked", through)
        stream = torch.cuda.Stream() if given else None
        codes, scale = G.alloc_kv_bounds(k.shape[0], DEV)
        score, chosen = torch.zeros(4, 8, 2 * paged.max_pages, device=DEV), torch.zeros_like(sel)
        a, z, st = torch.zeros_like(q), torch.zeros_like(q), status()
        torch.cuda.synchronize()
        G.kv_bounds_paged(k, table, zero, lens, max(paged.lens), codes, scale, st, stream)
        G.select_blocks_paged(q, codes, scale, table, lens, 1, 1, score, chosen, st, stream)
        G.decode_sparse_paged(q, k, v, table, lens, sel, G.alloc_decode_sparse_workspace(4, 3), a, st, stream)
        G.decode_shared_paged(q, k, v, table, lens, ints(starts), ints([2]),
                              G.alloc_decode_shared_workspace(4, paged.max_pages, 1), z, st, stream)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        results.append((codes, scale, score, chosen, a, z))
    for x, y in zip(*results):
        assert torch.equal(x, y) and x.any()


def test_tensors_that_are_not_contiguous_are_refused():
    paged, q = Paged([200], seed=32), queries(1, 51).to(DEV)
    k, v, table = paged.dev()
    sel, ws = ints(lists([200], 2, seed=12)), G.alloc_decode_sparse_workspace(1, 2)
    args = [q, k, v, table, ints([200]), sel, ws, torch.zeros_like(q)]
    for i in (0, 1, 2, 7):
        bad = list(args)
        bad[i] = torch.cat((args[i], args[i]), -1)[..., :128]
        with pytest.raises(ValueError, match="contiguous"):
            G.decode_sparse_paged(*bad)
    with pytest.raises(TypeError):
        G.decode_sparse_paged(q.half(), *args[1:])
    with pytest.raises(ValueError):
        G.decode_sparse_paged(q.cpu(), *args[1:])


@pytest.mark.parametrize("bits", [0xFFFFFFFF, 0x7FC00000, 0xFF800001, 0x7F800000, 0xFF800000, 0x80000000], ids=hex)
def test_choice_over_bounds_that_nobody_wrote(bits):
    """Whatever the scales hold, sel holds blocks of the sequence, ascending and each once, and its neighbours stay."""
    lens, budget = [3000, 2000], 7
    paged = Paged(lens, seed=33)
    codes, scale, _ = run_bounds(paged, [0, 0], lens, 3000)
    raw = scale.view(torch.int32)
    raw.view(-1)[::3] = bits - (1 << 32) if bits >> 31 else bits
    for every in (False, True):
        if every:
            raw[:] = raw.view(-1)[0]
            codes[:] = -128
        for sink, recent in ((0, 0), (1, 2), (3, 4)):
            around = torch.full((4, 8, budget), 99, dtype=torch.int32, device=DEV)
            score = torch.zeros(2, 8, 2 * paged.max_pages, device=DEV)
            G.select_blocks_paged(queries(2, 7).to(DEV), codes, scale, torch.tensor(paged.table).to(DEV), ints(lens), sink,
                                  recent, score, around[1:3])
            got = around.cpu().numpy()
            assert (got[[0, 3]] == 99).all()
            for b, n in enumerate(lens):
                for row in got[1 + b]:
                    blocks = -(-n // 64)
                    assert (np.diff(row) > 0).all() and row[0] >= 0 and row[-1] < blocks
                    assert set(range(sink)) | set(range(blocks - recent, blocks)) <= set(row.tolist())


def test_bounds_of_a_prefix_that_many_sequences_share():
    """All of them may be given to one call, each with the prefix's rows."""
    paged, _ = grouped([40], [3], lambda i: 1 + 11 * i, seed=34)
    codes, scale, st = run_bounds(paged, [0] * 40, paged.lens, max(paged.lens))
    assert st == 0
    touched = {}
    for b, n in enumerate(paged.lens):
        for blk in range(-(-n // 64)):
            touched[b, blk] = min(64, n - 64 * blk)
    check_bounds(paged, codes, scale, touched)


def test_integers_that_begin_anywhere():
    """Tables, lengths, lists, scores and groups need no more than their type's alignment."""
    paged, starts = grouped([3, 4], [2, 1], lambda i: 77 * i, seed=35)
    q = queries(7, 52)
    k, v, table = paged.dev()
    k.nan_to_num_(0.5)
    v.nan_to_num_(0.5)
    codes, scale, _ = run_bounds(paged, [0] * 7, paged.lens, max(paged.lens))
    sel = lists(paged.lens, 3, seed=13)

    def off(t, by):
        flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
        flat[by:] = t.reshape(-1)
        return flat[by:].view(t.shape)

    results = []
    for by in (0, 1, 3):
        tb, lens = off(table, by), off(ints(paged.lens), by)
        score, chosen = off(torch.zeros(7, 8, 2 * paged.max_pages, device=DEV), by), off(ints(np.zeros((7, 8, 3))), by)
        c, s = torch.zeros_like(codes), off(torch.zeros_like(scale), by)
        a, z = torch.zeros_like(q, device=DEV), torch.zeros_like(q, device=DEV)
        G.kv_bounds_paged(k, tb, off(ints([0] * 7), by), lens, max(paged.lens), c, s)
        G.select_blocks_paged(q.to(DEV), c, s, tb, lens, 1, 1, score, chosen)
        G.decode_sparse_paged(q.to(DEV), k, v, tb, lens, off(ints(sel), by), G.alloc_decode_sparse_workspace(7, 3), a)
        G.decode_shared_paged(q.to(DEV), k, v, tb, lens, off(ints(starts), by), off(ints([2, 1]), by),
                              G.alloc_decode_shared_workspace(7, paged.max_pages, 2), z)
        results.append((c, s, score, chosen, a, z))
    for other in results[1:]:
        for x, y in zip(results[0], other):
            assert torch.equal(x, y) and x.any()


@pytest.mark.parametrize("sizes,pages,mine", [
    ([40], [1], lambda i: 500 + 11 * i), ([3, 30, 7], [2, 30, 0], lambda i: 1100 - 17 * i), ([200], [110], lambda i: 65 + i % 64),
    ([2] * 30, [9] * 30, lambda i: 900 if i % 2 else 1)], ids=["short prefix", "unequal", "long prefix", "many groups"])
def test_many_own_rows_behind_prefixes(sizes, pages, mine):
    """More blocks than half of the CTAs take at once: the halves get unequal shares."""
    paged, starts = grouped(sizes, pages, mine, seed=36)
    B = len(paged.lens)
    q = queries(B, 53)
    out, st = run_shared(paged, q, starts, pages)
    assert st == 0
    some = sorted({0, 1, B // 3, B // 2, B // 2 + 1, B - 2, B - 1})
    want, spread = expected(paged, q, lambda b, g: np.arange(paged.lens[b]) if b in some else [])
    check(out[some], want[some], spread[some], 2.0 ** -10)
    # the others, against every sequence by itself: two roundings of outputs below 1 or so, weights off by 2^-10
    single, st = run_shared(paged, q, [0, B], [0])
    assert st == 0
    check(out, single.float().cpu().double().numpy(), np.full((B, 48, 128), 1.0), 2.0 ** -8)
