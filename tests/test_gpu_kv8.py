"""The 8-bit KV cache's calls against the oracle: append, decode with the blocks' weights, eviction, and a run of them."""
import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
from oracle import bf16, kv8
from oracle import rope as R
from tests.parity_util import assert_close

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
KINDS = ("int8", "e4m3")


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _bf16(x):
    return torch.from_numpy(bf16.from_f32(np.asarray(x, np.float32)).view(np.int16)).view(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make_cache(B, max_blocks, kind, seed=0, extra=5):
    """A cache whose blocks lie in random order in a larger pool; every byte and scale that nothing writes is junk
    (0x7f: the largest int8, an e4m3 NaN)."""
    g = torch.Generator().manual_seed(seed)
    n = B * 8 * max_blocks + extra
    table = torch.randperm(n, generator=g)[:B * 8 * max_blocks].to(torch.int32).view(B, 8, max_blocks).to(DEV)
    junk = lambda *s: torch.full((n,) + s, 0x7f, dtype=torch.uint8, device=DEV).view(DT[kind])  # noqa: E731
    nan = lambda *s, d=torch.float32: torch.full(s, float("nan"), dtype=d, device=DEV)  # noqa: E731
    return G.Kv8Cache(junk(2, 64, 64), junk(128, 64), nan(n), nan(n), table,
                      nan(B, 8, 64, 128, d=torch.bfloat16), nan(B, 8, 64, 128, d=torch.bfloat16))


def tables(n):
    return G.rope_cos_sin(0, n)


class Host:
    """The oracle's side of a cache: each sequence's rotated keys and values, bf16 bits [L, 8, 128]."""

    def __init__(self, B):
        self.k = [np.zeros((0, 8, 128), np.uint16) for _ in range(B)]
        self.v = [np.zeros((0, 8, 128), np.uint16) for _ in range(B)]

    def append(self, q, k, v, start, valid):
        k_rot = R.rotary_embedding(_bits(k), np.asarray(start))
        for b, n in enumerate(valid):
            self.k[b] = np.concatenate([self.k[b], k_rot[b, :n]])
            self.v[b] = np.concatenate([self.v[b], _bits(v)[b, :n]])
        return R.rotary_embedding(_bits(q), np.asarray(start))


def block_of(cache, b, g, i):
    """Codes [64, 128] (bytes) of K and V and the two scales of one block."""
    at = int(cache.table[b, g, i])
    k = cache.k_pool[at].view(torch.uint8).cpu().numpy()
    v = cache.v_pool[at].view(torch.uint8).cpu().numpy()
    return (np.concatenate([k[0], k[1]], 1), v.T, np.float32(cache.k_scale[at].item()),
            np.float32(cache.v_scale[at].item()))


def check_cache(cache, host, kind):
    for b in range(cache.B):
        L = len(host.k[b])
        for g in range(8):
            want_k, want_v = kv8.blocks(host.k[b][:, g], kind), kv8.blocks(host.v[b][:, g], kind)
            for i in range(cache.max_blocks):
                k, v, ks, vs = block_of(cache, b, g, i)
                if i >= len(want_k):
                    assert (k == 0x7f).all() and (v == 0x7f).all() and np.isnan(ks) and np.isnan(vs), (b, g, i)
                    continue
                (ck, sk), (cv, sv) = want_k[i], want_v[i]
                r = len(ck)
                assert np.array_equal(ks, sk, equal_nan=True) and np.array_equal(vs, sv, equal_nan=True), (b, g, i)
                assert np.array_equal(k[:r], ck) and np.array_equal(v[:r], cv), (b, g, i)
                assert (k[r:] == 0x7f).all() and (v[r:] == 0x7f).all(), (b, g, i)
        r = L % 64
        if r:
            got, want = _bits(cache.open_k[b])[:, :r], host.k[b][L - r:].transpose(1, 0, 2)
            nan = (want & 0x7fff) > 0x7f80  # (a rotated NaN is a NaN: the conversion to bf16 gives 0x7fff, the oracle 0x7fc0)
            assert np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7fff) > 0x7f80).all()
            assert np.array_equal(_bits(cache.open_v[b])[:, :r], host.v[b][L - r:].transpose(1, 0, 2))


def rows(rng, B, T, scale=3.0):
    q, k, v = (_bf16(rng.standard_normal((B, T, h, 128)) * scale) for h in (48, 8, 8))
    return q, k, v


def append(cache, host, q, k, v, start, valid, tab, valid_given=True):
    """One append on both sides; q_rot is compared."""
    B, T = q.shape[:2]
    lens = [len(x) for x in host.k]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_rot = torch.zeros_like(q, device=DEV)
    G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints(start), _ints(lens), _ints(valid) if valid_given else None,
                 *tab, q_rot, status)
    want = host.append(q, k, v, start, valid)
    assert int(status.item()) == 0
    assert np.array_equal(_bits(q_rot), want)
    return q_rot


# ------------------------------------------------------------------------------------------------- append
CHUNKS = {
    "one_by_one": [1] * 67,
    "whole": [200],
    "odd": [63, 1, 1, 130, 5],
    "closes_and_opens": [40, 100, 64, 3, 61, 65],
    "exact": [64, 128, 64],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("chunks", list(CHUNKS))
def test_append_any_chunks_give_the_rows_cache(kind, chunks):
    sizes = CHUNKS[chunks]
    rng = np.random.default_rng(len(sizes))
    B, total = 2, sum(sizes)
    cache, host, tab = make_cache(B, (total + 63) // 64 + 1, kind, seed=1), Host(B), tables(total + 1000)
    pos = np.array([0, 777])
    for T in sizes:
        q, k, v = rows(rng, B, T)
        append(cache, host, q, k, v, pos.tolist(), [T] * B, tab, valid_given=False)
        pos += T
    check_cache(cache, host, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_append_padded_batch(kind):
    rng = np.random.default_rng(5)
    B, T = 5, 150
    cache, host, tab = make_cache(B, 6, kind, seed=2), Host(B), tables(512)
    for valid in ([150, 1, 64, 65, 127], [2, 63, 150, 100, 1], [1, 1, 1, 1, 1]):
        q, k, v = rows(rng, B, T)
        append(cache, host, q, k, v, [len(x) for x in host.k], valid, tab)
    check_cache(cache, host, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_append_scales_grow_stay_and_break(kind):
    """Rows one by one whose magnitudes rise, fall, vanish and leave the finite numbers; each head its own."""
    rng = np.random.default_rng(6)
    cache, host, tab = make_cache(1, 3, kind, seed=3), Host(1), tables(256)
    factor = [0.0, 2.0 ** -110, 1e-20, 1.0, 0.5, 1.0, 1e4, 3e4, 1e-3, 1e30, 1.0] + [1.0] * 60
    for i, f in enumerate(factor):
        q, k, v = rows(rng, 1, 1)
        k, v = (k.float() * f).bfloat16(), (v.float() * f).bfloat16()
        if i == 40:
            k[0, 0, 2, 7] = float("nan")
            v[0, 0, 3, 9] = float("inf")
        append(cache, host, q, k, v, [i], [1], tab)
    check_cache(cache, host, kind)
    ks, vs = cache.k_scale[cache.table[0, 2, 0].long()], cache.v_scale[cache.table[0, 3, 0].long()]
    assert torch.isnan(ks) and torch.isnan(vs)


@pytest.mark.parametrize("kind", KINDS)
def test_append_of_single_tokens_to_many_sequences(kind):
    """Steps of 70 sequences of all lengths, magnitudes that rise and fall and leave the finite numbers."""
    rng = np.random.default_rng(60)
    B, T, tab = 70, 130, tables(512)
    cache, host = make_cache(B, 3, kind, seed=60), Host(B)
    append(cache, host, *rows(rng, B, T), [0] * B, rng.integers(1, T + 1, B).tolist(), tab)
    for i in range(7):
        q, k, v = rows(rng, B, 1)
        f, h = (torch.from_numpy(10.0 ** rng.integers(-2, 2, (B, 1, 8, 1))).float() for _ in range(2))
        k, v = (k.float() * f).bfloat16(), (v.float() * h).bfloat16()
        if i == 4:
            k[3, 0, 2, 7], v[5, 0, 3, 9] = float("nan"), float("inf")
        append(cache, host, q, k, v, [len(x) for x in host.k], [1] * B, tab, valid_given=i % 2 == 0)
    check_cache(cache, host, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_append_of_single_tokens_is_that_of_halves(kind):
    """A step of 126 sequences, some with bad integers and pages, against steps of its two halves over the same pools."""
    rng = np.random.default_rng(61)
    B, tab = 126, tables(256)
    lens = rng.integers(1, 129, B).tolist()
    cache, _ = filled(rng, lens, kind, 3, seed=61, tab=tab)
    table = cache.table.clone()
    table[7, 3, lens[7] // 64], table[90, 0, lens[90] // 64] = -1, cache.n_blocks
    start, valid = list(lens), [1] * B
    start[3], start[100], valid[11], valid[12], lens[20], lens[121] = -1, 256, 0, 2, -1, 192
    q, k, v = (x.to(DEV) for x in rows(rng, B, 1, 5.0))
    got = []
    for parts in ((slice(0, B),), (slice(0, 63), slice(63, B))):
        pools = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale)]
        open_k, open_v = cache.open_k.clone(), cache.open_v.clone()
        q_rot, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device=DEV)
        for s in parts:
            part = G.Kv8Cache(*pools, table[s].clone(), open_k[s].contiguous(), open_v[s].contiguous())
            x = torch.zeros_like(q[s])
            G.kv8_append(part, q[s].contiguous(), k[s].contiguous(), v[s].contiguous(), _ints(start[s]), _ints(lens[s]),
                         _ints(valid[s]), *tab, x, status)
            q_rot[s], open_k[s], open_v[s] = x, part.open_k, part.open_v
        got.append([x.view(torch.uint8) for x in (*pools, open_k, open_v, q_rot)] + [status])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert int(got[0][-1].item()) == G.DEV_BAD_START | G.DEV_BAD_VALID | G.DEV_BAD_KV_LEN | G.DEV_BAD_PAGE
    assert not torch.equal(got[0][0], cache.k_pool.view(torch.uint8))


def test_append_skips_bad_sequences():
    rng = np.random.default_rng(7)
    B, T = 6, 3
    tab = tables(64)
    q, k, v = rows(rng, B, T)
    for start, lens, valid, bit in (([0, -1, 0, 0, 0, 0], [0] * 6, [3] * 6, G.DEV_BAD_START),
                                    ([0, 62, 0, 0, 0, 0], [0] * 6, [3] * 6, G.DEV_BAD_START),
                                    ([0] * 6, [0, -1, 0, 0, 0, 0], [3] * 6, G.DEV_BAD_KV_LEN),
                                    ([0] * 6, [0, 126, 0, 0, 0, 0], [3] * 6, G.DEV_BAD_KV_LEN),
                                    ([0] * 6, [0] * 6, [3, 0, 3, 3, 3, 3], G.DEV_BAD_VALID),
                                    ([0] * 6, [0] * 6, [3, 4, 3, 3, 3, 3], G.DEV_BAD_VALID)):
        cache, host = make_cache(B, 2, "int8", seed=4), Host(B)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        q_rot = torch.full_like(q, 7.0, device=DEV)
        G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints(start), _ints(lens), _ints(valid), *tab, q_rot, status)
        assert int(status.item()) == bit
        start, valid = list(start), list(valid)
        start[1], valid[1] = 0, 0
        want = host.append(q, k, v, start, valid)
        got = _bits(q_rot)
        assert (q_rot[1] == 7.0).all() and np.array_equal(got[[0, 2, 3, 4, 5]], want[[0, 2, 3, 4, 5]])
        check_cache(cache, host, "int8")


def test_append_skips_blocks_outside_the_pool():
    rng = np.random.default_rng(8)
    q, k, v = rows(rng, 1, 70)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        cache, host, tab = make_cache(1, 2, "int8", seed=5), Host(1), tables(128)
        saved = cache.table.clone()
        cache.table[0, 3, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        q_rot = torch.zeros_like(q, device=DEV)
        G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints([0]), _ints([0]), None, *tab, q_rot, status)
        assert int(status.item()) == G.DEV_BAD_PAGE
        cache.table.copy_(saved)
        host.append(q, k, v, [0], [70])
        for g in range(8):
            kk, vv, ks, _ = block_of(cache, 0, g, 1)
            if g == 3:
                assert (kk == 0x7f).all() and (vv == 0x7f).all() and np.isnan(ks)
            else:
                assert np.array_equal(kk[:6], kv8.blocks(host.k[0][:, g], "int8")[1][0])


# ------------------------------------------------------------------------------------------------- decode
def filled(rng, lens, kind, max_blocks, seed, scale=3.0, tab=None):
    """A cache of lens[b] rows (0 allowed) and the oracle's rows."""
    B, T = len(lens), max(max(lens), 1)
    cache, host = make_cache(B, max_blocks, kind, seed=seed), Host(B)
    q, k, v = rows(rng, B, T, scale)
    lens1 = [max(n, 1) for n in lens]
    append(cache, host, q, k, v, [0] * B, lens1, tab or tables(T))
    return cache, host


def decode_reference(host, q, lens, kind, max_blocks):
    """Exact outputs, block weights, and per output the weighted sum of |v| (for the tolerance)."""
    B = len(lens)
    out, scale_v = np.zeros((B, 48, 128)), np.zeros((B, 48, 128))
    weight = np.zeros((B, 8, max_blocks))
    s_abs = 0.0
    x = bf16.to_f64(_bits(q))
    for b in range(B):
        for g in range(8):
            if lens[b] < 1:
                continue
            K, V = kv8.held(host.k[b][:lens[b], g], kind), kv8.held(host.v[b][:lens[b], g], kind)
            qs = x[b, 6 * g:6 * g + 6]
            o, w = kv8.attend(qs, K, V)
            out[b, 6 * g:6 * g + 6], scale_v[b, 6 * g:6 * g + 6] = o, w @ np.abs(V)
            weight[b, g] = kv8.block_weights(w, max_blocks)
            s_abs = max(s_abs, (np.abs(qs) @ np.abs(K).T).max() / 128 ** 0.5)
    return out, weight, scale_v, s_abs


def check_decode(got, out, scale_v, s_abs, L, live):
    """bf16 rounding of the result (half a step, 2^-8), and of a weight: its fp16 rounding (2^-11), its logit (a
    128-term fp32 sum, 128 * 2^-23 of the sum of magnitudes), and three approximate functions on log2 weights up to
    87 (2^-20 each of 87); a weight enters numerator and sum. fp16 below its normal range: 2^-25 of the largest
    weight per key."""
    got = got.float().cpu().numpy().astype(np.float64)
    delta = 2.0 ** -11 + 2 * (128 * 2.0 ** -23 * s_abs + 3 * 87 * 2.0 ** -20)
    tol = 2.0 ** -8 * np.abs(out) + delta * scale_v * (1 + 2.0 ** -8) + L * 2.0 ** -25 * scale_v.max()
    bad = np.abs(got - out) > tol
    assert not bad[live].any(), (np.abs(got - out) / tol)[live].max()


def run_decode(cache, q, lens, weight_in=None, weights=True):
    B = cache.B
    out = torch.full((B, 48, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    w_out = torch.full((B, 8, cache.max_blocks), 7.0, device=DEV) if weights else None
    ws = G.alloc_kv8_decode_workspace(cache, weights)
    ws.fill_(0xff)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    G.kv8_decode(cache, q, _ints(lens), ws, out, weight_in, w_out, status)
    torch.cuda.synchronize()
    return out, w_out, int(status.item())


LENS = {
    "short": [1, 2, 63, 64, 65, 128, 300],
    "one": [1],
    "one_long": [2000],
    "mixed": [700, 1, 129, 64, 640, 5],
    "many": [(37 * i) % 200 + 1 for i in range(70)],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(LENS))
def test_decode(kind, name):
    lens = LENS[name]
    rng = np.random.default_rng(11)
    max_blocks = (max(lens) + 63) // 64 + 1
    cache, host = filled(rng, lens, kind, max_blocks, seed=6)
    q = _bf16(rng.standard_normal((len(lens), 48, 128)) * 3).to(DEV)
    before = torch.rand(len(lens), 8, max_blocks, device=DEV)
    got, w, status = run_decode(cache, q, lens, before)
    assert status == 0
    out, weight, scale_v, s_abs = decode_reference(host, q, lens, kind, max_blocks)
    live = np.ones(len(lens), bool)
    check_decode(got, out, scale_v, s_abs, max(lens), live)
    assert_close(_bits(got), bf16.from_f64(out), f"kv8 decode {kind} {name}")
    # the weights are sums of fp32 weights: the same errors but for the fp16 rounding, and one fp32 sum
    exact = before.double().cpu().numpy() + weight
    delta = 2 * (128 * 2.0 ** -23 * s_abs + 3 * 87 * 2.0 ** -20) + 2.0 ** -20
    assert (np.abs(w.double().cpu().numpy() - exact) <= delta * weight + 2.0 ** -23 * exact).all()
    assert torch.equal(run_decode(cache, q, lens, weights=False)[0], got)
    # in place
    G.kv8_decode(cache, q, _ints(lens), G.alloc_kv8_decode_workspace(cache), got, before, before)
    assert torch.equal(before, w)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1e-6, 0.02, 8.0])
def test_decode_flat_and_peaked_logits(kind, scale):
    """Weights all alike, and logits far beyond the cap."""
    lens = [517, 64]
    rng = np.random.default_rng(12)
    cache, host = filled(rng, lens, kind, 9, seed=7, scale=scale)
    q = _bf16(rng.standard_normal((2, 48, 128)) * scale).to(DEV)
    got, _, _ = run_decode(cache, q, lens)
    out, _, scale_v, s_abs = decode_reference(host, q, lens, kind, 9)
    check_decode(got, out, scale_v, s_abs, 517, np.ones(2, bool))


def test_decode_unequal_query_heads():
    """Queries of very different magnitudes, one zero: each head is scaled to fp16 by its own power of two."""
    lens = [200]
    rng = np.random.default_rng(13)
    cache, host = filled(rng, lens, "int8", 4, seed=8)
    mag = 2.0 ** np.linspace(-40, 3, 48)[None, :, None]
    mag[0, 5] = 0
    q = _bf16(rng.standard_normal((1, 48, 128)) * mag).to(DEV)
    got, _, _ = run_decode(cache, q, lens)
    out, _, scale_v, s_abs = decode_reference(host, q, lens, "int8", 4)
    check_decode(got, out, scale_v, s_abs, 200, np.ones(1, bool))


def test_decode_bad_lengths_leave_the_outputs():
    rng = np.random.default_rng(14)
    lens = [100, 70, 3, 128]
    cache, host = filled(rng, lens, "e4m3", 2, seed=9)
    q = _bf16(rng.standard_normal((4, 48, 128)) * 3).to(DEV)
    given = [100, 0, 129, 128]
    got, w, status = run_decode(cache, q, given)
    assert status == G.DEV_BAD_KV_LEN
    assert (got[[1, 2]] == 7.0).all() and (w[[1, 2]] == 7.0).all()
    out, _, scale_v, s_abs = decode_reference(host, q, [100, 0, 0, 128], "e4m3", 2)
    check_decode(got, out, scale_v, s_abs, 128, np.array([True, False, False, True]))
    got, _, status = run_decode(cache, q, [0, -5, 2 ** 31 - 1, -2 ** 31])
    assert status == G.DEV_BAD_KV_LEN and (got == 7.0).all()


def test_decode_reports_blocks_outside_the_pool():
    rng = np.random.default_rng(15)
    cache, _ = filled(rng, [100, 100], "int8", 2, seed=10)
    q = _bf16(rng.standard_normal((2, 48, 128)) * 3).to(DEV)
    good, _, _ = run_decode(cache, q, [100, 100])
    for bad in (-1, cache.n_blocks, 2 ** 31 - 1):
        cache.table[1, 0, 1] = bad
        got, _, status = run_decode(cache, q, [100, 100])
        assert status == G.DEV_BAD_PAGE
        assert torch.equal(got[0], good[0]) and torch.equal(got[1, 6:], good[1, 6:])


def test_decode_of_a_non_finite_block_is_nan_for_its_head_alone():
    rng = np.random.default_rng(16)
    cache, host = filled(rng, [200, 200], "int8", 4, seed=11)
    q = _bf16(rng.standard_normal((2, 48, 128)) * 3).to(DEV)
    good, _, _ = run_decode(cache, q, [200, 200])
    cache.k_scale[cache.table[0, 1, 2].long()] = float("nan")
    cache.v_scale[cache.table[1, 4, 0].long()] = float("nan")
    got, _, _ = run_decode(cache, q, [200, 200])
    nan = torch.isnan(got).all(-1)
    want = torch.zeros_like(nan)
    want[0, 6:12] = True
    want[1, 24:30] = True
    assert torch.equal(nan, want) and torch.equal(got[~want], good[~want])


def test_decode_pool_past_2_gb():
    """Blocks behind byte 2^31 of both pools."""
    rng = np.random.default_rng(17)
    small, host = filled(rng, [150], "int8", 3, seed=12)
    n = 300000
    k = torch.empty((n, 2, 64, 64), dtype=torch.int8, device=DEV)
    v = torch.empty((n, 128, 64), dtype=torch.int8, device=DEV)
    ks, vs = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    shift = n - small.n_blocks
    k[shift:], v[shift:], ks[shift:], vs[shift:] = small.k_pool, small.v_pool, small.k_scale, small.v_scale
    cache = G.Kv8Cache(k, v, ks, vs, small.table + shift, small.open_k, small.open_v)
    q = _bf16(rng.standard_normal((1, 48, 128)) * 3).to(DEV)
    assert torch.equal(run_decode(cache, q, [150])[0], run_decode(small, q, [150])[0])
    del host


def random_cache(B, max_blocks, kind, seed):
    """A cache of random codes and scales in random order (no rows behind it: for long caches)."""
    g = torch.Generator(DEV).manual_seed(seed)
    n = B * 8 * max_blocks
    k, v = (torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            for shape in ((n, 2, 64, 64), (n, 128, 64)))
    if kind == "e4m3":
        k, v = (torch.where((x & 0x7f) == 0x7f, 0x11, x) for x in (k, v))  # no NaN
    scale = torch.rand(n, generator=g, device=DEV) * (3 / 127 if kind == "int8" else 3 / 448) + 1e-3
    table = torch.randperm(n, generator=g, device=DEV).to(torch.int32).view(B, 8, max_blocks)
    rows_open = torch.zeros(B, 8, 64, 128, dtype=torch.bfloat16, device=DEV)
    return G.Kv8Cache(k.view(DT[kind]), v.view(DT[kind]), scale, scale.flip(0).contiguous(), table, rows_open, rows_open)


def cache_values(cache, b, h, L):
    """Keys and values [L, 128] of one head in fp64."""
    ids = cache.table[b, h, :(L + 63) // 64].long()
    k = cache.k_pool.view(torch.uint8)[ids].view(cache.k_pool.dtype)
    v = cache.v_pool.view(torch.uint8)[ids].view(cache.v_pool.dtype)
    K = k.float().double().transpose(1, 2).flatten(2) * cache.k_scale[ids].double()[:, None, None]
    V = v.float().double().transpose(1, 2) * cache.v_scale[ids].double()[:, None, None]
    return K.reshape(-1, 128)[:L].cpu().numpy(), V.reshape(-1, 128)[:L].cpu().numpy()


def check_random_cache_decode(cache, lens, pick, what):
    q = (torch.randn(cache.B, 48, 128, generator=torch.Generator(DEV).manual_seed(9), device=DEV) * 3).bfloat16()
    got, w, status = run_decode(cache, q, lens)
    assert status == 0
    want, exact = [], []
    for b in pick:
        for h in range(8):
            o, p = kv8.attend(q[b, 6 * h:6 * h + 6].double().cpu().numpy(), *cache_values(cache, b, h, lens[b]))
            want.append(o)
            exact.append(kv8.block_weights(p, cache.max_blocks))
    assert_close(_bits(got[pick]).reshape(-1, 6, 128), bf16.from_f64(np.stack(want)), what)
    # sums of |q k| are about 40 here: logits off by at most 128 * 2^-23 * 40, weights by the functions' 3 * 87 * 2^-20, twice
    assert np.allclose(w[pick].double().cpu().numpy().reshape(-1, cache.max_blocks), np.stack(exact), rtol=2e-3, atol=1e-7)
    assert (w.sum(-1) - 6).abs().max() < 1e-3  # every head's weights add up to one: every block was read once
    assert torch.equal(run_decode(cache, q, lens, weights=False)[0], got)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_long_shares_in_two_waves(kind):
    """Enough blocks (24 and more for every resident warp) for the second wave of small shares."""
    lens = np.random.default_rng(50).integers(4000, 72 * 64 + 1, 80).tolist()
    lens[7], lens[40] = 1, 65
    check_random_cache_decode(random_cache(80, 72, kind, 50), lens, [0, 7, 40, 79], f"kv8 decode two waves {kind}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows_", [65536, 40001])
def test_decode_longest_cache(kind, rows_):
    """One sequence over the whole range: over a hundred partials for each head."""
    check_random_cache_decode(random_cache(1, 1024, kind, 51), [rows_], [0], f"kv8 decode {rows_} rows {kind}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,start", [(3, 65000), (32, 65504), (40, 65000)])
def test_prefill_behind_the_longest_cache(kind, T, start):
    """Tokens behind 65000 rows: passes over the codes to the last row; items in parts, kernels over 510 key tiles."""
    cache = random_cache(1, 1024, kind, 52)
    q = (torch.randn(1, T, 48, 128, generator=torch.Generator(DEV).manual_seed(10), device=DEV) * 3).bfloat16()
    got, status = run_prefill(cache, q, [start], [T], T)
    assert status == 0
    want = []
    for h in range(8):
        K, V = cache_values(cache, 0, h, start + T)
        for r in range(6):
            want.append(kv8.attend(q[0, :, 6 * h + r].double().cpu().numpy(), K, V, start + np.arange(T))[0])
    assert_close(_bits(got[0]), bf16.from_f64(np.stack(want, 1)), f"kv8 prefill of {T} behind {start} rows {kind}")


def test_calls_on_two_streams_at_once():
    """Decode and prefill over one cache from two streams, each with its own workspace and outputs."""
    cache = random_cache(4, 40, "int8", 53)
    lens = [2500, 700, 64, 1]
    gen = torch.Generator(DEV).manual_seed(11)
    q = (torch.randn(4, 48, 128, generator=gen, device=DEV) * 3).bfloat16()
    qp = (torch.randn(4, 130, 48, 128, generator=gen, device=DEV) * 3).bfloat16()
    want_d = run_decode(cache, q, lens, weights=False)[0]
    want_p = run_prefill(cache, qp, [2000, 500, 64, 1], None, 130)[0]
    kv, cl = _ints(lens), _ints([2000, 500, 64, 1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros_like(qp), G.alloc_kv8_decode_workspace(cache),
             G.alloc_kv8_prefill_workspace(cache)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (d, p, wd, wp) in zip(streams, outs):
            G.kv8_decode(cache, q, kv, wd, d, stream=s)
            G.kv8_prefill(cache, qp, cl, None, p, wp, stream=s)
    torch.cuda.synchronize()
    for d, p, _, _ in outs:
        assert torch.equal(d, want_d) and torch.equal(p, want_p)


def test_workspace_too_small_is_refused():
    rng = np.random.default_rng(18)
    cache, _ = filled(rng, [10], "int8", 1, seed=13)
    q = _bf16(rng.standard_normal((1, 48, 128))).to(DEV)
    out = torch.empty(1, 48, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.empty(1, 8, 1, device=DEV)
    ws = G.alloc_kv8_decode_workspace(cache, weights=False)
    with pytest.raises(G.GrokError, match="smaller"):
        G.kv8_decode(cache, q, _ints([10]), ws, out, None, w)
    with pytest.raises(G.GrokError, match="smaller"):
        G.kv8_decode(cache, q, _ints([10]), ws[:-256], out)


# ------------------------------------------------------------------------------------------------- prefill
def run_prefill(cache, q_rot, lens, valid, T):
    out = torch.full((cache.B, T, 48, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = G.alloc_kv8_prefill_workspace(cache)
    ws.fill_(0xff)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    G.kv8_prefill(cache, q_rot, _ints(lens), _ints(valid) if valid else None, out, ws, status)
    torch.cuda.synchronize()
    return out, int(status.item())


def check_prefill(host, q_rot, got, lens, valid, kind, what, picks=None, heads=range(48)):
    """The rows `picks` (default: edges of the tiles and the sequence) of every sequence against the oracle."""
    T = q_rot.shape[1]
    x, y = bf16.to_f64(_bits(q_rot)), _bits(got)
    want, have = [], []
    for b in range(len(lens)):
        n = valid[b]
        rows_ = sorted({i for i in (picks or (0, 1, 31, 63, 64, 65, 127, 128, 129, 200, 255, 256, n - 1, n, T - 1))
                        if 0 <= i < T})
        last = np.minimum(lens[b] + np.array(rows_), lens[b] + n - 1)
        for g in sorted({h // 6 for h in heads}):
            K, V = kv8.held(host.k[b][:, g], kind), kv8.held(host.v[b][:, g], kind)
            for h in range(6 * g, 6 * g + 6):
                o, _ = kv8.attend(x[b, rows_, h], K, V, last)
                want.append(o)
                have.append(y[b, rows_, h])
    return assert_close(np.concatenate(have), bf16.from_f64(np.concatenate(want)), what)


def logit_error(q, K):
    """A 128-term fp32 sum: at most 128 * 2^-23 of the sum of the terms' magnitudes."""
    return 128 * 2.0 ** -23 * (np.abs(q) @ np.abs(K).T).max() / 128 ** 0.5


PREFILLS = {
    # warm rows, valid tokens, padded T
    "tiny": ([0], [1], 1),
    "one_tile": ([0], [128], 128),
    "odd": ([0, 5, 64], [200, 77, 131], 200),
    "warm": ([130, 700, 63], [90, 33, 1], 90),
    "chunk_split": ([2100, 1900], [150, 61], 150),
    "ragged": ([0, 0, 0, 0], [300, 1, 64, 129], 300),
    # items split over the key range
    "split_few": ([2500], [1], 1),
    "split_unequal": ([2000, 64, 900], [300, 500, 7], 500),
    "split_causal": ([700], [1400], 1400),
    # the longest call that runs as single tokens, and the shortest that does not
    "last_few": ([2500, 63, 120], [32, 4, 17], 32),
    "first_many": ([2500, 63, 120], [33, 4, 17], 33),
    "last_few_of_nine": (list(range(40, 400, 40)), [16, 1, 2, 3, 4, 5, 11, 15, 16], 16),
    "first_many_of_nine": (list(range(40, 400, 40)), [17, 1, 2, 3, 4, 5, 11, 15, 16], 17),
    "last_few_of_one": ([700], [95], 96),
    "first_many_of_one": ([700], [96], 97),
    "last_few_of_one_tile": ([100, 1], [12, 5], 12),
    "first_many_of_one_tile": ([100, 1], [13, 5], 13),
    "few_over_many_shares": ([9000, 60, 0, 7000], [5, 7, 1, 2], 7),
    "few_over_many_sequences": (list(range(0, 320, 5)), [1 + i % 3 for i in range(64)], 3),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(PREFILLS))
def test_prefill(kind, name):
    lens, valid, T = PREFILLS[name]
    rng = np.random.default_rng(40)
    B = len(lens)
    max_blocks, tab = (max(lens) + T + 63) // 64, tables(max(lens) + T + 1)
    cache, host = make_cache(B, max_blocks, kind, seed=30), Host(B)
    if max(lens):
        warm = [max(n, 1) for n in lens]
        append(cache, host, *rows(rng, B, max(lens)), [0] * B, warm, tab)
        lens = warm
    q_rot = append(cache, host, *rows(rng, B, T), lens, valid, tab)
    got, status = run_prefill(cache, q_rot, lens, valid, T)
    assert status == 0
    check_prefill(host, q_rot, got, lens, valid, kind, f"kv8 prefill {kind} {name}")
    assert torch.equal(run_prefill(cache, q_rot, lens, valid, T)[0], got)


def test_prefill_of_one_token_is_the_decode():
    rng = np.random.default_rng(41)
    cache, host = filled(rng, [300, 65], "int8", 5, seed=31)
    q = _bf16(rng.standard_normal((2, 1, 48, 128)) * 3).to(DEV)
    a, _ = run_prefill(cache, q, [299, 64], [1, 1], 1)
    b, _, _ = run_decode(cache, q[:, 0].contiguous(), [300, 65])
    assert_close(_bits(a[:, 0]), _bits(b), "kv8 prefill against decode")


def test_prefill_of_few_tokens_is_that_of_many():
    """The same valid tokens in calls of 32 and of 33 tokens, which take different kernels."""
    rng = np.random.default_rng(48)
    cache, host = filled(rng, [700, 64, 32, 300], "e4m3", 11, seed=38)
    q = _bf16(rng.standard_normal((4, 33, 48, 128)) * 3).to(DEV)
    lens, valid = [668, 60, 0, 269], [32, 4, 32, 31]
    a, sa = run_prefill(cache, q[:, :32].contiguous(), lens, valid, 32)
    b, sb = run_prefill(cache, q, lens, valid, 33)
    assert sa == sb == 0
    assert_close(_bits(a), _bits(b[:, :32]), "kv8 prefill of 32 tokens against 33")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1e-6, 0.02, 8.0, "unequal"])
def test_prefill_of_few_tokens_flat_and_peaked_logits(kind, scale):
    """Seven tokens over a block's end: all weights alike, logits beyond the cap, queries of unequal magnitudes."""
    lens, T = [517, 66], 7
    rng = np.random.default_rng(52)
    cache, host = filled(rng, lens, kind, 9, seed=42, scale=3.0 if scale == "unequal" else scale)
    size = 2.0 ** rng.integers(-40, 4, (2, T, 48, 1)) if scale == "unequal" else scale
    q = _bf16(rng.standard_normal((2, T, 48, 128)) * size).to(DEV)
    got, status = run_prefill(cache, q, [n - T for n in lens], None, T)
    assert status == 0
    x = bf16.to_f64(_bits(q))
    out, scale_v = np.zeros((2, T, 48, 128)), np.zeros((2, T, 48, 128))
    s_abs = 0.0
    for b, n in enumerate(lens):
        for g in range(8):
            K, V = kv8.held(host.k[b][:n, g], kind), kv8.held(host.v[b][:n, g], kind)
            for h in range(6 * g, 6 * g + 6):
                o, w = kv8.attend(x[b, :, h], K, V, n - T + np.arange(T))
                out[b, :, h], scale_v[b, :, h] = o, w @ np.abs(V)
                s_abs = max(s_abs, (np.abs(x[b, :, h]) @ np.abs(K).T).max() / 128 ** 0.5)
    flat = lambda a: a.reshape(2 * T, 48, 128)  # noqa: E731
    check_decode(flat(got), flat(out), flat(scale_v), s_abs, 517, np.ones(2 * T, bool))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["k", "v"])
def test_prefill_of_few_tokens_non_finite_block_reaches_its_tokens_alone(kind, where):
    """Tokens 0 and 1 end the first block; token 3 makes the second one's scale a NaN, which tokens 2 to 5 see."""
    tab, T = tables(256), 6
    results = []
    for broken in (False, True):
        rng = np.random.default_rng(51)
        cache, _ = filled(rng, [62, 62], kind, 3, seed=41, tab=tab)
        q, k, v = rows(rng, 2, T)
        if broken:
            (k if where == "k" else v)[0, 3, 5, 17] = float("inf")
        q_rot = torch.empty_like(q, device=DEV)
        G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints([62, 62]), _ints([62, 62]), None, *tab, q_rot)
        got, status = run_prefill(cache, q_rot, [62, 62], None, T)
        assert status == 0
        results.append(got.float())
    good, bad = results
    head = slice(30, 36)
    assert torch.isnan(bad[0, 2:, head]).all() and torch.equal(bad[0, :2], good[0, :2])
    keep = [*range(30), *range(36, 48)]
    assert torch.equal(bad[0][:, keep], good[0][:, keep]) and torch.equal(bad[1], good[1])
    assert torch.isfinite(good).all()


def test_prefill_of_few_tokens_bad_integers():
    rng = np.random.default_rng(49)
    cache, host = filled(rng, [128] * 3, "int8", 2, seed=39)
    q = _bf16(rng.standard_normal((3, 5, 48, 128))).to(DEV)
    good, _ = run_prefill(cache, q, [100] * 3, [5] * 3, 5)
    for start, n, bit in ((-1, 5, G.DEV_BAD_KV_LEN), (124, 5, G.DEV_BAD_KV_LEN), (2 ** 31 - 1, 5, G.DEV_BAD_KV_LEN),
                          (100, 0, G.DEV_BAD_VALID), (100, -7, G.DEV_BAD_VALID), (100, 6, G.DEV_BAD_VALID),
                          (125, 6, G.DEV_BAD_VALID | G.DEV_BAD_KV_LEN),
                          (-1, 2 ** 31 - 1, G.DEV_BAD_VALID | G.DEV_BAD_KV_LEN)):
        got, status = run_prefill(cache, q, [100, start, 100], [5, n, 5], 5)
        assert status == bit
        assert (got[1] == 7.0).all() and torch.equal(got[[0, 2]], good[[0, 2]])
    got, status = run_prefill(cache, q, [110] * 3, [5, 1, 3], 5)
    assert status == 0
    got, status = run_prefill(cache, q, [-1] * 3, [5] * 3, 5)
    assert status == G.DEV_BAD_KV_LEN and (got == 7.0).all()
    cache.table[1, 7, 1] = cache.n_blocks
    got, status = run_prefill(cache, q, [100] * 3, [5] * 3, 5)
    assert status == G.DEV_BAD_PAGE and torch.equal(got[[0, 2]], good[[0, 2]])


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_block_magnitudes_apart(kind):
    """V blocks 2^-12 to 2^12 of one another, keys 2^-3 to 2^1: each element still within its own block's share."""
    rng = np.random.default_rng(42)
    L = 400
    cache, host, tab = make_cache(1, 7, kind, seed=32), Host(1), tables(512)
    q, k, v = rows(rng, 1, L)
    vm = 2.0 ** rng.integers(-12, 13, (1, 7, 8, 1)).repeat(64, 1)[:, :L]
    km = 2.0 ** rng.integers(-3, 2, (1, 7, 8, 1)).repeat(64, 1)[:, :L]
    v, k = (v.float() * torch.from_numpy(vm).float()).bfloat16(), (k.float() * torch.from_numpy(km).float()).bfloat16()
    q_rot = append(cache, host, q, k, v, [0], [L], tab)
    got, _ = run_prefill(cache, q_rot, [0], [L], L)
    x, y = bf16.to_f64(_bits(q_rot)), got.float().cpu().numpy().astype(np.float64)
    for h in range(0, 48, 5):
        K, V = kv8.held(host.k[0][:, h // 6], kind), kv8.held(host.v[0][:, h // 6], kind)
        o, w = kv8.attend(x[0, :, h], K, V, np.arange(L))
        # half a step of bf16; a weight is off by its fp16 rounding (2^-11), by tanh and exp2 (1e-5 of 30, that is 3e-4)
        # and by its logit (a 128-term fp32 sum), in the sum too; below fp16's normal range by 2^-17 of the row's
        # largest; V by 2^-11, or 2^-40 of the head's largest
        rel = 2.0 ** -11 + 2 * (3e-4 + logit_error(x[0, :, h], K)) + 2.0 ** -11
        tol = 2.0 ** -8 * np.abs(o) + rel * (w @ np.abs(V)) + 2.0 ** -17 * np.abs(V).sum(0) * w.max(1, keepdims=True) \
            + 2.0 ** -40 * np.abs(V).max()
        assert (np.abs(y[0, :, h] - o) <= tol).all(), h


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_weights_that_outgrow_fp16(kind):
    """A first tile of small logits and a later key at the cap: those items are computed again in bf16, V rounded to
    bf16 there (2^-9 of each value, within the tolerance of one bf16 step of the result)."""
    rng = np.random.default_rng(43)
    L = 300
    cache, host, tab = make_cache(2, 5, kind, seed=33), Host(2), tables(512)
    q, k, v = rows(rng, 2, L)
    k[0] = (k[0].float() * 0.02).bfloat16()
    q[0, :, :6] = q[0, 200, 0]
    k[0, 200, 0] = q[0, 200, 0]
    # the rotation keeps q . k only at equal positions: rotate by none
    tab = (torch.ones_like(tab[0]), torch.zeros_like(tab[1]))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_rot = torch.zeros_like(q, device=DEV)
    G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints([0, 0]), _ints([0, 0]), None, *tab, q_rot, status)
    assert torch.equal(q_rot.cpu(), q)
    for b in range(2):
        host.k[b], host.v[b] = _bits(k)[b], _bits(v)[b]
    got, st = run_prefill(cache, q_rot, [0, 0], [L, L], L)
    assert st == 0
    x, y = bf16.to_f64(_bits(q_rot)), got.float().cpu().numpy().astype(np.float64)
    for b in range(2):
        for h in (0, 5, 7, 47):
            K, V = kv8.held(host.k[b][:, h // 6], kind), kv8.held(host.v[b][:, h // 6], kind)
            o, w = kv8.attend(x[b, :, h], K, V, np.arange(L))
            # half a step of the result, 2^-8; of V 2^-8; weights as above (bf16 hi + lo: 2^-16)
            rel = 2.0 ** -8 + 2.0 ** -11 + 2 * (3e-4 + logit_error(x[b, :, h], K))
            tol = 2.0 ** -8 * np.abs(o) + rel * (w @ np.abs(V)) \
                + 2.0 ** -17 * np.abs(V).sum(0) * w.max(1, keepdims=True)
            assert (np.abs(y[b, :, h] - o) <= tol).all(), (b, h)


def test_prefill_non_finite_blocks_reach_their_rows_alone():
    rng = np.random.default_rng(44)
    cache, host = filled(rng, [300, 300], "int8", 5, seed=34)
    q = _bf16(rng.standard_normal((2, 300, 48, 128)) * 3).to(DEV)
    good, _ = run_prefill(cache, q, [0, 0], None, 300)
    for scale, b, g, blk in ((cache.k_scale, 0, 1, 1), (cache.v_scale, 1, 3, 2), (cache.v_scale, 1, 5, 4)):
        at = cache.table[b, g, blk].long()
        saved = scale[at].clone()
        scale[at] = float("nan")
        got, _ = run_prefill(cache, q, [0, 0], None, 300)
        scale[at] = saved
        nan = torch.isnan(got).all(-1)
        want = torch.zeros_like(nan)
        want[b, 64 * blk:, 6 * g:6 * g + 6] = True
        assert torch.equal(nan, want)
        assert torch.equal(got[~want], good[~want])


def test_prefill_split_items_of_good_and_bad_sequences():
    """A key-range split with a sequence that takes no part: its outputs stay."""
    rng = np.random.default_rng(46)
    cache, host = filled(rng, [1500, 1100, 1300], "int8", 32, seed=36)
    q = _bf16(rng.standard_normal((3, 140, 48, 128)) * 3).to(DEV)
    lens, valid = [1360, 960, 1160], [140, 130, 140]
    good, status = run_prefill(cache, q, lens, valid, 140)
    assert status == 0
    host.k[1], host.v[1] = host.k[1][:1090], host.v[1][:1090]
    check_prefill(host, q, good, lens, valid, "int8", "kv8 prefill shared", heads=(0, 47))
    for bad in (-1, 2 ** 31 - 1, 2000):
        got, status = run_prefill(cache, q, [1360, bad, 1160], valid, 140)
        assert status == G.DEV_BAD_KV_LEN and (got[1] == 7.0).all()
        # the split may fall elsewhere: the same within one bf16 step
        assert_close(_bits(got[[0, 2]]), _bits(good[[0, 2]]), "beside a bad sequence")
    got, status = run_prefill(cache, q, [-1, -1, -1], valid, 140)
    assert status == G.DEV_BAD_KV_LEN and (got == 7.0).all()


@pytest.mark.parametrize("T", [28, 40])
def test_prefill_bad_integers_leave_the_outputs(T):
    rng = np.random.default_rng(45)
    cache, host = filled(rng, [128] * 3, "int8", 2, seed=35)
    q = _bf16(rng.standard_normal((3, T, 48, 128))).to(DEV)
    good, _ = run_prefill(cache, q, [128 - T] * 3, [T] * 3, T)
    for lens, valid, bit in (([128 - T, -1, 128 - T], [T] * 3, G.DEV_BAD_KV_LEN),
                             ([128 - T, 129 - T, 128 - T], [T] * 3, G.DEV_BAD_KV_LEN),
                             ([128 - T] * 3, [T, 0, T], G.DEV_BAD_VALID),
                             ([128 - T] * 3, [T, T + 1, T], G.DEV_BAD_VALID | G.DEV_BAD_KV_LEN)):
        got, status = run_prefill(cache, q, lens, valid, T)
        assert status == bit
        assert (got[1] == 7.0).all() and torch.equal(got[[0, 2]], good[[0, 2]])
    # padding tokens past the capacity are no error
    got, status = run_prefill(cache, q, [110] * 3, [18, 1, 10], T)
    assert status == 0
    cache.table[1, 7, 1] = cache.n_blocks
    got, status = run_prefill(cache, q, [128 - T] * 3, [T] * 3, T)
    assert status == G.DEV_BAD_PAGE and torch.equal(got[[0, 2]], good[[0, 2]])


# ------------------------------------------------------------------------------------------------- evict
EVICTS = [dict(B=3, n=9, keep=4, sink=1, recent=2), dict(B=2, n=40, keep=33, sink=0, recent=0),
          dict(B=2, n=1024, keep=500, sink=4, recent=60), dict(B=4, n=33, keep=1, sink=0, recent=1),
          dict(B=2, n=64, keep=8, sink=4, recent=4), dict(B=1, n=1, keep=1, sink=0, recent=0),
          dict(B=3, n=5, keep=64, sink=3, recent=9)]


@pytest.mark.parametrize("case", EVICTS, ids=str)
@pytest.mark.parametrize("values", ["random", "ties", "special"])
def test_evict(case, values):
    B, n, keep, sink, recent = (case[x] for x in ("B", "n", "keep", "sink", "recent"))
    rng = np.random.default_rng(20)
    w = rng.standard_normal((B, 8, n)).astype(np.float32)
    if values == "ties":
        w = np.round(w).astype(np.float32) * np.float32(1.0)
    if values == "special":
        w = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 3.4e38, 1e-45], np.float32), (B, 8, n))
    lens = rng.integers(0, n * 64 + 1, B)
    lens[0] = n * 64
    if B > 2:
        lens[2] = min(keep, n) * 64
    table = torch.from_numpy(rng.permutation(B * 8 * n).astype(np.int32).reshape(B, 8, n)).to(DEV)
    weight, length = torch.from_numpy(w).to(DEV), _ints(lens.tolist())
    t_out, w_out, l_out = torch.empty_like(table), torch.empty_like(weight), torch.empty_like(length)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    G.kv8_evict(table, weight, length, keep, sink, recent, t_out, w_out, l_out, status)
    assert int(status.item()) == 0
    for b in range(B):
        for g in range(8):
            t, ww, m = kv8.evict(table[b, g].tolist(), w[b, g], int(lens[b]), keep, sink, recent)
            assert t_out[b, g].tolist() == t, (b, g)
            assert np.array_equal(w_out[b, g].cpu().numpy(), np.array(ww, np.float32), equal_nan=True)
            assert int(l_out[b]) == m
    # in place
    G.kv8_evict(table, weight, length, keep, sink, recent, table, weight, l_out, status)
    assert torch.equal(table, t_out) and torch.equal(torch.nan_to_num(weight), torch.nan_to_num(w_out))


def test_evict_bad_lengths_copy():
    table = torch.arange(2 * 8 * 3, dtype=torch.int32, device=DEV).view(2, 8, 3)
    weight = torch.rand(2, 8, 3, device=DEV)
    t_out, w_out, l_out = torch.empty_like(table), torch.empty_like(weight), _ints([0, 0])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    G.kv8_evict(table, weight, _ints([-1, 193]), 1, 0, 0, t_out, w_out, l_out, status)
    assert int(status.item()) == G.DEV_BAD_KV_LEN
    assert torch.equal(table, t_out) and torch.equal(weight, w_out) and l_out.tolist() == [-1, 193]


# ------------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("kind", KINDS)
def test_a_conversation_within_a_budget(kind):
    """Prompt, steps, eviction, and steps on: rows and positions part, the blocks that were freed are written again."""
    rng = np.random.default_rng(30)
    B, max_blocks, tab = 2, 8, tables(1024)
    cache, host = make_cache(B, max_blocks, kind, seed=20), Host(B)
    pos, valid = [0, 0], [450, 333]
    append(cache, host, *rows(rng, B, 450), pos, valid, tab)
    pos = list(valid)
    weight = torch.zeros(B, 8, max_blocks, device=DEV)
    total = np.zeros((B, 8, max_blocks))
    # per head from here on: the rows a head holds
    held = [[(host.k[b][:, g], host.v[b][:, g]) for g in range(8)] for b in range(B)]
    length = list(valid)
    ws = G.alloc_kv8_decode_workspace(cache)
    for step in range(70):
        q, k, v = rows(rng, B, 1)
        q_rot = torch.empty_like(q, device=DEV)
        G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), _ints(pos), _ints(length), None, *tab, q_rot)
        k_rot = R.rotary_embedding(_bits(k), np.array(pos))
        for b in range(B):
            held[b] = [(np.concatenate([kk, k_rot[b, :, g]]), np.concatenate([vv, _bits(v)[b, :, g]]))
                       for g, (kk, vv) in enumerate(held[b])]
            pos[b] += 1
            length[b] += 1
        out = torch.empty(B, 48, 128, dtype=torch.bfloat16, device=DEV)
        G.kv8_decode(cache, q_rot[:, 0], _ints(length), ws, out, weight, weight)
        if step % 23 == 0 or step == 69:
            got = out.float().cpu().numpy()
            x = bf16.to_f64(_bits(q_rot))[:, 0]
            exact = np.zeros((B, 48, 128))
            for b in range(B):
                for g in range(8):
                    K, V = (kv8.held(h, kind) for h in held[b][g])
                    exact[b, 6 * g:6 * g + 6], _ = kv8.attend(x[b, 6 * g:6 * g + 6], K, V)
            assert_close(_bits(out), bf16.from_f64(exact), f"conversation {kind} step {step}")
            assert np.isfinite(got).all()
        if step in (20, 55):
            keep = 4 if step == 20 else 2
            old, w = cache.table.clone(), weight.cpu().numpy()
            t_out, l_out = torch.empty_like(old), _ints(length)
            G.kv8_evict(old, weight, _ints(length), keep, 1, 1, t_out, weight, l_out)
            cache = cache.with_table(t_out)
            for b in range(B):
                for g in range(8):
                    t, _, m = kv8.evict(old[b, g].tolist(), w[b, g], length[b], keep, 1, 1)
                    assert t_out[b, g].tolist() == t
                    order = [old[b, g].tolist().index(x) for x in t[:(m + 63) // 64]]
                    held[b][g] = tuple(np.concatenate([h[64 * i:64 * i + 64] for i in order]) for h in held[b][g])
                    assert len(held[b][g][0]) == m
            length = l_out.tolist()
    del total


def test_a_captured_step_on_another_stream():
    """Append, decode and accumulation captured once and replayed with new inputs, on a side stream, equal the eager calls."""
    rng = np.random.default_rng(31)
    B, tab = 3, tables(512)
    lens = [100, 63, 300]
    cache, host = filled(rng, lens, "int8", 6, seed=21)
    twin = G.Kv8Cache(*(x.clone() for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale, cache.table,
                                            cache.open_k, cache.open_v)))
    ws, ws2 = G.alloc_kv8_decode_workspace(cache), G.alloc_kv8_decode_workspace(cache)
    q, k, v = (x.to(DEV) for x in rows(rng, B, 1))
    q_rot, out = torch.zeros_like(q), torch.zeros(B, 48, 128, dtype=torch.bfloat16, device=DEV)
    length, rows_now, weight = _ints(lens), _ints([n + 1 for n in lens]), torch.zeros(B, 8, 6, device=DEV)

    def step(c, w, x, o, wt, stream=None):
        G.kv8_append(c, q, k, v, length, length, None, *tab, x, stream=stream)
        G.kv8_decode(c, x[:, 0], rows_now, w, o, wt, wt, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache, ws, q_rot, out, weight)
    eager_x, eager_out, eager_w = torch.zeros_like(q), torch.zeros_like(out), torch.zeros_like(weight)
    for _ in range(4):
        q.copy_(rows(rng, B, 1)[0])
        k.copy_(rows(rng, B, 1)[1])
        v.copy_(rows(rng, B, 1)[2])
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step(twin, ws2, eager_x, eager_out, eager_w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, eager_out) and torch.equal(weight, eager_w) and torch.equal(q_rot, eager_x)
        length += 1
        rows_now += 1
    for a in ("k_pool", "v_pool"):
        assert torch.equal(getattr(cache, a).view(torch.uint8), getattr(twin, a).view(torch.uint8))


def test_captured_turns_that_share_workspaces():
    """A turn (12 and 3 tokens, a single one, an eviction in place) as two graphs over the same workspaces, by turns."""
    rng = np.random.default_rng(50)
    B, tab, keep = 2, tables(1024), 5
    cache, host = filled(rng, [400, 330], "e4m3", 8, seed=40)
    twin = G.Kv8Cache(*(x.clone() for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale, cache.table,
                                            cache.open_k, cache.open_v)))

    def state():
        return dict(pos=_ints([400, 330]), rows=_ints([400, 330]), next=_ints([0, 0]), weight=torch.zeros(B, 8, 8, device=DEV),
                    out=[torch.zeros(B, t, 48, 128, dtype=torch.bfloat16, device=DEV) for t in (12, 3, 1)],
                    status=torch.zeros(1, dtype=torch.int32, device=DEV))

    x = [[r.to(DEV) for r in rows(rng, B, t)] for t in (12, 3, 1)]
    rot = [torch.zeros_like(q) for q, _, _ in x]
    before = cache.table.clone()
    pre, dec = G.alloc_kv8_prefill_workspace(cache), G.alloc_kv8_decode_workspace(cache)

    def prompt(c, s):
        for i in (0, 1):
            G.kv8_append(c, *x[i], s["pos"], s["rows"], None, *tab, rot[i], s["status"])
            G.kv8_prefill(c, rot[i], s["rows"], None, s["out"][i], pre, s["status"])
            s["pos"] += x[i][0].shape[1]
            s["rows"] += x[i][0].shape[1]

    def answer(c, s):
        G.kv8_append(c, *x[2], s["pos"], s["rows"], None, *tab, rot[2], s["status"])
        s["pos"] += 1
        s["rows"] += 1
        G.kv8_decode(c, rot[2][:, 0], s["rows"], dec, s["out"][2][:, 0], s["weight"], s["weight"], s["status"])
        G.kv8_evict(c.table, s["weight"], s["rows"], keep, 1, 2, c.table, s["weight"], s["next"], s["status"])
        s["rows"].copy_(s["next"])

    mine, theirs = state(), state()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, call in zip(graphs, (prompt, answer)):
        with torch.cuda.graph(graph):
            call(cache, mine)
    for turn in range(3):
        for q, k, v in x:
            a, b, c = rows(rng, B, q.shape[1])
            q.copy_(a), k.copy_(b), v.copy_(c)
        for graph in graphs:
            graph.replay()
        prompt(twin, theirs)
        answer(twin, theirs)
        torch.cuda.synchronize()
        for name in ("pos", "rows", "weight", "status"):
            assert torch.equal(mine[name], theirs[name]), (turn, name)
        assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(mine["out"], theirs["out"]))
        assert torch.equal(cache.table, twin.table)
        assert int(mine["status"].item()) == 0 and mine["rows"].max().item() < (keep + 1) * 64
    assert not torch.equal(cache.table, before)


def test_readme_example_runs():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    scope = {}
    for block in re.findall(r"```python\n(.*?)```", text, re.S):
        exec(block, scope)  # noqa: S102
    torch.cuda.synchronize()
    assert int(scope["status"].item()) == 0
    assert scope["left"].tolist() == [48 * 64 + 1] and torch.isfinite(scope["out1"].float()).all()


def test_cache_tensors_are_fixed():
    cache = G.alloc_kv8_cache(1, 2)
    with pytest.raises(AttributeError, match="with_table"):
        cache.table = cache.table.clone()
    other = cache.table.flip(2).contiguous()
    assert cache.with_table(other).table is other and cache.with_table(other).k_pool is cache.k_pool
    with pytest.raises(ValueError, match="shape"):
        cache.with_table(other[:, :4].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        G.Kv8Cache(cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale, cache.table, cache.open_k.transpose(2, 3)
                   .contiguous().transpose(2, 3), cache.open_v)
