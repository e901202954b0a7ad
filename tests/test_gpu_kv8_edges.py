"""The 8-bit cache's calls at the ends of their ranges: magnitudes, workspaces, fallback, rows taken back."""
import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
from oracle import bf16, kv8
from tests.test_gpu_kv8 import (DEV, KINDS, Host, _bf16, _bits, _ints, append, check_cache, check_decode, filled,
                                make_cache, rows, run_decode, run_prefill, tables)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 3, 69])
def test_zero_keys_in_a_block_of_very_large_ones(kind, tokens):
    """Keys near 2^100, some exactly zero, queries near 2^60: the product of scale and query leaves fp32, the logits of
    the zero keys are 0 all the same and the others' are the cap."""
    rng = np.random.default_rng(1)
    L, tab = 70, tables(80)
    cache, host = make_cache(1, 2, kind, seed=1), Host(1)
    q, k, v = rows(rng, 1, L)
    k = (k.float() * 2.0 ** 100).bfloat16()
    k[0, 5:40] = 0
    append(cache, host, q, k, v, [0], [L], tab)
    x = _bf16(rng.standard_normal((1, tokens, 48, 128)) * 2.0 ** 60).to(DEV)
    if tokens == 1:
        got, _, status = run_decode(cache, x[:, 0].contiguous(), [L])
        got = got[:, None]
    else:
        got, status = run_prefill(cache, x, [L - tokens], None, tokens)
    assert status == 0
    out, scale_v = np.zeros((tokens, 48, 128)), np.zeros((tokens, 48, 128))
    y = bf16.to_f64(_bits(x[0]))
    for g in range(8):
        K, V = kv8.held(host.k[0][:, g], kind), kv8.held(host.v[0][:, g], kind)
        for h in range(6 * g, 6 * g + 6):
            out[:, h], w = kv8.attend(y[:, h], K, V, L - tokens + np.arange(tokens))
            scale_v[:, h] = w @ np.abs(V)
    assert torch.isfinite(got).all()
    # (every logit is 0 or far beyond the cap: none has an error of its own)
    check_decode(got[0], out, scale_v, 0.0, L, np.ones(tokens, bool))


def overflowing(kind, B, L, max_blocks, seed, first=0, v_of_the_key=None):
    """A cache whose items from sequence `first` on hold weights beyond fp16's range: a first tile of small logits and a
    later key at the cap (no rotation: it would keep q . k only at equal positions). v_of_the_key: that key's value."""
    rng = np.random.default_rng(seed)
    cache, host = make_cache(B, max_blocks, kind, seed=seed), Host(B)
    q, k, v = rows(rng, B, L)
    k[first:] = (k[first:].float() * 0.02).bfloat16()
    q[first:] = q[first:, L - 100, :1][:, None].expand(-1, L, 48, -1)
    k[first:, L - 100] = q[first:, L - 100, :1].expand(-1, 8, -1)
    if v_of_the_key is not None:
        v[first:, L - 100] = v_of_the_key
    tab = tables(L)
    tab = (torch.ones_like(tab[0]), torch.zeros_like(tab[1]))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_rot = torch.zeros_like(q, device=DEV)
    zero = _ints([0] * B)
    G.kv8_append(cache, q.to(DEV), k.to(DEV), v.to(DEV), zero, zero, None, *tab, q_rot, status)
    assert int(status.item()) == 0 and torch.equal(q_rot.cpu(), q)
    for b in range(B):
        host.k[b], host.v[b] = _bits(k)[b], _bits(v)[b]
    return cache, host, q_rot


def check_overflowing(host, q_rot, got, kind, picks, heads=(0, 7, 47)):
    """Half a step of the result, 2^-8; of V 2^-8; a weight's approximate functions 3e-4 and its logit, 128 * 2^-23 of the
    sum of the magnitudes, in the sum too; fp16 weights 2^-11, and 2^-10 of the sum for all small ones."""
    x, y = bf16.to_f64(_bits(q_rot)), got.float().cpu().numpy().astype(np.float64)
    for b in range(len(host.k)):
        for h in heads:
            K, V = kv8.held(host.k[b][:, h // 6], kind), kv8.held(host.v[b][:, h // 6], kind)
            o, w = kv8.attend(x[b, picks, h], K, V, np.array(picks))
            logit = 128 * 2.0 ** -23 * (np.abs(x[b, picks, h]) @ np.abs(K).T).max() / 128 ** 0.5
            rel = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -10 + 2 * (3e-4 + logit)
            assert (np.abs(y[b, picks, h] - o) <= 2.0 ** -8 * np.abs(o) + rel * (w @ np.abs(V))).all(), (b, h)


@pytest.mark.parametrize("kind", KINDS)
def test_fallback_touches_the_rows_of_the_call_alone(kind):
    """Two sequences of 300 rows with room for 32768: the workspace behind their copies keeps its bytes."""
    B, L, max_blocks = 2, 300, 512
    cache, host, q_rot = overflowing(kind, B, L, max_blocks, 3, first=1)
    out = torch.empty_like(q_rot)
    ws = G.alloc_kv8_prefill_workspace(cache)
    ws.fill_(0xff)  # as fp16 a NaN, which a conversion to bf16 would write as another one
    G.kv8_prefill(cache, q_rot, _ints([0] * B), None, out, ws)
    copies = 2 * B * 8 * 384 * 128 * 2  # K and V, rows up to the next 128
    assert int((ws != 0xff).sum()) <= copies + (1 << 16)
    check_overflowing(host, q_rot, out, kind, [0, 100, 199, 200, 250, 299])


@pytest.mark.parametrize("kind", KINDS)
def test_fallback_where_the_large_keys_value_is_zero(kind):
    """An infinite weight is seen in the outputs also where it meets zeros."""
    cache, host, q_rot = overflowing(kind, 2, 300, 8, 6, v_of_the_key=0.0)
    got, status = run_prefill(cache, q_rot, [0, 0], None, 300)
    assert status == 0 and torch.isfinite(got).all()
    check_overflowing(host, q_rot, got, kind, [0, 100, 199, 200, 250, 299])
    ck, cv = (torch.from_numpy(np.stack(x).view(np.int16)).view(torch.bfloat16).to(DEV) for x in (host.k, host.v))
    out, want = torch.empty_like(q_rot), torch.empty_like(q_rot)
    G.prefill_ws(q_rot, ck, cv, _ints([0, 0]), None, out, G.alloc_prefill_workspace(2, 300))
    G.prefill(q_rot, ck, cv, _ints([0, 0]), None, want)
    assert torch.equal(out[:, 200:], want[:, 200:])


def test_fallback_lists_an_item_once():
    """The items of rows 128 to 299 of every sequence overflow (key 200 is at the cap): each is computed again once. The
    workspace begins with their number (prefill_ws: behind a flag for each sequence)."""
    B, L = 4, 300
    cache, host, q_rot = overflowing("int8", B, L, 8, 4)
    out, ws = torch.empty_like(q_rot), G.alloc_kv8_prefill_workspace(cache)
    zero = _ints([0] * B)
    G.kv8_prefill(cache, q_rot, zero, None, out, ws)
    assert int(ws.view(torch.int32)[0]) == B * 2 * 24
    check_overflowing(host, q_rot, out, "int8", [0, 199, 200, 299])
    ck, cv = (torch.from_numpy(np.stack(x).view(np.int16)).view(torch.bfloat16).to(DEV) for x in (host.k, host.v))
    ws = G.alloc_prefill_workspace(B, L)
    G.prefill_ws(q_rot, ck, cv, zero, None, out, ws)
    assert int(ws.view(torch.int32)[B]) == B * 2 * 24


def test_a_workspace_serves_every_smaller_cache():
    """Sizes do not fall with the number of sequences or blocks; a call over 36 blocks in the workspace for 64."""
    Bs, blocks = [*range(1, 20), 31, 32, 33, 64, 100, 256], [*range(1, 41), 64, 100, 128, 511, 512, 1024]
    for size in (G.kv8_prefill_workspace, G.kv8_decode_workspace):
        n = np.array([[size(B, m) for m in blocks] for B in Bs])
        assert (np.diff(n, axis=0) >= 0).all() and (np.diff(n, axis=1) >= 0).all(), size.__name__
    rng = np.random.default_rng(5)
    cache, host = filled(rng, [300], "int8", 36, seed=5)
    q = _bf16(rng.standard_normal((1, 90, 48, 128))).to(DEV)
    want, _ = run_prefill(cache, q, [210], None, 90)
    ws = torch.empty(G.kv8_prefill_workspace(1, 64), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    G.kv8_prefill(cache, q, _ints([210]), None, out, ws)
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("many", [False, True])
def test_rows_taken_back_to_a_blocks_start(kind, many):
    """Lengths set back to a multiple of 64, from inside the block and from a later one: the next rows make the cache that
    they alone would have made, with scales that the dropped rows, larger ones, had raised. (64 and more sequences: single
    tokens by their own kernel.)"""
    rng = np.random.default_rng(8)
    B, tab = (65, tables(400)) if many else (3, tables(400))
    cache, host = make_cache(B, 5, kind, seed=8), Host(B)
    append(cache, host, *rows(rng, B, 100), [0] * B, [100] * B, tab)
    q, k, v = rows(rng, B, 130)
    append(cache, host, q, (k.float() * 50).bfloat16(), (v.float() * 50).bfloat16(), [100] * B, [130] * B, tab)
    for b in range(B):  # 230 rows: back to 64, to 192 or to nothing
        keep = (64, 192, 0)[b % 3]
        host.k[b], host.v[b] = host.k[b][:keep], host.v[b][:keep]
    for T in (1, 1, 40, 1, 30) if not many else (1, 1, 1):
        append(cache, host, *rows(rng, B, T), [len(x) for x in host.k], [T] * B, tab)
    for b in range(B if not many else 4):
        L = len(host.k[b])
        for g in range(8):
            for pool, scale, held_rows in ((cache.k_pool, cache.k_scale, host.k[b]), (cache.v_pool, cache.v_scale, host.v[b])):
                for i, (codes, s) in enumerate(kv8.blocks(held_rows[:, g], kind)):
                    at = int(cache.table[b, g, i])
                    got = pool[at].view(torch.uint8).cpu().numpy()
                    got = np.concatenate([got[0], got[1]], 1) if pool is cache.k_pool else got.T
                    assert np.float32(scale[at].item()) == s and np.array_equal(got[:len(codes)], codes), (b, g, i)
    lens = [len(x) for x in host.k]
    q = _bf16(rng.standard_normal((B, 48, 128)) * 3).to(DEV)
    out, _, status = run_decode(cache, q, lens, weights=False)
    assert status == 0 and torch.isfinite(out).all()


@pytest.mark.parametrize("T,start", [(2200, 0), (200, 2300)])
def test_non_finite_blocks_among_the_sampled_keys(T, start):
    """Rows 1664 to 1791 are a key tile that rows' references look at ahead of the rest (whole items, and parts of items):
    a block of it without finite values is NaN for the rows that see it, and nothing to the others."""
    rng = np.random.default_rng(9)
    L = start + T
    cache, _ = filled(rng, [L], "int8", 40, seed=9)
    q = _bf16(rng.standard_normal((1, T, 48, 128)) * 3).to(DEV)
    good, status = run_prefill(cache, q, [start], None, T)
    assert status == 0 and torch.isfinite(good).all()
    for scale in (cache.k_scale, cache.v_scale):
        at = cache.table[0, 2, 27].long()
        saved = scale[at].clone()
        scale[at] = float("nan")
        got, _ = run_prefill(cache, q, [start], None, T)
        scale[at] = saved
        want = torch.zeros(1, T, 48, dtype=torch.bool, device=DEV)
        want[0, max(0, 64 * 27 - start):, 12:18] = True
        assert torch.equal(torch.isnan(got).all(-1), want) and torch.equal(got[~want], good[~want])


@pytest.mark.parametrize("kind", KINDS)
def test_outputs_of_flat_peaked_and_unequal_logits_are_finite(kind, monkeypatch):
    """The cases of those tests again: a comparison with a NaN is false, so their bound alone lets one pass."""
    from tests import test_gpu_kv8 as T

    def strict(got, out, scale_v, s_abs, L, live):
        assert torch.isfinite(got[torch.from_numpy(live).to(got.device)]).all()
        check_decode(got, out, scale_v, s_abs, L, live)

    monkeypatch.setattr(T, "check_decode", strict)
    for scale in (1e-6, 0.02, 8.0):
        T.test_decode_flat_and_peaked_logits(kind, scale)
        T.test_prefill_of_few_tokens_flat_and_peaked_logits(kind, scale)
    T.test_prefill_of_few_tokens_flat_and_peaked_logits(kind, "unequal")
    T.test_decode_unequal_query_heads()
    T.test_decode_bad_lengths_leave_the_outputs()
