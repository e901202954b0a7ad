"""Rows whose softmax has a few large weights in the first keys and most of its mass in thousands of small ones.

The usual case in use: the first keys of a sequence draw attention far above the rest, and the rest is nearly flat.
A weight of the rest is 2^-13 to 2^-23 of the largest one, yet together they are a few percent to half of the row.
"""
import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
from oracle import bf16, kv8

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
KINDS = ("int8", "e4m3")
MULT = 128 ** -0.5

# How far the rest lies below the first keys' capped logit, and the deviation of its logits (nats).
TAILS = {"9.2": (9.2, 0.0), "10.3": (10.3, 0.0), "11.9": (11.9, 0.0), "13 spread": (13.0, 1.0)}
SINK = 22.0  # capped logit of the first keys


def raw(c):
    """The logit before the cap."""
    return 30.0 * np.arctanh(np.asarray(c) / 30.0)


def levels(n, tail, n_sinks, late=None):
    """Logits before the cap of n keys: n_sinks large ones, then the rest; key `late` is at the cap."""
    below, spread = TAILS[tail]
    c = SINK - below + spread * np.random.default_rng(n).standard_normal(n)
    c[:n_sinks] = SINK
    x = raw(np.clip(c, -25, SINK))
    if late is not None:
        x[late] = 200.0
    return x


def values(n, rng):
    """V whose mean is not zero, and other in the first keys than in the rest."""
    v = 1.0 + rng.standard_normal((n, 128)) * 0.25
    v[:4] = -1.0
    return v


def check(got, x, K, V, last, what, v_rounding):
    """got [n, 6, 128] against fp64, queries x over K, V. The tolerance: half a bf16 step of the result (2^-8); a weight's
    relative error in the numerator and in the sum: fp16 rounding (2^-11, numerator only), tanh and exp2 (tanh.approx is
    off by 8e-6 at most, times 30; 3e-4 in all) and a 128-term fp32 sum of the logit; the rounding of V; and what
    weights below fp16's normal range lose, which must not grow with the number of keys: 2^-10 of the row's sum, at
    mean |V|."""
    s_abs = (np.abs(x).reshape(-1, 128) @ np.abs(K).T).max() * MULT
    for h in range(6):
        o, w = kv8.attend(x[:, h], K, V, last)
        rel = 2.0 ** -11 + 2 * (3e-4 + 128 * 2.0 ** -23 * s_abs) + v_rounding
        tol = 2.0 ** -8 * np.abs(o) + rel * (w @ np.abs(V)) + 2.0 ** -10 * np.abs(V).mean(0)
        bad = np.abs(got[:, h] - o) / tol
        assert bad.max() <= 1.0, (what, h, float(bad.max()))


# ------------------------------------------------------------------------------------------- 8-bit cache
def cache8(kind, n, max_blocks, tail, late=None):
    """A cache whose keys are constant over the features, so a query of ones meets the logits of levels(); codes and
    scales are written here, as an append would leave them. n_sinks: four."""
    rng = np.random.default_rng(7)
    x = levels(n, tail, 4, late) / (128 * MULT)  # key values, for a query of ones
    blocks = -(-n // 64)
    xp = np.concatenate([x, np.zeros(blocks * 64 - n)]).reshape(blocks, 64)
    vp = np.concatenate([values(n, rng), np.zeros((blocks * 64 - n, 128))]).reshape(blocks, 64, 128)
    top = kv8.TOP[kind]

    def codes(y):  # [blocks, 64, 128] -> codes of the tensor's type, scales
        s = torch.from_numpy(np.abs(y).max((1, 2)) / top).float()
        z = torch.from_numpy(y).float() / s[:, None, None]
        return (torch.round(z).to(torch.int8) if kind == "int8" else z.to(torch.float8_e4m3fn)), s

    kc, ks = codes(np.repeat(xp[:, :, None], 128, 2))
    vc, vs = codes(vp)
    k1 = kc.view(torch.uint8).view(blocks, 64, 2, 64).transpose(1, 2).contiguous().to(DEV)
    v1 = vc.view(torch.uint8).transpose(1, 2).contiguous().to(DEV)
    open_ = torch.zeros(1, 8, 64, 128, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, 8, max_blocks, dtype=torch.int32, device=DEV)
    table[..., :blocks] = torch.arange(blocks, dtype=torch.int32, device=DEV)  # the heads share the blocks
    cache = G.Kv8Cache(k1.view(DT[kind]), v1.view(DT[kind]), ks.to(DEV), vs.to(DEV), table, open_, open_.clone())
    K = (kc.double() * ks.double()[:, None, None]).reshape(-1, 128)[:n].numpy()
    V = (vc.double() * vs.double()[:, None, None]).reshape(-1, 128)[:n].numpy()
    return cache, K, V


def queries(B, T):
    """Ones, each head a little larger or smaller."""
    size = torch.linspace(0.97, 1.0, 48)[None, None, :, None]
    return (torch.ones(B, T, 48, 128) * size).bfloat16().to(DEV)


def picks(T):
    return np.array(sorted({0, 1, T // 3, T // 2, T - 129 if T > 129 else 0, T - 1}))


def run_prefill8(cache, q, start, T):
    out = torch.full_like(q, 7.0)
    ws = G.alloc_kv8_prefill_workspace(cache)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([start], dtype=torch.int32, device=DEV)
    G.kv8_prefill(cache, q, lens, None, out, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


# rows before the call, tokens, capacity in blocks: few tokens on the codes, items split over the key range, whole
# items (more than two for each SM), one key tile past the sampled ones, a prompt in an empty cache
SHAPES8 = {
    "few": (8176, 16, 160),
    "split": (8000, 192, 128),
    "whole": (6200, 1992, 128),
    "prompt": (0, 2100, 40),
    "short": (300, 300, 10),
    "longest few": (65520, 16, 1024),
    "longest split": (65496, 40, 1024),
    "longest whole": (63736, 1800, 1024),
}


@pytest.mark.parametrize("tail", list(TAILS))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", list(SHAPES8))
def test_kv8_prefill(shape, kind, tail):
    start, T, max_blocks = SHAPES8[shape]
    cache, K, V = cache8(kind, start + T, max_blocks, tail)
    q = queries(1, T)
    got = run_prefill8(cache, q, start, T).float().cpu().numpy().astype(np.float64)
    rows = picks(T)
    x = bf16.to_f64(q[0].cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    for g in (0, 7):
        check(got[0, rows, 6 * g:6 * g + 6], x[rows, 6 * g:6 * g + 6], K, V, start + rows, f"{shape} {kind} {tail}",
              2.0 ** -11)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", ["split", "whole", "longest split", "longest whole"])
def test_kv8_prefill_with_a_late_key_at_the_cap(shape, kind):
    """A key behind the first ones that rises 8 nats above them, and rows that do not see it. (V is rounded to bf16
    where an item is computed again: 2^-8.)"""
    start, T, max_blocks = SHAPES8[shape]
    n = start + T
    cache, K, V = cache8(kind, n, max_blocks, "10.3", late=n - 33)
    q = queries(1, T)
    got = run_prefill8(cache, q, start, T).float().cpu().numpy().astype(np.float64)
    rows = picks(T)
    x = bf16.to_f64(q[0].cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    check(got[0, rows, :6], x[rows, :6], K, V, start + rows, f"{shape} {kind} late", 2.0 ** -8)


@pytest.mark.parametrize("tail", list(TAILS))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [300, 8200, 65536])
def test_kv8_decode(kind, tail, n):
    """One token: as above, but for V, whose codes are exact there."""
    cache, K, V = cache8(kind, n, 1024, tail)
    q = queries(1, 1)[:, 0].contiguous()
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    G.kv8_decode(cache, q, torch.tensor([n], dtype=torch.int32, device=DEV), G.alloc_kv8_decode_workspace(cache, False),
                 out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = out.float().cpu().numpy().astype(np.float64)
    x = bf16.to_f64(q.cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    for g in (0, 7):
        check(got[:, 6 * g:6 * g + 6], x[:, 6 * g:6 * g + 6], K, V, np.array([n - 1]), f"decode {kind} {tail} {n}", 0.0)


# ------------------------------------------------------------------------------------------- bf16 cache
SHAPES16 = {
    "split": (8000, 192, 8192),
    "whole": (6200, 1992, 8192),
    "prompt": (0, 2100, 2560),
    "short": (300, 300, 640),
    "longest split": (65408, 128, 65536),
    "longest whole": (63736, 1800, 65536),
}


@pytest.mark.parametrize("tail", list(TAILS))
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES16))
def test_prefill_ws(shape, paged, tail):
    start, T, rows_max = SHAPES16[shape]
    n = start + T
    k = torch.from_numpy(np.repeat((levels(n, tail, 4) / (128 * MULT))[:, None], 128, 1)).bfloat16()
    v = torch.from_numpy(values(n, np.random.default_rng(8))).bfloat16()
    ck, cv = (torch.zeros(1, rows_max, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ck[0, :n], cv[0, :n] = k.to(DEV)[:, None], v.to(DEV)[:, None]
    q = queries(1, T)
    out = torch.full_like(q, 7.0)
    lens = torch.tensor([start], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = G.alloc_prefill_workspace(1, rows_max)
    if paged:
        pages = rows_max // 128
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(DEV)
        pool_k, pool_v = (torch.empty(pages, 128, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        pool_k[order], pool_v[order] = ck.view(pages, 128, 8, 128), cv.view(pages, 128, 8, 128)
        G.prefill_ws_paged(q, pool_k, pool_v, order.to(torch.int32)[None].contiguous(), lens, None, out, ws, status)
    else:
        G.prefill_ws(q, ck, cv, lens, None, out, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = out.float().cpu().numpy().astype(np.float64)
    rows = picks(T)
    x = bf16.to_f64(q[0].cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    K, V = k.double().numpy(), v.double().numpy()
    for g in (0, 7):
        check(got[0, rows, 6 * g:6 * g + 6], x[rows, 6 * g:6 * g + 6], K, V, start + rows, f"{shape} {tail}", 2.0 ** -11)


@pytest.mark.parametrize("kind", KINDS)
def test_kv8_decode_of_many_long_caches_keeps_the_smallest_weights(kind):
    """256 sequences, so that a warp reads a head's whole range: one key 17.4 nats above 65535 equal ones, each 2^-25.1
    of it, together 0.18 % of the sum. The 128 outputs' mean difference from the rounded exact ones shows what a bf16
    step hides: without the small weights it is about -1.8e-3. The weights' own errors (tanh and exp2 at 3 * 87 * 2^-20,
    a 128-term fp32 logit) move the large key's share by less than 2e-6; ten outputs next to a midpoint that round the
    other way are 10 * 2^-8 / 128 = 3e-4."""
    B, n = 256, 65536
    rng = np.random.default_rng(9)
    c = np.full(n, SINK - 17.4)
    c[0] = SINK
    x = raw(c) / (128 * MULT)
    vp = 1.0 + rng.standard_normal((n, 128)) * 0.25
    vp[0] = -1.0 + rng.standard_normal(128) * 0.25
    top = kv8.TOP[kind]

    def codes(y):
        s = torch.from_numpy(np.abs(y).max((1, 2)) / top).float()
        z = torch.from_numpy(y).float() / s[:, None, None]
        return (torch.round(z).to(torch.int8) if kind == "int8" else z.to(torch.float8_e4m3fn)), s

    xb = np.repeat(x.reshape(-1, 64, 1), 128, 2)
    xb[0, 1:] = xb[1, 0]
    kc, ks = codes(xb)
    vc, vs = codes(vp.reshape(-1, 64, 128))
    k1 = kc.view(torch.uint8).view(-1, 64, 2, 64).transpose(1, 2).contiguous().to(DEV)
    v1 = vc.view(torch.uint8).transpose(1, 2).contiguous().to(DEV)
    open_ = torch.zeros(B, 8, 64, 128, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(1024, dtype=torch.int32, device=DEV).expand(B, 8, 1024).contiguous()  # all share the blocks
    cache = G.Kv8Cache(k1.view(DT[kind]), v1.view(DT[kind]), ks.to(DEV), vs.to(DEV), table, open_, open_.clone())
    q = torch.ones(B, 48, 128, dtype=torch.bfloat16, device=DEV)  # (all heads alike)
    out = torch.full_like(q, 7.0)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    G.kv8_decode(cache, q, lens, G.alloc_kv8_decode_workspace(cache, False), out)
    K = (kc.double() * ks.double()[:, None, None]).reshape(-1, 128).numpy()
    V = (vc.double() * vs.double()[:, None, None]).reshape(-1, 128).numpy()
    qx = bf16.to_f64(q[0].cpu().contiguous().view(torch.int16).numpy().view(np.uint16))
    o, w = kv8.attend(qx, K, V)
    assert 1.2e-3 < 1 - w[:, 0].min() < 2.5e-3
    delta = (out.float().cpu().numpy().astype(np.float64) - bf16.to_f64(bf16.from_f64(o))[None]).mean()
    assert abs(delta) < 3e-4, float(delta)
