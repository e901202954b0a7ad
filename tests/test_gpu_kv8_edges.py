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
