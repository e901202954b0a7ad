"""The 8-bit cache's calls refuse bad arguments before any device call (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from grok_gqa_attention_gb300 import build
    build.build()
    import grok_gqa_attention_gb300 as G
    return G.load()


A = 1 << 20  # an aligned address that nothing dereferences


def _cache(**kw):
    from grok_gqa_attention_gb300.kv8 import _Cache
    f = dict(k_pool=A, v_pool=A, k_scale=A, v_scale=A, table=A, open_k=A, open_v=A, kind=0, B=2, max_blocks=4, n_blocks=64)
    f.update(kw)
    return ctypes.byref(_Cache(*f.values()))


def _append(lib, cache=None, q=A, k=A, v=A, start=A, length=A, valid=None, T=4, cos=A, sin=A, n=128, q_rot=2 * A):
    return lib.grok_kv8_append(_cache() if cache is None else cache, q, k, v, start, length, valid, T, cos, sin, n, q_rot,
                               None, None)


def _decode(lib, cache=None, q=A, length=A, ws=A, nbytes=1 << 30, out=A, w_in=None, w_out=None):
    return lib.grok_kv8_decode(_cache() if cache is None else cache, q, length, ws, nbytes, out, w_in, w_out, None, None)


def _evict(lib, table=A, w=A, length=A, B=2, n=4, keep=2, sink=0, recent=0, t_out=A, w_out=A, l_out=2 * A):
    return lib.grok_kv8_evict(table, w, length, B, n, keep, sink, recent, t_out, w_out, l_out, None, None)


def _prefill(lib, cache=None, q=A, length=A, valid=None, T=4, out=2 * A, ws=A, nbytes=1 << 40):
    return lib.grok_kv8_prefill(_cache() if cache is None else cache, q, length, valid, T, out, ws, nbytes, None, None)


BAD_CACHES = [dict(k_pool=None), dict(v_pool=None), dict(k_scale=None), dict(v_scale=None), dict(table=None),
              dict(open_k=None), dict(open_v=None), dict(k_pool=A + 8), dict(open_v=A + 2), dict(table=A + 4),
              dict(kind=2), dict(kind=-1), dict(B=0), dict(B=65536), dict(max_blocks=0), dict(max_blocks=1025),
              dict(n_blocks=0)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad):
    assert _append(lib, _cache(**bad)) == 1
    assert _decode(lib, _cache(**bad)) == 1
    assert _prefill(lib, _cache(**bad)) == 1


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=None), dict(start=None), dict(length=None),
                                 dict(cos=None), dict(sin=None), dict(q_rot=None), dict(q=A + 8), dict(q_rot=A),
                                 dict(sin=A + 4), dict(T=0), dict(T=65537), dict(n=0), dict(n=65537)], ids=str)
def test_bad_appends(lib, bad):
    assert _append(lib, **bad) == 1
    assert b"grok_kv8_append" in lib.grok_last_error()


@pytest.mark.parametrize("bad", [dict(q=None), dict(length=None), dict(ws=None), dict(out=None), dict(q=A + 8),
                                 dict(out=A + 8), dict(ws=A + 16), dict(w_in=A)], ids=str)
def test_bad_decodes(lib, bad):
    assert _decode(lib, **bad) == 1
    assert b"grok_kv8_decode" in lib.grok_last_error()


@pytest.mark.parametrize("bad", [dict(q=None), dict(length=None), dict(ws=None), dict(out=None), dict(q=A + 8),
                                 dict(out=A + 8), dict(out=A), dict(ws=A + 16), dict(T=0), dict(T=257)], ids=str)
def test_bad_prefills(lib, bad):
    assert _prefill(lib, **bad) == 1
    assert b"grok_kv8_prefill" in lib.grok_last_error()


@pytest.mark.parametrize("bad", [dict(table=None), dict(w=None), dict(length=None), dict(t_out=None), dict(w_out=None),
                                 dict(l_out=None), dict(l_out=A), dict(B=0), dict(B=65536), dict(n=0), dict(n=1025),
                                 dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=2, recent=1)], ids=str)
def test_bad_evictions(lib, bad):
    assert _evict(lib, **bad) == 1
    assert b"grok_kv8_evict" in lib.grok_last_error()


def test_null_cache_and_workspace_sizes(lib):
    assert lib.grok_kv8_append(None, A, A, A, A, A, None, 1, A, A, 1, 2 * A, None, None) == 1
    n = ctypes.c_size_t(0)
    assert lib.grok_kv8_decode_workspace(0, 4, 0, ctypes.byref(n)) == 1
    assert lib.grok_kv8_decode_workspace(1, 1025, 0, ctypes.byref(n)) == 1
    assert lib.grok_kv8_decode_workspace(1, 4, 0, None) == 1
    assert lib.grok_kv8_prefill_workspace(0, 4, ctypes.byref(n)) == 1
    assert lib.grok_kv8_prefill_workspace(65535, 1024, ctypes.byref(n)) == 1
    assert lib.grok_kv8_prefill_workspace(1, 4, None) == 1


def test_binding_constants_and_cpu_tensors():
    import os
    import re

    import grok_gqa_attention_gb300 as G
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "grok_attn.h")).read()
    defines = {m.group(1): int(m.group(2)) for m in re.finditer(r"^#define GROK_(KV8_\w+) (\d+)\b", text, re.M)}
    assert defines == {"KV8_BLOCK": G.KV8_BLOCK, "KV8_INT8": G.KV8_INT8, "KV8_E4M3": G.KV8_E4M3}
    B, n, m = 1, 16, 2
    args = dict(k_pool=torch.zeros(n, 2, 64, 64, dtype=torch.int8), v_pool=torch.zeros(n, 128, 64, dtype=torch.int8),
                k_scale=torch.zeros(n), v_scale=torch.zeros(n), table=torch.zeros(B, 8, m, dtype=torch.int32),
                open_k=torch.zeros(B, 8, 64, 128, dtype=torch.bfloat16),
                open_v=torch.zeros(B, 8, 64, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.Kv8Cache(**args)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        G.Kv8Cache(**{**args, "k_pool": args["k_pool"].float()})
    with pytest.raises(ValueError, match="table"):
        G.Kv8Cache(**{**args, "table": args["table"][0]})
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.kv8_evict(args["table"], torch.zeros(B, 8, m), torch.zeros(B, dtype=torch.int32), 1, 0, 0, args["table"],
                    torch.zeros(B, 8, m), torch.zeros(B, dtype=torch.int32))
