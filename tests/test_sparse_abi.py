"""The calls that read part of a paged cache refuse bad arguments before any device call (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

A = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    from grok_gqa_attention_gb300 import build
    build.build()
    import grok_gqa_attention_gb300 as G
    return G.load()


def _bounds(lib, k=A, n=8, table=A, mp=4, start=A, valid=None, B=2, T=1, codes=A, scale=A):
    return lib.grok_kv_bounds_paged(k, n, table, mp, start, valid, B, T, codes, scale, None, None)


def _select(lib, q=A, codes=A, scale=A, n=8, table=A, mp=4, length=A, B=2, budget=4, sink=1, recent=1, score=A, sel=A):
    return lib.grok_attn_select_paged(q, codes, scale, n, table, mp, length, B, budget, sink, recent, score, sel, None, None)


def _sparse(lib, q=A, k=A, v=A, n=8, table=A, mp=4, length=A, sel=A, budget=4, B=2, ws=A, nbytes=1 << 40, out=A):
    return lib.grok_attn_decode_sparse_paged(q, k, v, n, table, mp, length, sel, budget, B, ws, nbytes, out, None, None)


def _shared(lib, q=A, k=A, v=A, n=8, table=A, mp=4, length=A, B=2, start=A, pages=A, groups=1, ws=A, nbytes=1 << 40, out=A):
    return lib.grok_attn_decode_shared_paged(q, k, v, n, table, mp, length, B, start, pages, groups, ws, nbytes, out, None,
                                             None)


SIZES = [dict(n=0), dict(n=1 << 24), dict(mp=0), dict(mp=513), dict(B=0), dict(B=65536)]
BAD = {_bounds: [dict(k=None), dict(table=None), dict(start=None), dict(codes=None), dict(scale=None), dict(k=A + 8),
                 dict(codes=A + 8), dict(T=0), dict(T=513)],
       _select: [dict(q=None), dict(codes=None), dict(scale=None), dict(table=None), dict(length=None), dict(score=None),
                 dict(sel=None), dict(q=A + 8), dict(codes=A + 4), dict(budget=0), dict(budget=1025), dict(sink=-1),
                 dict(recent=-1), dict(sink=3, recent=2)],
       _sparse: [dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(length=None), dict(sel=None),
                 dict(ws=None), dict(out=None), dict(q=A + 2), dict(k=A + 8), dict(v=A + 8), dict(out=A + 8),
                 dict(ws=A + 16), dict(budget=0), dict(budget=1025)],
       _shared: [dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(length=None), dict(start=None),
                 dict(pages=None), dict(ws=None), dict(out=None), dict(q=A + 2), dict(k=A + 8), dict(v=A + 8),
                 dict(out=A + 8), dict(ws=A + 16), dict(groups=0), dict(groups=257)]}


@pytest.mark.parametrize("call,bad", [(c, b) for c, bads in BAD.items() for b in bads + SIZES],
                         ids=lambda x: x.__name__ if callable(x) else str(x))
def test_bad_arguments(lib, call, bad):
    assert call(lib, **bad) == 1
    assert lib.grok_last_error()


def test_bad_workspace_questions(lib):
    n = ctypes.c_size_t(0)
    assert lib.grok_attn_decode_sparse_workspace(2, 4, None) == 1
    assert lib.grok_attn_decode_shared_workspace(2, 4, 1, None) == 1
    for B, budget in ((0, 4), (65536, 4), (2, 0), (2, 1025)):
        assert lib.grok_attn_decode_sparse_workspace(B, budget, ctypes.byref(n)) == 1
    for B, mp, groups in ((0, 4, 1), (65536, 4, 1), (2, 0, 1), (2, 513, 1), (2, 4, 0), (2, 4, 257)):
        assert lib.grok_attn_decode_shared_workspace(B, mp, groups, ctypes.byref(n)) == 1


def test_binding_constants():
    import grok_gqa_attention_gb300 as G
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "grok_attn.h")).read()
    defines = {m.group(1): int(m.group(2), 0) for m in re.finditer(r"^#define (GROK_\w+) (0x[0-9a-fA-F]+|\d+)\b", text, re.M)}
    for name in ("DEV_BAD_BLOCK", "DEV_BAD_GROUP", "SPARSE_BLOCK"):
        assert getattr(G, name) == defines["GROK_" + name]


def test_binding_refuses_cpu_tensors():
    import grok_gqa_attention_gb300 as G
    q, pool = torch.zeros(2, 48, 128, dtype=torch.bfloat16), torch.zeros(4, 128, 8, 128, dtype=torch.bfloat16)
    table, one = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    codes, scale = G.alloc_kv_bounds(4, "cpu")
    sel, ws = torch.zeros(2, 8, 2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    calls = [lambda: G.kv_bounds_paged(pool, table, one, None, 1, codes, scale),
             lambda: G.select_blocks_paged(q, codes, scale, table, one, 0, 0, torch.zeros(2, 8, 4), sel),
             lambda: G.decode_sparse_paged(q, pool, pool, table, one, sel, ws, q),
             lambda: G.decode_shared_paged(q, pool, pool, table, one, one, one[:1], ws, q)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_the_extension_hands_back_what_it_does_not_take(lib):
    """Whatever is not a call as it should be comes back as None, without an error left over and without references kept."""
    import sys

    from grok_gqa_attention_gb300 import sparse
    m = sparse._binding()
    q, pool = torch.zeros(2, 48, 128, dtype=torch.bfloat16), torch.zeros(4, 128, 8, 128, dtype=torch.bfloat16)
    table, one, ws = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    codes, scale = torch.zeros(4, 2, 8, 2, 128, dtype=torch.int8), torch.zeros(4, 2, 8)
    sel, score = torch.zeros(2, 8, 2, dtype=torch.int32), torch.zeros(2, 8, 4)
    calls = {"kv_bounds_paged": (pool, table, one, None, 1, codes, scale, None, None),
             "select_blocks_paged": (q, codes, scale, table, one, 0, 0, score, sel, None, None),
             "decode_sparse_paged": (q, pool, pool, table, one, sel, ws, q, None, None),
             "decode_shared_paged": (q, pool, pool, table, one, one, one[:1], ws, q, None, None)}
    odd = [None, 3, 2 ** 70, 1.5, "x", [], object(), torch.zeros(3), torch.zeros(2, 2, 2, 2, 2, 2), torch.Size([1]),
           torch.zeros(2, 48, 128, dtype=torch.bfloat16, device="meta")]
    kept = [q, pool, table, one, ws, codes, scale, sel, score] + odd[5:]
    before = [sys.getrefcount(y) for y in kept]
    for name, args in calls.items():
        f = getattr(m, name)
        assert f() is None and f(*args) is None and f(*args, None) is None  # (CPU tensors)
        for i in range(len(args)):
            for x in odd:
                assert f(*args[:i], x, *args[i + 1:]) is None
    del x  # (the loop's own reference)
    assert [sys.getrefcount(y) for y in kept] == before
    with pytest.raises(TypeError):
        m.bind(1)
