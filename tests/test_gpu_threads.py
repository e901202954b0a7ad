"""Calls from host threads that have made no other CUDA call, and from several threads at once."""
import threading

import numpy as np
import pytest
import torch

import grok_gqa_attention_gb300 as G
from tests.test_gpu_sparse import DEV, grouped, ints, lists, queries, status

pytestmark = pytest.mark.gpu


def in_thread(call):
    """The call in a thread of its own; what it raised is raised here."""
    raised = []

    def body():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if raised:
        raise raised[0]


def calls():
    """(name, function of an output and a stream, the output's shape): calls whose kernels load by tensor maps, and others."""
    paged, starts = grouped([6], [2], lambda i: 100 * i, seed=80)
    B, T = 6, paged.max_pages * 128
    k, v, table = paged.dev()
    k.nan_to_num_(0.5)
    v.nan_to_num_(0.5)
    q, lens, sel = queries(B, 81).to(DEV), ints(paged.lens), ints(lists(paged.lens, 5, seed=82))
    zero, st = ints([0] * B), status()
    q4 = q.view(B, 1, 48, 128)
    ws = {"decode": G.alloc_decode_workspace(B, T, DEV), "sparse": G.alloc_decode_sparse_workspace(B, 5),
          "shared": G.alloc_decode_shared_workspace(B, paged.max_pages, 1), "prefill": G.alloc_prefill_workspace(B, T, DEV)}
    g, p = ints(starts), ints([2])
    x = queries(1, 83).view(6, 1024).to(DEV)
    w = torch.randn(1024, 256, generator=torch.Generator().manual_seed(84)).bfloat16().to(DEV)
    w8, scales = (w * 40).clamp(-127, 127).to(torch.int8), torch.rand(256, device=DEV)
    big = torch.empty(G.linear_int8_workspace(1024, 256) + 256, dtype=torch.uint8, device=DEV)

    def whole(out, s):
        G.decode_paged(q, k, v, table, lens, ws["decode"], st, s)
        G.combine(ws["decode"], lens, out, T, st, s)

    heads, codes = (B, 48, 128), (k.shape[0], 2, 8, 2, 128)
    scale = torch.zeros(k.shape[0], 2, 8, device=DEV)
    return [
        ("decode_sparse_paged", lambda o, s: G.decode_sparse_paged(q, k, v, table, lens, sel, ws["sparse"], o, st, s), heads,
         torch.bfloat16),
        ("decode_shared_paged", lambda o, s: G.decode_shared_paged(q, k, v, table, lens, g, p, ws["shared"], o, st, s), heads,
         torch.bfloat16),
        ("decode_paged", whole, heads, torch.bfloat16),
        ("prefill_paged", lambda o, s: G.prefill_paged(q4, k, v, table, lens - 1, None, o, st, s), (B, 1, 48, 128),
         torch.bfloat16),
        ("prefill_ws_paged", lambda o, s: G.prefill_ws_paged(q4, k, v, table, lens - 1, None, o, ws["prefill"], st, s),
         (B, 1, 48, 128), torch.bfloat16),
        ("linear", lambda o, s: G.linear(x, w, o, st, s), (6, 256), torch.bfloat16),
        ("linear_int8", lambda o, s: G.linear_int8(x, w8, scales, o, big, st, s), (6, 256), torch.bfloat16),
        ("kv_bounds_paged", lambda o, s: G.kv_bounds_paged(k, table, zero, lens, max(paged.lens), o, scale, st, s), codes,
         torch.int8)], st


def test_calls_from_a_new_thread():
    """A thread that has no CUDA context yet gets its device's, as with the runtime's own calls."""
    todo, st = calls()
    stream = torch.cuda.Stream()
    for name, call, shape, dtype in todo:
        want, got = (torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(2))
        call(want, None)
        torch.cuda.synchronize()
        in_thread(lambda: call(got, stream))
        torch.cuda.synchronize()
        assert torch.equal(want, got) and got.any(), name
    assert int(st.item()) == 0


@pytest.mark.parametrize("streams", [1, 4])
def test_calls_of_four_threads_at_once(streams):
    """Each with its own workspace and outputs, on one stream (where their kernels mix) or on four."""
    on = [torch.cuda.Stream() for _ in range(streams)] * (4 // streams)
    jobs = []
    for i in range(4):
        paged, starts = grouped([5 + 7 * i, 2], [4, 1], lambda b: 40 * b, seed=90 + i)
        B = len(paged.lens)
        k, v, table = paged.dev()
        q, lens, budget = queries(B, 94 + i).to(DEV), ints(paged.lens), (3, 40)[i % 2]
        sel, g, p = ints(lists(paged.lens, budget, seed=98)), ints(starts), ints([4, 1])
        wa, wb = G.alloc_decode_sparse_workspace(B, budget), G.alloc_decode_shared_workspace(B, paged.max_pages, 2)
        outs = [[torch.zeros_like(q) for _ in range(2)] for _ in range(2)]

        def job(a, z, s, q=q, k=k, v=v, table=table, lens=lens, sel=sel, g=g, p=p, wa=wa, wb=wb):
            G.decode_sparse_paged(q, k, v, table, lens, sel, wa, a, None, s)
            G.decode_shared_paged(q, k, v, table, lens, g, p, wb, z, None, s)

        job(*outs[0], None)
        jobs.append((job, outs))
    torch.cuda.synchronize()
    raised = []

    def body(i):
        try:
            for _ in range(100):
                jobs[i][0](*jobs[i][1][1], on[i])
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not raised, raised[0]
    for _, (want, got) in jobs:
        assert all(torch.equal(a, b) and np.isfinite(a.float().cpu().numpy()).all() for a, b in zip(want, got))
