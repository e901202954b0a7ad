"""Decode that reads part of a paged cache: argument marshalling, as in the package's other calls.

Bounds of the keys of each 64-token block, the choice of the blocks that a query reads, attention over a list of
blocks, and attention for a batch whose sequences share prefixes (see grok_kv_bounds_paged in include/grok_attn.h).
Every call runs on the device of its pools, on that device's current stream unless one is given. A call's arguments are
checked by the extension _binding where all is as it should be, and by the functions here otherwise, which say what is not. (Where
the library was built without Python's headers there is none: a call then takes about 3 us more.)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import HEAD_DIM, N_KV_HEADS, N_Q_HEADS, PAGE_TOKENS, SPARSE_BLOCK, _check, load
from .kv8 import _call, _maybe, _need, _raw_device, _raw_stream

_BF16, _F32, _I32, _I8, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8
_PAGE_BLOCKS = PAGE_TOKENS // SPARSE_BLOCK


class _Unchecked:
    """Stands for an extension that was not built: hands every call back to the checks here."""

    def __getattr__(self, name: str):
        return lambda *args: None


_checked = None


def _binding():
    """The extension's checks, with the library's functions."""
    global _checked
    if _checked is None:
        from .build import BINDING  # (here: the package does not import what builds it)
        lib = load()
        if not os.path.exists(BINDING):
            _checked = _Unchecked()
            return _checked
        spec = importlib.util.spec_from_file_location("_binding", BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        calls = (lib.grok_kv_bounds_paged, lib.grok_attn_select_paged, lib.grok_attn_decode_sparse_paged,
                 lib.grok_attn_decode_shared_paged)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in calls), _BF16, _F32, _I32, _I8, _U8, _raw_device,
                    _raw_stream)
        _checked = module
    return _checked


def _index(t, name: str) -> int:
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return at


def _table(block_table, B: int, at: int) -> tuple[int, int]:
    """(address, max_pages) of a block table [B, max_pages]."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    n = block_table.shape[1]
    return _need(block_table, "block_table", _I32, (B, n), at), n


def _pool(pool, name: str, n: int, at: int) -> int:
    return _need(pool, name, _BF16, (n, PAGE_TOKENS, N_KV_HEADS, HEAD_DIM), at)


def alloc_kv_bounds(n_pages: int, device=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Empty bounds of a pool of n_pages pages: codes int8 [n_pages, 2, 8, 2, 128], scale float32 [n_pages, 2, 8]."""
    dev = device or "cuda"
    return (torch.zeros((n_pages, _PAGE_BLOCKS, N_KV_HEADS, 2, HEAD_DIM), dtype=_I8, device=dev),
            torch.zeros((n_pages, _PAGE_BLOCKS, N_KV_HEADS), dtype=_F32, device=dev))


def kv_bounds_paged(k_pool, block_table, start_pos, valid_len, T: int, codes, scale, dev_status=None,
                    stream=None) -> None:
    """Bounds of the keys of every block that rows [start_pos[b], start_pos[b] + valid_len[b]) touch (after an append).

    valid_len may be None (T rows of every sequence). codes, scale as from alloc_kv_bounds(k_pool.shape[0]).
    """
    status = (_checked or _binding()).kv_bounds_paged(k_pool, block_table, start_pos, valid_len, T, codes, scale, dev_status,
                                                        stream)
    if status is not None:
        return _check(status)
    at, n, B = _index(k_pool, "k_pool"), k_pool.shape[0], start_pos.shape[0]
    table, max_pages = _table(block_table, B, at)
    _call(at, stream, "grok_kv_bounds_paged", _pool(k_pool, "k_pool", n, at), n, table, max_pages,
          _need(start_pos, "start_pos", _I32, (B,), at), _maybe(valid_len, "valid_len", _I32, (B,), at), B, int(T),
          _need(codes, "codes", _I8, (n, _PAGE_BLOCKS, N_KV_HEADS, 2, HEAD_DIM), at),
          _need(scale, "scale", _F32, (n, _PAGE_BLOCKS, N_KV_HEADS), at),
          _maybe(dev_status, "dev_status", _I32, (1,), at))


def select_blocks_paged(q_rot, codes, scale, block_table, kv_len, sink: int, recent: int, score, sel, dev_status=None,
                        stream=None) -> None:
    """score [B, 8, 2 * max_pages] float32: a bound of q . k over each block; sel [B, 8, budget] int32: the blocks to
    read, ascending, -1 behind them: the first `sink`, the last `recent`, then the largest scores.
    """
    status = (_checked or _binding()).select_blocks_paged(q_rot, codes, scale, block_table, kv_len, sink, recent, score,
                                                            sel, dev_status, stream)
    if status is not None:
        return _check(status)
    at, n, B = _index(q_rot, "q_rot"), codes.shape[0], q_rot.shape[0]
    if sel.dim() != 3:
        raise ValueError("sel must be [B, 8, budget]")
    budget = sel.shape[2]
    table, max_pages = _table(block_table, B, at)
    _call(at, stream, "grok_attn_select_paged", _need(q_rot, "q_rot", _BF16, (B, N_Q_HEADS, HEAD_DIM), at),
          _need(codes, "codes", _I8, (n, _PAGE_BLOCKS, N_KV_HEADS, 2, HEAD_DIM), at),
          _need(scale, "scale", _F32, (n, _PAGE_BLOCKS, N_KV_HEADS), at), n, table, max_pages,
          _need(kv_len, "kv_len", _I32, (B,), at), B, budget, int(sink), int(recent),
          _need(score, "score", _F32, (B, N_KV_HEADS, _PAGE_BLOCKS * max_pages), at),
          _need(sel, "sel", _I32, (B, N_KV_HEADS, budget), at), _maybe(dev_status, "dev_status", _I32, (1,), at))


def decode_sparse_workspace(B: int, budget: int) -> int:
    """Bytes of workspace for decode_sparse_paged() on the current device."""
    n = ctypes.c_size_t(0)
    _check(load().grok_attn_decode_sparse_workspace(int(B), int(budget), ctypes.byref(n)))
    return n.value


def alloc_decode_sparse_workspace(B: int, budget: int, device=None) -> torch.Tensor:
    with torch.cuda.device(device):  # (None: the current one)
        return torch.empty(decode_sparse_workspace(B, budget), dtype=_U8, device="cuda")


def decode_sparse_paged(q_rot, k_pool, v_pool, block_table, kv_len, sel, workspace, out, dev_status=None,
                        stream=None) -> None:
    """out [B, 48, 128] = attention of q_rot [B, 48, 128] over the rows below kv_len[b] of the blocks in sel
    [B, 8, budget] (per KV head; negative entries are passed over).
    """
    status = (_checked or _binding()).decode_sparse_paged(q_rot, k_pool, v_pool, block_table, kv_len, sel, workspace, out,
                                                            dev_status, stream)
    if status is not None:
        return _check(status)
    at, n, B = _index(k_pool, "k_pool"), k_pool.shape[0], q_rot.shape[0]
    if sel.dim() != 3:
        raise ValueError("sel must be [B, 8, budget]")
    budget, nbytes = sel.shape[2], workspace.numel()
    table, max_pages = _table(block_table, B, at)
    heads = (B, N_Q_HEADS, HEAD_DIM)
    _call(at, stream, "grok_attn_decode_sparse_paged", _need(q_rot, "q_rot", _BF16, heads, at),
          _pool(k_pool, "k_pool", n, at), _pool(v_pool, "v_pool", n, at), n, table, max_pages,
          _need(kv_len, "kv_len", _I32, (B,), at), _need(sel, "sel", _I32, (B, N_KV_HEADS, budget), at), budget, B,
          _need(workspace, "workspace", _U8, (nbytes,), at), nbytes, _need(out, "out", _BF16, heads, at),
          _maybe(dev_status, "dev_status", _I32, (1,), at))


def decode_shared_workspace(B: int, max_pages: int, n_groups: int) -> int:
    """Bytes of workspace for decode_shared_paged() on the current device."""
    n = ctypes.c_size_t(0)
    _check(load().grok_attn_decode_shared_workspace(int(B), int(max_pages), int(n_groups), ctypes.byref(n)))
    return n.value


def alloc_decode_shared_workspace(B: int, max_pages: int, n_groups: int, device=None) -> torch.Tensor:
    with torch.cuda.device(device):  # (None: the current one)
        return torch.empty(decode_shared_workspace(B, max_pages, n_groups), dtype=_U8, device="cuda")


def decode_shared_paged(q_rot, k_pool, v_pool, block_table, kv_len, group_start, shared_pages, workspace, out,
                        dev_status=None, stream=None) -> None:
    """out [B, 48, 128] = attention of q_rot [B, 48, 128] over rows [0, kv_len[b]), common rows read once.

    Sequences [group_start[i], group_start[i + 1]) have the first shared_pages[i] entries of block_table in common;
    group_start [n_groups + 1], shared_pages [n_groups] int32.
    """
    status = (_checked or _binding()).decode_shared_paged(q_rot, k_pool, v_pool, block_table, kv_len, group_start,
                                                            shared_pages, workspace, out, dev_status, stream)
    if status is not None:
        return _check(status)
    at, n, B = _index(k_pool, "k_pool"), k_pool.shape[0], q_rot.shape[0]
    n_groups, nbytes = shared_pages.numel(), workspace.numel()
    table, max_pages = _table(block_table, B, at)
    heads = (B, N_Q_HEADS, HEAD_DIM)
    _call(at, stream, "grok_attn_decode_shared_paged", _need(q_rot, "q_rot", _BF16, heads, at),
          _pool(k_pool, "k_pool", n, at), _pool(v_pool, "v_pool", n, at), n, table, max_pages,
          _need(kv_len, "kv_len", _I32, (B,), at), B, _need(group_start, "group_start", _I32, (n_groups + 1,), at),
          _need(shared_pages, "shared_pages", _I32, (n_groups,), at), n_groups,
          _need(workspace, "workspace", _U8, (nbytes,), at), nbytes, _need(out, "out", _BF16, heads, at),
          _maybe(dev_status, "dev_status", _I32, (1,), at))
