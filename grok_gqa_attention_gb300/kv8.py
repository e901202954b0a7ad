"""The 8-bit KV cache of libgrok_attn.so: argument marshalling, as in the package's other calls.

A cache is blocks of 64 tokens of one KV head, int8 or e4m3 codes with one fp32
scale per block (see grok_kv8_cache in include/grok_attn.h). Every call runs on
the device of its tensors, on that device's current stream unless one is given.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import (HEAD_DIM, KV8_BLOCK, KV8_E4M3, KV8_INT8, MAX_POSITION, N_KV_HEADS, N_Q_HEADS, _check, _ptr, _want, load)

_KINDS = {torch.int8: KV8_INT8, torch.float8_e4m3fn: KV8_E4M3}


class _Cache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("open_k", ctypes.c_void_p),
                ("open_v", ctypes.c_void_p), ("kind", ctypes.c_int), ("B", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("n_blocks", ctypes.c_int)]


def _same_device(device: torch.device, **tensors: Optional[torch.Tensor]) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


@contextlib.contextmanager
def _on(device: torch.device):
    with torch.cuda.device(device):
        yield


def _call(device: torch.device, stream: Optional[torch.cuda.Stream], name: str, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    lib = load()
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    s = (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream
    if torch.cuda.current_device() == device.index:
        _check(getattr(lib, name)(*args, ctypes.c_void_p(s)))
    else:
        with _on(device):
            _check(getattr(lib, name)(*args, ctypes.c_void_p(s)))


class Kv8Cache:
    """The tensors of an 8-bit cache, checked once; the calls below read and write them in place.

    k_pool [n_blocks, 2, 64, 64] (half of the features, token, feature), v_pool [n_blocks, 128, 64] (feature,
    token): torch.int8 or torch.float8_e4m3fn. k_scale, v_scale [n_blocks] float32. table [B, 8, max_blocks]
    int32: the block of rows [64 i, 64 i + 64) of each sequence and KV head. open_k, open_v [B, 8, 64, 128]
    bfloat16: the unrounded rows of the block that is not full yet.
    """

    __slots__ = ("k_pool", "v_pool", "k_scale", "v_scale", "table", "open_k", "open_v", "B", "max_blocks", "n_blocks",
                 "device", "_c", "_ref")

    def __init__(self, k_pool, v_pool, k_scale, v_scale, table, open_k, open_v):
        if k_pool.dtype not in _KINDS:
            raise TypeError(f"k_pool must be torch.int8 or torch.float8_e4m3fn, got {k_pool.dtype}")
        if table.dim() != 3:
            raise ValueError("table must be [B, 8, max_blocks]")
        n, (B, _, max_blocks) = k_pool.shape[0], table.shape
        half = HEAD_DIM // 2
        _want(k_pool, "k_pool", k_pool.dtype, (n, 2, KV8_BLOCK, half))
        _want(v_pool, "v_pool", k_pool.dtype, (n, HEAD_DIM, KV8_BLOCK))
        _want(k_scale, "k_scale", torch.float32, (n,))
        _want(v_scale, "v_scale", torch.float32, (n,))
        _want(table, "table", torch.int32, (B, N_KV_HEADS, max_blocks))
        _want(open_k, "open_k", torch.bfloat16, (B, N_KV_HEADS, KV8_BLOCK, HEAD_DIM))
        _want(open_v, "open_v", torch.bfloat16, (B, N_KV_HEADS, KV8_BLOCK, HEAD_DIM))
        if not 1 <= max_blocks <= MAX_POSITION // KV8_BLOCK:
            raise ValueError(f"max_blocks must be 1 to {MAX_POSITION // KV8_BLOCK}, got {max_blocks}")
        self.device = k_pool.device
        _same_device(self.device, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale, table=table, open_k=open_k,
                     open_v=open_v)
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = k_pool, v_pool, k_scale, v_scale
        self.table, self.open_k, self.open_v = table, open_k, open_v
        self.B, self.max_blocks, self.n_blocks = B, max_blocks, n
        self._c = _Cache(k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         table.data_ptr(), open_k.data_ptr(), open_v.data_ptr(), _KINDS[k_pool.dtype], B, max_blocks, n)
        self._ref = ctypes.byref(self._c)

    def __setattr__(self, name, value):
        if hasattr(self, "_ref"):  # the C struct holds the tensors' addresses
            raise AttributeError("a Kv8Cache's tensors are fixed; make another (with_table) for others")
        object.__setattr__(self, name, value)

    def with_table(self, table) -> "Kv8Cache":
        """The same blocks under another table (what kv8_evict returned)."""
        return Kv8Cache(self.k_pool, self.v_pool, self.k_scale, self.v_scale, table, self.open_k, self.open_v)


def alloc_kv8_cache(B: int, max_blocks: int, dtype: torch.dtype = torch.int8, device=None) -> Kv8Cache:
    """An empty cache of B sequences of max_blocks * 64 rows, each with its own blocks."""
    dev = torch.device(device or "cuda")
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    n = B * N_KV_HEADS * max_blocks
    pool = lambda *shape: torch.zeros((n,) + shape, dtype=torch.uint8, device=dev).view(dtype)  # noqa: E731
    rows = lambda: torch.zeros((B, N_KV_HEADS, KV8_BLOCK, HEAD_DIM), dtype=torch.bfloat16, device=dev)  # noqa: E731
    return Kv8Cache(pool(2, KV8_BLOCK, HEAD_DIM // 2), pool(HEAD_DIM, KV8_BLOCK), torch.zeros(n, device=dev),
                    torch.zeros(n, device=dev),
                    torch.arange(n, dtype=torch.int32, device=dev).view(B, N_KV_HEADS, max_blocks), rows(), rows())


def kv8_append(cache: Kv8Cache, q, k, v, start_pos, cache_len, valid_len, cos_tab, sin_tab, q_rot, dev_status=None,
               stream=None) -> None:
    """RoPE on q and k at positions start_pos[b] + i; tokens i < valid_len[b] become rows cache_len[b] + i.

    valid_len may be None (all T tokens). cos_tab, sin_tab [n, 64] as from rope_cos_sin(0, n). The caller advances
    cache_len and start_pos (see grok_kv8_append).
    """
    B, T, n = cache.B, q.shape[1], cos_tab.shape[0]
    _want(q, "q", torch.bfloat16, (B, T, N_Q_HEADS, HEAD_DIM))
    _want(k, "k", torch.bfloat16, (B, T, N_KV_HEADS, HEAD_DIM))
    _want(v, "v", torch.bfloat16, (B, T, N_KV_HEADS, HEAD_DIM))
    _want(start_pos, "start_pos", torch.int32, (B,))
    _want(cache_len, "cache_len", torch.int32, (B,))
    if valid_len is not None:
        _want(valid_len, "valid_len", torch.int32, (B,))
    _want(cos_tab, "cos_tab", torch.float32, (n, 64))
    _want(sin_tab, "sin_tab", torch.float32, (n, 64))
    _want(q_rot, "q_rot", torch.bfloat16, (B, T, N_Q_HEADS, HEAD_DIM))
    if dev_status is not None:
        _want(dev_status, "dev_status", torch.int32, (1,))
    _same_device(cache.device, q=q, k=k, v=v, start_pos=start_pos, cache_len=cache_len, valid_len=valid_len,
                 cos_tab=cos_tab, sin_tab=sin_tab, q_rot=q_rot, dev_status=dev_status)
    _call(cache.device, stream, "grok_kv8_append", cache._ref, _ptr(q), _ptr(k), _ptr(v), _ptr(start_pos),
          _ptr(cache_len), _ptr(valid_len), T, _ptr(cos_tab), _ptr(sin_tab), n, _ptr(q_rot), _ptr(dev_status))


def kv8_decode_workspace(B: int, max_blocks: int, weights: bool = True) -> int:
    """Bytes of workspace for kv8_decode() on the current device; weights: room for the blocks' weights."""
    n = ctypes.c_size_t(0)
    _check(load().grok_kv8_decode_workspace(int(B), int(max_blocks), 1 if weights else 0, ctypes.byref(n)))
    return n.value


def alloc_kv8_decode_workspace(cache: Kv8Cache, weights: bool = True) -> torch.Tensor:
    with _on(cache.device):
        return torch.empty(kv8_decode_workspace(cache.B, cache.max_blocks, weights), dtype=torch.uint8,
                           device=cache.device)


def kv8_decode(cache: Kv8Cache, q_rot, kv_len, workspace, out, weight_in=None, weight_out=None, dev_status=None,
               stream=None) -> None:
    """out [B, 48, 128] = attention of q_rot [B, 48, 128] over rows [0, kv_len[b]) of the cache.

    weight_out [B, 8, max_blocks] float32 (optional): weight_in (None: zero; may be weight_out) plus the softmax
    weight each block received, summed over the KV head's query heads.
    """
    B = cache.B
    _want(q_rot, "q_rot", torch.bfloat16, (B, N_Q_HEADS, HEAD_DIM))
    _want(kv_len, "kv_len", torch.int32, (B,))
    _want(out, "out", torch.bfloat16, (B, N_Q_HEADS, HEAD_DIM))
    _want(workspace, "workspace", torch.uint8, (workspace.numel(),))
    if weight_in is not None:
        _want(weight_in, "weight_in", torch.float32, (B, N_KV_HEADS, cache.max_blocks))
    if weight_out is not None:
        _want(weight_out, "weight_out", torch.float32, (B, N_KV_HEADS, cache.max_blocks))
    if dev_status is not None:
        _want(dev_status, "dev_status", torch.int32, (1,))
    _same_device(cache.device, q_rot=q_rot, kv_len=kv_len, out=out, workspace=workspace, weight_in=weight_in,
                 weight_out=weight_out, dev_status=dev_status)
    _call(cache.device, stream, "grok_kv8_decode", cache._ref, _ptr(q_rot), _ptr(kv_len), _ptr(workspace),
          workspace.numel(), _ptr(out), _ptr(weight_in), _ptr(weight_out), _ptr(dev_status))


def kv8_prefill_workspace(B: int, max_blocks: int) -> int:
    """Bytes of workspace for kv8_prefill() on the current device."""
    n = ctypes.c_size_t(0)
    _check(load().grok_kv8_prefill_workspace(int(B), int(max_blocks), ctypes.byref(n)))
    return n.value


def alloc_kv8_prefill_workspace(cache: Kv8Cache) -> torch.Tensor:
    with _on(cache.device):
        return torch.empty(kv8_prefill_workspace(cache.B, cache.max_blocks), dtype=torch.uint8, device=cache.device)


def kv8_prefill(cache: Kv8Cache, q_rot, cache_len, valid_len, out, workspace, dev_status=None, stream=None) -> None:
    """out [B, T, 48, 128]: token i of sequence b attends rows j <= cache_len[b] + i, j < cache_len[b] + valid_len[b].

    The tokens' own rows are in the cache already (kv8_append with the same cache_len and valid_len, which may be None).
    """
    B, T = cache.B, q_rot.shape[1]
    _want(q_rot, "q_rot", torch.bfloat16, (B, T, N_Q_HEADS, HEAD_DIM))
    _want(cache_len, "cache_len", torch.int32, (B,))
    if valid_len is not None:
        _want(valid_len, "valid_len", torch.int32, (B,))
    _want(out, "out", torch.bfloat16, (B, T, N_Q_HEADS, HEAD_DIM))
    _want(workspace, "workspace", torch.uint8, (workspace.numel(),))
    if dev_status is not None:
        _want(dev_status, "dev_status", torch.int32, (1,))
    _same_device(cache.device, q_rot=q_rot, cache_len=cache_len, valid_len=valid_len, out=out, workspace=workspace,
                 dev_status=dev_status)
    _call(cache.device, stream, "grok_kv8_prefill", cache._ref, _ptr(q_rot), _ptr(cache_len), _ptr(valid_len), T,
          _ptr(out), _ptr(workspace), workspace.numel(), _ptr(dev_status))


def kv8_evict(table, weight, kv_len, keep: int, sink: int, recent: int, table_out, weight_out, kv_len_out,
              dev_status=None, stream=None) -> None:
    """Down to `keep` full blocks per sequence and head: the first `sink`, the last `recent`, then by weight.

    table_out may be table, weight_out weight; kv_len_out is another tensor than kv_len (see grok_kv8_evict).
    """
    if table.dim() != 3:
        raise ValueError("table must be [B, 8, max_blocks]")
    B, _, n = table.shape
    _want(table, "table", torch.int32, (B, N_KV_HEADS, n))
    _want(weight, "weight", torch.float32, (B, N_KV_HEADS, n))
    _want(kv_len, "kv_len", torch.int32, (B,))
    _want(table_out, "table_out", torch.int32, (B, N_KV_HEADS, n))
    _want(weight_out, "weight_out", torch.float32, (B, N_KV_HEADS, n))
    _want(kv_len_out, "kv_len_out", torch.int32, (B,))
    if dev_status is not None:
        _want(dev_status, "dev_status", torch.int32, (1,))
    _same_device(table.device, weight=weight, kv_len=kv_len, table_out=table_out, weight_out=weight_out,
                 kv_len_out=kv_len_out, dev_status=dev_status)
    _call(table.device, stream, "grok_kv8_evict", _ptr(table), _ptr(weight), _ptr(kv_len), B, n, int(keep), int(sink),
          int(recent), _ptr(table_out), _ptr(weight_out), _ptr(kv_len_out), _ptr(dev_status))
