"""The 8-bit KV cache of libgrok_attn.so: argument marshalling, as in the package's other calls.

A cache is blocks of 64 tokens of one KV head, int8 or e4m3 codes with one fp32
scale per block (see grok_kv8_cache in include/grok_attn.h). Every call runs on
the device of its tensors, on that device's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import HEAD_DIM, KV8_BLOCK, KV8_E4M3, KV8_INT8, MAX_POSITION, N_KV_HEADS, N_Q_HEADS, _check, _want, load

_KINDS = {torch.int8: KV8_INT8, torch.float8_e4m3fn: KV8_E4M3}


class _Cache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("open_k", ctypes.c_void_p),
                ("open_v", ctypes.c_void_p), ("kind", ctypes.c_int), ("B", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("n_blocks", ctypes.c_int)]


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _need(t, name: str, dtype: torch.dtype, shape: tuple, index: int) -> int:
    """The address of t, which must be a contiguous tensor of this type and shape on CUDA device `index`.

    One pass of cheap comparisons (a decode step's calls are short); _want says what is wrong otherwise.
    """
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _want(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the cache's or the other tensors on cuda:{index}")


def _maybe(t, name: str, dtype: torch.dtype, shape: tuple, index: int) -> Optional[int]:
    return None if t is None else _need(t, name, dtype, shape, index)


# The raw forms of torch.cuda.current_stream(i).cuda_stream and torch.cuda.current_device(), where torch has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_calls: dict = {}


def _call(index: int, stream: Optional[torch.cuda.Stream], name: str, *args) -> None:
    """The library's call `name` on `stream` (None: the device's current one), with device `index` current."""
    fn = _calls.get(name)
    if fn is None:
        fn = _calls[name] = getattr(load(), name)
    if stream is None:
        s = _raw_stream(index)
    elif stream.device.index == index:
        s = stream.cuda_stream
    else:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    if _raw_device() == index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    if status:
        _check(status)


class Kv8Cache:
    """The tensors of an 8-bit cache, checked once; the calls below read and write them in place.

    k_pool [n_blocks, 2, 64, 64] (half of the features, token, feature), v_pool [n_blocks, 128, 64] (feature,
    token): torch.int8 or torch.float8_e4m3fn. k_scale, v_scale [n_blocks] float32. table [B, 8, max_blocks]
    int32: the block of rows [64 i, 64 i + 64) of each sequence and KV head. open_k, open_v [B, 8, 64, 128]
    bfloat16: the unrounded rows of the block that is not full yet.
    """

    __slots__ = ("k_pool", "v_pool", "k_scale", "v_scale", "table", "open_k", "open_v", "B", "max_blocks", "n_blocks",
                 "index", "_c", "_ref")

    def __init__(self, k_pool, v_pool, k_scale, v_scale, table, open_k, open_v):
        if k_pool.dtype not in _KINDS:
            raise TypeError(f"k_pool must be torch.int8 or torch.float8_e4m3fn, got {k_pool.dtype}")
        if table.dim() != 3:
            raise ValueError("table must be [B, 8, max_blocks]")
        n, (B, _, max_blocks) = k_pool.shape[0], table.shape
        half, pool = HEAD_DIM // 2, k_pool.dtype
        _want(k_pool, "k_pool", pool, (n, 2, KV8_BLOCK, half))
        if not 1 <= max_blocks <= MAX_POSITION // KV8_BLOCK:
            raise ValueError(f"max_blocks must be 1 to {MAX_POSITION // KV8_BLOCK}, got {max_blocks}")
        rows, index = (B, N_KV_HEADS, KV8_BLOCK, HEAD_DIM), k_pool.get_device()
        self.index = index
        self._c = _Cache(k_pool.data_ptr(), _need(v_pool, "v_pool", pool, (n, HEAD_DIM, KV8_BLOCK), index),
                         _need(k_scale, "k_scale", torch.float32, (n,), index),
                         _need(v_scale, "v_scale", torch.float32, (n,), index),
                         _need(table, "table", torch.int32, (B, N_KV_HEADS, max_blocks), index),
                         _need(open_k, "open_k", torch.bfloat16, rows, index),
                         _need(open_v, "open_v", torch.bfloat16, rows, index), _KINDS[pool], B, max_blocks, n)
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = k_pool, v_pool, k_scale, v_scale
        self.table, self.open_k, self.open_v = table, open_k, open_v
        self.B, self.max_blocks, self.n_blocks = B, max_blocks, n
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
    cache_len and start_pos, and sets cache_len back, if at all, to a multiple of 64 (see grok_kv8_append).
    """
    B, T, n, at = cache.B, q.shape[1], cos_tab.shape[0], cache.index
    kv = (B, T, N_KV_HEADS, HEAD_DIM)
    heads = (B, T, N_Q_HEADS, HEAD_DIM)
    _call(at, stream, "grok_kv8_append", cache._ref, _need(q, "q", _BF16, heads, at),
          _need(k, "k", _BF16, kv, at), _need(v, "v", _BF16, kv, at),
          _need(start_pos, "start_pos", _I32, (B,), at), _need(cache_len, "cache_len", _I32, (B,), at),
          _maybe(valid_len, "valid_len", _I32, (B,), at), T,
          _need(cos_tab, "cos_tab", _F32, (n, 64), at), _need(sin_tab, "sin_tab", _F32, (n, 64), at),
          n, _need(q_rot, "q_rot", _BF16, heads, at), _maybe(dev_status, "dev_status", _I32, (1,), at))


def kv8_decode_workspace(B: int, max_blocks: int, weights: bool = True) -> int:
    """Bytes of workspace for kv8_decode() on the current device; weights: room for the blocks' weights."""
    n = ctypes.c_size_t(0)
    _check(load().grok_kv8_decode_workspace(int(B), int(max_blocks), 1 if weights else 0, ctypes.byref(n)))
    return n.value


def alloc_kv8_decode_workspace(cache: Kv8Cache, weights: bool = True) -> torch.Tensor:
    with torch.cuda.device(cache.index):
        return torch.empty(kv8_decode_workspace(cache.B, cache.max_blocks, weights), dtype=torch.uint8, device="cuda")


def kv8_decode(cache: Kv8Cache, q_rot, kv_len, workspace, out, weight_in=None, weight_out=None, dev_status=None,
               stream=None) -> None:
    """out [B, 48, 128] = attention of q_rot [B, 48, 128] over rows [0, kv_len[b]) of the cache.

    weight_out [B, 8, max_blocks] float32 (optional): weight_in (None: zero; may be weight_out) plus the softmax
    weight each block received, summed over the KV head's query heads.
    """
    B, at = cache.B, cache.index
    heads, blocks = (B, N_Q_HEADS, HEAD_DIM), (B, N_KV_HEADS, cache.max_blocks)
    nbytes = workspace.numel()
    _call(at, stream, "grok_kv8_decode", cache._ref, _need(q_rot, "q_rot", _BF16, heads, at),
          _need(kv_len, "kv_len", _I32, (B,), at), _need(workspace, "workspace", _U8, (nbytes,), at),
          nbytes, _need(out, "out", _BF16, heads, at),
          _maybe(weight_in, "weight_in", _F32, blocks, at),
          _maybe(weight_out, "weight_out", _F32, blocks, at),
          _maybe(dev_status, "dev_status", _I32, (1,), at))


def kv8_prefill_workspace(B: int, max_blocks: int) -> int:
    """Bytes of workspace for kv8_prefill() on the current device."""
    n = ctypes.c_size_t(0)
    _check(load().grok_kv8_prefill_workspace(int(B), int(max_blocks), ctypes.byref(n)))
    return n.value


def alloc_kv8_prefill_workspace(cache: Kv8Cache) -> torch.Tensor:
    with torch.cuda.device(cache.index):
        return torch.empty(kv8_prefill_workspace(cache.B, cache.max_blocks), dtype=torch.uint8, device="cuda")


def kv8_prefill(cache: Kv8Cache, q_rot, cache_len, valid_len, out, workspace, dev_status=None, stream=None) -> None:
    """out [B, T, 48, 128]: token i of sequence b attends rows j <= cache_len[b] + i, j < cache_len[b] + valid_len[b].

    The tokens' own rows are in the cache already (kv8_append with the same cache_len and valid_len, which may be None).
    """
    B, T, at = cache.B, q_rot.shape[1], cache.index
    heads, nbytes = (B, T, N_Q_HEADS, HEAD_DIM), workspace.numel()
    _call(at, stream, "grok_kv8_prefill", cache._ref, _need(q_rot, "q_rot", _BF16, heads, at),
          _need(cache_len, "cache_len", _I32, (B,), at), _maybe(valid_len, "valid_len", _I32, (B,), at), T,
          _need(out, "out", _BF16, heads, at), _need(workspace, "workspace", _U8, (nbytes,), at), nbytes,
          _maybe(dev_status, "dev_status", _I32, (1,), at))


def kv8_evict(table, weight, kv_len, keep: int, sink: int, recent: int, table_out, weight_out, kv_len_out,
              dev_status=None, stream=None) -> None:
    """Down to `keep` full blocks per sequence and head: the first `sink`, the last `recent`, then by weight.

    table_out may be table, weight_out weight; kv_len_out is another tensor than kv_len (see grok_kv8_evict).
    """
    if table.dim() != 3:
        raise ValueError("table must be [B, 8, max_blocks]")
    B, _, n = table.shape
    row, at = (B, N_KV_HEADS, n), table.get_device()
    if at < 0:
        raise ValueError("table must be a CUDA tensor")
    _call(at, stream, "grok_kv8_evict", _need(table, "table", _I32, row, at),
          _need(weight, "weight", _F32, row, at), _need(kv_len, "kv_len", _I32, (B,), at), B, n,
          int(keep), int(sink), int(recent), _need(table_out, "table_out", _I32, row, at),
          _need(weight_out, "weight_out", _F32, row, at),
          _need(kv_len_out, "kv_len_out", _I32, (B,), at),
          _maybe(dev_status, "dev_status", _I32, (1,), at))
