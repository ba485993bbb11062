"""Python binding of the paged 8-bit context cache (include/dflash.h): block tables, the quantising
append and attention over the cache. Argument marshalling and checks only, as in the package's
``Handle``; every tensor is the caller's, on one CUDA device."""
from __future__ import annotations

import ctypes

from . import (DFLASH_BF16, DFLASH_EINVAL, DFLASH_F16, DFLASH_F32, DFLASH_POOL_SCRATCH, DFlashError, _check, _stream_ptr,
               dflash_attention, dflash_cache_config, dflash_pool, dflash_rows, lib)


def _row_dtype(t) -> int:
    import torch
    codes = {torch.float32: DFLASH_F32, torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_F16}
    if t.dtype not in codes:
        raise ValueError(f"rows are fp32, bf16 or f16, not {t.dtype}")
    return codes[t.dtype]


def _ints(name, t, n, device):
    """The address of a contiguous int32 tensor of n elements (None: NULL)."""
    import torch
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device or (n is not None and t.numel() != n):
        raise ValueError(f"{name}: a contiguous int32 tensor{'' if n is None else f' of {n} elements'} on {device} is wanted")
    return t.data_ptr()


def _rows(name, t, shape, device, dtype):
    """dflash_rows of a [..., rows, heads, head_dim] tensor with contiguous last dimension."""
    if t is None:
        return dflash_rows(None, 0, 0, 0)
    if tuple(t.shape[-len(shape):]) != tuple(shape) or t.dim() > 4 or t.dtype != dtype or t.device != device or t.stride(-1) != 1:
        raise ValueError(f"{name}: {dtype} rows of shape {tuple(shape)} on {device} are wanted, contiguous in the last dimension")
    return dflash_rows(t.data_ptr(), t.stride(0) if t.dim() == 4 else 0, t.stride(-3), t.stride(-2))


class BlockPool:
    """Block tables over a pool of blocks of ``block_tokens`` tokens (dflash_pool_reserve and
    dflash_pool_truncate). Holds the calls' 256 bytes of device scratch; lens, table and the stack of
    free blocks are the caller's tensors:

      lens int32 [rows], table int32 [rows][blocks per request], free int32 [blocks], free_count int32 [1]
    """

    def __init__(self, block_tokens: int, max_requests: int | None = None, ring: bool = False, device="cuda"):
        import torch
        if block_tokens not in (16, 32, 64, 128) or (max_requests is not None and not 0 < max_requests <= 1024):
            raise DFlashError(DFLASH_EINVAL, "BlockPool")
        self.block_tokens, self.ring, self.max_requests = block_tokens, bool(ring), max_requests
        self.scratch = torch.zeros(DFLASH_POOL_SCRATCH, dtype=torch.uint8, device=device)
        self.device = self.scratch.device

    def _pool(self, lens, table, free, free_count):
        rows, blocks = table.shape
        return dflash_pool(self.block_tokens, free.numel(), rows, blocks, int(self.ring), _ints("lens", lens, rows, self.device),
                           _ints("table", table, None, self.device), _ints("free", free, None, self.device),
                           _ints("free_count", free_count, 1, self.device), self.scratch.data_ptr())

    def reserve(self, n_new, lens, table, free, free_count, slots, row_start, granted, requests=None, stream=None) -> int:
        """n_new[i] more tokens for table row requests[i] (None: row i); fills slots, row_start and granted."""
        n = n_new.numel()
        p = self._pool(lens, table, free, free_count)
        d = self.device
        return _check(lib().dflash_pool_reserve(ctypes.byref(p), n, _ints("requests", requests, n, d), _ints("n_new", n_new, n, d),
                                                _ints("slots", slots, None, d), slots.numel(), _ints("row_start", row_start, n + 1, d),
                                                _ints("granted", granted, n, d), _stream_ptr(stream)), "dflash_pool_reserve")

    def truncate(self, new_len, lens, table, free, free_count, requests=None, stream=None) -> int:
        """Shorten table row requests[i] to new_len[i] tokens and give the blocks behind them back."""
        n = new_len.numel()
        p = self._pool(lens, table, free, free_count)
        return _check(lib().dflash_pool_truncate(ctypes.byref(p), n, _ints("requests", requests, n, self.device),
                                                 _ints("new_len", new_len, n, self.device), _stream_ptr(stream)), "dflash_pool_truncate")


class Cache:
    """A dflash_cache over the caller's codes and scales.

    k, v: e4m3 codes (torch.float8_e4m3fn or uint8) [layers][blocks][KV heads][block tokens][head_dim], the same
    strides for both, contiguous in the last dimension (any order of the others: permuted views are
    taken as they are). k_scale, v_scale: fp32 [layers][blocks][KV heads], contiguous.
    max_requests, max_q and n_q_heads bound the attention calls and size their workspace; without
    them the object appends only."""

    def __init__(self, k, v, k_scale, v_scale, max_requests: int = 0, max_q: int = 0, n_q_heads: int = 0, stream=None):
        import torch
        layers, blocks, heads, tokens, head_dim = k.shape
        for name, t in (("k", k), ("v", v)):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.shape != k.shape or t.stride() != k.stride() or t.stride(-1) != 1 \
                    or t.device != k.device:
                raise ValueError(f"{name}: e4m3 codes [layers][blocks][heads][tokens][head_dim] are wanted, K and V alike")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or tuple(t.shape) != (layers, blocks, heads) or not t.is_contiguous() or t.device != k.device:
                raise ValueError(f"{name}: contiguous fp32 [layers][blocks][heads] is wanted")
        self.tensors = (k, v, k_scale, v_scale)
        self.device, self.heads, self.head_dim = k.device, heads, head_dim
        self.n_q_heads, self.max_q = n_q_heads, max_q
        cfg = dflash_cache_config(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), layers, blocks, tokens,
                                  heads, head_dim, *k.stride()[:4], n_q_heads, max_requests, max_q)
        nbytes = lib().dflash_cache_workspace_bytes(ctypes.byref(cfg))
        if nbytes == 0:
            raise DFlashError(DFLASH_EINVAL, "dflash_cache_workspace_bytes")
        self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=k.device)
        base = (self.workspace.data_ptr() + 255) // 256 * 256
        h = ctypes.c_void_p()
        _check(lib().dflash_cache_create(ctypes.byref(cfg), base, nbytes, _stream_ptr(stream), ctypes.byref(h)), "dflash_cache_create")
        self.h = h

    def append(self, slots, k_rows, v_rows, layer: int = 0, stream=None) -> int:
        """Quantise rows [layers'][n][KV heads][head_dim] (or [n][KV heads][head_dim]: one layer) into their
        slots, for layers layer .. layer + layers' - 1."""
        n = slots.numel()
        shape = (n, self.heads, self.head_dim)
        dtype = _row_dtype(k_rows)
        n_layers = k_rows.shape[0] if k_rows.dim() == 4 else 1
        if v_rows.shape != k_rows.shape:
            raise ValueError("k_rows and v_rows have different shapes")
        k = _rows("k_rows", k_rows, shape, self.device, k_rows.dtype)
        v = _rows("v_rows", v_rows, shape, self.device, k_rows.dtype)
        return _check(lib().dflash_cache_append(self.h, layer, n_layers, n, _ints("slots", slots, n, self.device), ctypes.byref(k),
                                                ctypes.byref(v), dtype, _stream_ptr(stream)), "dflash_cache_append")

    def attention(self, q, lens, table, out, layer: int = 0, row_start=None, max_q: int | None = None, k_own=None, v_own=None,
                  window: int = 0, causal: bool = False, scale: float | None = None, requests=None, stream=None) -> int:
        """out[row][head] = softmax attention of q [rows][query heads][head_dim] over the cached rows of each
        request (and its own rows k_own, v_own [rows][KV heads][head_dim]). row_start int32 [requests + 1]:
        the rows of each request (None: max_q rows each). max_q defaults to the limit given at creation
        when row_start is given, else to rows / requests. scale defaults to head_dim ** -0.5."""
        if not self.max_q:
            raise DFlashError(DFLASH_EINVAL, "dflash_cache_attention (the cache was made without attention limits)")
        d, dt, n_rows = self.device, q.dtype, q.shape[0]
        dtype = _row_dtype(q)
        table_rows, table_blocks = table.shape
        if requests is not None:
            n_req = requests.numel()
        elif row_start is not None:
            n_req = row_start.numel() - 1
        else:
            n_req = lens.numel()
        if max_q is None:
            max_q = self.max_q if row_start is not None else n_rows // max(n_req, 1)
        q_shape, kv_shape = (n_rows, self.n_q_heads, self.head_dim), (n_rows, self.heads, self.head_dim)
        a = dflash_attention(layer, n_req, n_rows, max_q, table_rows, table_blocks, _ints("requests", requests, n_req, d),
                             _ints("lens", lens, table_rows, d), _ints("table", table, None, d),
                             _ints("row_start", row_start, n_req + 1, d), dtype, _rows("q", q, q_shape, d, dt),
                             _rows("out", out, q_shape, d, dt), _rows("k_own", k_own, kv_shape, d, dt),
                             _rows("v_own", v_own, kv_shape, d, dt), int(causal), window,
                             self.head_dim ** -0.5 if scale is None else scale)
        return _check(lib().dflash_cache_attention(self.h, ctypes.byref(a), _stream_ptr(stream)), "dflash_cache_attention")

    def check_errors(self, stream=None) -> int:
        return _check(lib().dflash_cache_check_errors(self.h, _stream_ptr(stream)), "dflash_cache_check_errors")

    def close(self):
        if getattr(self, "h", None):
            lib().dflash_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
