"""Python binding of the paged 8-bit context cache (include/dflash.h): block tables, the quantising
append and attention over the cache. Argument marshalling and checks only, as in the package's
``Handle``; every tensor is the caller's, on one CUDA device."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import (DFLASH_BF16, DFLASH_EINVAL, DFLASH_F16, DFLASH_F32, DFLASH_POOL_MAX_REQUESTS, DFLASH_POOL_SCRATCH, DFlashError, _check,
               dflash_attention, dflash_cache_config, dflash_pool, dflash_rows, lib)

_ROW_DTYPES = {torch.float32: DFLASH_F32, torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_F16}
# dflash_attention, dflash_pool and dflash_rows as one struct.pack each: a call's arguments are a few dozen words, and
# setting them one by one through ctypes takes longer than the kernels of a small call
_ATTENTION, _POOL, _ROWS = struct.Struct("@6i4Qi4Q4Q4Q4Q2if"), struct.Struct("@5i5Q"), struct.Struct("@4Q")
_NO_ROWS = (0, 0, 0, 0)


def _row_dtype(t) -> int:
    code = _ROW_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"rows are fp32, bf16 or f16, not {t.dtype}")
    return code


def _ints(name, t, n, device):
    """The address of a contiguous int32 tensor of n elements on CUDA device number `device` (None: NULL)."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != device or (n is not None and t.numel() != n):
        raise ValueError(f"{name}: a contiguous int32 tensor{'' if n is None else f' of {n} elements'} on CUDA device {device} is wanted")
    return t.data_ptr()


def _rows(name, t, n, heads, head_dim, device, dtype):
    """The words of dflash_rows for a [..., n rows, heads, head_dim] tensor with contiguous last dimension."""
    if t is None:
        return _NO_ROWS
    shape, stride = t.shape, t.stride()
    if not 3 <= len(shape) <= 4 or shape[-3] != n or shape[-2] != heads or shape[-1] != head_dim or t.dtype is not dtype \
            or t.get_device() != device or stride[-1] != 1:
        raise ValueError(f"{name}: {dtype} rows of shape {(n, heads, head_dim)} on CUDA device {device} are wanted, contiguous in the last dimension")
    return t.data_ptr(), stride[0] if len(shape) == 4 else 0, stride[-3], stride[-2]


class _OnStreams:
    """Device memory of the object's own, and the streams that its calls ran on: PyTorch hands memory of a dropped object out again
    once the work that was on them then is done. (Not for a stream given as a number, which may be gone by then:
    whoever passes one keeps the object until its calls have run, as for calls captured into a graph.)"""

    def _own(self, memory):
        self._memory, self._streams = memory, {torch._C._cuda_getCurrentRawStream(memory.get_device())}

    def _stream(self, stream) -> int:
        """A cudaStream_t: the given stream's, or the one current on the tensors' device."""
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(self.device)
        elif hasattr(stream, "cuda_stream"):
            raw = stream.cuda_stream
        else:
            return int(stream)
        if raw not in self._streams:
            self._memory.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
            self._streams.add(raw)
        return raw


class BlockPool(_OnStreams):
    """Block tables over a pool of blocks of ``block_tokens`` tokens (dflash_pool_reserve and
    dflash_pool_truncate). Holds the calls' 256 bytes of device scratch; lens, table and the stack of
    free blocks are the caller's tensors:

      lens int32 [rows], table int32 [rows][blocks per request], free int32 [blocks], free_count int32 [1]

    ring: requests may grow without end, and a window of w needs ceil((w + n - 1) / block_tokens) + 1 blocks per
    request, n the most rows of a call that are attended causally or given back (dflash_pool.ring).
    """

    def __init__(self, block_tokens: int, max_requests: int | None = None, ring: bool = False, device="cuda"):
        if block_tokens not in (16, 32, 64, 128) or (max_requests is not None and not 0 < max_requests <= DFLASH_POOL_MAX_REQUESTS):
            raise DFlashError(DFLASH_EINVAL, "BlockPool")
        if torch.device(device).type != "cuda":
            raise ValueError(f"BlockPool: its tensors are on a CUDA device, not on {device}")
        self.block_tokens, self.ring, self.max_requests = block_tokens, int(ring), max_requests
        self.scratch = torch.zeros(DFLASH_POOL_SCRATCH, dtype=torch.uint8, device=device)
        self.device = self.scratch.get_device()
        self._own(self.scratch)
        self.p = dflash_pool()
        self._reserve, self._truncate = lib().dflash_pool_reserve, lib().dflash_pool_truncate

    def _pool(self, n, lens, table, free, free_count):
        if self.max_requests is not None and n > self.max_requests:
            raise DFlashError(DFLASH_EINVAL, f"BlockPool: {n} requests, limit {self.max_requests}")
        (rows, blocks), d = table.shape, self.device
        _POOL.pack_into(self.p, 0, self.block_tokens, free.numel(), rows, blocks, self.ring, _ints("lens", lens, rows, d),
                        _ints("table", table, None, d), _ints("free", free, None, d), _ints("free_count", free_count, 1, d),
                        self.scratch.data_ptr())
        return ctypes.byref(self.p)

    def reserve(self, n_new, lens, table, free, free_count, slots, row_start, granted, requests=None, stream=None) -> int:
        """n_new[i] more tokens for table row requests[i] (None: row i); fills slots, row_start and granted."""
        n, d = n_new.numel(), self.device
        return _check(self._reserve(self._pool(n, lens, table, free, free_count), n, _ints("requests", requests, n, d),
                                    _ints("n_new", n_new, n, d), _ints("slots", slots, None, d), slots.numel(),
                                    _ints("row_start", row_start, n + 1, d), _ints("granted", granted, n, d),
                                    self._stream(stream)), "dflash_pool_reserve")

    def truncate(self, new_len, lens, table, free, free_count, requests=None, stream=None) -> int:
        """Shorten table row requests[i] to new_len[i] tokens and give the blocks behind them back."""
        n, d = new_len.numel(), self.device
        return _check(self._truncate(self._pool(n, lens, table, free, free_count), n, _ints("requests", requests, n, d),
                                     _ints("new_len", new_len, n, d), self._stream(stream)), "dflash_pool_truncate")


class Cache(_OnStreams):
    """A dflash_cache over the caller's codes and scales.

    k, v: e4m3 codes (torch.float8_e4m3fn or uint8) [layers][blocks][KV heads][block tokens][head_dim], the same
    strides for both, contiguous in the last dimension (any order of the others: permuted views are
    taken as they are). k_scale, v_scale: fp32 [layers][blocks][KV heads], contiguous.
    max_requests, max_q and n_q_heads bound the attention calls and size their workspace; without
    them the object appends only."""

    def __init__(self, k, v, k_scale, v_scale, max_requests: int = 0, max_q: int = 0, n_q_heads: int = 0, stream=None):
        layers, blocks, heads, tokens, head_dim = k.shape
        for name, t in (("k", k), ("v", v)):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or t.shape != k.shape or t.stride() != k.stride() or t.stride(-1) != 1 \
                    or t.device != k.device:
                raise ValueError(f"{name}: e4m3 codes [layers][blocks][heads][tokens][head_dim] are wanted, K and V alike")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or tuple(t.shape) != (layers, blocks, heads) or not t.is_contiguous() or t.device != k.device:
                raise ValueError(f"{name}: contiguous fp32 [layers][blocks][heads] is wanted")
        self.tensors = (k, v, k_scale, v_scale)
        self.device, self.heads, self.head_dim = k.get_device(), heads, head_dim
        self.n_q_heads, self.max_q = n_q_heads, max_q
        cfg = dflash_cache_config(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), layers, blocks, tokens,
                                  heads, head_dim, *k.stride()[:4], n_q_heads, max_requests, max_q)
        nbytes = lib().dflash_cache_workspace_bytes(ctypes.byref(cfg))
        if nbytes == 0:
            raise DFlashError(DFLASH_EINVAL, "dflash_cache_workspace_bytes")
        if not k.is_cuda or self.device != torch.cuda.current_device():
            raise ValueError(f"the codes are on {k.device}, not on the current CUDA device")
        self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=k.device)
        self._own(self.workspace)
        base = (self.workspace.data_ptr() + 255) // 256 * 256
        h = ctypes.c_void_p()
        _check(lib().dflash_cache_create(ctypes.byref(cfg), base, nbytes, self._stream(stream), ctypes.byref(h)),
               "dflash_cache_create")
        self.h = h
        self._k, self._v, self._a = dflash_rows(), dflash_rows(), dflash_attention()
        self._append, self._attention = lib().dflash_cache_append, lib().dflash_cache_attention

    def append(self, slots, k_rows, v_rows, layer: int = 0, stream=None) -> int:
        """Quantise rows [layers'][n][KV heads][head_dim] (or [n][KV heads][head_dim]: one layer) into their
        slots, for layers layer .. layer + layers' - 1."""
        n, d, dt = slots.numel(), self.device, k_rows.dtype
        if v_rows.shape != k_rows.shape:
            raise ValueError("k_rows and v_rows have different shapes")
        _ROWS.pack_into(self._k, 0, *_rows("k_rows", k_rows, n, self.heads, self.head_dim, d, dt))
        _ROWS.pack_into(self._v, 0, *_rows("v_rows", v_rows, n, self.heads, self.head_dim, d, dt))
        return _check(self._append(self.h, layer, k_rows.shape[0] if k_rows.dim() == 4 else 1, n, _ints("slots", slots, n, d),
                                   ctypes.byref(self._k), ctypes.byref(self._v), _row_dtype(k_rows), self._stream(stream)),
                      "dflash_cache_append")

    def attention(self, q, lens, table, out, layer: int = 0, row_start=None, max_q: int | None = None, k_own=None, v_own=None,
                  window: int = 0, causal: bool = False, scale: float | None = None, requests=None, stream=None) -> int:
        """out[row][head] = softmax attention of q [rows][query heads][head_dim] over the cached rows of each
        request (and its own rows k_own, v_own [rows][KV heads][head_dim]). row_start int32 [requests + 1]:
        the rows of each request (None: max_q rows each). max_q defaults to the limit given at creation
        when row_start is given, else to rows / requests. scale defaults to head_dim ** -0.5."""
        if not self.max_q:
            raise DFlashError(DFLASH_EINVAL, "dflash_cache_attention (the cache was made without attention limits)")
        d, dt, n_rows, heads, hd = self.device, q.dtype, q.shape[0], self.heads, self.head_dim
        table_rows, table_blocks = table.shape
        if requests is not None:
            n_req = requests.numel()
        elif row_start is not None:
            n_req = row_start.numel() - 1
        else:
            n_req = lens.numel()
        if max_q is None:
            max_q = self.max_q if row_start is not None else n_rows // max(n_req, 1)
        _ATTENTION.pack_into(self._a, 0, layer, n_req, n_rows, max_q, table_rows, table_blocks, _ints("requests", requests, n_req, d),
                             _ints("lens", lens, table_rows, d), _ints("table", table, None, d),
                             _ints("row_start", row_start, n_req + 1, d), _row_dtype(q), *_rows("q", q, n_rows, self.n_q_heads, hd, d, dt),
                             *_rows("out", out, n_rows, self.n_q_heads, hd, d, dt), *_rows("k_own", k_own, n_rows, heads, hd, d, dt),
                             *_rows("v_own", v_own, n_rows, heads, hd, d, dt), causal, window, hd ** -0.5 if scale is None else scale)
        return _check(self._attention(self.h, ctypes.byref(self._a), self._stream(stream)), "dflash_cache_attention")

    def check_errors(self, stream=None) -> int:
        return _check(lib().dflash_cache_check_errors(self.h, self._stream(stream)), "dflash_cache_check_errors")

    def set_wait_limit(self, limit_us: int) -> int:
        """Test hook: limit of the attention's bounded waits in microseconds (0: the 1 s default)."""
        return _check(lib().dflash_cache_set_wait_limit(self.h, limit_us), "dflash_cache_set_wait_limit")

    def debug_stall(self, cta: int) -> int:
        """Test hook: CTA `cta` of the next attention call gets no keys (cta < 0 disarms)."""
        return _check(lib().dflash_cache_debug_stall(self.h, cta), "dflash_cache_debug_stall")

    def close(self):
        if getattr(self, "h", None):
            lib().dflash_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
