"""Binding of the paged key/value cache calls (``include/cccl_kv.h``): append
tokens, take tokens out, attend.

A serving program keeps one ``KvCache`` per layer and one workspace, makes a
``KvBatch`` per step, and enqueues ``cccl_kv_write`` and ``cccl_kv_attention``
with it.  Nothing here computes, and there is no fallback.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (CCCL_DTYPE_BF16, CCCL_DTYPE_FP16, CCCL_ERR_INVALID_ARG, CcclError, _check, _lib, _stream,
               cccl_get_result)

CCCL_KV_16BIT, CCCL_KV_INT8, CCCL_KV_E4M3 = 0, 1, 2
KV_MAX_BATCH, KV_MAX_DIM, KV_MAX_HEADS = 1024, 128, 4096

_i32, _i64, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("dtype", _i32), ("format", _i32),
                ("kv_heads", _i32), ("head_dim", _i32), ("page_tokens", _i32), ("reserved", _i32), ("pages", _i64),
                ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64), ("scale_page_stride", _i64),
                ("scale_token_stride", _i64), ("scale_head_stride", _i64)]


class _Batch(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("cu_tokens", _vp), ("kv_lens", _vp), ("table_stride", _i64), ("n_tokens", _i64),
                ("batch", _i32), ("table_pages", _i32), ("max_new", _i32), ("max_len", _i32)]


# the current stream's handle without a Stream object (a decoding step makes many calls)
_current_stream = torch._C._cuda_getCurrentRawStream
_lib.cccl_kv_clear_status.argtypes = [_vp, _sz, _vp]
_lib.cccl_kv_clear_status.restype = ctypes.c_int
_lib.cccl_kv_workspace_bytes.argtypes = [_vp, _vp, ctypes.c_int]
_lib.cccl_kv_workspace_bytes.restype = _sz
for _f in (_lib.cccl_kv_write, _lib.cccl_kv_read):
    _f.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _sz, _vp]
    _f.restype = ctypes.c_int
_lib.cccl_kv_attention.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i64, _i64, ctypes.c_float, ctypes.c_int, _i64, _vp,
                                   _i64, _i64, _vp, _vp, _sz, _vp]
_lib.cccl_kv_attention.restype = ctypes.c_int

_write, _read, _attention = _lib.cccl_kv_write, _lib.cccl_kv_read, _lib.cccl_kv_attention
_DTYPE = {torch.bfloat16: CCCL_DTYPE_BF16, torch.float16: CCCL_DTYPE_FP16}
_CODES = (torch.int8, torch.uint8, torch.float8_e4m3fn)


class KvCache:
    """One layer's paged cache: tensors k and v of shape [pages, page_tokens,
    kv_heads, head_dim] with equal strides (any order of the first three axes;
    the last is contiguous), 16-bit values or one-byte codes, and for codes the
    binary32 scales [pages, page_tokens, kv_heads].  ``dtype`` is the type of
    the values passed in and out."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None, *, dtype: torch.dtype | None = None, fmt: int = CCCL_KV_16BIT):
        if dtype is None:
            dtype = k.dtype
        if dtype not in _DTYPE:
            raise TypeError("values are bfloat16 or float16, got %s" % (dtype,))
        if fmt not in (CCCL_KV_16BIT, CCCL_KV_INT8, CCCL_KV_E4M3):
            raise ValueError("unknown cache format %r" % (fmt,))
        if fmt == CCCL_KV_16BIT:
            if k.dtype != dtype or v.dtype != dtype:
                raise TypeError("a 16-bit cache holds values of its dtype")
            if k_scale is not None or v_scale is not None:
                raise ValueError("a 16-bit cache has no scales")
        elif k.dtype not in _CODES or v.dtype not in _CODES:
            raise TypeError("codes are one-byte tensors (int8, uint8 or float8_e4m3fn)")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or k.stride(3) != 1:
            raise ValueError("k and v are [pages, page_tokens, kv_heads, head_dim] with equal strides, "
                             "the last axis contiguous")
        if fmt != CCCL_KV_16BIT:
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.float32 or s.shape != k.shape[:3] or s.stride() != k_scale.stride():
                    raise ValueError("scales are float32 [pages, page_tokens, kv_heads] with equal strides")
        self.k, self.v, self.k_scale, self.v_scale, self.dtype, self.fmt = k, v, k_scale, v_scale, dtype, fmt
        pages, page_tokens, heads, dim = k.shape
        ss = k_scale.stride() if k_scale is not None else (0, 0, 0)
        self.kv_heads, self.head_dim, self.page_tokens, self.pages = heads, dim, page_tokens, pages
        self._c = _Cache(k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
                         None if v_scale is None else v_scale.data_ptr(), _DTYPE[dtype], fmt, heads, dim, page_tokens,
                         0, pages, k.stride(0), k.stride(1), k.stride(2), *ss)
        self._ref = ctypes.addressof(self._c)
        self._device, self._scale = k.get_device(), 1.0 / math.sqrt(dim)

    @classmethod
    def empty(cls, pages: int, page_tokens: int, kv_heads: int, head_dim: int, *, dtype: torch.dtype = torch.bfloat16,
              fmt: int = CCCL_KV_16BIT, device=None) -> "KvCache":
        """A new cache, tokens outermost in a page; its contents are undefined until written."""
        device = device or "cuda"
        store = {CCCL_KV_16BIT: dtype, CCCL_KV_INT8: torch.int8, CCCL_KV_E4M3: torch.float8_e4m3fn}.get(fmt)
        if store is None:
            raise ValueError("unknown cache format %r" % (fmt,))
        k, v = (torch.empty(pages, page_tokens, kv_heads, head_dim, dtype=store, device=device) for _ in range(2))
        ks = vs = None
        if fmt != CCCL_KV_16BIT:  # a head's scales lie together: attention reads one head at a time
            ks, vs = (torch.empty(pages, kv_heads, page_tokens, device=device).transpose(1, 2) for _ in range(2))
        return cls(k, v, ks, vs, dtype=dtype, fmt=fmt)


class KvBatch:
    """The sequences of one call: ``page_table`` [batch, pages of the longest],
    ``cu_tokens`` [batch + 1] and ``kv_lens`` [batch], all int32 on the device.
    ``n_tokens`` rows are in the packed tensors; ``max_new`` and ``max_len`` are
    the most new tokens and the longest length the program expects of a
    sequence (they choose kernels and how work is divided: results may differ
    in their rounding and no more)."""

    def __init__(self, page_table: torch.Tensor, cu_tokens: torch.Tensor, kv_lens: torch.Tensor, *, n_tokens: int,
                 max_new: int, max_len: int):
        for t, what, axes in ((page_table, "page_table", 2), (cu_tokens, "cu_tokens", 1), (kv_lens, "kv_lens", 1)):
            if t.dtype != torch.int32 or t.dim() != axes or (t.numel() > 0 and t.stride(-1) != 1):
                raise TypeError("%s is a %d-dimensional int32 tensor, contiguous in its last axis" % (what, axes))
        batch = kv_lens.numel()
        if cu_tokens.numel() != batch + 1 or page_table.shape[0] != batch:
            raise ValueError("page_table has a row, kv_lens an entry and cu_tokens one more for each sequence")
        width = page_table.shape[1]
        row = page_table.stride(0) if batch > 1 else width
        if row < width:
            raise ValueError("page_table's rows overlap (an expanded table has to be copied: .contiguous())")
        self.page_table, self.cu_tokens, self.kv_lens = page_table, cu_tokens, kv_lens
        self.n_tokens, self.batch = int(n_tokens), batch
        self._c = _Batch(page_table.data_ptr(), cu_tokens.data_ptr(), kv_lens.data_ptr(),
                         row, self.n_tokens, batch, width, int(max_new), int(max_len))
        self._ref = ctypes.addressof(self._c)


def cccl_kv_workspace_bytes(cache: KvCache, batch: KvBatch, q_heads: int = 0) -> int:
    """Bytes of a workspace for these calls; 0 for arguments they refuse."""
    return int(_lib.cccl_kv_workspace_bytes(cache._ref, batch._ref, q_heads))


def cccl_kv_clear_status(ws: torch.Tensor, stream=None) -> None:
    """Enqueue zeroing of the workspace's status header (once, before its first use)."""
    _check(_lib.cccl_kv_clear_status(ws.data_ptr(), ws.nbytes, _stream(stream)), "cccl_kv_clear_status")


def _raw_stream(cache: KvCache, stream) -> int:
    return _current_stream(cache._device) if stream is None else stream.cuda_stream


def _packed(x: torch.Tensor, cache: KvCache, n_tokens: int, heads: int, what: str) -> tuple[int, int]:
    """Token and head stride of a packed [n_tokens, heads, head_dim] tensor."""
    if x.dtype is not cache.dtype:
        raise TypeError("%s: expected %s, got %s" % (what, cache.dtype, x.dtype))
    if x.shape == (n_tokens, heads, cache.head_dim):
        token, head, inner = x.stride()
        if inner == 1:
            return token, head
    raise ValueError("%s: expected [n_tokens, heads, head_dim], contiguous in its last axis" % what)


def cccl_kv_write(cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor, ws: torch.Tensor,
                  stream=None) -> None:
    """Enqueue storing of ``k`` and ``v`` [n_tokens, kv_heads, head_dim] in the cache."""
    kt, kh = _packed(k, cache, batch.n_tokens, cache.kv_heads, "k")
    vt, vh = _packed(v, cache, batch.n_tokens, cache.kv_heads, "v")
    status = _write(cache._ref, batch._ref, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, ws.data_ptr(), ws.nbytes,
                    _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_kv_write")


def cccl_kv_read(cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor, ws: torch.Tensor,
                 stream=None) -> None:
    """Enqueue reading of the batch's tokens into ``k`` and ``v`` [n_tokens, kv_heads, head_dim]."""
    kt, kh = _packed(k, cache, batch.n_tokens, cache.kv_heads, "k")
    vt, vh = _packed(v, cache, batch.n_tokens, cache.kv_heads, "v")
    status = _read(cache._ref, batch._ref, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, ws.data_ptr(), ws.nbytes,
                   _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_kv_read")


def cccl_kv_attention(cache: KvCache, batch: KvBatch, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *,
                      scale: float | None = None, causal: bool = True, window: int = 0,
                      lse: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue attention of ``q`` [n_tokens, q_heads, head_dim] over the cache
    into ``out`` (same shape); ``lse`` (float32 [n_tokens, q_heads], contiguous)
    receives the log of each row's sum.  ``scale`` defaults to head_dim ** -0.5."""
    heads = q.shape[1]
    qt, qh = _packed(q, cache, batch.n_tokens, heads, "q")
    ot, oh = _packed(out, cache, batch.n_tokens, heads, "out")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse: expected a contiguous float32 [n_tokens, q_heads]")
    status = _attention(cache._ref, batch._ref, q.data_ptr(), heads, qt, qh, cache._scale if scale is None else scale,
                        1 if causal else 0, window, out.data_ptr(), ot, oh, None if lse is None else lse.data_ptr(),
                        ws.data_ptr(), ws.nbytes, _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_kv_attention")


# ---------------------------------------------------------------- conveniences
def empty_kv_workspace(cache: KvCache, batch: KvBatch, q_heads: int = 0) -> torch.Tensor:
    """A workspace for these calls, its status header zeroed."""
    n = cccl_kv_workspace_bytes(cache, batch, q_heads)
    if n == 0:
        raise CcclError(CCCL_ERR_INVALID_ARG, "cccl_kv_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.k.device)
    ws[:16].zero_()
    return ws


def _finish(ws: torch.Tensor, what: str) -> None:
    _, dev = cccl_get_result(ws, None)
    _check(dev, what + " (device)")


def _hand_over(stream, *outs: torch.Tensor) -> None:
    """Results that `stream`'s memory holds are used on the current stream from here on."""
    if stream is not None:
        for t in outs:
            t.record_stream(torch.cuda.current_stream(t.device))


def kv_write(cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Store and wait."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch)
        cccl_kv_write(cache, batch, k, v, ws)
        _finish(ws, "cccl_kv_write")


def kv_read(cache: KvCache, batch: KvBatch, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Read and wait; returns k and v [n_tokens, kv_heads, head_dim] (rows of no sequence: undefined)."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch)
        shape = (batch.n_tokens, cache.kv_heads, cache.head_dim)
        k, v = (torch.empty(shape, dtype=cache.dtype, device=cache.k.device) for _ in range(2))
        cccl_kv_read(cache, batch, k, v, ws)
        _finish(ws, "cccl_kv_read")
    _hand_over(stream, k, v)
    return k, v


def kv_attention(cache: KvCache, batch: KvBatch, q: torch.Tensor, *, scale: float | None = None, causal: bool = True,
                 window: int = 0, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Attend and wait; returns the result [n_tokens, q_heads, head_dim] and each row's log-sum-exp (rows of no
    sequence: undefined)."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch, q.shape[1])
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        cccl_kv_attention(cache, batch, q, out, ws, scale=scale, causal=causal, window=window, lse=lse)
        _finish(ws, "cccl_kv_attention")
    _hand_over(stream, out, lse)
    return out, lse
