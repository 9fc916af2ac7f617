"""Binding of a step with drafted tokens (``include/cccl_step.h``): plan, write
with rotary positions, attend over a tree, verify, keep.

A serving program keeps a ``StepTables`` for all sequences, a ``StepRotary``
for its model and one workspace, and enqueues, a step: ``cccl_step_plan``, and
with the ``KvBatch`` of what it wrote, for every layer ``cccl_step_write`` and
``cccl_step_attention``; then ``cccl_step_verify``, and for every layer
``cccl_step_keep``.  Nothing here computes, and there is no fallback.
"""

from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check, _lib
from .kv import KvBatch, KvCache, _current_stream, _finish, _hand_over, _packed, _raw_stream, empty_kv_workspace

STEP_MAX_DRAFT, STEP_MAX_VOCAB = 1024, 1 << 20
_int32 = torch.int32

_i32, _i64, _vp, _sz, _int = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int


class _Tables(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("held", _vp), ("free_pages", _vp), ("free_count", _vp), ("table_stride", _i64),
                ("free_capacity", _i64), ("batch", _i32), ("table_pages", _i32), ("page_tokens", _i32),
                ("reserved", _i32)]


class _Out(ctypes.Structure):
    _fields_ = [("cu_tokens", _vp), ("kv_lens", _vp), ("held", _vp), ("free_count", _vp), ("slots", _vp),
                ("positions", _vp), ("mask", _vp), ("mask_stride", _i64), ("rows", _i64), ("mask_words", _i32),
                ("reserved", _i32)]


class _Rotary(ctypes.Structure):
    _fields_ = [("turns", _vp), ("magnitude", ctypes.c_float), ("rot_dim", _i32), ("interleaved", _i32),
                ("reserved", _i32)]


class _Draft(ctypes.Structure):
    _fields_ = [("p", _vp), ("q", _vp), ("p_stride", _i64), ("q_stride", _i64), ("tokens", _vp), ("parents", _vp),
                ("uniform", _vp), ("cu_tokens", _vp), ("rows", _i64), ("batch", _i32), ("vocab", _i32)]


_double = ctypes.c_double
_lib.cccl_step_plan.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.cccl_step_rotary_turns.argtypes = [_int, _double, _double, _double, _double, _double, _vp]
_lib.cccl_step_write.argtypes = [_vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                                 _i64, _vp, _sz, _vp]
_lib.cccl_step_attention.argtypes = [_vp, _vp, _vp, _int, _i64, _i64, ctypes.c_float, _vp, _i64, _int, _i64, _vp, _i64,
                                     _i64, _vp, _vp, _sz, _vp]
_lib.cccl_step_verify.argtypes = [_vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.cccl_step_keep.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
for _f in (_lib.cccl_step_plan, _lib.cccl_step_rotary_turns, _lib.cccl_step_write, _lib.cccl_step_attention,
           _lib.cccl_step_verify, _lib.cccl_step_keep):
    _f.restype = _int
_plan, _write, _attention = _lib.cccl_step_plan, _lib.cccl_step_write, _lib.cccl_step_attention
_verify, _keep = _lib.cccl_step_verify, _lib.cccl_step_keep


# a call's host structures as bytes, which take less time to fill than ctypes' fields (their layouts are tested alike)
_pack_out = struct.Struct("@7P2q2i").pack
_pack_draft = struct.Struct("@2P2q4Pq2i").pack


def _numbers(t: torch.Tensor, dtype: torch.dtype, n: int | None, device: int, what: str) -> int:
    """The address of a contiguous [n] tensor on the call's device."""
    if t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    if t.dtype is not dtype or t.dim() != 1 or (n is not None and t.shape[0] != n) or \
            (t.shape[0] > 1 and t.stride(0) != 1):
        raise TypeError("%s: expected a contiguous %s of %s numbers" % (what, dtype, "some" if n is None else n))
    if t.get_device() != device:
        raise ValueError("%s is on another device" % what)
    return t.data_ptr()


def _maybe(t: torch.Tensor | None, dtype: torch.dtype, n: int, device: int, what: str) -> int:
    return 0 if t is None else _numbers(t, dtype, n, device, what)


def _stream_on(device: int, stream) -> int:
    if device < 0:
        raise ValueError("all tensors of a call are on one CUDA device")
    return _current_stream(device) if stream is None else stream.cuda_stream


def _strides(x: torch.Tensor, cache: KvCache, shape: tuple, what: str) -> tuple:
    """Token, head and value stride of a packed tensor of that shape, on the cache's device."""
    if x.get_device() != cache._device:
        raise ValueError("%s: all tensors of a call are on the cache's device" % what)
    if x.dtype is cache.dtype and x.shape == shape:
        s = x.stride()
        if s[2] == 1:
            return s
    return *_packed(x, cache, shape[0], shape[1], what), 1  # (says what is wrong)


def empty_step_workspace(device=None) -> torch.Tensor:
    """A workspace for any of these calls but attention, its status header zeroed."""
    return torch.zeros(16, dtype=torch.uint8, device=device or "cuda")


class StepTables:
    """Who holds which page: ``page_table`` [batch, most pages], ``held``
    [batch] (how many entries of its row a sequence holds), ``free_pages`` and
    ``free_count`` [1] (the first so many are nobody's), all int32 on one
    device."""

    def __init__(self, page_table: torch.Tensor, held: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                 *, page_tokens: int):
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
                (page_table.numel() > 0 and page_table.stride(1) != 1):
            raise TypeError("page_table is a 2-dimensional int32 tensor, contiguous in its last axis")
        batch, width = page_table.shape
        row = page_table.stride(0) if batch > 1 else width
        if row < width:
            raise ValueError("page_table's rows overlap (an expanded table has to be copied: .contiguous())")
        self._device = page_table.get_device()
        _numbers(held, torch.int32, batch, self._device, "held")
        _numbers(free_pages, torch.int32, None, self._device, "free_pages")
        _numbers(free_count, torch.int32, 1, self._device, "free_count")
        self.page_table, self.held, self.free_pages, self.free_count = page_table, held, free_pages, free_count
        self.page_tokens, self.batch = int(page_tokens), batch
        self._c = _Tables(page_table.data_ptr(), held.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), row,
                          free_pages.numel(), batch, width, self.page_tokens, 0)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, batch: int, table_pages: int, pages: int, page_tokens: int, device=None) -> "StepTables":
        """Nobody holds any of the pool's ``pages`` pages yet; they are given from page 0 on."""
        device = device or "cuda"
        return cls(torch.zeros(batch, table_pages, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device),
                   torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.full((1,), pages, dtype=torch.int32, device=device), page_tokens=page_tokens)


class StepRotary:
    """A model's rotary positions: the first ``rot_dim`` values of a head turn,
    in pairs half of that apart or side by side (``interleaved``), by
    base^(-2 i / rot_dim) radians a position.  Stretched for long contexts by
    ``factor``: all pairs alike, or with ``original_length`` by parts (pairs that
    turn fewer than ``few`` times over that length are slowed, those that turn
    more than ``many`` times are not, the others are mixed).  ``magnitude``
    multiplies what was turned."""

    def __init__(self, rot_dim: int, *, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
                 original_length: float = 0, few: float = 1.0, many: float = 32.0, magnitude: float = 1.0, device=None):
        host = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.int64)
        _check(_lib.cccl_step_rotary_turns(rot_dim, base, factor, original_length, few, many, host.data_ptr()),
               "cccl_step_rotary_turns")
        if not math.isfinite(magnitude):
            raise ValueError("magnitude is a finite number")
        self.turns, self.rot_dim, self.interleaved = host.to(device or "cuda"), int(rot_dim), bool(interleaved)
        self.magnitude = float(magnitude)
        self._device = self.turns.get_device()
        self._c = _Rotary(self.turns.data_ptr(), self.magnitude, self.rot_dim, 1 if interleaved else 0, 0)
        self._ref = ctypes.addressof(self._c)


def cccl_step_plan(tables: StepTables, lens: torch.Tensor, new: torch.Tensor, ws: torch.Tensor, *,
                   cu_tokens: torch.Tensor, kv_lens: torch.Tensor, held: torch.Tensor | None = None,
                   free_count: torch.Tensor | None = None, parents: torch.Tensor | None = None,
                   slots: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                   mask: torch.Tensor | None = None, rows: int | None = None, stream=None) -> None:
    """Enqueue the plan of ``new`` [batch] tokens on top of ``lens`` [batch] into
    ``cu_tokens`` [batch + 1], ``kv_lens`` [batch] and what else is given:
    ``slots`` (int64) and ``positions`` [rows], ``mask`` [rows, words] (int32).
    ``held`` and ``free_count`` receive the tables' new counts (default: in
    place).  ``parents`` [rows]: the trees; without, chains.  ``rows``: the rows
    of the packed tensors, where none of these says it."""
    dev, batch, i32 = tables._device, tables.batch, _int32
    if ws.get_device() != dev:
        raise ValueError("ws is on another device")
    held = tables.held if held is None else held
    free_count = tables.free_count if free_count is None else free_count
    if rows is None:
        for t in (slots, positions, mask, parents):
            if t is not None:
                rows = t.shape[0]
                break
        else:
            raise ValueError("rows: how many rows the packed tensors have")
    words, stride = (0, 0) if mask is None else _mask_of(mask, rows, dev)
    if rows == 0:  # an empty tensor has no address: no mask
        words = 0
    out = _pack_out(_numbers(cu_tokens, i32, batch + 1, dev, "cu_tokens"), _numbers(kv_lens, i32, batch, dev, "kv_lens"),
                    _numbers(held, i32, batch, dev, "held"), _numbers(free_count, i32, 1, dev, "free_count"),
                    _maybe(slots, torch.int64, rows, dev, "slots"), _maybe(positions, i32, rows, dev, "positions"),
                    0 if mask is None else mask.data_ptr(), stride, rows, words, 0)
    status = _plan(tables._ref, _numbers(lens, i32, batch, dev, "lens"), _numbers(new, i32, batch, dev, "new"),
                   _maybe(parents, i32, rows, dev, "parents"), out, ws.data_ptr(), ws.nbytes, _stream_on(dev, stream))
    if status:
        _check(status, "cccl_step_plan")


def _mask_of(mask: torch.Tensor, rows: int, device: int) -> tuple[int, int]:
    """Words of a mask's rows and the stride between them."""
    shape, stride = mask.shape, mask.stride()
    if mask.dtype is not _int32 or len(shape) != 2 or shape[0] != rows or shape[1] < 1 or stride[1] != 1:
        raise TypeError("mask: expected int32 [rows, words], contiguous in its last axis")
    if mask.get_device() != device:
        raise ValueError("mask is on another device")
    return shape[1], stride[0] if rows > 1 else shape[1]


def cccl_step_write(cache: KvCache, batch: KvBatch, rotary: StepRotary, q: torch.Tensor | None, k: torch.Tensor,
                    v: torch.Tensor, q_out: torch.Tensor | None, ws: torch.Tensor, *,
                    positions: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue rotation of ``q`` [n_tokens, q_heads, head_dim] into ``q_out``
    (the same tensor or another; both None: no queries) and of ``k``
    [n_tokens, kv_heads, head_dim], and storing of ``k`` and ``v`` in the cache.
    ``positions`` [n_tokens]: where rows stand (default: their places)."""
    n, dev = batch.n_tokens, cache._device
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if ws.get_device() != dev or rotary._device != dev:
        raise ValueError("all tensors of a call are on the cache's device")
    shape = (n, cache.kv_heads, cache.head_dim)
    kt, kh, _ = _strides(k, cache, shape, "k")
    vt, vh, _ = _strides(v, cache, shape, "v")
    heads = qt = qh = ot = oh = q_at = out_at = 0
    if q is not None:
        heads = q.shape[1]
        shape = (n, heads, cache.head_dim)
        qt, qh, _ = _strides(q, cache, shape, "q")
        ot, oh, _ = _strides(q_out, cache, shape, "q_out")
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    status = _write(cache._ref, batch._ref, rotary._ref, _maybe(positions, _int32, n, dev, "positions"), q_at, heads, qt, qh,
                    out_at, ot, oh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, ws.data_ptr(), ws.nbytes,
                    _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_step_write")


def cccl_step_attention(cache: KvCache, batch: KvBatch, q: torch.Tensor, mask: torch.Tensor, out: torch.Tensor,
                        ws: torch.Tensor, *, scale: float | None = None, window: int = 0,
                        lse: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue attention of drafted tokens ``q`` [n_tokens, q_heads, head_dim]
    over what was cached before them and the ones among themselves whose bits
    are set in ``mask`` [n_tokens, words] (int32), into ``out`` (same shape);
    ``lse`` (float32 [n_tokens, q_heads], contiguous) receives the log of each
    row's sum.  ``scale`` defaults to head_dim ** -0.5."""
    heads, dev = q.shape[1], cache._device
    shape = (batch.n_tokens, heads, cache.head_dim)
    qt, qh, _ = _strides(q, cache, shape, "q")
    ot, oh, _ = _strides(out, cache, shape, "out")
    words, stride = _mask_of(mask, batch.n_tokens, dev)
    if ws.get_device() != dev or (lse is not None and lse.get_device() != dev):
        raise ValueError("all tensors of a call are on the cache's device")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse: expected a contiguous float32 [n_tokens, q_heads]")
    status = _attention(cache._ref, batch._ref, q.data_ptr(), heads, qt, qh, cache._scale if scale is None else scale,
                        mask.data_ptr(), stride, words, window, out.data_ptr(), ot, oh,
                        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_step_attention")


def _probabilities(x: torch.Tensor, rows: int, vocab: int, what: str) -> int:
    """The stride between rows."""
    shape, stride = x.shape, x.stride()
    if x.dtype is not torch.float32 or len(shape) != 2 or shape[0] != rows or shape[1] != vocab or \
            (vocab > 1 and stride[1] != 1):
        raise TypeError("%s: expected float32 [rows, vocab], contiguous in its last axis" % what)
    return stride[0] if rows > 1 else vocab


def cccl_step_verify(p: torch.Tensor, q: torch.Tensor | None, tokens: torch.Tensor, parents: torch.Tensor | None,
                     uniform: torch.Tensor, cu_tokens: torch.Tensor, path: torch.Tensor, n_kept: torch.Tensor,
                     next_token: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Enqueue verification of drafted ``tokens`` [rows] against the target's
    probabilities ``p`` [rows, vocab], with the draft's ``q`` (or None) and the
    random numbers ``uniform`` [rows] (float32, 0 <= u < 1), into ``path``
    [rows], ``n_kept`` and ``next_token`` [batch] (int32)."""
    rows, vocab = p.shape
    dev, batch, i32 = p.get_device(), n_kept.numel(), _int32
    p_stride = _probabilities(p, rows, vocab, "p")
    q_stride = 0 if q is None else _probabilities(q, rows, vocab, "q")
    if q is not None and q.get_device() != dev:
        raise ValueError("q is on another device")
    if ws.get_device() != dev:
        raise ValueError("ws is on another device")
    draft = _pack_draft(p.data_ptr(), 0 if q is None else q.data_ptr(), p_stride, q_stride,
                        _numbers(tokens, i32, rows, dev, "tokens"), _maybe(parents, i32, rows, dev, "parents"),
                        _numbers(uniform, torch.float32, rows, dev, "uniform"),
                        _numbers(cu_tokens, i32, batch + 1, dev, "cu_tokens"), rows, batch, vocab)
    status = _verify(draft, _numbers(path, i32, rows, dev, "path"), _numbers(n_kept, i32, batch, dev, "n_kept"),
                     _numbers(next_token, i32, batch, dev, "next_token"), ws.data_ptr(), ws.nbytes,
                     _stream_on(dev, stream))
    if status:
        _check(status, "cccl_step_verify")


def cccl_step_keep(cache: KvCache, batch: KvBatch, path: torch.Tensor, n_kept: torch.Tensor,
                   lens: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """Enqueue moving of the kept tokens' keys and values together; ``lens``
    [batch] (or None) receives the lengths without the others."""
    dev, i32 = cache._device, _int32
    if ws.get_device() != dev:
        raise ValueError("all tensors of a call are on the cache's device")
    status = _keep(cache._ref, batch._ref, _numbers(path, i32, batch.n_tokens, dev, "path"),
                   _numbers(n_kept, i32, batch.batch, dev, "n_kept"),
                   None if lens is None else _numbers(lens, i32, batch.batch, dev, "lens"), ws.data_ptr(), ws.nbytes,
                   _raw_stream(cache, stream))
    if status:
        _check(status, "cccl_step_keep")


# ---------------------------------------------------------------- conveniences
def step_plan(tables: StepTables, lens: torch.Tensor, new: torch.Tensor, rows: int, *,
              parents: torch.Tensor | None = None, mask_words: int | None = None, stream=None) -> dict:
    """Plan and wait: the tables' counts change in place, the rest is returned
    as ``cu_tokens``, ``kv_lens``, ``slots``, ``positions`` and (with
    ``mask_words``) ``mask``."""
    dev = tables.page_table.device
    with torch.cuda.stream(stream):
        ws = empty_step_workspace(dev)

        def empty(*shape, dtype=torch.int32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        out = {"cu_tokens": empty(tables.batch + 1), "kv_lens": empty(tables.batch),
               "slots": empty(rows, dtype=torch.int64), "positions": empty(rows)}
        if mask_words is not None:
            out["mask"] = empty(rows, mask_words)
        cccl_step_plan(tables, lens, new, ws, parents=parents, rows=rows, **out)
        _finish(ws, "cccl_step_plan")
    _hand_over(stream, *out.values())
    return out


def step_write(cache: KvCache, batch: KvBatch, rotary: StepRotary, q: torch.Tensor | None, k: torch.Tensor,
               v: torch.Tensor, *, positions: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotate, store and wait; returns the rotated queries (rows of no sequence: undefined)."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch)
        q_out = None if q is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
        cccl_step_write(cache, batch, rotary, q, k, v, q_out, ws, positions=positions)
        _finish(ws, "cccl_step_write")
    if q_out is not None:
        _hand_over(stream, q_out)
    return q_out


def step_attention(cache: KvCache, batch: KvBatch, q: torch.Tensor, mask: torch.Tensor, *, scale: float | None = None,
                   window: int = 0, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Attend and wait; returns the result and each row's log-sum-exp (rows of no sequence: undefined)."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch, q.shape[1])
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        cccl_step_attention(cache, batch, q, mask, out, ws, scale=scale, window=window, lse=lse)
        _finish(ws, "cccl_step_attention")
    _hand_over(stream, out, lse)
    return out, lse


def step_verify(p: torch.Tensor, q: torch.Tensor | None, tokens: torch.Tensor, parents: torch.Tensor | None,
                uniform: torch.Tensor, cu_tokens: torch.Tensor,
                stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Verify and wait; returns path [rows] (rows of no sequence: undefined), the
    numbers kept and the next tokens [batch]."""
    with torch.cuda.stream(stream):
        ws = empty_step_workspace(p.device)
        path = torch.empty(p.shape[0], dtype=torch.int32, device=p.device)
        n_kept, next_token = (torch.empty(cu_tokens.numel() - 1, dtype=torch.int32, device=p.device) for _ in range(2))
        cccl_step_verify(p, q, tokens, parents, uniform, cu_tokens, path, n_kept, next_token, ws)
        _finish(ws, "cccl_step_verify")
    _hand_over(stream, path, n_kept, next_token)
    return path, n_kept, next_token


def step_keep(cache: KvCache, batch: KvBatch, path: torch.Tensor, n_kept: torch.Tensor, stream=None) -> torch.Tensor:
    """Move and wait; returns the lengths [batch] without what was not kept."""
    with torch.cuda.stream(stream):
        ws = empty_kv_workspace(cache, batch)
        lens = torch.empty(batch.batch, dtype=torch.int32, device=cache.k.device)
        cccl_step_keep(cache, batch, path, n_kept, lens, ws)
        _finish(ws, "cccl_step_keep")
    _hand_over(stream, lens)
    return lens
