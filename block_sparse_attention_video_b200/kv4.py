"""The paged 4-bit key/value cache (include/fvattn.h, "Paged 4-bit key/value cache").

``KV4Cache`` owns a pool of pages, ``KV4Batch`` describes the sequences of a call,
the ``fvattn_kv4_*`` functions are the C calls of those names, and ``KV4Path`` strings
them into the step of a growing sequence: write the new rows, choose pages, attend.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (FVATTN_OP_KV4_APPEND, FVATTN_OP_KV4_ATTN, FVATTN_OP_KV4_SELECT, _c_float, _c_int,
               _c_size_t, _c_void_p, _call, _check, _dtype_code, _expect, _expect_ws, _lib, _stream,
               alloc_workspace)

_c_int64 = ctypes.c_int64


class _CacheStruct(ctypes.Structure):
    """fvattn_kv4_cache."""
    _fields_ = [("pages", _c_void_p), ("ksum", _c_void_p), ("k_scale", _c_void_p), ("v_scale", _c_void_p),
                ("num_pages", _c_int), ("H", _c_int), ("d", _c_int), ("block", _c_int)]


class _BatchStruct(ctypes.Structure):
    """fvattn_kv4_batch."""
    _fields_ = [("table", _c_void_p), ("kv_len", _c_void_p), ("cu", _c_void_p), ("B", _c_int), ("max_pages", _c_int),
                ("rows", _c_int), ("max_q", _c_int)]


_P = [ctypes.POINTER(_CacheStruct), ctypes.POINTER(_BatchStruct)]
_WS = [_c_void_p, _c_size_t, _c_void_p]
_lib.fvattn_kv4_workspace_bytes.argtypes = [_c_int, *_P, _c_int]
_lib.fvattn_kv4_workspace_bytes.restype = _c_size_t
_lib.fvattn_kv4_append.argtypes = [*_P, _c_void_p, _c_void_p, _c_int64, _c_int64, _c_int, *_WS]
_lib.fvattn_kv4_append.restype = _c_int
_lib.fvattn_kv4_read.argtypes = [*_P, _c_void_p, _c_void_p, _c_int, *_WS]
_lib.fvattn_kv4_read.restype = _c_int
_lib.fvattn_kv4_select.argtypes = [*_P, _c_void_p, _c_int64, _c_int, _c_int, _c_float, _c_float, _c_int, _c_void_p,
                                   _c_void_p, *_WS]
_lib.fvattn_kv4_select.restype = _c_int
_lib.fvattn_kv4_attn.argtypes = [*_P, _c_void_p, _c_int64, _c_int, _c_void_p, _c_void_p, _c_int, _c_float, _c_int,
                                 _c_void_p, _c_void_p, *_WS]
_lib.fvattn_kv4_attn.restype = _c_int


class KV4Cache:
    """A pool of ``num_pages`` pages of ``block`` tokens for ``H`` KV heads of ``d`` channels:
    ``pages`` [num_pages, H, block*(d+d/8)] uint8 and ``ksum`` [num_pages, H, d] int32 (allocated
    here unless given), with optional fp32 head scales [H]. The tensors stay the cache's for its
    lifetime; their contents may change."""

    def __init__(self, num_pages, H, d, block, device="cuda", k_scale=None, v_scale=None, pages=None, ksum=None):
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        if d not in (64, 128) or block not in (64, 128):
            raise ValueError("d and block must be 64 or 128")
        if num_pages < 1 or H < 1:
            raise ValueError("num_pages and H must be positive")
        self.num_pages, self.H, self.d, self.block = int(num_pages), int(H), int(d), int(block)
        self.record = self.block * (self.d + self.d // 8)
        if pages is None:
            pages = torch.zeros((num_pages, H, self.record), dtype=torch.uint8, device=dev)
        if ksum is None:
            ksum = torch.zeros((num_pages, H, d), dtype=torch.int32, device=dev)
        _expect(pages, "pages", dev, (num_pages, H, self.record), torch.uint8)
        _expect(ksum, "ksum", dev, (num_pages, H, d), torch.int32)
        _expect(k_scale, "k_scale", dev, (H,), torch.float32, optional=True)
        _expect(v_scale, "v_scale", dev, (H,), torch.float32, optional=True)
        self._tensors = (pages, ksum, k_scale, v_scale)
        self.device = dev
        p = lambda t: None if t is None else t.data_ptr()
        self._struct = _CacheStruct(p(pages), p(ksum), p(k_scale), p(v_scale), self.num_pages, self.H, self.d, self.block)
        self._ref = ctypes.byref(self._struct)

    pages = property(lambda self: self._tensors[0])
    ksum = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])


class KV4Batch:
    """The sequences of a call: ``table`` [B, max_pages], ``kv_len`` [B] and ``cu`` [B+1], all int32
    CUDA tensors, and ``max_q``, the most rows any of them has. The tensors stay the batch's for its
    lifetime; their contents may change. Lengths and row starts are checked on the device, where they
    are used (``fvattn_workspace_status``)."""

    def __init__(self, table, kv_len, cu, max_q):
        for t, name in ((table, "table"), (kv_len, "kv_len"), (cu, "cu")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
        if table.dim() != 2 or min(table.shape) < 1:
            raise ValueError(f"table has shape {tuple(table.shape)}, expected [B, max_pages]")
        B = table.shape[0]
        dev = table.device
        _expect(table, "table", dev, None, torch.int32)
        _expect(kv_len, "kv_len", dev, (B,), torch.int32)
        _expect(cu, "cu", dev, (B + 1,), torch.int32)
        if int(max_q) < 1:
            raise ValueError("max_q must be positive")
        self._tensors = (table, kv_len, cu)
        self.max_q, self.B, self.max_pages, self.device = int(max_q), B, table.shape[1], dev
        self._args = (table.data_ptr(), kv_len.data_ptr(), cu.data_ptr(), self.B, self.max_pages)

    table = property(lambda self: self._tensors[0])
    kv_len = property(lambda self: self._tensors[1])
    cu = property(lambda self: self._tensors[2])

    def _ref(self, rows):
        return ctypes.byref(_BatchStruct(*self._args, rows, self.max_q))


def _rows(t, name, dev, heads, d, dtype=None):
    """A [rows, heads, d] input whose rows may lie apart (columns of a wider projection);
    returns (rows, heads, row stride in elements, dtype code)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [rows, {heads or 'heads'}, {d}]")
    code = _dtype_code(t)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    rows, H = shape[0], shape[1]
    if t.is_contiguous():
        return rows, H, H * d, code
    stride, head, one = t.stride()
    if one != 1 or (H > 1 and head != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if rows == 1:
        stride = H * d
    if stride < H * d or (stride * t.element_size()) % 16:
        raise ValueError(f"{name}: row stride {stride} must be at least {H * d} and a multiple of 16 bytes")
    return rows, H, stride, code


def _common(cache, batch, workspace):
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    _expect_ws(workspace, cache.device)
    return cache.device


def _lists(cache, batch, rows, kv_idx, kv_cnt):
    _expect(kv_idx, "kv_idx", cache.device, (rows, cache.H, batch.max_pages), torch.int32)
    _expect(kv_cnt, "kv_cnt", cache.device, (rows, cache.H), torch.int32)


def _ws(workspace):
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _at(t):
    return None if t is None else t.data_ptr()


def fvattn_kv4_workspace_bytes(op: int, cache: KV4Cache, batch: KV4Batch, rows: int, H_q: int = 0) -> int:
    """Workspace bytes of an FVATTN_OP_KV4_* call over ``rows`` rows with ``H_q`` query heads (the
    attention's grows with the batch's max_q)."""
    return int(_lib.fvattn_kv4_workspace_bytes(op, cache._ref, batch._ref(int(rows)), int(H_q)))


def fvattn_kv4_append(cache: KV4Cache, batch: KV4Batch, k, v, workspace, stream=None):
    """Quantizes k, v [rows, H, d] (bf16 or fp32) into the pages at the rows' positions."""
    dev = _common(cache, batch, workspace)
    rows, _, ks, code = _rows(k, "k", dev, cache.H, cache.d)
    vrows, _, vs, _ = _rows(v, "v", dev, cache.H, cache.d, k.dtype)
    if vrows != rows:
        raise ValueError(f"v has {vrows} rows, k {rows}")
    _check(_call(dev, _lib.fvattn_kv4_append, cache._ref, batch._ref(rows), k.data_ptr(), v.data_ptr(), ks, vs,
                 code, *_ws(workspace), _stream(stream, dev)), "fvattn_kv4_append")
    return cache


def fvattn_kv4_read(cache: KV4Cache, batch: KV4Batch, k_out, v_out, workspace, stream=None):
    """Reads the rows back into k_out, v_out [rows, H, d] (bf16 or fp32, contiguous)."""
    dev = _common(cache, batch, workspace)
    rows, _, _, code = _rows(k_out, "k_out", dev, cache.H, cache.d)
    _expect(k_out, "k_out", dev)
    _expect(v_out, "v_out", dev, (rows, cache.H, cache.d), k_out.dtype)
    _check(_call(dev, _lib.fvattn_kv4_read, cache._ref, batch._ref(rows), k_out.data_ptr(), v_out.data_ptr(),
                 code, *_ws(workspace), _stream(stream, dev)), "fvattn_kv4_read")
    return k_out, v_out


def fvattn_kv4_select(cache: KV4Cache, batch: KV4Batch, q, p: float, k_min: int, kv_idx, kv_cnt, workspace,
                      scale=None, stream=None):
    """The pages each row of q [rows, H_q, d] attends, per KV head: kv_idx [rows, H, max_pages] and
    kv_cnt [rows, H] (Top-p with a Top-k floor over the softmax on the pages' mean keys)."""
    dev = _common(cache, batch, workspace)
    rows, H_q, qs, code = _rows(q, "q", dev, None, cache.d)
    _lists(cache, batch, rows, kv_idx, kv_cnt)
    sc = 1.0 / math.sqrt(cache.d) if scale is None else float(scale)
    _check(_call(dev, _lib.fvattn_kv4_select, cache._ref, batch._ref(rows), q.data_ptr(), qs, H_q, code, sc,
                 float(p), int(k_min), kv_idx.data_ptr(), kv_cnt.data_ptr(), *_ws(workspace),
                 _stream(stream, dev)), "fvattn_kv4_select")
    return kv_idx, kv_cnt


def fvattn_kv4_attn(cache: KV4Cache, batch: KV4Batch, q, out, workspace, scale=None, causal: bool = True, lse=None,
                    kv_idx=None, kv_cnt=None, stream=None):
    """Attention of q [rows, H_q, d] over the cache (or over the pages of the lists) into out, with
    an optional lse [rows, H_q] fp32."""
    dev = _common(cache, batch, workspace)
    rows, H_q, qs, code = _rows(q, "q", dev, None, cache.d)
    _expect(out, "out", dev, (rows, H_q, cache.d), q.dtype)
    _expect(lse, "lse", dev, (rows, H_q), torch.float32, optional=True)
    if (kv_idx is None) != (kv_cnt is None):
        raise ValueError("kv_idx and kv_cnt go together")
    if kv_idx is not None:
        _lists(cache, batch, rows, kv_idx, kv_cnt)
    sc = 1.0 / math.sqrt(cache.d) if scale is None else float(scale)
    _check(_call(dev, _lib.fvattn_kv4_attn, cache._ref, batch._ref(rows), q.data_ptr(), qs, H_q, out.data_ptr(),
                 _at(lse), code, sc, 1 if causal else 0, _at(kv_idx), _at(kv_cnt), *_ws(workspace),
                 _stream(stream, dev)), "fvattn_kv4_attn")
    return out


class KV4Path:
    """One attention layer's step over a KV4Cache with buffers allocated once.

    ``__call__(batch, q, k, v)`` writes the rows' k and v into the cache, chooses the pages of every
    row (``p``, ``k_min``) and attends; ``p=None`` attends the whole cache. Choosing is for few rows a
    sequence (tokens, drafts): lists are read row by row, and for a chunk's rows attending the whole
    cache is faster. At most ``max_rows`` rows a call; the returned output is the path's buffer,
    overwritten by the next call. What the path refuses it refuses before anything is written."""

    def __init__(self, cache: KV4Cache, H_q, max_rows, max_batch, max_pages, dtype, p=None, k_min=1, causal=True,
                 scale=None):
        if p is not None and not 0.0 < p <= 1.0:
            raise ValueError(f"p = {p} is not in (0, 1]")
        if int(k_min) < 1:
            raise ValueError("k_min must be positive")
        if scale is not None and not 0.0 < scale < math.inf:
            raise ValueError("scale must be positive and finite")
        self.cache, self.H_q, self.p, self.k_min, self.causal, self.scale = cache, int(H_q), p, int(k_min), causal, scale
        self.max_rows, self.max_batch, self.max_pages = int(max_rows), int(max_batch), int(max_pages)
        dev = cache.device
        self.out = torch.empty((max_rows, H_q, cache.d), dtype=dtype, device=dev)
        self.lse = torch.empty((max_rows, H_q), dtype=torch.float32, device=dev)
        self.kv_idx = self.kv_cnt = None
        if p is not None:
            self.kv_idx = torch.empty((max_rows, cache.H, max_pages), dtype=torch.int32, device=dev)
            self.kv_cnt = torch.empty((max_rows, cache.H), dtype=torch.int32, device=dev)
        b = _BatchStruct(None, None, None, self.max_batch, self.max_pages, self.max_rows, self.max_rows)

        def workspace(op):
            n = int(_lib.fvattn_kv4_workspace_bytes(op, cache._ref, ctypes.byref(b), self.H_q))
            if n == 0:
                raise ValueError("unsupported sizes")
            return alloc_workspace(n, dev)

        self.ws_append = workspace(FVATTN_OP_KV4_APPEND)
        self.ws_select = None if p is None else workspace(FVATTN_OP_KV4_SELECT)
        self.ws_attn = workspace(FVATTN_OP_KV4_ATTN)

    def __call__(self, batch: KV4Batch, q, k, v):
        rows = q.shape[0]
        if rows > self.max_rows or batch.B > self.max_batch or batch.max_pages != self.max_pages:
            raise ValueError(f"{rows} rows of {batch.B} sequences with {batch.max_pages} pages do not fit the path "
                             f"({self.max_rows}, {self.max_batch}, {self.max_pages})")
        # all of it before the first call writes into the cache (which looks at k and v itself)
        _, heads, stride, _ = _rows(q, "q", self.cache.device, self.H_q, self.cache.d, self.out.dtype)
        at, out, es, row = q.data_ptr(), self.out.data_ptr(), q.element_size(), heads * self.cache.d
        if at % 16:
            raise ValueError("q must be 16-byte aligned")
        if at < out + rows * row * es and out < at + ((rows - 1) * stride + row) * es:
            raise ValueError("q overlaps the path's output")
        if batch.max_q > self.max_rows:              # claimed, not there: the kernel for many rows may need more workspace
            need = fvattn_kv4_workspace_bytes(FVATTN_OP_KV4_ATTN, self.cache, batch, rows, self.H_q)
            if need > self.ws_attn.numel():
                raise ValueError(f"the batch's max_q {batch.max_q} does not fit the path's {self.max_rows} rows")
        if k.shape[0] != rows or v.shape[0] != rows:
            raise ValueError(f"q has {rows} rows, k {k.shape[0]} and v {v.shape[0]}")
        fvattn_kv4_append(self.cache, batch, k, v, self.ws_append)
        idx = cnt = None
        if self.p is not None:
            idx, cnt = self.kv_idx[:rows], self.kv_cnt[:rows]
            fvattn_kv4_select(self.cache, batch, q, self.p, self.k_min, idx, cnt, self.ws_select, scale=self.scale)
        out, lse = self.out[:rows], self.lse[:rows]
        return fvattn_kv4_attn(self.cache, batch, q, out, self.ws_attn, scale=self.scale, causal=self.causal, lse=lse,
                               kv_idx=idx, kv_cnt=cnt)
