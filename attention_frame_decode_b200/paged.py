"""Binding of the paged KV cache (vc_paged_kv in vc.h): windowed attention with sinks over pages, and the
page calls resize, fork and compact.  Argument marshalling only; every computation is in libvc.so.

    cache = PagedCache.empty(layers=4, pages=4096, page_size=64, kv_heads=8, head_dim=128, seqs=16,
                             columns=1024, q_heads=40, window=4096, sinks=64)
    cache.resize(seqs, add=1, pos=pos)                      # room for one more frame of each session
    for layer in range(4):
        cache.attend(layer, q, k, v, out, pos, seqs=seqs)   # append its key and value, attend
    cache.fork(src, dst, parts=session_parts([state.ssm, state.conv, state.ctx_len]))
    cache.resize(ended, lens=zeros)                         # give an ended session's pages back
"""
from __future__ import annotations

import ctypes as C

import torch

from . import VcAttnRows, VcError, VcPagedKv, VcSessionPart, VC_ERR_INVALID_ARG, _check, lib

_lib = lib()


# the handle of a device's current stream; without the Stream object where torch has that (3 us of a call's 12 otherwise)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


class SessionParts:
    """Dense per-session tensors that a fork copies beside the pages (see session_parts)."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if len(self.tensors) > 8:
            raise ValueError("at most 8 parts")
        self.c = (VcSessionPart * max(len(self.tensors), 1))()
        self.seqs = None
        for part, t in zip(self.c, self.tensors):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("a part is a contiguous CUDA tensor")
            outer, seqs = (1, t.shape[0]) if t.dim() == 1 else (t.shape[0], t.shape[1])
            if self.seqs not in (None, seqs):
                raise ValueError("parts of different numbers of sessions")
            self.seqs = seqs
            size = t.element_size() * (t.numel() // max(outer * seqs, 1))
            part.base, part.bytes, part.stride = t.data_ptr(), size, size
            part.outer_stride, part.outer = size * seqs, outer


def session_parts(tensors) -> SessionParts:
    """tensors: [seqs] or [outer][seqs][...] (e.g. State's ctx_len, ssm, conv), at most 8"""
    return SessionParts(tensors)


class PagedCache:
    """A paged KV cache over the caller's tensors (layouts as in vc_paged_kv)."""

    def __init__(self, k, v, table, lens, refs, *, q_heads: int, window: int = 0, sinks: int = 0, status=None):
        if k.dtype not in (torch.bfloat16, torch.float16) or k.dim() != 5 or v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError("k and v are bf16 or fp16 [layers][pages][kv_heads][page_size][head_dim]")
        layers, pages, kv_heads, page, head_dim = k.shape
        seqs, columns = table.shape
        if tuple(lens.shape) != (seqs,) or tuple(refs.shape) != (pages,):
            raise ValueError("lens is [seqs] and refs [pages]")
        self.device, self.dtype = k.device, k.dtype
        if status is None:
            status = torch.zeros((1,), dtype=torch.int32, device=k.device)
        for t in (table, lens, refs, status):
            if t.dtype != torch.int32:
                raise ValueError("table, lens, refs and status are int32")
        for t in (k, v, table, lens, refs, status):
            if t.device != k.device or not t.is_cuda or not t.is_contiguous():
                raise ValueError("the cache's tensors are contiguous CUDA tensors of one device")
        self.k, self.v, self.table, self.lens, self.refs, self.status = k, v, table, lens, refs, status
        self.layers, self.pages, self.kv_heads, self.page_size, self.head_dim = layers, pages, kv_heads, page, head_dim
        self.seqs, self.columns, self.q_heads, self.window, self.sinks = seqs, columns, q_heads, window, sinks
        c = VcPagedKv()
        c.k, c.v, c.table, c.len, c.refs, c.status = (t.data_ptr() for t in (k, v, table, lens, refs, status))
        c.layers, c.pages, c.page_size, c.kv_heads, c.head_dim = layers, pages, page, kv_heads, head_dim
        c.q_heads, c.f16, c.seqs, c.columns = q_heads, int(k.dtype == torch.float16), seqs, columns
        c.window, c.sinks = window, sinks
        n = int(_lib.vc_paged_workspace_bytes(C.byref(c)))
        if n == 0:
            raise VcError(VC_ERR_INVALID_ARG, "vc_paged_workspace_bytes")
        self.workspace = torch.zeros((n,), dtype=torch.uint8, device=k.device)
        c.workspace, c.workspace_bytes = self.workspace.data_ptr(), n
        self.c = c
        self._ref = C.byref(c)
        self._q_shape, self._kv_shape = (q_heads, head_dim), (kv_heads, head_dim)

    @classmethod
    def empty(cls, *, layers, pages, page_size, kv_heads, head_dim, seqs, columns, q_heads, window=0, sinks=0,
              dtype=torch.bfloat16, device="cuda", status=None):
        """a new cache without sessions"""
        k = torch.zeros((layers, pages, kv_heads, page_size, head_dim), dtype=dtype, device=device)
        ints = dict(dtype=torch.int32, device=device)
        return cls(k, torch.zeros_like(k), torch.full((seqs, columns), -1, **ints), torch.zeros((seqs,), **ints),
                   torch.zeros((pages,), **ints), q_heads=q_heads, window=window, sinks=sinks,
                   status=status)

    def _call(self, fn, where, *args, stream=None):
        """fn(cache, *args, stream) on the cache's device"""
        index = self.device.index
        s = stream.cuda_stream if stream is not None else _current_stream(index)
        if torch.cuda.current_device() == index:
            _check(fn(self._ref, *args, s), where)
        else:
            with torch.cuda.device(index):
                _check(fn(self._ref, *args, s), where)

    def _index(self, t, n, name):
        """an int32 tensor of n values on the cache's device"""
        if t is not None and (t.dtype != torch.int32 or t.device != self.device or t.dim() != 1 or t.shape[0] != n or
                              not t.is_contiguous()):
            raise ValueError(f"{name}: a contiguous int32 tensor of {n} on {self.device}")
        return _ptr(t)

    def resize(self, seqs=None, lens=None, add: int = 0, pos=None, stream=None):
        """sets sessions (seqs, or the first len(lens), or all) to the lengths lens + add (lens None: theirs + add);
        pos gets each one's first new position, or -1 (see vc_paged_resize)"""
        n = seqs.shape[0] if seqs is not None else lens.shape[0] if lens is not None else self.seqs
        self._call(_lib.vc_paged_resize, "vc_paged_resize", n, self._index(seqs, n, "seqs"), self._index(lens, n, "lens"),
                   add, self._index(pos, n, "pos"), stream=stream)

    def fork(self, src, dst, parts: SessionParts | None = None, done=None, stream=None):
        """makes the sessions dst copies of the sessions src (see vc_paged_fork)"""
        n = src.shape[0]
        if parts is not None and parts.tensors and parts.seqs != self.seqs:
            raise ValueError(f"parts of {parts.seqs} sessions; the cache has {self.seqs}")
        if parts is not None and any(t.device != self.device for t in parts.tensors):
            raise ValueError("parts on another device than the cache's")
        self._call(_lib.vc_paged_fork, "vc_paged_fork", n, self._index(src, n, "src"), self._index(dst, n, "dst"),
                   parts.c if parts is not None else None, len(parts.tensors) if parts is not None else 0,
                   self._index(done, n, "done"), stream=stream)

    def compact(self, live=None, stream=None):
        """moves the pages in use to the front; live (int32 [1]) gets how many there are"""
        self._call(_lib.vc_paged_compact, "vc_paged_compact", self._index(live, 1, "live"), stream=stream)

    def _rows(self, t, rows, shape, name):
        """the row stride of a 16-bit tensor [rows][heads][head_dim] whose rows are contiguous"""
        s = t.stride()
        if (t.dtype != self.dtype or t.device != self.device or t.shape != (rows, *shape) or
                (shape[1] > 1 and s[2] != 1) or (shape[0] > 1 and s[1] != shape[1])):
            raise ValueError(f"{name}: {self.dtype} {(rows, *shape)} on {self.device} with contiguous rows")
        return s[0] if rows > 1 else shape[0] * shape[1]

    def attend(self, layer: int, q, k, v, out, pos, seqs=None, cu_rows=None, scale: float = 0.0, stream=None):
        """appends the rows' keys and values (None: they are there) to the layer's pages and attends (see
        vc_paged_attend): q, out [rows][q_heads][head_dim], k, v [rows][kv_heads][head_dim], pos int32 [batch]"""
        rows, batch = q.shape[0], pos.shape[0]
        a = VcAttnRows()
        a.q_stride = self._rows(q, rows, self._q_shape, "q")
        a.out_stride = self._rows(out, rows, self._q_shape, "out")
        a.q, a.out, a.pos = q.data_ptr(), out.data_ptr(), self._index(pos, batch, "pos")
        if k is not None or v is not None:
            if k is None or v is None:
                raise ValueError("k and v come together")
            a.k_stride = self._rows(k, rows, self._kv_shape, "k")
            a.v_stride = self._rows(v, rows, self._kv_shape, "v")
            a.k, a.v = k.data_ptr(), v.data_ptr()
        if seqs is not None:
            a.seqs = self._index(seqs, batch, "seqs")
        if cu_rows is not None:
            a.cu_rows = self._index(cu_rows, batch + 1, "cu_rows")
        a.batch, a.rows, a.scale = batch, rows, scale
        self._call(_lib.vc_paged_attend, "vc_paged_attend", layer, C.byref(a), stream=stream)
        return out
