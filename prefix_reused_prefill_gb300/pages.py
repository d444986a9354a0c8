"""ctypes binding of the paged 4-bit cache (include/kvr.h): argument marshalling only.

A step of a serving loop plans its rows once and then runs, layer by layer, append and attend:

    pg = PagedKv(paged_config(n_pages=4096, n_layers=36, n_q_heads=32, n_kv_heads=8, head_dim=128,
                              max_seqs=64, max_len=32768, max_rows=512))
    pg.kvr_page_plan(keep, add, rows)            # device int32: tokens each sequence keeps, rows it gains
    for l in range(36):
        q = pg.kvr_page_append(l, q, k, v, norm_q[l], norm_k[l])
        o = pg.kvr_page_attend(l, q)
    pg.kvr_pages_sync()                          # once per step or later: was a plan refused?

Torch provides the memory and the streams.  There is no fallback without the built library.
"""
from __future__ import annotations

import ctypes
import types
from typing import Optional, Tuple

import torch

from .kvr import KVR_OK, KvrError, KvrPagesConfig, KvrPageTables, load_library

PAGE_TOKENS = 64
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle (a Stream object costs 2 us)
_ACTS = {"bf16": (0, torch.bfloat16), "fp16": (1, torch.float16)}


def paged_config(n_pages: int, n_layers: int, n_q_heads: int, n_kv_heads: int, head_dim: int, max_seqs: int,
                 max_len: int, max_rows: int, act: str = "bf16", rope_theta: float = 1.0e6,
                 norm_eps: float = 1.0e-6) -> KvrPagesConfig:
    return KvrPagesConfig(n_pages, n_layers, n_q_heads, n_kv_heads, head_dim, max_seqs, max_len, max_rows,
                          _ACTS[act][0], rope_theta, norm_eps)


class PagedKv:
    """One kvr_pages handle over a torch-allocated pool and work area.

    ``state`` holds views of the device tables: table, lens, free, count, cu, row_seq, row_pos, row_slot
    (read them on the stream of the calls; write none of them).
    """

    def __init__(self, cfg: KvrPagesConfig, device="cuda"):
        self.ctx = None
        self.lib = load_library()
        self.cfg = cfg
        pb = self.lib.kvr_pages_pool_bytes(ctypes.byref(cfg))
        wb = self.lib.kvr_pages_work_bytes(ctypes.byref(cfg))
        if pb == 0 or wb == 0:
            raise KvrError(-1, "invalid configuration")
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.device, self._index = device, device.index
        self.dtype = {i: t for i, t in _ACTS.values()}[cfg.act]
        with torch.cuda.device(device):
            self.pool = torch.empty(pb, dtype=torch.uint8, device=device)
            self.work = torch.empty(wb, dtype=torch.uint8, device=device)
            # the buffers may hold memory that other work on this stream still uses
            torch.cuda.current_stream(device).synchronize()
            ctx = ctypes.c_void_p()
            rc = self.lib.kvr_pages_create(ctypes.byref(cfg), self.pool.data_ptr(), pb, self.work.data_ptr(), wb,
                                           ctypes.byref(ctx))
        if rc != KVR_OK:
            raise KvrError(rc, "kvr_pages_create failed")
        self.ctx = ctx
        self._rows = 0
        self._streams = {torch.cuda.current_stream(device).cuda_stream}   # whose memory pool and work are
        self._scale = cfg.head_dim ** -0.5
        t = KvrPageTables()
        self.lib.kvr_pages_tables(ctx, ctypes.byref(t))
        words, base = self.work.view(torch.int32), self.work.data_ptr()

        def view(ptr, *shape):
            n = 1
            for s in shape:
                n *= s
            return words[(ptr - base) // 4:(ptr - base) // 4 + n].view(shape)

        self.state = types.SimpleNamespace(
            table=view(t.table, cfg.max_seqs, t.table_width), lens=view(t.lens, cfg.max_seqs),
            free=view(t.free_list, cfg.n_pages), count=view(t.count, 1), cu=view(t.cu_rows, cfg.max_seqs + 1),
            row_seq=view(t.row_seq, cfg.max_rows), row_pos=view(t.row_pos, cfg.max_rows),
            row_slot=view(t.row_slot, cfg.max_rows))

    # -------------------------------------------------------------- helpers
    def close(self):
        if self.ctx:
            self.lib.kvr_pages_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc: int):
        if rc != KVR_OK:
            raise KvrError(rc, self.lib.kvr_pages_error(self.ctx).decode())

    def _stream(self, stream=None):
        raw = stream.cuda_stream if stream is not None else _raw_stream(self._index)
        if raw not in self._streams:
            # pool and work are not handed out anew before this stream's work is done
            stream = stream if stream is not None else torch.cuda.current_stream(self.device)
            self.pool.record_stream(stream)
            self.work.record_stream(stream)
            self._streams.add(raw)
        return raw

    def _rows_arg(self, name: str, x: torch.Tensor, heads: int) -> int:
        """Row stride of x [rows][heads][head_dim], the heads of a row contiguous."""
        d = self.cfg.head_dim
        if x.dtype is not self.dtype or x.get_device() != self._index:
            raise KvrError(-1, f"{name} must be {self.dtype} on {self.device}")
        if x.shape != (self._rows, heads, d):
            raise KvrError(-1, f"{name} has shape {tuple(x.shape)}, the plan needs {(self._rows, heads, d)}")
        if self._rows == 0:
            return heads * d
        s = x.stride()
        if s[2] != 1 or (heads > 1 and s[1] != d):
            raise KvrError(-1, f"{name}: the heads of a row must be contiguous")
        return s[0] if self._rows > 1 else heads * d   # (one row's stride means nothing)

    def _gain(self, name: str, x: Optional[torch.Tensor]) -> Optional[int]:
        if x is None:
            return None
        if x.dtype is not self.dtype or x.get_device() != self._index or x.shape != (self.cfg.head_dim,) \
                or not x.is_contiguous():
            raise KvrError(-1, f"{name} must be {self.dtype} [{self.cfg.head_dim}] on {self.device}")
        return x.data_ptr()

    def _out(self, name: str, x: Optional[torch.Tensor], heads: int, dtype, stream) -> torch.Tensor:
        shape = (self._rows, heads, self.cfg.head_dim)
        if x is None:
            if stream is None:
                return torch.empty(shape, dtype=dtype, device=self.device)
            with torch.cuda.stream(stream):   # memory that the stream may write at once
                return torch.empty(shape, dtype=dtype, device=self.device)
        if x.dtype is not dtype or x.get_device() != self._index or x.shape != shape or not x.is_contiguous():
            raise KvrError(-1, f"{name} must be a contiguous {dtype} tensor of shape {shape} on {self.device}")
        return x

    # -------------------------------------------------------------- C ABI
    def kvr_page_plan(self, keep: torch.Tensor, add: torch.Tensor, rows: int, max_add: int = 0, stream=None):
        """Sequence b keeps keep[b] tokens and gains add[b] rows (device int32 [n_seq]); the step's buffers
        have ``rows`` rows, no add[b] is larger than max_add (0: no closer bound than rows)."""
        n = keep.numel()
        if keep.dtype is not torch.int32 or add.dtype is not torch.int32 or keep.get_device() != self._index \
                or add.get_device() != self._index or keep.dim() != 1 or add.dim() != 1 or add.numel() != n \
                or not keep.is_contiguous() or not add.is_contiguous():
            raise KvrError(-1, f"keep and add must be contiguous int32 vectors of one length on {self.device}")
        rc = self.lib.kvr_page_plan(self.ctx, n, keep.data_ptr(), add.data_ptr(), rows, max_add, self._stream(stream))
        if rc:
            self._check(rc)
        self._rows = rows

    def kvr_page_append(self, layer: int, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                        norm_q: Optional[torch.Tensor] = None, norm_k: Optional[torch.Tensor] = None,
                        rotate: bool = True, out: Optional[torch.Tensor] = None, stream=None):
        """Norm, rotate and store the planned rows; returns the rotated q (None without q)."""
        c = self.cfg
        ks, vs = self._rows_arg("k", k, c.n_kv_heads), self._rows_arg("v", v, c.n_kv_heads)
        qs, qp, op = 0, None, None
        if q is not None:
            qs, qp = self._rows_arg("q", q, c.n_q_heads), q.data_ptr()
            out = self._out("out", out, c.n_q_heads, self.dtype, stream)
            op = out.data_ptr()
        elif out is not None:
            raise KvrError(-1, "out without q")
        self._check(self.lib.kvr_page_append(self.ctx, layer, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs,
                                             self._gain("norm_q", norm_q), self._gain("norm_k", norm_k),
                                             1 if rotate else 0, op, self._rows, self._stream(stream)))
        return out

    def kvr_page_read(self, layer: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """What the cache holds for the planned rows: k and v [rows][n_kv_heads][head_dim]."""
        k = self._out("k", None, self.cfg.n_kv_heads, self.dtype, stream)
        v = self._out("v", None, self.cfg.n_kv_heads, self.dtype, stream)
        self._check(self.lib.kvr_page_read(self.ctx, layer, k.data_ptr(), v.data_ptr(), self._rows,
                                           self._stream(stream)))
        return k, v

    def kvr_page_attend(self, layer: int, q: torch.Tensor, out: Optional[torch.Tensor] = None,
                        scale: Optional[float] = None, stream=None) -> torch.Tensor:
        """Causal attention of the planned rows over their sequences (scale: 1 / sqrt(head_dim))."""
        H = self.cfg.n_q_heads
        qs = self._rows_arg("q", q, H)
        out = self._out("out", out, H, self.dtype, stream)
        self._check(self.lib.kvr_page_attend(self.ctx, layer, q.data_ptr(), qs, out.data_ptr(), 0,
                                             self._scale if scale is None else scale, self._rows,
                                             self._stream(stream)))
        return out

    def kvr_pages_sync(self, stream=None):
        """Wait for the stream; raises KvrError for a plan that the device refused or a wait that gave up."""
        self._check(self.lib.kvr_pages_sync(self.ctx, self._stream(stream)))
