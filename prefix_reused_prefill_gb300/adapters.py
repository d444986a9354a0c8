"""ctypes binding of low-rank adapters (include/kvr.h): argument marshalling only.

    site = Adapters([(a0, b0, scale0), (a1, b1, scale1)], cols=[3584, 512, 512])   # q, k and v of one layer
    qkv = site.kvr_adapt(x, cu_rows, which, qkv)                                   # which: the sequences' adapters

There is no fallback without the built library.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from .kvr import KvrAdapterSite, KvrError, load_library
from .sampling import _check, _check_stream, _current_device, _raw_stream, _work_alloc, _work_free

MAX_RANK = 128
_TYPES = {torch.bfloat16: 0, torch.float16: 1}
_ENTRY = np.dtype([("a", np.uint64), ("b", np.uint64), ("rank", np.int32), ("scale", np.float32)])


def kvr_batch_sync(stream=None):
    """Wait for the stream (None: the current one); raises KvrError if a wait in a kernel of kvr_adapt on its device has
    given up since the last such report (what was formed since then may read NaN)."""
    lib = load_library()
    with torch.cuda.stream(stream):
        _check(lib, lib.kvr_batch_sync(_raw_stream(_current_device())))


class Adapters:
    """The adapters of one projection: entries (a [n_parts * rank][k], b [sum of cols][rank], scale), of one type
    (bf16 or fp16) on one device, contiguous; ``cols``: the outputs of its parts.  The tensors are kept alive."""

    def __init__(self, adapters: Sequence[Tuple[torch.Tensor, torch.Tensor, float]], cols: Sequence[int]):
        self.lib = load_library()
        cols = [int(c) for c in cols]
        if not adapters or not 1 <= len(cols) <= 3 or any(c < 8 or c % 8 for c in cols):
            raise KvrError(-1, "one to three parts of a multiple of 8 outputs, and at least one adapter")
        a0 = adapters[0][0]
        self.dtype, self._index, self.device = a0.dtype, a0.get_device(), a0.device
        if self.dtype not in _TYPES or not a0.is_cuda or a0.dim() != 2:
            raise KvrError(-1, "adapters must be bf16 or fp16 matrices on a device")
        self.k, self.cols, self.n = a0.shape[1], cols, sum(cols)
        table = np.zeros(len(adapters), _ENTRY)
        for i, (a, b, scale) in enumerate(adapters):
            rank = b.shape[1] if b.dim() == 2 else 0
            if rank < 8 or rank % 8 or rank > MAX_RANK or a.shape != (len(cols) * rank, self.k) \
                    or b.shape != (self.n, rank):
                raise KvrError(-1, f"adapter {i}: a {tuple(a.shape)} and b {tuple(b.shape)} do not fit "
                                   f"[{len(cols)} rank][{self.k}] and [{self.n}][rank], rank 8, 16 .. {MAX_RANK}")
            for x in (a, b):
                if x.dtype is not self.dtype or x.get_device() != self._index or not x.is_contiguous() \
                        or x.data_ptr() % 16:
                    raise KvrError(-1, f"adapter {i}: contiguous {self.dtype} matrices on {self.device}")
            table[i] = (a.data_ptr(), b.data_ptr(), rank, scale)
        self._table = torch.from_numpy(table.view(np.uint8)).to(self.device)
        self._keep = [self._table] + [t for a, b, _ in adapters for t in (a, b)]
        self._streams = set()
        self.site = KvrAdapterSite(self._table.data_ptr(), len(adapters), int(table["rank"].max()), self.k, len(cols),
                                   (ctypes.c_int * 3)(*cols), _TYPES[self.dtype])
        if self.lib.kvr_adapt_work_bytes(ctypes.byref(self.site), 1) == 0:
            raise KvrError(-1, "a site's adapters, ranks, widths or type are out of their range")
        self._site = ctypes.byref(self.site)
        self._call, self._work_bytes = self.lib.kvr_adapt, self.lib.kvr_adapt_work_bytes
        torch.cuda.current_stream(self.device).synchronize()   # the table is there for every stream

    def used_on(self, raw: int):
        """Work on the current stream (handle raw) reads the adapters: their memory is not handed out anew before it
        is done."""
        if raw not in self._streams:
            stream = torch.cuda.current_stream(self.device)
            for t in self._keep:
                t.record_stream(stream)
            self._streams.add(raw)

    def _stride(self, x: torch.Tensor, rows: int, n: int) -> int:
        """Row stride of x [rows][n], -1 where it is none."""
        if x.get_device() != self._index or x.shape != (rows, n):
            return -1
        if x.is_contiguous():
            return n
        return x.stride(0) if x.stride(1) == 1 or n == 1 else -1

    def _vector(self, x: torch.Tensor, n: int) -> bool:
        return x.dtype is torch.int32 and x.get_device() == self._index and x.shape == (n,) and x.is_contiguous()

    def kvr_adapt(self, x: torch.Tensor, cu_rows: torch.Tensor, which: torch.Tensor,
                  base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """base (zeros of x's type if None) + the sequences' adapters of x [rows][k].  cu_rows [n_seq + 1] and which
        [n_seq] are device int32; base and out are [rows][sum of cols] of x's type or float32, and may be one."""
        index = self._index
        if stream is not None or _current_device() != index:   # (memory that the stream may write at once)
            _check_stream(stream, index)
            with torch.cuda.device(index), torch.cuda.stream(stream):
                return self.kvr_adapt(x, cu_rows, which, base, out)
        rows, n_seq = x.shape[0] if x.dim() == 2 else -1, which.numel()
        like = self.dtype if base is None else base.dtype
        if out is None:
            out = torch.empty((rows, self.n), dtype=like, device=self.device) if rows >= 0 else x
        elif base is None:
            like = out.dtype
        xs, os = self._stride(x, rows, self.k), self._stride(out, rows, self.n)
        bs, bp = (self.n, None) if base is None else (self._stride(base, rows, self.n), base.data_ptr())
        if xs < 0 or os < 0 or bs < 0 or x.dtype is not self.dtype or out.dtype is not like \
                or (like is not self.dtype and like is not torch.float32) or not self._vector(cu_rows, n_seq + 1) \
                or not self._vector(which, n_seq):
            raise KvrError(-1, f"x [rows][{self.k}] of {self.dtype}, base and out [rows][{self.n}] of it or float32, cu_rows "
                               f"[n_seq + 1] and which [n_seq] of int32, all on {self.device}, a row's elements contiguous")
        raw, wb = _raw_stream(index), self._work_bytes(self._site, rows)
        if raw not in self._streams:
            self.used_on(raw)
        work = _work_alloc(max(wb, 16), raw)
        try:
            rc = self._call(self._site, x.data_ptr(), xs, cu_rows.data_ptr(), which.data_ptr(), n_seq, rows, bp, bs,
                            out.data_ptr(), os, 2 if like is torch.float32 else self.site.type, work, wb, raw)
        finally:
            _work_free(work)
        if rc:
            _check(self.lib, rc)
        return out
