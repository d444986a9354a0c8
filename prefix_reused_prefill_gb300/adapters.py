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
from .sampling import _check, _elsewhere, _raw_stream, _vec

MAX_RANK = 128
_TYPES = {torch.bfloat16: 0, torch.float16: 1}
_ENTRY = np.dtype([("a", np.uint64), ("b", np.uint64), ("rank", np.int32), ("scale", np.float32)])


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
        self._keep = [t for a, b, _ in adapters for t in (a, b)]
        self._table = torch.from_numpy(table.view(np.uint8)).to(self.device)
        self.site = KvrAdapterSite(self._table.data_ptr(), len(adapters), int(table["rank"].max()), self.k, len(cols),
                                   (ctypes.c_int * 3)(*cols), _TYPES[self.dtype])
        if self.lib.kvr_adapt_work_bytes(ctypes.byref(self.site), 1) == 0:
            raise KvrError(-1, "a site's adapters, ranks, widths or type are out of their range")
        torch.cuda.current_stream(self.device).synchronize()   # the table is there for every stream

    def _rows(self, name: str, x: torch.Tensor, n: int, dtypes) -> int:
        if x.dtype not in dtypes or x.get_device() != self._index or x.dim() != 2 or x.shape[1] != n \
                or (n > 1 and x.numel() and x.stride(1) != 1):
            raise KvrError(-1, f"{name} must be [rows][{n}] of {dtypes} on {self.device}, a row's elements contiguous")
        return x.stride(0) if x.shape[0] > 1 else n   # (one row's stride means nothing)

    def kvr_adapt(self, x: torch.Tensor, cu_rows: torch.Tensor, which: torch.Tensor,
                  base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """base (zeros of x's type if None) + the sequences' adapters of x [rows][k].  cu_rows [n_seq + 1] and which
        [n_seq] are device int32; base and out are [rows][sum of cols] of x's type or float32, and may be one."""
        if _elsewhere(self._index, stream):   # (memory that the stream may write at once)
            with torch.cuda.device(self._index), torch.cuda.stream(stream):
                return self.kvr_adapt(x, cu_rows, which, base, out)
        types = (self.dtype, torch.float32)
        xs = self._rows("x", x, self.k, (self.dtype,))
        rows, n_seq = x.shape[0], which.numel()
        wp, cp = _vec("which", which, n_seq, torch.int32, self._index), _vec("cu_rows", cu_rows, n_seq + 1, torch.int32,
                                                                             self._index)
        bp, bs = None, self.n
        if base is not None:
            bs, bp = self._rows("base", base, self.n, types), base.data_ptr()
        if out is None:
            out = torch.empty((rows, self.n), dtype=self.dtype if base is None else base.dtype, device=self.device)
        os = self._rows("out", out, self.n, types if base is None else (base.dtype,))
        if out.shape[0] != rows or (base is not None and base.shape[0] != rows):
            raise KvrError(-1, f"base and out must have x's {rows} rows")
        wb = self.lib.kvr_adapt_work_bytes(self.site, rows)
        work = torch.empty(wb, dtype=torch.uint8, device=self.device)
        rc = self.lib.kvr_adapt(self.site, x.data_ptr(), xs, cp, wp, n_seq, rows, bp, bs, out.data_ptr(), os,
                                2 if out.dtype is torch.float32 else self.site.type, work.data_ptr(), wb,
                                _raw_stream(self._index))
        if rc:
            _check(self.lib, rc)
        return out
