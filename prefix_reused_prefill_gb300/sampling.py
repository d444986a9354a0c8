"""ctypes binding of sampling and speculative sampling (include/kvr.h): argument marshalling only.

    token, prob = kvr_sample(logits, torch.rand(rows, device="cuda"), temperature=t, top_k=k, top_p=p)
    accepted, following = kvr_accept(logits, tokens, cu_rows, u, u_next, draft_probs=q, temperature=t, top_p=p)

Settings are tensors with one entry per request, numbers that hold for all of them, or None.  There is no fallback
without the built library.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from .kvr import KvrError, KvrSampling, load_library

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle (a Stream object costs 2 us)
Setting = Optional[Union[torch.Tensor, float, int]]


def _elsewhere(index: int, stream) -> bool:
    """Whether a call has to make the tensors' device, or the given stream, the current one first."""
    return stream is not None or _current_device() != index


def _check(lib, rc: int):
    if rc:
        raise KvrError(rc, lib.kvr_batch_error().decode())


def _rows(name: str, x: torch.Tensor, shape, dtypes, index: int) -> int:
    """Row stride of x [rows][n], the elements of a row contiguous."""
    if x.dtype not in dtypes or x.get_device() != index or x.dim() != 2 or (shape is not None and x.shape != shape):
        raise KvrError(-1, f"{name}: a device tensor {shape or '[rows][n]'} of {dtypes}, all on one device")
    if x.shape[1] > 1 and x.numel() and x.stride(1) != 1:
        raise KvrError(-1, f"{name}: the elements of a row must be contiguous")
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]   # (one row's stride means nothing)


def _vec(name: str, x: torch.Tensor, n: int, dtype, index: int) -> int:
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.get_device() != index or x.shape != (n,) \
            or not x.is_contiguous():
        raise KvrError(-1, f"{name} must be a contiguous {dtype} vector [{n}] on the logits' device")
    return x.data_ptr()


def _settings(n: int, index: int, temperature, top_k, min_p, top_p):
    """The struct, and what it points to (kept until the call is made)."""
    keep = [None if x is None else x if isinstance(x, torch.Tensor) else torch.full((n,), x, dtype=t, device=index)
            for x, t in ((temperature, torch.float32), (top_k, torch.int32), (min_p, torch.float32), (top_p, torch.float32))]
    t, k, m, p = keep
    return KvrSampling(None if t is None else _vec("temperature", t, n, torch.float32, index),
                       None if k is None else _vec("top_k", k, n, torch.int32, index),
                       None if m is None else _vec("min_p", m, n, torch.float32, index),
                       None if p is None else _vec("top_p", p, n, torch.float32, index)), keep


def _logits(x: torch.Tensor) -> Tuple[int, int]:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise KvrError(-1, "logits: a device tensor [rows][vocab]")
    index = x.get_device()
    return index, _rows("logits", x, None, tuple(_TYPES), index)


def kvr_sample(logits: torch.Tensor, u: torch.Tensor, temperature: Setting = None, top_k: Setting = None,
               min_p: Setting = None, top_p: Setting = None, dist: Union[bool, torch.Tensor] = False, stream=None):
    """A token of each row of logits [rows][vocab] (fp32, bf16 or fp16) by u [rows] in [0, 1): (token int32, its
    probability float32), and with ``dist`` (True, or a float32 tensor to fill) every token's probability.  Settings:
    [rows].  A row without a distribution has token -1."""
    index, ls = _logits(logits)
    if _elsewhere(index, stream):   # (memory that the stream may write at once)
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return kvr_sample(logits, u, temperature, top_k, min_p, top_p, dist)
    lib = load_library()
    rows, vocab = logits.shape
    up = _vec("u", u, rows, torch.float32, index)
    st, keep = _settings(rows, index, temperature, top_k, min_p, top_p)
    token = torch.empty(rows, dtype=torch.int32, device=logits.device)
    prob = torch.empty(rows, dtype=torch.float32, device=logits.device)
    ds, dp = vocab, None
    if dist is not False:
        if dist is True:
            dist = torch.empty((rows, vocab), dtype=torch.float32, device=logits.device)
        ds, dp = _rows("dist", dist, (rows, vocab), (torch.float32,), index), dist.data_ptr()
    rc = lib.kvr_sample(logits.data_ptr(), _TYPES[logits.dtype], ls, rows, vocab, st, up, token.data_ptr(),
                        prob.data_ptr(), dp, ds, _raw_stream(index))
    if rc:
        _check(lib, rc)
    return (token, prob) if dp is None else (token, prob, dist)


def kvr_accept(logits: torch.Tensor, tokens: torch.Tensor, cu_rows: torch.Tensor, u: torch.Tensor,
               u_next: torch.Tensor, draft_probs: Optional[torch.Tensor] = None, temperature: Setting = None,
               top_k: Setting = None, min_p: Setting = None, top_p: Setting = None, stream=None):
    """Speculative sampling: rows cu_rows[b] .. cu_rows[b + 1] - 1 of logits [rows][vocab] and of tokens (int32; the
    last committed token, then the drafts) are sequence b's.  Returns per sequence (drafts that stay, the token after
    them), int32.  u [rows] judges the drafts, u_next [n_seq] draws; draft_probs: float32 [rows][vocab], the
    distribution of the draft after each row (None: the drafts were certain).  Settings: [n_seq]."""
    index, ls = _logits(logits)
    if _elsewhere(index, stream):
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return kvr_accept(logits, tokens, cu_rows, u, u_next, draft_probs, temperature, top_k, min_p, top_p)
    lib = load_library()
    rows, vocab = logits.shape
    n = cu_rows.numel() - 1
    if n < 1:
        raise KvrError(-1, "cu_rows must have an entry more than there are sequences")
    cp, tp = _vec("cu_rows", cu_rows, n + 1, torch.int32, index), _vec("tokens", tokens, rows, torch.int32, index)
    up, np = _vec("u", u, rows, torch.float32, index), _vec("u_next", u_next, n, torch.float32, index)
    qp, qs = None, vocab
    if draft_probs is not None:
        qs, qp = _rows("draft_probs", draft_probs, (rows, vocab), (torch.float32,), index), draft_probs.data_ptr()
    st, keep = _settings(n, index, temperature, top_k, min_p, top_p)
    accepted = torch.empty(n, dtype=torch.int32, device=logits.device)
    following = torch.empty(n, dtype=torch.int32, device=logits.device)
    wb = lib.kvr_accept_work_bytes(rows)
    work = torch.empty(wb, dtype=torch.uint8, device=logits.device)
    rc = lib.kvr_accept(logits.data_ptr(), _TYPES[logits.dtype], ls, rows, vocab, st, n, cp, tp, qp, qs, up, np,
                        accepted.data_ptr(), following.data_ptr(), work.data_ptr(), wb, _raw_stream(index))
    if rc:
        _check(lib, rc)
    return accepted, following
