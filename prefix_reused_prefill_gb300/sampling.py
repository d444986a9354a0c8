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
# A call's working memory: from torch's allocator without a tensor around it (which costs as much as a
# launch), given back when the call has been made; work on the stream that follows may have it then.
_work_alloc, _work_free = torch._C._cuda_cudaCachingAllocator_raw_alloc, torch._C._cuda_cudaCachingAllocator_raw_delete
Setting = Optional[Union[torch.Tensor, float, int]]


def _check(lib, rc: int):
    if rc:
        raise KvrError(rc, lib.kvr_batch_error().decode())


def _check_stream(stream, index: int):
    if stream is not None and stream.device.index != index:
        raise KvrError(-1, f"the stream is of {stream.device}, the tensors are on device {index}")


def _refuse(what: str, x, shape, dtypes, index: int):
    raise KvrError(-1, f"{what} must be {shape} of {dtypes} on device {index}, a row's elements contiguous; it is "
                       f"{tuple(x.shape)} of {x.dtype} on {x.device}" if isinstance(x, torch.Tensor) else f"{what}: {x}")


def _rows(name: str, x: torch.Tensor, shape, dtypes, index: int) -> int:
    """Row stride of x [rows][n], the elements of a row contiguous."""
    if x.dtype not in dtypes or x.get_device() != index or x.shape != shape:
        _refuse(name, x, shape, dtypes, index)
    if x.is_contiguous():
        return shape[1]
    if shape[1] > 1 and x.stride(1) != 1:
        _refuse(name, x, shape, dtypes, index)
    return x.stride(0) if shape[0] > 1 else shape[1]   # (one row's stride means nothing)


def _vec(name: str, x: torch.Tensor, shape, dtype, index: int) -> int:
    """Address of a vector of that shape."""
    if x.dtype is not dtype or x.get_device() != index or x.shape != shape or not x.is_contiguous():
        _refuse(name, x, shape, dtype, index)
    return x.data_ptr()


def _settings(shape, index: int, temperature, top_k, min_p, top_p):
    """The struct, and what it points to (kept until the call is made)."""
    f32, keep = torch.float32, None
    if not (isinstance(temperature, torch.Tensor) and isinstance(top_k, torch.Tensor) and isinstance(min_p, torch.Tensor)
            and isinstance(top_p, torch.Tensor)):
        keep = [x if x is None or isinstance(x, torch.Tensor) else torch.full(shape, x, dtype=t, device=index)
                for x, t in ((temperature, f32), (top_k, torch.int32), (min_p, f32), (top_p, f32))]
        temperature, top_k, min_p, top_p = keep
    return KvrSampling(None if temperature is None else _vec("temperature", temperature, shape, f32, index),
                       None if top_k is None else _vec("top_k", top_k, shape, torch.int32, index),
                       None if min_p is None else _vec("min_p", min_p, shape, f32, index),
                       None if top_p is None else _vec("top_p", top_p, shape, f32, index)), keep


def _logits(x: torch.Tensor):
    """(device, type, row stride) of logits [rows][vocab]."""
    kind = _TYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if kind is None or not x.is_cuda or x.dim() != 2:
        _refuse("logits", x, "[rows][vocab]", tuple(_TYPES), -1)
    index = x.get_device()
    return index, kind, x.shape[1] if x.is_contiguous() else _rows("logits", x, x.shape, (x.dtype,), index)


def kvr_sample(logits: torch.Tensor, u: torch.Tensor, temperature: Setting = None, top_k: Setting = None,
               min_p: Setting = None, top_p: Setting = None, dist: Union[bool, torch.Tensor] = False, stream=None):
    """A token of each row of logits [rows][vocab] (fp32, bf16 or fp16) by u [rows] in [0, 1): (token int32, its
    probability float32), and with ``dist`` (True, or a float32 tensor to fill) every token's probability.  Settings:
    [rows].  A row without a distribution has token -1."""
    index, kind, ls = _logits(logits)
    if stream is not None or _current_device() != index:   # (memory that the stream may write at once)
        _check_stream(stream, index)
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return kvr_sample(logits, u, temperature, top_k, min_p, top_p, dist)
    lib = load_library()
    rows, vocab = logits.shape
    shape, device = (rows,), logits.device
    up = _vec("u", u, shape, torch.float32, index)
    st, keep = _settings(shape, index, temperature, top_k, min_p, top_p)
    token = torch.empty(shape, dtype=torch.int32, device=device)
    prob = torch.empty(shape, dtype=torch.float32, device=device)
    ds, dp = vocab, None
    if dist is not False:
        if dist is True:
            dist = torch.empty((rows, vocab), dtype=torch.float32, device=device)
        else:
            ds = _rows("dist", dist, (rows, vocab), (torch.float32,), index)
        dp = dist.data_ptr()
    rc = lib.kvr_sample(logits.data_ptr(), kind, ls, rows, vocab, st, up, token.data_ptr(), prob.data_ptr(), dp, ds,
                        _raw_stream(index))
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
    index, kind, ls = _logits(logits)
    if stream is not None or _current_device() != index:
        _check_stream(stream, index)
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return kvr_accept(logits, tokens, cu_rows, u, u_next, draft_probs, temperature, top_k, min_p, top_p)
    lib = load_library()
    rows, vocab = logits.shape
    n = u_next.numel()
    shape, device, i32, f32 = (n,), logits.device, torch.int32, torch.float32
    cp, tp = _vec("cu_rows", cu_rows, (n + 1,), i32, index), _vec("tokens", tokens, (rows,), i32, index)
    up, np = _vec("u", u, (rows,), f32, index), _vec("u_next", u_next, shape, f32, index)
    qp, qs = None, vocab
    if draft_probs is not None:
        qs, qp = _rows("draft_probs", draft_probs, (rows, vocab), (f32,), index), draft_probs.data_ptr()
    st, keep = _settings(shape, index, temperature, top_k, min_p, top_p)
    accepted = torch.empty(shape, dtype=i32, device=device)
    following = torch.empty(shape, dtype=i32, device=device)
    raw, wb = _raw_stream(index), lib.kvr_accept_work_bytes(rows)
    work = _work_alloc(max(wb, 16), raw)
    try:
        rc = lib.kvr_accept(logits.data_ptr(), kind, ls, rows, vocab, st, n, cp, tp, qp, qs, up, np,
                            accepted.data_ptr(), following.data_ptr(), work, wb, raw)
    finally:
        _work_free(work)
    if rc:
        _check(lib, rc)
    return accepted, following
