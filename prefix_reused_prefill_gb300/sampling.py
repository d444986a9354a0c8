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
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle (a Stream object costs 2 us)
Setting = Optional[Union[torch.Tensor, float, int]]


class _On:
    """The tensors' device for the length of a call, where another one is current."""

    def __init__(self, index: int):
        self.other = torch.cuda.device(index) if index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()

    def __exit__(self, *args):
        if self.other is not None:
            self.other.__exit__(*args)


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


def _settings(n: int, index: int, **given):
    st, keep = KvrSampling(), []
    for name, x in given.items():
        if x is None:
            continue
        dtype = torch.int32 if name == "top_k" else torch.float32
        if not isinstance(x, torch.Tensor):
            x = torch.full((n,), x, dtype=dtype, device=index)
        setattr(st, name, _vec(name, x, n, dtype, index))
        keep.append(x)
    return st, keep


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
    lib = load_library()
    index, ls = _logits(logits)
    rows, vocab = logits.shape
    up = _vec("u", u, rows, torch.float32, index)
    with _On(index), torch.cuda.stream(stream):   # (where one is given) memory that it may write at once
        st, keep = _settings(rows, index, temperature=temperature, top_k=top_k, min_p=min_p, top_p=top_p)
        token = torch.empty(rows, dtype=torch.int32, device=logits.device)
        prob = torch.empty(rows, dtype=torch.float32, device=logits.device)
        ds = vocab
        if dist is True:
            dist = torch.empty((rows, vocab), dtype=torch.float32, device=logits.device)
        elif dist is False:
            dist = None
        else:
            ds = _rows("dist", dist, (rows, vocab), (torch.float32,), index)
        _check(lib, lib.kvr_sample(logits.data_ptr(), _TYPES[logits.dtype], ls, rows, vocab, ctypes.byref(st), up,
                                   token.data_ptr(), prob.data_ptr(), None if dist is None else dist.data_ptr(), ds,
                                   stream.cuda_stream if stream is not None else _raw_stream(index)))
    return (token, prob) if dist is None else (token, prob, dist)


def kvr_accept(logits: torch.Tensor, tokens: torch.Tensor, cu_rows: torch.Tensor, u: torch.Tensor,
               u_next: torch.Tensor, draft_probs: Optional[torch.Tensor] = None, temperature: Setting = None,
               top_k: Setting = None, min_p: Setting = None, top_p: Setting = None, stream=None):
    """Speculative sampling: rows cu_rows[b] .. cu_rows[b + 1] - 1 of logits [rows][vocab] and of tokens (int32; the
    last committed token, then the drafts) are sequence b's.  Returns per sequence (drafts that stay, the token after
    them), int32.  u [rows] judges the drafts, u_next [n_seq] draws; draft_probs: float32 [rows][vocab], the
    distribution of the draft after each row (None: the drafts were certain).  Settings: [n_seq]."""
    lib = load_library()
    index, ls = _logits(logits)
    rows, vocab = logits.shape
    n = cu_rows.numel() - 1
    if n < 1:
        raise KvrError(-1, "cu_rows must have an entry more than there are sequences")
    args = (_vec("cu_rows", cu_rows, n + 1, torch.int32, index), _vec("tokens", tokens, rows, torch.int32, index))
    us = (_vec("u", u, rows, torch.float32, index), _vec("u_next", u_next, n, torch.float32, index))
    qp, qs = None, vocab
    if draft_probs is not None:
        qs, qp = _rows("draft_probs", draft_probs, (rows, vocab), (torch.float32,), index), draft_probs.data_ptr()
    with _On(index), torch.cuda.stream(stream):
        st, keep = _settings(n, index, temperature=temperature, top_k=top_k, min_p=min_p, top_p=top_p)
        accepted = torch.empty(n, dtype=torch.int32, device=logits.device)
        following = torch.empty(n, dtype=torch.int32, device=logits.device)
        wb = lib.kvr_accept_work_bytes(rows)
        work = torch.empty(wb, dtype=torch.uint8, device=logits.device)
        _check(lib, lib.kvr_accept(logits.data_ptr(), _TYPES[logits.dtype], ls, rows, vocab, ctypes.byref(st), n,
                                   *args, qp, qs, *us, accepted.data_ptr(), following.data_ptr(), work.data_ptr(), wb,
                                   stream.cuda_stream if stream is not None else _raw_stream(index)))
    return accepted, following
