"""What low-rank adapters lose before the output's own rounding, on the GPU against 64-bit arithmetic (GB300).

Outputs of 16 bits hide it: so base is the negated product, rounded, and of what is left the elements next to zero are
looked at, whose own rounding is far below.  All factors are positive, so nothing cancels, and a relative bound holds.
A product of the matrix units (16 inputs) cuts at most 2^-23 of the sum that it is added to."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def relative_errors(lens, k, cols, dtype, out, seed):
    """Of the elements next to zero, (what the kernel adds - the exact product) / the product.  B has one element a row, so
    an output is one element of the low-rank product, times a number of the type."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(seed)
    pos = lambda *n: torch.randn(*n, generator=g, device=DEV).abs().clamp_min(0.05)
    rank, rows = 8, sum(lens)
    a = (pos(rank, k) * k ** -0.5).to(dtype)
    b = torch.zeros(cols, rank, device=DEV)
    at = torch.arange(cols, device=DEV)
    b[at, at % rank] = pos(cols)
    b = b.to(dtype)
    x = pos(rows, k).to(dtype)
    s = torch.cat([part.double() @ a.double().t() for part in x.split(2048)])
    product = s @ b.double().t()
    cu = i32([0] + np.cumsum(lens).tolist())
    base = None if out is F32 else (-product).to(out)
    got = Adapters([(a, b, 1.0)], [cols]).kvr_adapt(x, cu, i32([0] * len(lens)), base,
                                                     out=torch.empty(rows, cols, dtype=out, device=DEV))
    left = product + (0 if base is None else base.double())
    off = (got.double() - left) / product
    return off if base is None else off[left.abs() <= product * 2.0 ** (-15 if out is BF else -13)]


@pytest.mark.parametrize("lens", [[20], [300, 40]])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_the_low_rank_product_goes_on_in_24_bits(dtype, out, lens):
    """In steps of 2^-23: four products of 16 inputs, 4, three (one a term) with B, 3; the terms and the last addition,
    1/2 each; the rounding of an output that is 2^-15 (fp16: 2^-13) of the product, 1 (1/2).  9 in all; two terms of bf16
    leave 2^-16, of fp16 2^-22."""
    off = relative_errors(lens, 64, 2048, dtype, out, len(lens))
    assert off.numel() > 200 and off.abs().max() <= 9 * STEP, (off.numel(), off.abs().max() / STEP)
