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


def relative_errors(lens, k, cols, dtype, out, seed, less=1.0, size=(0, 0, 0, 1.0)):
    """Of the elements next to zero, (what the kernel adds - the exact product) / the product.  B has one element a row, so
    an output is one element of the low-rank product, times a number of the type.  All of A but its first row is `less`
    times the usual size, and B's part of it that much larger; x, A and B are 2^size[:3] of theirs, and the adapter's
    scale is size[3]."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(seed)
    pos = lambda *n: torch.randn(*n, generator=g, device=DEV).abs().clamp_min(0.05)
    rank, rows = 8, sum(lens)
    a = pos(rank, k) * k ** -0.5
    a[1:] *= less
    a = (a * 2.0 ** size[1]).to(dtype)
    b = torch.zeros(cols, rank, device=DEV)
    at = torch.arange(cols, device=DEV)
    b[at, at % rank] = pos(cols)
    b[:, 1:] /= less
    b = (b * 2.0 ** size[2]).to(dtype)
    x = (pos(rows, k) * 2.0 ** size[0]).to(dtype)
    s = torch.cat([part.double() @ a.double().t() for part in x.split(2048)])
    product = s @ b.double().t() * float(np.float32(size[3]))
    cu = i32([0] + np.cumsum(lens).tolist())
    base = None if out is F32 else (-product).to(out)
    got = Adapters([(a, b, size[3])], [cols]).kvr_adapt(x, cu, i32([0] * len(lens)), base,
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


@pytest.mark.parametrize("lens,k", [([1, 1, 1], 8192), ([60, 250, 3], 8192), ([7424], 8192), ([3000, 900, 4000], 1000)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_long_sums_lose_nothing_to_their_length(dtype, out, lens, k):
    """Sums of equal signs, whose cut bits add up: the mean of the errors.  In steps of 2^-23 at most: chains of 128 inputs
    are eight products, which on average are added to 9/16 of the chain, 4.5; three products with B, 3; additions and
    roundings have no bias.  8 with room for what they leave.  (One chain of 8192 inputs would cut 512 times.)  7424 rows
    are tiles enough that none shares its inputs with another CTA."""
    off = relative_errors(lens, k, 2048 if sum(lens) < 100 else 64, dtype, out, k + len(lens))
    assert off.numel() > 20 and off.mean().abs() <= 8 * STEP, (off.numel(), off.mean() / STEP)


@pytest.mark.parametrize("lens", [[5, 2], [300, 40]])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sums_of_either_sign(dtype, lens):
    """Outputs of 32 bits, rms error over rms output.  A chain's eight sums are on average 0.57 of its last one, each cut by
    half a step at most in the mean and all the same way: 0.57 x 8 x 2^-24; the chains' sums are added with errors
    of 2^-25 of the running sum, 64 of them: 4 x 2^-24; three terms times the rank's products with B the same as one
    chain of 3: 3 x 2^-24.  In all 11.6 x 2^-24 = 7e-7."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(3)
    k, rank, rows, cols = 8192, 16, sum(lens), 512
    a = (torch.randn(2 * rank, k, generator=g, device=DEV) * k ** -0.5).to(dtype)
    b = torch.randn(2 * cols, rank, generator=g, device=DEV).to(dtype)
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    got = Adapters([(a, b, 1.0)], [cols, cols]).kvr_adapt(x, i32([0] + np.cumsum(lens).tolist()), i32([0] * len(lens)),
                                                           out=torch.empty(rows, 2 * cols, device=DEV)).double()
    s = x.double() @ a.double().t()
    want = torch.cat([s[:, j * rank:(j + 1) * rank] @ b[j * cols:(j + 1) * cols].double().t() for j in (0, 1)], 1)
    assert ((got - want).pow(2).mean() / want.pow(2).mean()).sqrt() <= 7e-7


@pytest.mark.parametrize("lens", [[20], [300, 40]])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_small_elements_beside_large_ones(dtype, out, lens):
    """Elements of the low-rank product 2^-9 of their row's largest, by B as large as that one: as exact as alone."""
    off = relative_errors(lens, 64, 2048, dtype, out, len(lens), less=2.0 ** -9)
    assert off.numel() > 200 and off.abs().max() <= 9 * STEP, (off.numel(), off.abs().max() / STEP)


@pytest.mark.parametrize("lens", [[20], [300, 40]])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("size", [(60, 62, -110, 1000.0), (63, 60, -120, 3e20), (-58, -58, 100, 3e-12), (-40, -50, 120, 1e-38),
                                  (0, 0, 100, 2e-38), (10, 0, -110, 1.7e38)])
def test_magnitudes_whose_product_is_ordinary(size, out, lens):
    """Low-rank products and scales next to the ends of the 32-bit floats' range, and B that brings them back.  One step
    more than above: the scale is no power of two."""
    off = relative_errors(lens, 64, 2048, BF, out, len(lens), size=size)
    assert off.numel() > 200 and off.abs().max() <= 10 * STEP, (off.numel(), off.abs().max() / STEP)


@pytest.mark.parametrize("lens", [[1, 19], [300, 40]])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
def test_infinities_of_b_are_those_of_the_formula(dtype, out, lens):
    """An infinity in B is the output's, with the sign of its low-rank element; NaN where that is 0, where two of them
    meet with other signs, and where B is NaN.  All other outputs are as they were."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(8)
    k, rank, rows, cols = 256, 16, sum(lens), [200, 72]
    a = (torch.randn(2 * rank, k, generator=g, device=DEV) * k ** -0.5).to(dtype)
    b = torch.randn(sum(cols), rank, generator=g, device=DEV).to(dtype)
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    x[1] = 0
    base = torch.randn(rows, sum(cols), generator=g, device=DEV).to(out)
    cu, which = i32([0] + np.cumsum(lens).tolist()), i32([0, 0])
    clean = Adapters([(a, b, -2.0)], cols).kvr_adapt(x, cu, which, base)
    b = b.clone()
    inf = float("inf")
    for n, j, v in ((0, 0, inf), (7, 3, -inf), (64, 15, inf), (131, 8, inf), (131, 9, inf), (199, 1, float("nan")), (200, 0, inf),
                    (271, 5, -inf)):
        b[n, j] = v
    for same in (False, True):
        to = base.clone() if same else None
        got = Adapters([(a, b, -2.0)], cols).kvr_adapt(x, cu, which, base if to is None else to, out=to).double().cpu()
        s = (x.double() @ a.double().t()).cpu()
        bd, hit = b.double().cpu(), [0, 7, 64, 131, 199, 200, 271]
        for n in hit:
            part = s[:, :rank] if n < 200 else s[:, rank:]
            want = base[:, n].double().cpu() - 2.0 * (part * bd[n]).sum(1)
            assert torch.equal(got[:, n].isnan(), want.isnan()), n
            assert torch.equal(got[:, n][~want.isnan()], want[~want.isnan()]), n
        rest = [n for n in range(sum(cols)) if n not in hit]
        assert torch.equal(got[:, rest], clean.double().cpu()[:, rest])
