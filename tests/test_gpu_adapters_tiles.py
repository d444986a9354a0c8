"""Low-rank adapters over batches that fill the GPU several times (GB300), against 64-bit arithmetic on the device.

A CTA takes runs of tiles here: the next tile's products under the last one's outputs, buffers and their barriers used
again, from one part of the outputs to the next and from one sequence to the next.  Bound of an element, in steps of
2^-23 of sum |B| sum |A| |x|: eight products of a chain, half a step for each of the chains' sums, three products (one a
term) for 16 ranks, and four for the terms and the last roundings; and the output's own rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run(lens, which, k, cols, ranks, dtype, out, seed, same=False):
    """A call with random operands, checked whole; returns what it wrote and how far it was off at most, in bounds."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, rows = sum(cols), sum(lens)
    entries = [((torch.randn(len(cols) * r, k, generator=g, device=DEV) * k ** -0.5).to(dtype),
                torch.randn(n, r, generator=g, device=DEV).to(dtype), [1.0, -0.5, 3.0][i % 3]) for i, r in enumerate(ranks)]
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    base = torch.randn(rows, n, generator=g, device=DEV).to(out)
    want, bound = base.double(), torch.zeros(rows, n, dtype=torch.float64, device=DEV)
    at = 0
    for b, m in enumerate(lens):
        if 0 <= which[b] < len(entries):
            A, B, scale = entries[which[b]]
            rank, col = B.shape[1], 0
            steps = 8 + k / 256 + 3 * rank / 16 + 4
            for j, c in enumerate(cols):
                Aj, Bj = A[j * rank:(j + 1) * rank].double(), B[col:col + c].double()
                xs, to = x[at:at + m].double(), (slice(at, at + m), slice(col, col + c))
                want[to] += scale * ((xs @ Aj.t()) @ Bj.t())
                bound[to] = abs(scale) * steps * 2.0 ** -23 * ((xs.abs() @ Aj.abs().t()) @ Bj.abs().t())
                col += c
        at += m
    cu = i32([0] + np.cumsum(lens).tolist())
    if same:
        base = base.clone()
    got = Adapters(entries, cols).kvr_adapt(x, cu, i32(which), base, out=base if same else None)
    tol = bound + torch.finfo(out).eps / 2 * (want.abs() + bound) + (2.0 ** -25 if out is HF else 2.0 ** -133)
    off = ((got.double() - want).abs() / tol).max().item()
    assert off <= 1, off
    return got


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("lens,which,cols,ranks", [
    ([3000, 1, 1900, 2715], [1, 0, -1, 2], [2056, 264, 264], [16, 64, 128]),     # runs over parts, sequences and ranks
    ([2999, 2000, 129, 2560], [0, 1, 0, 2], [1032], [8, 40, 24]),                # one part, its last tile of 8 outputs
    ([700, 0, 64, 1, 65, 900, 128, 300], [0, 3, 1, 2, 2, 0, 1, -1], [4096, 4096], [24, 16, 64]),
])
def test_runs_of_many_tiles(lens, which, cols, ranks, dtype, out):
    for same in (False, True):
        got = run(lens, which, 512, cols, ranks, dtype, out, len(lens), same)
    assert torch.equal(got, run(lens, which, 512, cols, ranks, dtype, out, len(lens)))


@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("k", [72, 520, 4096])
def test_inputs_that_no_cta_shares(k, dtype, out):
    """Tiles enough that each has one CTA for all inputs."""
    run([4000, 3500, 500], [1, 0, 1], k, [64, 64], [32, 8], dtype, out, k)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF)])
@pytest.mark.parametrize("long", [512, 2048])
def test_one_long_sequence_beside_many_short_ones(long, dtype, out):
    """A prompt in one step with a token of each of 150 others: tiles of eight rows for all (2048), and the other way."""
    run([1] * 70 + [long] + [1] * 80, [i % 5 - 1 for i in range(151)], 1024, [512, 72], [16, 64, 8, 32], dtype, out, long)
    run([1] * 7 + [long] + [1] * 8, [i % 5 - 1 for i in range(16)], 1024, [512, 72], [16, 64, 8, 32], dtype, out, long)
