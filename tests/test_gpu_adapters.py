"""Low-rank adapters on the GPU against 64-bit arithmetic (GB300).

The bound of an element, from the arithmetic that include/kvr.h states: the output's rounding (half a step of it); the
32-bit sums, cut by the tensor cores to 2^-23 of what they hold at each of K / 16 products and at the few additions that
join the parts; and the low-rank product's terms (bf16 2^-8 each, fp16 2^-11 each; elements next to zero lose 2^-25 of
the largest of their row)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(k, cols, ranks, dtype, seed):
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator().manual_seed(seed)
    n = sum(cols)
    entries = [((torch.randn(len(cols) * r, k, generator=g) * k ** -0.5).to(dtype).to(DEV),
                torch.randn(n, r, generator=g).to(dtype).to(DEV), [1.0, 2.0, -0.5, 0.0][i % 4])
               for i, r in enumerate(ranks)]
    return Adapters(entries, cols), entries


def oracle(x, entries, cols, which, cu, base):
    """(value, bound without the output's own rounding) in 64 bits; rows of no sequence are base's."""
    out = base.double().cpu().clone()
    err = torch.zeros_like(out)
    x = x.double().cpu()
    dt = entries[0][0].dtype
    terms = 2.0 ** -22 if dt is HF else (2.0 ** -24 if base.dtype is F32 else 2.0 ** -16)
    for b, a in enumerate(which):
        r0, r1 = cu[b], cu[b + 1]
        if not 0 <= a < len(entries) or r0 == r1:
            continue
        A, B, scale = entries[a][0].double().cpu(), entries[a][1].double().cpu(), entries[a][2]
        rank, at = B.shape[1], 0
        for j, n in enumerate(cols):
            Aj, Bj = A[j * rank:(j + 1) * rank], B[at:at + n]
            s = x[r0:r1] @ Aj.t()
            out[r0:r1, at:at + n] += scale * (s @ Bj.t())
            big = x[r0:r1].abs() @ Aj.abs().t()
            cut = (x.shape[1] / 16 + 80) * 2.0 ** -23
            err[r0:r1, at:at + n] += abs(scale) * ((big @ Bj.abs().t()) * (cut + terms + (rank / 16 + 4) * 2.0 ** -22)
                                                  + 2.0 ** -24 * s.abs().amax(1, keepdim=True) * Bj.abs().sum(1)[None])
            at += n
    return out, err


def check(x, entries, cols, which, cu, base, got):
    want, err = oracle(x, entries, cols, which, cu, base)
    tol = err + torch.finfo(got.dtype).eps / 2 * (want.abs() + err) + (2.0 ** -25 if got.dtype is HF else 2.0 ** -133)
    off = (got.double().cpu() - want).abs()
    assert (off <= tol).all(), ((off / tol).max(), (off > tol).nonzero()[:4])


PATTERNS = {
    "one": ([1], [0]),
    "tokens": ([1] * 9, [0, 1, 2, 0, -1, 1, 1, 2, 0]),
    "verify": ([4, 8, 1, 3, 5], [2, 2, 0, -1, 1]),
    "ragged": ([0, 17, 0, 1, 40, 7, 130, 0], [0, 1, 2, 0, 2, 7, 1, 1]),
    "long": ([300, 2, 77], [1, 0, 2]),
}


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("k,cols,ranks", [(8, [8], [8, 8, 8]), (1000, [520, 72], [8, 24, 40]), (512, [512, 128, 128], [16, 64, 128]),
                                          (2560, [264], [128, 8, 16]), (4096, [1024, 256, 256], [16, 32, 48])])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_against_64_bits(pattern, k, cols, ranks, dtype, out):
    lens, which = PATTERNS[pattern]
    rows = sum(lens)
    site, entries = make(k, cols, ranks, dtype, k + rows)
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, k, generator=g).to(dtype).to(DEV)
    base = torch.randn(rows, sum(cols), generator=g).to(out).to(DEV)
    cu = [0] + np.cumsum(lens).tolist()
    got = site.kvr_adapt(x, i32(cu), i32(which), base)
    check(x, entries, cols, which, cu, base, got)
    again = site.kvr_adapt(x, i32(cu), i32(which), base)
    assert torch.equal(got, again)
    zero = torch.zeros_like(base)
    none = site.kvr_adapt(x, i32(cu), i32(which), out=torch.full_like(base, 7.0))
    check(x, entries, cols, which, cu, zero, none)
    same = base.clone()
    assert site.kvr_adapt(x, i32(cu), i32(which), same, out=same) is same and torch.equal(same, got)


def test_rows_of_no_sequence_and_sequences_without_an_adapter():
    site, entries = make(256, [64, 64], [16, 8], BF, 3)
    x = torch.randn(40, 256, device=DEV).to(BF)
    x[:3], x[33:] = float("nan"), float("nan")
    base = torch.randn(40, 128, device=DEV).to(BF)
    base[12, :5] = torch.tensor([float("inf"), float("nan"), -0.0, 1e-40, -float("inf")])
    cu, which = [3, 10, 20, 33], [1, -1, 5]
    out = torch.full_like(base, 9.0)
    got = site.kvr_adapt(x, i32(cu), i32(which), base, out=out)
    assert (got[:3] == 9).all() and (got[33:] == 9).all()
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(bits(got[10:33]), bits(base[10:33]))    # base's own bits
    check(x[3:10], entries, [64, 64], [1], [0, 7], base[3:10], got[3:10])
    out.fill_(9.0)
    site.kvr_adapt(x, i32([0, 0, 0, 0]), i32(which), base, out=out)
    assert (out == 9).all()


def test_what_is_not_finite_stays_in_its_rows():
    from prefix_reused_prefill_gb300 import Adapters
    site, entries = make(512, [128], [16, 16, 16], BF, 4)
    x = torch.randn(24, 512, device=DEV).to(BF)
    cu, which = [0, 2, 3, 5, 16, 24], [0, 1, 2, 0, 2]
    base = torch.randn(24, 128, device=DEV).to(BF)
    clean = site.kvr_adapt(x, i32(cu), i32(which), base)
    x[2, 5], x[6, 1] = float("nan"), float("inf")
    got = site.kvr_adapt(x, i32(cu), i32(which), base)
    bad = [2, 6]
    good = [r for r in range(24) if r not in bad]
    assert got[bad].isnan().all() and torch.equal(got[good], clean[good])
    entries[1][0][3, 7] = float("nan")         # an adapter's own: only its rows
    entries[2][1][5, 3] = float("inf")
    x[2, 5], x[6, 1] = 1.0, 1.0
    got = Adapters(entries, [128]).kvr_adapt(x, i32(cu), i32(which), base)
    zero = [0, 1] + list(range(5, 16))
    again = site.kvr_adapt(x, i32(cu), i32([0, -1, -1, 0, -1]), base)
    assert torch.equal(got[zero], again[zero]) and got[2].isnan().all()


def test_magnitudes_beyond_16_bits():
    """Low-rank products far above and below what fp16 holds."""
    for dtype in (BF, HF):
        site, entries = make(256, [64], [16], dtype, 5)
        for size in (2.0 ** 13, 2.0 ** -14):
            x = (torch.randn(5, 256, device=DEV) * size).to(dtype)
            entries[0][0].mul_(64.0 if size > 1 else 2.0 ** -8)
            base = torch.zeros(5, 64, device=DEV)
            got = site.kvr_adapt(x, i32([0, 5]), i32([0]), base)
            check(x, entries, [64], [0], [0, 5], base, got)
            entries[0][0].mul_(1 / 64.0 if size > 1 else 2.0 ** 8)


def test_strides():
    site, entries = make(264, [72, 8], [24], HF, 6)
    wide = torch.randn(21, 264 + 40, device=DEV).to(HF)
    x = wide[::3, 16:280]
    bw = torch.randn(7, 80 + 24, device=DEV)
    ow = torch.full((14, 96), 3.0, device=DEV)
    got = site.kvr_adapt(x, i32([0, 7]), i32([0]), bw[:, 8:88], out=ow[::2, 8:88])
    check(x, entries, [72, 8], [0], [0, 7], bw[:, 8:88], got)
    assert (ow[1::2] == 3).all() and (ow[:, :8] == 3).all() and (ow[:, 88:] == 3).all()


def test_many_sequences_one_adapter_and_many():
    n = 2048
    site, entries = make(128, [64], [8] * 37, BF, 7)
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 3, (n,), generator=g).tolist()
    which = torch.randint(-1, 38, (n,), generator=g).tolist()
    cu = [0] + np.cumsum(lens).tolist()
    x = torch.randn(cu[-1], 128, device=DEV).to(BF)
    base = torch.randn(cu[-1], 64, device=DEV).to(BF)
    check(x, entries, [64], which, cu, base, site.kvr_adapt(x, i32(cu), i32(which), base))
    check(x, entries, [64], [3] * n, cu, base, site.kvr_adapt(x, i32(cu), i32([3] * n), base))


def test_no_rows():
    site, _ = make(64, [8], [8], BF, 9)
    out = site.kvr_adapt(torch.zeros(0, 64, dtype=BF, device=DEV), i32([0, 0]), i32([0]))
    assert out.shape == (0, 8)


def test_captured_on_another_stream_and_two_at_once():
    site, entries = make(1024, [256, 64], [16, 64], BF, 10)
    x = torch.randn(50, 1024, device=DEV).to(BF)
    base = torch.randn(50, 320, device=DEV).to(BF)
    cu, which = i32([0, 1, 30, 50]), i32([0, 1, 0])
    want = site.kvr_adapt(x, cu, which, base)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(4)]
    outs = [site.kvr_adapt(x, cu, which, base, stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = site.kvr_adapt(x, cu, which, base)
    x.copy_(torch.randn(50, 1024, device=DEV))
    which.copy_(i32([1, 0, -1]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, site.kvr_adapt(x, cu, which, base))


def test_refusals():
    from prefix_reused_prefill_gb300 import Adapters, KvrError
    site, entries = make(64, [16, 16], [8], BF, 11)
    a, b, s = entries[0]
    x, cu, which = torch.zeros(4, 64, dtype=BF, device=DEV), i32([0, 4]), i32([0])
    base = torch.zeros(4, 32, dtype=BF, device=DEV)
    zeros = lambda *n: torch.zeros(*n, dtype=BF, device=DEV)
    for bad in (lambda: Adapters([], [16]), lambda: Adapters(entries, [16, 20]), lambda: Adapters(entries, [16, 8]),
                lambda: Adapters([(a.float(), b.float(), s)], [16, 16]), lambda: Adapters([(a, b.half(), s)], [16, 16]),
                lambda: Adapters([(a, b.t(), s)], [16, 16]), lambda: Adapters([(a.cpu(), b, s)], [16, 16]),
                lambda: Adapters([(zeros(2 * 136, 64), zeros(32, 136), 1.0)], [16, 16]),
                lambda: site.kvr_adapt(x.half(), cu, which, base), lambda: site.kvr_adapt(x[:, :56], cu, which, base),
                lambda: site.kvr_adapt(x, cu.long(), which, base), lambda: site.kvr_adapt(x, cu[:1], which, base),
                lambda: site.kvr_adapt(x, cu, which, base.half()), lambda: site.kvr_adapt(x, cu, which, base[:3]),
                lambda: site.kvr_adapt(x, cu, which, base, out=base.float()), lambda: site.kvr_adapt(x.cpu(), cu, which, base)):
        with pytest.raises(KvrError):
            bad()
    both = zeros(5, 32)
    with pytest.raises(KvrError):
        site.kvr_adapt(x, cu, which, both[:4], out=both[1:])
    torch.cuda.synchronize()
