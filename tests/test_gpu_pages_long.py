"""Attention over long histories in 4-bit pages against the formula in 64 bits (needs a GB300): runs of many pages in
one warp, segments that many CTAs share or that end inside a run, and values far quieter than the keys' weights.

The reference is plain float64 on the GPU over the values that the cache stands for: codes c = clamp(round(x / s), -8, 7)
and scales s = fp16(max|x| / 7) of groups of 32, softmax, weighted sum.

Bound, per element (u = eps / 2 of the output type; w the row's weights, largest w_max; v_top the largest |v| of the
element's group of 32 dims):
* weights and values c s are fp16 numbers, 2^-11 each relative to themselves (c s of less than 2^-14 is exact: s is a
  multiple of 2^-24); scores in fp32 sums move a weight by less than 2^-13 (|scale q k| <= 90): (2 * 2^-11 + 2^-13) sum w|v|;
* a weight below fp16's normal numbers is rounded by 2^-25 absolutely, and the largest weight of a warp's run is held at
  2^14 or more: 2^-25 / 2^14 v_top w_max, 2^-38 with its sum's, per key;
* sums over the n keys of a run are n / 16 + 2 additions, each dropping at most 2^-22 of the sum so far: with |v| in place
  of v, (n / 16 + 2) 2^-22 sum w|v|; the parts of the runs are joined by a few operations of 2^-24 more;
  (The tensor-memory kernel, for more than 64 rows of a KV head, holds the weight of a row's reference at 2^7, which
  the largest is at most a factor of 2 below: 2^-25 / 2^6.)
  (That kernel also rounds c s of the keys to fp16 for bf16 activations: a score is off by the sum of d errors of at most
  2^-11 each times scale q_d, at most 6 * 2^-11 scale |q k|_2 but for odds of 2 exp(-18) (Hoeffding), a weight by
  twice that.)
* the output is rounded once: u |o|, for fp16 half of its least number, 2^-25, at the least (below 2^-14 all fp16
  numbers are 2^-24 apart).
"""
import numpy as np
import pytest
import torch

from test_gpu_pages import TYPES, handle, ints

pytestmark = pytest.mark.gpu
STEP = 1 << 18


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def warps():
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count


def stands_for(x):
    g = x.double().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1, keepdim=True) / 7).half().double().clamp(max=8188)
    return torch.where(s > 0, torch.round(g / s.clamp(min=2.0 ** -24)).clamp(-8, 7) * s, 0).flatten(-2)


class Long:
    """Sequences of given lengths, the last m[b] tokens of each being the step's rows; k and v of sequence b from
    kv(b, n) (device tensors [n][kv heads][d])."""

    def __init__(self, lens, m, heads, kv_heads, d, act, kv):
        self.lens, self.m, self.heads, self.kv_heads, self.d, self.act = lens, m, heads, kv_heads, d, act
        n_pages = sum(-(-x // 64) for x in lens)
        self.pg = handle(heads, kv_heads, d, act, n_pages=n_pages, max_seqs=len(lens), max_len=max(max(lens), 1 << 17),
                         max_rows=max(STEP, sum(m)), n_layers=1)
        self.kv = []
        at = [0] * len(lens)
        for b, n in enumerate(lens):
            k, v = kv(b, n)
            self.kv.append((k, v))
            for i in range(0, n, STEP):
                add = [0] * len(lens)
                add[b] = min(STEP, n - i)
                self.pg.kvr_page_plan(ints(at), ints(add), add[b])
                self.pg.kvr_page_append(0, None, k[i:i + STEP], v[i:i + STEP], rotate=False)
                at[b] += add[b]
        self.rows = sum(m)
        self.pg.kvr_page_plan(ints([x - y for x, y in zip(lens, m)]), ints(m), self.rows, max(m))
        self.pg.kvr_pages_sync()

    def check(self, q, run, lost=2.0 ** -38, rounds_k=False):
        """run: keys of a warp's run, at most; lost: of the largest weight, per key; rounds_k: the keys are rounded."""
        got = self.pg.kvr_page_attend(0, q)
        self.pg.kvr_pages_sync()
        scale = self.d ** -0.5
        u, row, worst = torch.finfo(TYPES[self.act]).eps / 2, 0, 0.0
        group = self.heads // self.kv_heads
        for (k, v), n, m in zip(self.kv, self.lens, self.m):
            qs, gs = q[row:row + m].double(), got[row:row + m].double()
            seen = torch.arange(n, device="cuda") <= torch.arange(n - m, n, device="cuda")[:, None]
            for j in range(self.kv_heads):
                kk, vv = stands_for(k[:, j]), stands_for(v[:, j])
                top = vv.abs().amax(0).unflatten(0, (-1, 32)).amax(-1).repeat_interleave(32)
                for h in range(j * group, (j + 1) * group):
                    w = torch.softmax((scale * qs[:, h] @ kk.T).masked_fill(~seen, -np.inf), -1)
                    ref, mag, w_max = w @ vv, w @ vv.abs(), w.amax(-1, keepdim=True)
                    spread = 0.0
                    if rounds_k and self.act == "bf16":
                        spread = scale * ((qs[:, h] ** 2) @ (kk ** 2).T).amax(-1, keepdim=True).sqrt()
                    tol = ((12 * 2.0 ** -11 * spread + 2 * 2.0 ** -11 + 2.0 ** -13 + (run / 16 + 2) * 2.0 ** -22) * mag + n * lost * top * w_max
                           + u * ref.abs() + (2.0 ** -25 if self.act == "fp16" else 0.0))
                    off = ((gs[:, h] - ref).abs() / tol).nan_to_num(nan=np.inf)
                    worst = max(worst, off.max().item())
            row += m
        assert worst <= 1, worst


def with_sinks(kv_heads, d, act, v_size, seed):
    """Keys that all score 0 but for one in 1024, whose score is that of one element of q; quiet values around v_size, 0
    at those keys.  (The key is 7 * 2^-2 in one place: one code, an exact scale.)"""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(b, n):
        k = torch.zeros(n, kv_heads, d, dtype=TYPES[act], device="cuda")
        k[::1024, :, 5] = 1.75
        v = v_size * (1 + 0.3 * torch.randn(n, kv_heads, d, device="cuda", generator=g))
        v[::1024] = 0
        return k, v.to(TYPES[act])
    return make


def sink_queries(rows, heads, d, act, gaps):
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(rows, heads, d, device="cuda", generator=g)
    q[:, :, 5] = torch.linspace(gaps[0], gaps[1], rows * heads, device="cuda").view(rows, heads) * d ** 0.5 / 1.75
    return q.to(TYPES[act])


@pytest.mark.parametrize("act,d", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("log_v", [0, -9, -12, -15, -17])
def test_quiet_values_under_sinks(act, d, log_v):
    """At least 4096 keys in a warp's run, a sink among every 1024, the others 6 to 16 nats below it: attention is linear
    in v, so the tail counts the same however quiet the values are."""
    rows, heads, n = 8, 8, 6
    tokens = 64 * (-(-warps() * 64 // (8 * n)) + 1)   # pages of a sequence, with 8 row tiles each
    w = Long([tokens] * n, [rows] * n, heads, 1, d, act, with_sinks(1, d, act, 2.0 ** log_v, 3))
    w.check(sink_queries(n * rows, heads, d, act, (6, 16)), 64 * 66)


@pytest.mark.parametrize("act,d", [("bf16", 128), ("bf16", 64), ("fp16", 128), ("fp16", 64)])
def test_many_rows_under_sinks(act, d):
    """The same for 160 rows of a KV head (the tensor-memory kernel), the others 12 to 19 nats below the sinks.  The
    keys' c s are fp16 numbers, so that their scores are exact."""
    rows, heads, n = 20, 8, 2
    w = Long([131072, 130011], [rows] * n, heads, 1, d, act, with_sinks(1, d, act, 1.0, 4))
    w.check(sink_queries(n * rows, heads, d, act, (12, 19)), 128 * 16, lost=2.0 ** -31)


def growing(kv_heads, d, act, seed):
    """Keys whose scores spread more and more, so that a row's maximum moves again and again."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(b, n):
        size = torch.linspace(0.3, 1.5, n, device="cuda")[:, None, None]
        k = torch.randn(n, kv_heads, d, device="cuda", generator=g) * size
        return k.to(TYPES[act]), torch.randn(n, kv_heads, d, device="cuda", generator=g).to(TYPES[act])
    return make


def some_queries(n, heads, d, act):
    return torch.randn(n, heads, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(TYPES[act])


@pytest.mark.parametrize("act,d,heads,kv_heads,rows", [("bf16", 128, 8, 1, 8), ("bf16", 64, 8, 1, 8), ("fp16", 128, 8, 1, 8),
                                                       ("fp16", 64, 8, 1, 8), ("bf16", 128, 16, 4, 1), ("fp16", 64, 8, 8, 1)])
def test_runs_of_many_pages(act, d, heads, kv_heads, rows):
    """More than 32 pages in every warp's run (its list of pages is fetched 32 at a time, its ring wraps many times), with
    sequences of 1 to 900 pages: segments that end inside runs, that follow one another in them, and that
    several CTAs share."""
    rng = np.random.Generator(np.random.PCG64([d, rows]))
    units_of = -(-rows * heads // kv_heads // 8) * kv_heads       # of a page: row tiles of 8, KV heads
    lens, units = [], 0
    while units < 36 * warps():
        lens.append(rows + int(64 * 900 ** rng.random()))
        units += units_of * -(-lens[-1] // 64)
    w = Long(lens, [rows] * len(lens), heads, kv_heads, d, act, growing(kv_heads, d, act, 5))
    w.check(some_queries(w.rows, heads, d, act), 64 * 40)


@pytest.mark.parametrize("act,d,heads,kv_heads", [("bf16", 128, 7, 1), ("fp16", 64, 4, 1), ("bf16", 64, 8, 2)])
@pytest.mark.parametrize("lens", [[20011], [131071], [70001, 3000, 65]])
def test_one_row_over_a_long_history(act, d, heads, kv_heads, lens):
    """Few pages a warp and many CTAs a segment: its parts are joined in the CTAs, then by the last of them."""
    w = Long(lens, [1] * len(lens), heads, kv_heads, d, act, growing(kv_heads, d, act, 6))
    w.check(some_queries(w.rows, heads, d, act), 131072 // 64)


@pytest.mark.parametrize("act,d,heads,kv_heads", [("bf16", 128, 28, 4), ("fp16", 128, 8, 2), ("bf16", 64, 8, 2), ("fp16", 64, 7, 1)])
@pytest.mark.parametrize("lens,rows", [([16001], [30]), ([16400], [130]), ([40000, 300, 5000], [33, 260, 1])])
def test_many_rows_over_a_long_history(act, d, heads, kv_heads, lens, rows):
    """The tensor-memory kernel, with segments of parts from many CTAs."""
    w = Long(lens, rows, heads, kv_heads, d, act, growing(kv_heads, d, act, 7))
    w.check(some_queries(w.rows, heads, d, act), 40000, lost=2.0 ** -31, rounds_k=True)
