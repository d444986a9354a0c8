"""The paged 4-bit cache against its float64 oracle (needs a GB300).

Bounds, per element (u = half a step of the output type, 2^-9 relative for bf16's 8 bits counted as eps / 2 = 2^-8):
* plan: exact.
* q of append: 32-bit arithmetic, a few roundings of 2^-24 on each of the two terms of a rotated element, each term at
  most |x| + |x'| in size: 2^-20 (|x| + |x'|) + eps/2 |y|.
* v of append (and k without norm and rotation): exact, the cache of a 16-bit value has one answer.
* k of append: the cache holds y (rounded to the type) to half a scale, 7 scales being the group's largest, with s
  rounded to fp16 (2^-11, or 2^-25 absolutely) and the largest code clamped to 7 s >= (1 - 2^-11) top; read back in the
  type: s/2 + 7 s 2^-11 + 2 eps/2 |y|, plus the 2^-20 of y.
* attend, on known K and V: the weights p and p s are fp16 (eps/2 = 2^-11 each; below 2^-14 half of 2^-24
  absolutely, where the largest p is 4), the scores are fp32 sums whose error moves a weight by less than
  2^-13 for the scores here (|scale q k| <= 90, 2^-20 relative), the output is rounded once.  The values are summed
  in n / 16 + 2 fp32 additions that may each drop 2^-22 of the running sum, itself at most max|v|:
  (2 * 2^-11 + 2^-13) sum w|v| + n (2^-27 max|v| + 2^-24) + (n / 16 + 2) 2^-22 max|v| + eps/2 |o|.
  Sequences with many rows of a KV head (the tensor-memory kernel: more than 64, or more than 16 in a step where one has
  more than 64, where the sequences may be long) read k as fp16 too where the activations are bf16: c s has 14 bits, each
  rounded by at most 2^-11.  A score is off by the sum of d such errors times scale q_d: at most
  6 * 2^-11 scale |q k|_2 but for odds of 2 exp(-18) (Hoeffding), and a weight by twice that of its row's largest.
"""
import numpy as np
import pytest
import torch

from oracle import pages as op

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def half_step(act):
    return torch.finfo(TYPES[act]).eps / 2


def rand(rng, shape, act, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).to(TYPES[act])


def handle(heads=8, kv_heads=2, d=64, act="bf16", n_pages=64, max_seqs=8, max_len=1 << 17, max_rows=512,
           n_layers=2, **kw):
    """(max_len: at the default the step may be long, and many rows go to the tensor-memory kernel.)"""
    from prefix_reused_prefill_gb300 import PagedKv, paged_config
    return PagedKv(paged_config(n_pages=n_pages, n_layers=n_layers, n_q_heads=heads, n_kv_heads=kv_heads, head_dim=d,
                                max_seqs=max_seqs, max_len=max_len, max_rows=max_rows, act=act, **kw))


def code_of(call):
    from prefix_reused_prefill_gb300 import KvrError
    with pytest.raises(KvrError) as e:
        call()
    return e.value.code


# --------------------------------------------------------------------------- plan
def check_tables(pg, t, n, rows):
    s = pg.state
    torch.cuda.synchronize()
    assert s.lens.tolist() == t.lens
    assert s.free[:s.count.item()].tolist() == t.free
    for b, pages in enumerate(t.pages):
        assert s.table[b].tolist() == pages + [-1] * (s.table.shape[1] - len(pages)), b
    got = list(zip(s.row_seq[:rows].tolist(), s.row_pos[:rows].tolist(), s.row_slot[:rows].tolist()))
    assert got == t.rows + [(-1, -1, -1)] * (rows - len(t.rows))
    cu = s.cu[:n + 1].tolist()
    assert cu[0] == 0 and cu[-1] == len(t.rows)
    assert [b for b in range(n) for _ in range(cu[b + 1] - cu[b])] == [r[0] for r in t.rows]


@pytest.mark.parametrize("n,max_rows,n_pages", [(1, 40, 9), (5, 200, 30), (33, 1024, 400), (300, 1025, 2000),
                                                (2048, 6000, 9000)])
def test_plan_follows_the_oracle(n, max_rows, n_pages):
    """Random steps: growth, cut drafts, ended and restarted sequences, padding, and steps that must be refused."""
    rng = np.random.Generator(np.random.PCG64(n))
    pg = handle(n_pages=n_pages, max_seqs=n, max_len=700, max_rows=max_rows)
    t = op.Tables(n_pages, n, 700)
    refused = 0
    for step in range(25):
        m = int(rng.integers(1, n + 1)) if step % 3 == 2 else n
        keep = [int(rng.choice([x, max(0, x - int(rng.integers(0, 9))), 0], p=[.6, .3, .1])) for x in t.lens[:m]]
        big = max_rows // m + 1
        add = [int(rng.choice([0, 1, int(rng.integers(0, big + 1)), int(rng.integers(0, 2 * big + 1))], p=[.2, .4, .2, .2]))
               for _ in range(m)]
        add = [min(a, 700 - k) for a, k in zip(add, keep)]
        rows = min(max_rows, sum(add) + int(rng.integers(0, 4)))
        if step == 7:
            keep[0] += 701
        if step == 8:
            add[-1] = -1
        ok = t.plan(keep, add, rows)
        pg.kvr_page_plan(ints(keep), ints(add), rows)
        check_tables(pg, t, m, rows)
        if ok:
            pg.kvr_pages_sync()
        else:
            refused += 1
            assert code_of(pg.kvr_pages_sync) in (-1, -2)
            pg.kvr_pages_sync()   # reported once
    assert 0 < refused < 25


def test_plan_takes_the_state_itself_as_keep():
    """keep may be the handle's own lengths: every sequence goes on."""
    pg, t = handle(max_len=1024), op.Tables(64, 8, 1024)
    for add in ([3, 0, 70, 1, 0, 0, 5, 64], [1] * 8, [0, 0, 64, 0, 1, 0, 0, 1]):
        t.plan(list(t.lens), add, 512)
        pg.kvr_page_plan(pg.state.lens, ints(add), 512)
        check_tables(pg, t, 8, 512)


def test_a_step_longer_than_promised_is_refused():
    pg = handle()
    pg.kvr_page_plan(ints([0, 0]), ints([3, 9]), 12, 8)
    assert code_of(pg.kvr_pages_sync) == -1
    pg.kvr_page_plan(ints([0, 0]), ints([8, 2]), 12, 8)
    pg.kvr_pages_sync()
    assert pg.state.lens.tolist()[:2] == [8, 2]


# --------------------------------------------------------------------------- append and read
def step_rows(lens):
    return [(b, i) for b, n in enumerate(lens) for i in range(n)]


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (6, 2, 128), (28, 4, 128), (1, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("norm,rotate", [(True, True), (False, True), (True, False)])
def test_append_matches_the_definition(act, heads, kv_heads, d, norm, rotate):
    rng = np.random.Generator(np.random.PCG64([heads, d]))
    pg = handle(heads, kv_heads, d, act, rope_theta=1e4, norm_eps=1e-5)
    keep, add = [0, 67, 0, 130], [3, 1, 65, 62]
    pg.kvr_page_plan(ints([0] * 4), ints(keep), 512)
    pg.kvr_page_plan(ints(keep), ints(add), sum(add))
    n = sum(add)
    # one row of a projection's output: q, k, v, and columns of something else behind
    qkv = rand(rng, (n, (heads + 2 * kv_heads) * d + 24), act, 1.5)
    qkv[0, :heads * d] = 0                                   # a head of zeros under the norm
    dev = qkv.cuda()
    q, k, v = (dev[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in
               ((0, heads), (heads, heads + kv_heads), (heads + kv_heads, heads + 2 * kv_heads)))
    gq, gk = (rand(rng, (d,), act) + 1 if norm else None for _ in range(2))
    got = f64(pg.kvr_page_append(1, q, k, v, gq.cuda() if norm else None, gk.cuda() if norm else None, rotate=rotate))
    kc, vc = (f64(x) for x in pg.kvr_page_read(1))
    pg.kvr_pages_sync()
    u = half_step(act)
    assert np.array_equal(vc, f64(torch.from_numpy(op.values(f64(v))).to(TYPES[act])))
    row = 0
    for b, (p0, m) in enumerate(zip(keep, add)):
        for i in range(m):
            for name, x, gain in (("q", f64(q[row]), gq), ("k", f64(k[row]), gk)):
                g = f64(gain) if norm else None
                y = op.norm_rotate(x, p0 + i, 1e4, g, 1e-5, rotate)
                z = np.abs(op.norm_rotate(x, 0, 1e4, g, 1e-5, False))
                size = z + np.roll(z, d // 2, axis=-1)
                if name == "q":
                    bad = np.abs(got[row] - y) > 2.0 ** -20 * size + u * np.abs(y) + 2.0 ** -25
                else:
                    s = np.max(np.abs(y).reshape(-1, d // 32, 32), axis=-1) / 7
                    s = np.repeat(s, 32, axis=-1) * (1 + 2 * u + 2.0 ** -11) + 2.0 ** -25
                    bad = np.abs(kc[row] - y) > s / 2 + 7 * s * 2.0 ** -11 + 2 * u * np.abs(y) + 2.0 ** -20 * size
                assert not bad.any(), (name, b, i, int(bad.sum()))
            row += 1


@pytest.mark.parametrize("act,d", [("bf16", 128), ("fp16", 64)])
def test_stored_values_are_exact(act, d):
    """k without norm and rotation and v have one answer; halves between codes, saturation, tiny and empty groups,
    infinities and NaN among them."""
    rng = np.random.Generator(np.random.PCG64(3))
    pg = handle(2, 2, d, act)
    pg.kvr_page_plan(ints([0, 0]), ints([100, 33]), 133)
    x = rand(rng, (133, 2, d), act, 3.0)
    x[:20] = torch.from_numpy(rng.integers(-14, 15, (20, 2, d)) / 2).to(TYPES[act])      # many exact halves
    x[:20, :, ::32] = 7
    x[20:24] *= 2.0 ** -20
    x[24] = 0
    x[25, 0, 5] = float("inf")
    x[25, 1, 37] = float("nan")
    x[26, 1, d - 1] = -float("inf")
    if act == "bf16":
        x[27] = 1e6
        x[28, :, :32] *= 1e38
    want = torch.from_numpy(op.values(f64(x))).to(TYPES[act])
    assert pg.kvr_page_append(0, None, x.cuda(), x.flip(0).contiguous().cuda(), rotate=False) is None
    k, v = (y.cpu() for y in pg.kvr_page_read(0))
    for got, ref in ((k, want), (v, want.flip(0))):
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(), ref.nan_to_num())


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("d,norm,rotate", [(128, True, True), (64, True, True), (128, False, True), (64, True, False)])
def test_keys_are_those_of_64_bits(act, d, norm, rotate):
    """A normed and rotated key next to the border of two activation values or codes takes the side that 64 bits
    (then 32, then the type) give: it is formed to about 2^-45, which decides all but one in 2^35 of the values here."""
    rng = np.random.Generator(np.random.PCG64([d, norm, rotate]))
    pg = handle(2, 2, d, act, rope_theta=1e6, norm_eps=1e-6)
    pg.kvr_page_plan(ints([0, 0]), ints([500, 12]), 512)
    pg.kvr_page_plan(ints([500, 12]), ints([0, 500]), 500)
    k, v = rand(rng, (500, 2, d), act, 2.0), rand(rng, (500, 2, d), act, 0.3)
    gain = rand(rng, (d,), act) + 1 if norm else None
    pg.kvr_page_append(0, None, k.cuda(), v.cuda(), None, gain.cuda() if norm else None, rotate=rotate)
    got = [x.cpu() for x in pg.kvr_page_read(0)]
    pg.kvr_pages_sync()
    y = np.stack([op.norm_rotate(f64(k[i]), 12 + i, 1e6, f64(gain) if norm else None, 1e-6, rotate) for i in range(500)])
    y = f64(torch.from_numpy(y).float().to(TYPES[act]))
    for x, ref in zip(got, (y, f64(v))):
        assert torch.equal(x, torch.from_numpy(op.values(ref)).to(TYPES[act]))


def test_padded_rows_stay_as_they_were():
    rng = np.random.Generator(np.random.PCG64(5))
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0, 0, 0]), ints([2, 0, 3]), 9)
    q, k, v = (rand(rng, (9, h, 64), "bf16").cuda() for h in (8, 2, 2))
    out = torch.full((9, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = pg.pool.clone()
    r = pg.kvr_page_append(0, q, k, v, out=out)
    assert r is out and (out[5:] == 7).all() and (out[:5] != 7).any()
    touched = (pg.pool != pool).view(-1, 2 * (64 * 32 + 64 * 4)).any(1).nonzero().flatten().tolist()
    assert touched == [0, 1, 2, 3]                           # layer 0, pages 0 and 1, both heads
    out.fill_(7)
    pg.kvr_page_attend(0, q, out=out)
    assert (out[5:] == 7).all() and (out[:5] != 7).any()


def test_append_in_place():
    rng = np.random.Generator(np.random.PCG64(6))
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0]), ints([70]), 70)
    q, k, v = (rand(rng, (70, h, 64), "bf16").cuda() for h in (8, 2, 2))
    want = pg.kvr_page_append(0, q, k, v)
    assert pg.kvr_page_append(0, q, k, v, out=q) is q and torch.equal(q, want)


# --------------------------------------------------------------------------- attend
MANY, BESIDE = 64, 16


def bound(n, mag, v, ref, u, spread=0.0):
    """spread: the largest scale |q k|_2 of each head [heads][1], for rows whose k is rounded."""
    top = np.abs(v).max()
    return ((2 * 2.0 ** -11 + 2.0 ** -13 + 12 * 2.0 ** -11 * spread) * mag + n * (2.0 ** -27 * top + 2.0 ** -24)
            + (n / 16 + 2) * 2.0 ** -22 * top + u * np.abs(ref))


class World:
    """A handle and, beside it, the values that each sequence's cache stands for (k without rotation)."""
    rounds_k = True

    def __init__(self, heads, kv_heads, d, act, seed=0, layer=1, **kw):
        self.pg = handle(heads, kv_heads, d, act, **kw)
        self.heads, self.kv_heads, self.d, self.act, self.layer = heads, kv_heads, d, act, layer
        self.rng = np.random.Generator(np.random.PCG64(seed))
        n = self.pg.cfg.max_seqs
        self.k = [np.zeros((kv_heads, 0, d)) for _ in range(n)]
        self.v = [np.zeros((kv_heads, 0, d)) for _ in range(n)]

    def step(self, keep, add, pad=0, k_scale=1.0, v_scale=1.0, edit=None, max_add=0):
        n = sum(add) + pad
        self.pg.kvr_page_plan(ints(keep), ints(add), n, max_add)
        k = rand(self.rng, (n, self.kv_heads, self.d), self.act, k_scale)
        v = rand(self.rng, (n, self.kv_heads, self.d), self.act, v_scale)
        if edit:
            edit(k, v)
        self.pg.kvr_page_append(self.layer, None, k.cuda(), v.cuda(), rotate=False)
        row = 0
        for b, (p, m) in enumerate(zip(keep, add)):
            for store, x in ((self.k, k), (self.v, v)):
                new = op.values(f64(x[row:row + m])).transpose(1, 0, 2)
                store[b] = np.concatenate([store[b][:, :p], new], axis=1)
            row += m
        self.keep, self.add, self.rows = keep, add, n

    def q(self, scale=1.0):
        return rand(self.rng, (self.rows, self.heads, self.d), self.act, scale)

    def check(self, q, out, scale=None, skip=()):
        got, qn = f64(out), f64(q)
        scale = self.d ** -0.5 if scale is None else scale
        u, row = half_step(self.act), 0
        for b, (p, m) in enumerate(zip(self.keep, self.add)):
            for i in range(m):
                if (b, i) not in skip:
                    n = p + i + 1
                    k, v = self.k[b][:, :n], self.v[b][:, :n]
                    ref, mag = op.attend(qn[row], k, v, scale)
                    spread = 0.0
                    group = self.heads // self.kv_heads
                    many = BESIDE if self.rows * group > MANY else MANY
                    if self.rounds_k and self.act == "bf16" and m * group > many:
                        kk = np.repeat(k, self.heads // self.kv_heads, axis=0)
                        spread = scale * np.sqrt(np.max((kk * qn[row][:, None]) ** 2 @ np.ones(self.d), axis=1))[:, None]
                    tol = bound(n, mag, v, ref, u, spread)
                    bad = ~(np.abs(got[row] - ref) <= tol)
                    assert not bad.any(), (b, i, int(bad.sum()), float(np.nanmax(np.abs(got[row] - ref) / tol)))
                row += 1


SHAPES = [(8, 2, 64), (6, 2, 128), (28, 4, 128), (32, 8, 128), (1, 1, 64), (16, 1, 128), (4, 4, 64)]


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
def test_attend_one_token(act, heads, kv_heads, d):
    w = World(heads, kv_heads, d, act, seed=d + heads)
    lens = [0, 62, 63, 64, 191, 700, 5, 128]
    w.step([0] * 8, [max(x, 0) for x in lens[:4]] + [0] * 4)
    w.step(lens[:4] + [0] * 4, [0] * 4 + [191, 0, 5, 128])
    w.step(lens[:5] + [0] + lens[6:], [0] * 5 + [512, 0, 0])
    w.step(lens[:5] + [512] + lens[6:], [0] * 5 + [188, 0, 0])
    w.step(lens, [1] * 8, pad=3)
    q = w.q(2.0)
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("keep,add", [
    ([0], [1]), ([0], [2]), ([0], [64]), ([0], [65]), ([63], [2]), ([64], [1]), ([300], [8]), ([0], [200]), ([130], [129]),
    ([5, 0, 130, 64, 200], [3, 0, 7, 1, 40]), ([0, 0, 0], [1, 130, 17]), ([150, 2], [33, 150]),
])
def test_attend_rows(act, heads, kv_heads, d, keep, add):
    w = World(heads, kv_heads, d, act, seed=sum(add))
    if sum(keep):
        w.step([0] * len(keep), keep)
    for most in (max(add), 0):       # a close bound on the rows of a sequence, and none
        w.step(keep, add, max_add=most)
        q = w.q(1.5)
        w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (28, 4, 128), (16, 1, 128)])
@pytest.mark.parametrize("keep,add", [([0], [200]), ([130], [129]), ([5, 0, 130, 64, 200], [3, 0, 7, 1, 40])])
def test_attend_rows_of_sequences_that_cannot_be_long(act, heads, kv_heads, d, keep, add):
    """(one launch, k as it is)"""
    w = World(heads, kv_heads, d, act, seed=sum(add), max_len=384)
    w.rounds_k = False
    if sum(keep):
        w.step([0] * len(keep), keep)
    w.step(keep, add)
    q = w.q(1.5)
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()


@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (6, 2, 128)])
def test_attend_rows_in_fp16_round_weights_and_outputs_only(heads, kv_heads, d):
    """Root mean square error, relative to the outputs': an fp16 rounding is off by at most 2^-11 of the value, evenly
    spread, so by 2^-11 / sqrt(3) in the mean square; that of the weights, with values of random sign, and that of the
    output are independent: sqrt(2 / 3) 2^-11 together, and a hundredth for the sums in 32 bits."""
    w = World(heads, kv_heads, d, "fp16", seed=7)
    w.step([0] * 8, [400] + [0] * 7)
    w.step([400] + [0] * 7, [150] + [0] * 7)
    q = w.q(3.0)
    got, qn = f64(w.pg.kvr_page_attend(1, q.cuda())), f64(q)
    err = size = 0.0
    for i in range(150):
        ref, _ = op.attend(qn[i], w.k[0][:, :401 + i], w.v[0][:, :401 + i], d ** -0.5)
        err, size = err + ((got[i] - ref) ** 2).sum(), size + (ref ** 2).sum()
    assert (err / size) ** 0.5 <= 1.01 * (2 / 3) ** 0.5 * 2.0 ** -11


@pytest.mark.parametrize("d,heads,kv_heads", [(64, 32, 8), (128, 16, 4)])
@pytest.mark.parametrize("rows", [[20, 40], [40, 20], [17, 33, 100, 20], [30]])
@pytest.mark.parametrize("act", ["bf16", "fp16"])
def test_attend_many_segments_in_a_run(act, d, heads, kv_heads, rows):
    """More work than CTAs: a run goes through whole sequences with one and with two row tiles (80 and 160 rows of a
    KV head), in either order, over several key blocks each."""
    n = 36
    w = World(heads, kv_heads, d, act, seed=17, max_seqs=n, n_pages=n * 12, max_rows=n * 600)
    keep = [300 + 37 * (b % 9) for b in range(n)]
    add = [rows[b % len(rows)] for b in range(n)]
    w.step([0] * n, keep)
    w.step(keep, add)
    q = w.q(1.5)
    out = w.pg.kvr_page_attend(1, q.cuda())
    w.pg.kvr_pages_sync()
    w.check(q, out)


@pytest.mark.parametrize("long_rows", [1, 120])
def test_attend_all_the_sequences_there_can_be(long_rows):
    """2048 sequences of a few tokens, one of them with many rows."""
    w = World(4, 1, 64, "bf16", seed=31, max_seqs=2048, n_pages=2100, max_rows=8192)
    keep = [int(x) for x in w.rng.integers(0, 4, 2048)]
    add = [int(x) for x in w.rng.integers(0, 2, 2048)]
    keep[1500], add[1500], add[2047] = 130, long_rows, 1
    w.step([0] * 2048, keep)
    w.step(keep, add, pad=5)
    q = w.q(1.5)
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()


@pytest.mark.parametrize("max_len", [512, 1 << 17])
@pytest.mark.parametrize("keep,add", [([300], [1]), ([63, 0], [3, 5])])
def test_attend_groups_of_64(keep, add, max_len):
    w = World(64, 1, 128, "bf16", seed=33, max_len=max_len)
    w.step([0] * len(keep), keep)
    w.step(keep, add)
    q = w.q(1.5)
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()


def test_two_handles_at_once_on_two_streams():
    """Each handle has its own work area: calls of both in flight together give the bits of calls one after another."""
    made = []
    for i in range(2):
        w = World(8, 2, 64, "bf16", seed=40 + i, layer=0)
        w.step([0] * 8, [100 + 50 * i] + [20] * 7)
        w.step([100 + 50 * i] + [20] * 7, [150, 1, 3, 1, 1, 1, 40, 1])
        q = w.q(1.5).cuda()
        made.append((w.pg, q, w.pg.kvr_page_attend(0, q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    for _ in range(20):
        for i, (pg, q, _) in enumerate(made):
            got[i].append(pg.kvr_page_attend(0, q, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (pg, _, want) in enumerate(made):
        assert all(torch.equal(x, want) for x in got[i])
        pg.kvr_pages_sync()


def test_attend_peaked_flat_and_scaled():
    w = World(28, 4, 128, "bf16", seed=9)
    w.step([0, 0], [300, 140], k_scale=2.0)
    w.step([300, 140], [2, 1])
    for qs, scale in ((6.0, None), (0.0, None), (1.0, 0.3), (1e-3, 1.0), (1e4, 1e-5)):
        q = w.q(qs)
        w.check(q, w.pg.kvr_page_attend(1, q.cuda(), scale=scale), scale)


@pytest.mark.parametrize("rows", [1, 150])
def test_attend_extreme_magnitudes(rows):
    """q beyond fp16's range, values next to the largest and the smallest scales, groups of zeros."""
    w = World(8, 2, 64, "bf16", seed=10)
    w.step([0], [200], k_scale=2.0 ** -20, v_scale=1.0)

    def zero_k(k, v):
        k.zero_()
    w.step([200], [rows], edit=zero_k)      # so that the scores stay ordinary: (2^20 q) (2^-20 k)
    q = w.q(2.0 ** 20)
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))
    for vs in (8000.0, 2.0 ** -12):
        w.step([0], [200], v_scale=vs)

        def zeros(k, v):
            v[:, :, :32] = 0
        w.step([200], [rows], v_scale=vs, edit=zeros)
        q = w.q()
        w.check(q, w.pg.kvr_page_attend(1, q.cuda()))


@pytest.mark.parametrize("rows", [3, 100])
def test_nan_reaches_only_the_rows_that_see_it(rows):
    for what in ("k", "v"):
        w = World(8, 2, 64, "bf16", seed=11)
        w.step([0, 0], [90, 90])

        def edit(k, v):
            (k if what == "k" else v)[rows - 1, 1, 3] = float("nan")   # the last row of sequence 0, KV head 1
        w.step([90, 90], [rows, rows], edit=edit)
        q = w.q()
        got = w.pg.kvr_page_attend(1, q.cuda())
        w.check(q, got, skip=[(0, rows - 1)])
        last = got[rows - 1].float().cpu()
        # heads 4 .. 7 read KV head 1; the NaN is in its first group of 32 dims
        assert last[4:, :32].isnan().all() and not last[:4].isnan().any()


@pytest.mark.parametrize("rows", [1, 60])
def test_what_pages_held_before_does_not_show(rows):
    """Places behind the last token hold another sequence's values, NaN among them."""
    w = World(8, 2, 64, "bf16", seed=12)

    def poison(k, v):
        k[:] = float("nan")
        v[:] = float("inf")
    w.step([0], [512], edit=poison)
    w.step([0], [0])
    w.step([0, 0], [70, 1])
    w.step([70, 1], [rows, rows])
    q = w.q()
    w.check(q, w.pg.kvr_page_attend(1, q.cuda()))


def test_attend_strided_q_and_other_layer():
    w = World(8, 2, 64, "bf16", seed=13, layer=0)
    w.step([0, 0], [100, 3])
    w.step([100, 3], [5, 2])
    q = w.q()
    wide = torch.zeros(7, 8 * 64 + 40, dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = q.cuda().flatten(1)
    w.check(q, w.pg.kvr_page_attend(0, wide[:, :512].unflatten(1, (8, 64))))


def test_same_call_same_bits():
    w = World(32, 8, 128, "bf16", seed=14, max_len=2048, n_pages=200, max_rows=1700)
    w.step([0, 0, 0], [1000, 600, 3])
    w.step([1000, 600, 3], [4, 130, 1])
    q = w.q().cuda()
    first = w.pg.kvr_page_attend(1, q)
    for _ in range(5):
        assert torch.equal(w.pg.kvr_page_attend(1, q), first)


def test_pool_offsets_beyond_32_bits():
    """The last pages of a pool larger than 2^32 bytes (9216 bytes a page)."""
    from prefix_reused_prefill_gb300 import PagedKv, paged_config
    n_pages = 480000
    pg = PagedKv(paged_config(n_pages=n_pages, n_layers=1, n_q_heads=4, n_kv_heads=1, head_dim=128, max_seqs=9,
                              max_len=1 << 22, max_rows=1 << 22))
    used = 0
    for b in range(7):               # seven sequences of 2^22 tokens hold 458752 pages; their contents do not matter
        add = [0] * 9
        add[b] = 1 << 22
        pg.kvr_page_plan(pg.state.lens, ints(add), 1 << 22)
        used += (1 << 22) // 64
    add = [0] * 7 + [(n_pages - used - 3) * 64, 0]
    pg.kvr_page_plan(pg.state.lens, ints(add), 1 << 22)
    pg.kvr_page_plan(pg.state.lens, ints([0] * 8 + [150]), 150)
    pg.kvr_pages_sync()
    assert pg.state.table[8, :3].tolist() == [n_pages - 3, n_pages - 2, n_pages - 1]
    rng = np.random.Generator(np.random.PCG64(15))
    k, v = rand(rng, (150, 1, 128), "bf16"), rand(rng, (150, 1, 128), "bf16")
    q = rand(rng, (150, 4, 128), "bf16")
    pg.kvr_page_append(0, None, k.cuda(), v.cuda(), rotate=False)
    got = f64(pg.kvr_page_attend(0, q.cuda()))
    kk, vv = (op.values(f64(x)).transpose(1, 0, 2) for x in (k, v))
    for i in (0, 63, 64, 149):
        ref, mag = op.attend(f64(q[i]), kk[:, :i + 1], vv[:, :i + 1], 128 ** -0.5)
        spread = 128 ** -0.5 * np.sqrt(np.max(((kk[:, :i + 1] * f64(q[i])[:, None]) ** 2).sum(-1), axis=1))[:, None]
        tol = bound(i + 1, mag, vv, ref, 2.0 ** -8, spread)
        assert (np.abs(got[i] - ref) <= tol).all(), i


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (6, 2, 128)])
def test_steps_of_a_server(heads, kv_heads, d):
    """Prompts, single tokens, speculative rows that are cut back, an ended and a new sequence: plan, append and attend
    on two layers.  The reference keeps every sequence's rows itself, from the formulas; only where a k lies next to
    the border of two codes does it take the code that the cache read back (which may be off by one there).  Held to
    1 % of a row's norm: q and k rounded to bf16 the other way (2^-8 of one element) move a score by at most
    2^-8 * 4 * 4 / 8 < 2^-7, its weight by less than 1 %, besides the elementwise bound's 2^-10 + 2^-8."""
    rng = np.random.Generator(np.random.PCG64(d))
    pg = handle(heads, kv_heads, d, "bf16", max_seqs=3, rope_theta=1e4)
    gains = [[rand(rng, (d,), "bf16", 0.2) + 1 for _ in range(2)] for _ in range(2)]
    stores = [[[np.zeros((kv_heads, 0, d))] * 2 for _ in range(3)] for _ in range(2)]
    rnd = lambda x: f64(torch.from_numpy(x).to(torch.bfloat16))
    steps = [([0, 0, 0], [70, 9, 0]), ([70, 9, 0], [1, 4, 0]), ([71, 10, 0], [4, 4, 30]), ([72, 0, 30], [1, 64, 1]),
             ([73, 64, 31], [130, 1, 1])]
    for keep, add in steps:
        n = sum(add)
        pg.kvr_page_plan(ints(keep), ints(add), n + 2)
        for layer in range(2):
            q, k, v = (rand(rng, (n + 2, h, d), "bf16") for h in (heads, kv_heads, kv_heads))
            gq, gk = gains[layer]
            rot = pg.kvr_page_append(layer, q.cuda(), k.cuda(), v.cuda(), gq.cuda(), gk.cuda())
            held = f64(pg.kvr_page_read(layer)[0])
            got = f64(pg.kvr_page_attend(layer, rot))
            row = 0
            for b, (p, m) in enumerate(zip(keep, add)):
                kb, vb = (x[:, :p] for x in stores[layer][b])
                for i in range(m):
                    y = rnd(op.norm_rotate(f64(k[row]), p + i, 1e4, f64(gk), 1e-6))
                    c, s = op.quantise(y)
                    back = np.round(held[row].reshape(c.shape) / s)
                    exact = y.reshape(c.shape) / s
                    near = np.abs(np.abs(exact - np.floor(exact)) - 0.5) < 0.05
                    assert (back == c)[~near].all() and (np.abs(back - c) <= 1).all()
                    kb = np.concatenate([kb, (back * s).reshape(kv_heads, 1, d)], axis=1)
                    vb = np.concatenate([vb, op.values(f64(v[row]))[:, None]], axis=1)
                    ref, _ = op.attend(rnd(op.norm_rotate(f64(q[row]), p + i, 1e4, f64(gq), 1e-6)), kb, vb, d ** -0.5)
                    err = np.linalg.norm(got[row] - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
                    assert err.max() < 0.01, (keep, add, layer, b, i, err.max())
                    row += 1
                stores[layer][b] = [kb, vb]
    pg.kvr_pages_sync()


@pytest.mark.parametrize("max_len", [400, 1 << 17])
def test_captured_steps_and_two_graphs(max_len):
    """A captured step (plan, append, attend) replayed over growing lengths gives the bits of eager calls; a second
    graph of another handle and an eager step in between do not disturb it."""
    rng = np.random.Generator(np.random.PCG64(21))
    made = []
    for _ in range(3):
        pg = handle(8, 2, 64, max_seqs=4, max_len=max_len)
        pg.kvr_page_plan(ints([0] * 4), ints([60, 1, 130, 7]), 198)
        k, v = (rand(np.random.Generator(np.random.PCG64([22, i])), (198, 2, 64), "bf16").cuda() for i in range(2))
        pg.kvr_page_append(0, None, k, v)
        made.append(pg)
    one = ints([2, 1, 0, 1])
    q, k, v = (torch.empty(6, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))

    def step(pg):
        pg.kvr_page_plan(pg.state.lens, one, 6, 2)
        return pg.kvr_page_attend(0, pg.kvr_page_append(0, q, k, v))
    inputs = [[rand(rng, x.shape, "bf16") for x in (q, k, v)] for _ in range(12)]
    want = []
    for x in inputs:
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        want.append(step(made[0])[:4].clone())
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for pg in made[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(pg)
        graphs.append((g, out, pg))
    for i, x in enumerate(inputs):
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        for g, out, pg in graphs if i % 2 else graphs[::-1]:
            if i == 5:
                got = step(pg)[:4]               # an eager step among the replays
            else:
                g.replay()
                got = out[:4]
            assert torch.equal(got, want[i]), i
    for pg in made:
        pg.kvr_pages_sync()
        assert pg.state.lens.tolist() == made[0].state.lens.tolist()


def test_calls_on_another_stream():
    w = World(8, 2, 64, "bf16", seed=23)
    w.step([0], [100])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, k, v = (rand(w.rng, (4, h, 64), "bf16") for h in (8, 2, 2))
    dev = [x.cuda() for x in (q, k, v)]
    torch.cuda.synchronize()
    w.pg.kvr_page_plan(ints([100]), ints([4]), 4, stream=s)
    w.pg.kvr_page_append(1, None, dev[1], dev[2], rotate=False, stream=s)
    out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    w.pg.kvr_page_attend(1, dev[0], out=out, stream=s)
    w.pg.kvr_pages_sync(stream=s)
    for store, x in ((w.k, k), (w.v, v)):
        store[0] = np.concatenate([store[0], op.values(f64(x)).transpose(1, 0, 2)], axis=1)
    w.keep, w.add = [100], [4]
    w.check(q, out)


# --------------------------------------------------------------------------- refusals
def test_results_on_another_stream_take_memory_of_that_stream():
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0]), ints([200]), 200)
    q, k, v = (torch.ones(200, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    pg.kvr_page_append(0, None, k, v)
    side = torch.cuda.Stream()
    for call in (lambda: pg.kvr_page_attend(0, q, stream=side), lambda: pg.kvr_page_append(0, q, k, v, stream=side)):
        torch.cuda.synchronize()
        x = torch.full_like(q, 5)
        torch.cuda._sleep(100_000_000)
        y = x.clone()                       # waits behind the sleep; x's memory is free for this stream's next tensor
        del x
        out = call()
        torch.cuda.synchronize()
        assert (y == 5).all() and not (out == 5).any()
    pg.kvr_pages_sync()


def test_a_captured_attend_after_a_plan_of_longer_additions_is_reported():
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0] * 8), ints([5] * 8), 40, 5)
    rng = np.random.Generator(np.random.PCG64(11))
    q, k, v = (rand(rng, (40, h, 64), "bf16").cuda() for h in (8, 2, 2))
    pg.kvr_page_append(0, None, k, v)
    out = torch.empty_like(q)
    pg.kvr_page_attend(0, q, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pg.kvr_page_attend(0, q, out=out)
    graph.replay()
    pg.kvr_pages_sync()
    pg.kvr_page_plan(ints([0] * 8), ints([38, 2] + [0] * 6), 40, 38)
    pg.kvr_page_append(0, None, k, v)
    want = pg.kvr_page_attend(0, q)
    pg.kvr_pages_sync()
    out.fill_(7)
    graph.replay()
    assert code_of(pg.kvr_pages_sync) == -1
    assert (out[:38] == 7).all() and torch.equal(out[38:], want[38:])
    assert torch.equal(pg.kvr_page_attend(0, q), want)
    pg.kvr_pages_sync()


def test_refused_calls_change_nothing():
    rng = np.random.Generator(np.random.PCG64(30))
    pg = handle(8, 2, 64, max_seqs=4)
    pg.kvr_page_plan(ints([0, 0]), ints([3, 2]), 5)
    q, k, v = (rand(rng, (5, h, 64), "bf16").cuda() for h in (8, 2, 2))
    rot = pg.kvr_page_append(0, q, k, v)
    want = pg.kvr_page_attend(0, rot)
    pool, tables = pg.pool.clone(), pg.state.table.clone()
    z = ints([0, 0])
    gain = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    refused = [
        lambda: pg.kvr_page_plan(ints([0] * 5), ints([0] * 5), 0), lambda: pg.kvr_page_plan(z[:0], z[:0], 0),
        lambda: pg.kvr_page_plan(z, z, -1), lambda: pg.kvr_page_plan(z, z, 513),
        lambda: pg.kvr_page_plan(z.long(), z, 1), lambda: pg.kvr_page_plan(z, z[:1], 1),
        lambda: pg.kvr_page_plan(z.cpu(), z, 1), lambda: pg.kvr_page_plan(ints([0] * 4)[::2], z, 1),
        lambda: pg.kvr_page_append(2, q, k, v), lambda: pg.kvr_page_append(-1, q, k, v),
        lambda: pg.kvr_page_append(0, q[:4], k, v), lambda: pg.kvr_page_append(0, q, k[:, :1], v),
        lambda: pg.kvr_page_append(0, q.float(), k, v), lambda: pg.kvr_page_append(0, q, k.cpu(), v),
        lambda: pg.kvr_page_append(0, q.transpose(1, 2).contiguous().transpose(1, 2), k, v),
        lambda: pg.kvr_page_append(0, q, k, v, gain[:32]), lambda: pg.kvr_page_append(0, q, k, v, None, gain.half()),
        lambda: pg.kvr_page_append(0, None, k, v, out=rot), lambda: pg.kvr_page_append(0, q, k, v, out=rot[:4]),
        lambda: pg.kvr_page_attend(2, rot), lambda: pg.kvr_page_attend(0, rot, out=rot),
        lambda: pg.kvr_page_attend(0, rot, scale=0.0), lambda: pg.kvr_page_attend(0, rot, scale=float("nan")),
        lambda: pg.kvr_page_attend(0, rot[:, :4]), lambda: pg.kvr_page_read(5),
        # rows that do not start on 16 bytes, and a row stride that is no multiple of 8
        lambda: pg.kvr_page_attend(0, torch.zeros(5 * 512 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(5, 8, 64)),
        lambda: pg.kvr_page_append(0, torch.zeros(5, 516, dtype=torch.bfloat16, device="cuda")[:, :512].unflatten(1, (8, 64)), k, v),
    ]
    for i, call in enumerate(refused):
        assert code_of(call) in (-1, -2), i
    assert torch.equal(pg.pool, pool) and torch.equal(pg.state.table, tables)
    assert torch.equal(pg.kvr_page_attend(0, rot), want)
    pg.kvr_pages_sync()


def test_a_refused_plan_has_no_rows():
    """Out of pages: append, read and attend of that step touch nothing, and the next plan works."""
    pg = handle(8, 2, 64, n_pages=3, max_seqs=2)
    pg.kvr_page_plan(ints([0, 0]), ints([64, 64]), 128)
    rng = np.random.Generator(np.random.PCG64(31))
    q, k, v = (rand(rng, (130, h, 64), "bf16").cuda() for h in (8, 2, 2))
    pg.kvr_page_append(0, None, k[:128], v[:128])
    pool = pg.pool.clone()
    pg.kvr_page_plan(ints([64, 64]), ints([1, 129]), 130)
    out = torch.full_like(q, 5.0)
    pg.kvr_page_append(0, q, k, v, out=out)
    pg.kvr_page_attend(0, q, out=out)
    pg.kvr_page_read(0)
    assert code_of(pg.kvr_pages_sync) == -2
    assert (out == 5).all() and torch.equal(pg.pool, pool) and pg.state.lens.tolist() == [64, 64]
    pg.kvr_page_plan(ints([64, 64]), ints([1, 0]), 1)
    pg.kvr_pages_sync()
    assert pg.state.lens.tolist() == [65, 64]


def test_steps_without_rows():
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0, 0]), ints([0, 0]), 0)
    e = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert pg.kvr_page_append(0, e, kv, kv).shape == (0, 8, 64)
    assert pg.kvr_page_attend(0, e).shape == (0, 8, 64)
    pg.kvr_pages_sync()
