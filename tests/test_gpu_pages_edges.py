"""The paged 4-bit cache where its types end: NaN values under vanishing weights, queries and scales next to the largest
and the least numbers, steps without rows through the stack, waits that gave up (needs a GB300)."""
import numpy as np
import pytest
import torch

from oracle import pages as op
from test_gpu_pages import World, f64, handle, ints, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("where", [10, 64, 127, 128, 130])
@pytest.mark.parametrize("rows,max_len", [(3, 512), (3, 1 << 17), (100, 1 << 17)])
def test_nan_values_show_however_small_their_weight(where, rows, max_len):
    """A token whose v holds a NaN, 60 nats below the others: the heads that see it read NaN in that group of dims,
    wherever the page ends; the rows before it do not."""
    w = World(8, 2, 64, "bf16", seed=3, max_len=max_len)

    def edit(k, v):
        k[where, 1] = -8                       # (q is 8 below: a score of -8 * 8 * 64 / 8 = -512)
        v[where, 1, 40] = float("nan")
    first = max(1, 131 - rows)                 # the first row's position
    w.step([0, 0], [131, 20], edit=edit)
    w.pg.kvr_page_plan(ints([first, 17]), ints([131 - first, 3]), 131 - first + 3)
    n = 131 - first
    q = torch.full((n + 3, 8, 64), 8.0, dtype=torch.bfloat16)
    got = f64(w.pg.kvr_page_attend(1, q.cuda()))
    w.pg.kvr_pages_sync()
    for i in range(n):
        pos = first + i
        sees = pos >= where
        assert np.isnan(got[i, 4:, 32:]).all() == sees and not np.isnan(got[i, :4]).any(), (pos, where)
        if not sees:
            assert not np.isnan(got[i]).any()
    assert not np.isnan(got[n:]).any()


@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("log_q", [114, 117, 121, 125])
def test_queries_next_to_the_largest_number(rows, log_q):
    """q of about 2^log_q over small k, with a scale that leaves ordinary scores."""
    w = World(8, 2, 64, "bf16", seed=15)
    w.step([0], [200 + rows], k_scale=2.0 ** -20)
    w.pg.kvr_page_plan(ints([200]), ints([rows]), rows)
    w.keep, w.add, w.rows = [200], [rows], rows
    q, scale = w.q(2.0 ** log_q), 2.0 ** (18 - log_q)
    assert torch.isfinite(q).all()
    w.check(q, w.pg.kvr_page_attend(1, q.cuda(), scale=scale), scale)
    w.pg.kvr_pages_sync()


@pytest.mark.parametrize("rows", [2, 150])
@pytest.mark.parametrize("q_size,scale", [(2.0 ** -100, 2.0 ** -60), (2.0 ** -120, 1e-38), (1.0, 1e-38), (2.0 ** -100, 2.0 ** 100),
                                          (2.0 ** -110, 2.2e38)])
def test_queries_and_scales_next_to_zero(rows, q_size, scale):
    """Tiny q under tiny and large scales: scores next to equal, or far apart; rows that see only a part of a page among
    them."""
    w = World(8, 2, 64, "bf16", seed=16)
    w.step([0], [200 + rows], k_scale=0.1)
    w.pg.kvr_page_plan(ints([200]), ints([rows]), rows)
    w.keep, w.add, w.rows = [200], [rows], rows
    q = w.q(q_size)
    out = w.pg.kvr_page_attend(1, q.cuda(), scale=scale)
    w.pg.kvr_pages_sync()
    if scale < 1e38:
        return w.check(q, out, scale)
    # Scores of 2^-110 2^127.4 0.1 sqrt(64) = 1.4e5: the bound holds to 90 only.  k rounded to fp16 (2^-11) moves such a
    # score by tens, so any of several keys may have the weight; what is left is that the output is a mean of
    # values: between the least and the largest of them, rounded by 2^-8 for the type, 2^-10 for weights and values.
    got = f64(out)
    for i in range(rows):
        v = np.repeat(w.v[0][:, :201 + i], 4, axis=0)
        top = np.abs(v).max()
        assert (got[i] >= v.min(axis=1) - 2.0 ** -7 * top).all() and (got[i] <= v.max(axis=1) + 2.0 ** -7 * top).all()


def test_a_scale_beyond_the_largest_is_refused():
    from prefix_reused_prefill_gb300 import KvrError
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0]), ints([1]), 1)
    q, k, v = (torch.ones(1, h, 64, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    pg.kvr_page_append(0, None, k, v)
    for scale in (3e38, float("inf")):
        with pytest.raises(KvrError) as e:
            pg.kvr_page_attend(0, q, scale=scale)
        assert e.value.code == -1
    pg.kvr_page_attend(0, q, scale=2.2e38)
    pg.kvr_pages_sync()


@pytest.mark.parametrize("rows", [2, 150])
@pytest.mark.parametrize("scale", [1e3, 1e4, 3e5, 1e7, 1e20, 1e33])
def test_large_equal_scores(rows, scale):
    """All keys alike: every score of a row is the same number, and the output the mean of the values.  (With equal weights
    w the products' and sums' errors are relative to sum w|v|, as for any other scores.)  Scores above 1.8e8 read
    NaN, those below -1.8e8 have no weight."""
    w = World(8, 2, 64, "bf16", seed=18, max_rows=1024)

    def alike(k, v):
        k[:] = k[:1]
    w.step([0], [500 + rows], edit=alike)
    w.pg.kvr_page_plan(ints([500]), ints([rows]), rows)
    w.keep, w.add, w.rows = [500], [rows], rows
    q = w.q(2.0)
    out = w.pg.kvr_page_attend(1, q.cuda(), scale=scale)
    w.pg.kvr_pages_sync()
    if scale <= 3e5:
        return w.check(q, out, scale)
    got, k = f64(out), np.repeat(w.k[0][:, 0], 4, axis=0)
    score = scale * (f64(q) * k).sum(-1)                     # [rows][heads]
    assert np.isnan(got[score > 1.87e8]).all() and (got[score < -1.87e8] == 0).all()
    assert np.isfinite(got[np.abs(score) < 1.85e8]).all()
    assert (np.abs(score) > 1e3).mean() > 0.9


@pytest.mark.parametrize("act", ["bf16", "fp16"])
def test_norms_of_the_largest_numbers(act):
    """A head whose squares' sum passes the largest 32-bit number: it is normed to 0, k as q; an infinity is normed to
    NaN in its own place only (and so in its group of the cache), other heads as ever."""
    pg = handle(2, 2, 64, act)
    pg.kvr_page_plan(ints([0]), ints([6]), 6)
    x = torch.ones(6, 2, 64, dtype=torch.float32)
    if act == "bf16":
        x[1, 1] = 2.0 ** 70
        x[2, 0, 3] = 2.0 ** 100
        x[3, 0] = 3e38
    x[4, 1, 40] = float("inf")
    x = x.to(torch.bfloat16 if act == "bf16" else torch.float16)
    g = torch.ones(64, dtype=x.dtype, device="cuda")
    q = f64(pg.kvr_page_append(0, x.cuda(), x.cuda(), x.cuda(), g, g, rotate=False))
    k = f64(pg.kvr_page_read(0)[0])
    want = np.ones((6, 2, 64))
    if act == "bf16":
        want[1, 1] = want[2, 0] = want[3, 0] = 0
    want[4, 1] = 0
    want[4, 1, 40] = np.nan
    assert np.allclose(q, want, rtol=2.0 ** -7, equal_nan=True)
    want[4, 1, 32:] = np.nan
    assert np.allclose(k, want, rtol=2.0 ** -7, equal_nan=True)


TIMEOUT = -4


@pytest.mark.parametrize("rows,max_len", [(1, 1 << 17), (3, 512), (150, 1 << 17)])
def test_a_wait_that_gave_up(rows, max_len):
    """The status word as a wait that gave up leaves it, with arrivals of an unfinished merge, written by the host: the
    attention returns without a result, sync reports it once and clears both, and the next call is right."""
    from prefix_reused_prefill_gb300 import KvrError
    w = World(8, 1, 64, "bf16", seed=19, max_len=max_len, n_pages=96, max_rows=4608)
    n = min(max_len, 4500) - rows
    w.step([0], [n])
    w.step([n], [rows])
    q = w.q()
    want = w.pg.kvr_page_attend(1, q.cuda())
    w.pg.kvr_pages_sync()
    w.check(q, want)
    words = w.pg.work.view(torch.int32)            # status, then (from byte 512 on) the arrival counters
    assert words[0] == 0 and (words[128:128 + 152] == 0).all()
    words[0] = 1
    words[128:128 + 152] = 1
    out = torch.full_like(want, 7.0)
    w.pg.kvr_page_attend(1, q.cuda(), out=out)
    with pytest.raises(KvrError) as e:
        w.pg.kvr_pages_sync()
    assert e.value.code == TIMEOUT and (out == 7).all()
    w.pg.kvr_pages_sync()
    assert words[0] == 0 and (words[128:128 + 152] == 0).all()
    assert torch.equal(w.pg.kvr_page_attend(1, q.cuda()), want)
    w.pg.kvr_pages_sync()


def test_one_row_of_any_stride():
    """One row out of a wider buffer: its stride says nothing, odd or not."""
    pg = handle(8, 2, 64)
    pg.kvr_page_plan(ints([0]), ints([1]), 1)
    rng = np.random.Generator(np.random.PCG64(20))
    q, k, v = (rand(rng, (1, h, 64), "bf16").cuda() for h in (8, 2, 2))
    want = pg.kvr_page_attend(0, pg.kvr_page_append(0, q, k, v))
    wide = []
    for x in (q, k, v):
        buf = torch.zeros(2, x.numel() + 5, dtype=torch.bfloat16, device="cuda")
        buf[:1, :x.numel()] = x.flatten(1)
        wide.append(torch.as_strided(buf, x.shape, (buf.shape[1], 64, 1)))
        assert wide[-1].stride(0) % 8
    assert torch.equal(pg.kvr_page_attend(0, pg.kvr_page_append(0, *wide)), want)
    pg.kvr_pages_sync()


def test_results_that_share_memory_with_inputs_are_refused():
    """Rows are read and written by blocks in no order, so a result over an input would hold either; q in place (each
    head by its own lanes) and a result between the rows of a strided input stay possible."""
    from prefix_reused_prefill_gb300 import KvrError
    pg = handle(2, 2, 64)
    n, w = 6, 128
    pg.kvr_page_plan(ints([0]), ints([n]), n)
    rng = np.random.Generator(np.random.PCG64(22))
    x = rand(rng, (3, n + 2, 2, 64), "bf16").cuda()
    q, k, v = (y[:n] for y in x)
    rot = pg.kvr_page_append(0, q, k, v)
    want = pg.kvr_page_attend(0, rot)
    pool, before = pg.pool.clone(), x.clone()
    refused = [lambda: pg.kvr_page_append(0, q, k, v, out=k), lambda: pg.kvr_page_append(0, q, k, v, out=v),
               lambda: pg.kvr_page_append(0, q, k, v, out=x[0, 1:n + 1]), lambda: pg.kvr_page_append(0, q, k, v, out=x[1, 2:]),
               lambda: pg.kvr_page_attend(0, q, out=q), lambda: pg.kvr_page_attend(0, q, out=x[0, 2:]),
               lambda: pg.kvr_page_attend(0, x[0, 1:n + 1], out=q),
               lambda: pg._check(pg.lib.kvr_page_read(pg.ctx, 0, k.data_ptr(), x[1, 1:].data_ptr(), n, None))]
    for i, call in enumerate(refused):
        with pytest.raises(KvrError) as e:
            call()
        assert e.value.code == -1, i
    assert torch.equal(x, before) and torch.equal(pg.pool, pool)
    # rows of q far apart, the result between the first two of them, and right behind the last
    wide = torch.zeros(n * (n + 1) * w + n * w, dtype=torch.bfloat16, device="cuda")
    far = wide[:n * (n + 1) * w].view(n, (n + 1) * w)[:, :w].unflatten(1, (2, 64))
    far.copy_(rot)
    for at in (w, (n - 1) * (n + 1) * w + w):
        out = wide[at:at + n * w].view(n, 2, 64)
        assert torch.equal(pg.kvr_page_attend(0, far, out=out), want)
        assert torch.equal(far, rot)
    pg.kvr_pages_sync()


@pytest.mark.parametrize("given", [True, False])
def test_a_handle_dropped_while_another_stream_works(given):
    """Its pool and work area are not handed out again before that stream is done.  (Only addresses are looked at: nothing
    writes to the memory that the stream's call still uses.)"""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pg = handle(8, 2, 64, n_pages=4096, max_rows=64)
    keep, add = ints([0]), ints([5])
    pool, work = (t.data_ptr() for t in (pg.pool, pg.work))
    sizes = pg.pool.numel(), pg.work.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)
    if given:
        pg.kvr_page_plan(keep, add, 5, stream=side)
    else:
        with torch.cuda.stream(side):
            pg.kvr_page_plan(keep, add, 5)
    del pg
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not side.query()
    assert late[0].data_ptr() != pool and late[1].data_ptr() != work
    torch.cuda.synchronize()
