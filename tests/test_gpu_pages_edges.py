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
