"""The layer stack over pages at its edges: steps without rows, layers without a norm (needs a GB300)."""
import pytest
import torch

import workloads
from test_gpu_prefill_pages import ints, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_a_step_without_rows():
    """A decode loop whose sequences have all ended: the stack returns no rows, as the operators do, and goes on."""
    shape = workloads.SHAPES["small"]
    kv, pg = make(shape)
    w = kv.weights(workloads.weights_to(workloads.stack_weights(shape, 21), "cuda"))
    x = workloads.hidden_for_tokens(list(range(5)), shape.hidden, 5).cuda()
    pg.kvr_page_plan(ints([0, 0]), ints([3, 2]), 5)
    want = kv.kvr_prefill_pages(pg, x, w)
    pg.kvr_page_plan(ints([0, 0]), ints([0, 0]), 0)
    pool = pg.pool.clone()
    none = torch.empty(0, shape.hidden, dtype=torch.bfloat16, device="cuda")
    assert kv.kvr_prefill_pages(pg, none, w).shape == (0, shape.hidden)
    kv.kvr_sync_status()
    pg.kvr_pages_sync()
    assert torch.equal(pg.pool, pool) and pg.state.lens.tolist() == [0, 0, 0]
    pg.kvr_page_plan(ints([0, 0]), ints([3, 2]), 5)
    assert torch.equal(kv.kvr_prefill_pages(pg, x, w), want)
