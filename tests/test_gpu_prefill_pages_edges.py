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


def test_a_layer_without_a_norm():
    """Gains are given per layer; None stands for a layer without the norm, as a null pointer does."""
    shape = workloads.SHAPES["small"]
    kv, pg = make(shape)
    w = kv.weights(workloads.weights_to(workloads.stack_weights(shape, 21), "cuda"))
    x = workloads.hidden_for_tokens(list(range(5)), shape.hidden, 5).cuda()
    L, g = shape.n_layers, torch.full((shape.head_dim,), 0.75, dtype=torch.bfloat16, device="cuda")
    assert L > 1

    def run(norm_q, norm_k):
        pg.kvr_page_plan(ints([0, 0]), ints([3, 2]), 5)
        out = kv.kvr_prefill_pages(pg, x, w, norm_q, norm_k)
        return out, [t.clone() for l in range(L) for t in pg.kvr_page_read(l)]
    bare, normed = run(None, None), run([g] * L, [g] * L)
    some = run([g] + [None] * (L - 1), [None] * L)
    # k and v of the first layer are those without norms, its q is not
    assert all(torch.equal(a, b) for a, b in zip(some[1][:2], bare[1][:2])) and not torch.equal(some[0], bare[0])
    assert not torch.equal(some[0], normed[0])
    nothing = run([None] * L, [None] * L)
    assert torch.equal(nothing[0], bare[0]) and all(torch.equal(a, b) for a, b in zip(nothing[1], bare[1]))
    kv.kvr_sync_status()
    pg.kvr_pages_sync()
