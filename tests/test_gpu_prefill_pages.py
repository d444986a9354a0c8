"""The layer stack over the paged 4-bit cache (kvr_prefill_pages) against the float64 oracle (needs a GB300).

Each layer is checked on its own: from the traced residual stream before it, with the oracle's projections, norms,
rotation and attention, over the K and V that the cache holds (read back, in bf16).  The stream after the layer is held
to the stack tests' bar |gpu - oracle| <= 1e-2 + 2e-2 |oracle|; the rows that the layer stored to half a quantiser step
(0.5 s, s = max|x| / 7 of its group) beside the same bar.
"""
import numpy as np
import pytest
import torch

import workloads
from conftest import oracle_dims, oracle_weights
from oracle import model as om
from oracle import pages as op
from oracle.numerics import round_bf16, silu

pytestmark = pytest.mark.gpu
ATOL, RTOL = 1e-2, 2e-2


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def close(got, ref, what, more=0.0):
    err = np.abs(got - ref)
    bad = ~(err <= ATOL + RTOL * np.abs(ref) + more)
    assert not bad.any(), f"{what}: {int(bad.sum())}/{bad.size} out of tolerance, max err {err.max():.4g}"


def make(shape, max_rows=160, n_layers=None, **kw):
    from prefix_reused_prefill_gb300 import Kvr, PagedKv, config_for_shape, paged_config
    kv = Kvr(config_for_shape(shape, 1, 256, max_rows, n_layers=n_layers), device="cuda")
    pg = PagedKv(paged_config(**{**dict(
        n_pages=32, n_layers=kv.cfg.n_layers, n_q_heads=shape.n_q_heads, n_kv_heads=shape.n_kv_heads,
        head_dim=shape.head_dim, max_seqs=3, max_len=1 << 17, max_rows=max_rows, rope_theta=shape.rope_theta), **kw}))
    return kv, pg


@pytest.mark.parametrize("shape_name,norms", [("small", True), ("small", False), ("small_d128", True),
                                              ("small_bf16", True), ("small_q4k", False), ("small_g4", True)])
def test_stack_over_pages(shape_name, norms):
    """Prompts (the GEMM and, with 80 rows, both attention kernels), single tokens and verify rows (the GEMV), a
    rollback and a sequence that ends and starts again."""
    shape = workloads.SHAPES[shape_name]
    H, L, Hq, Hkv, d = shape.hidden, shape.n_layers, shape.n_q_heads, shape.n_kv_heads, shape.head_dim
    lws = workloads.stack_weights(shape, 21)
    kv, pg = make(shape)
    w = kv.weights(workloads.weights_to(lws, "cuda"))
    W = [oracle_weights(shape, lw) for lw in lws]
    rng = np.random.Generator(np.random.PCG64(8))
    gain = lambda: torch.from_numpy(0.5 + rng.random(d)).to(torch.bfloat16)
    gq, gk = ([gain() for _ in range(L)] if norms else None for _ in range(2))
    trace = torch.zeros(L + 1, 160, H, device="cuda")
    kv.kvr_trace_set(trace)
    stores = [[[np.zeros((Hkv, 0, d))] * 2 for _ in range(3)] for _ in range(L)]
    steps = [([0, 0, 0], [80, 9, 0]), ([80, 9, 0], [1, 3, 0]), ([81, 10, 0], [4, 1, 30]), ([82, 0, 30], [1, 40, 1])]
    for step, (keep, add) in enumerate(steps):
        n, pad = sum(add), step % 3
        pg.kvr_page_plan(ints(keep), ints(add), n + pad)
        x = torch.from_numpy(rng.standard_normal((n + pad, H)).astype(np.float32)).to(torch.bfloat16)
        dev = lambda g: None if g is None else [y.cuda() for y in g]
        out = kv.kvr_prefill_pages(pg, x.cuda(), w, dev(gq), dev(gk))
        kv.kvr_sync_status()
        pg.kvr_pages_sync()
        hs = trace.cpu().to(torch.float64).numpy()
        assert np.array_equal(hs[0, :n], workloads.bf16_to_f64(x[:n]))
        close(workloads.bf16_to_f64(out[:n]), hs[L, :n], "output")
        for l in range(L):
            h = hs[l, :n]
            a = round_bf16(om.rmsnorm(h, W[l]["norm_attn"], shape.rms_eps))
            q, k, v = (round_bf16(om.linear(a, W[l][name])).reshape(n, -1, d) for name in ("wq", "wk", "wv"))
            held_k, held_v = (workloads.bf16_to_f64(y)[:n] for y in pg.kvr_page_read(l))
            o, row = np.empty((n, Hq, d)), 0
            for b, (p, m) in enumerate(zip(keep, add)):
                kb, vb = (y[:, :p] for y in stores[l][b])
                for i in range(m):
                    g = [None if not norms else workloads.bf16_to_f64(y[l]) for y in (gq, gk)]
                    kr = op.norm_rotate(k[row], p + i, shape.rope_theta, g[1], 1e-6)
                    for got, ref, what in ((held_k[row], kr, "k"), (held_v[row], v[row], "v")):
                        s = np.repeat(np.max(np.abs(ref).reshape(Hkv, -1, 32), axis=-1), 32, axis=-1) / 7
                        close(got, ref, f"step {step} layer {l} sequence {b} row {i} {what}", 0.5 * s)
                    kb, vb = (np.concatenate([y, z[row][:, None]], axis=1) for y, z in ((kb, held_k), (vb, held_v)))
                    qr = round_bf16(op.norm_rotate(q[row], p + i, shape.rope_theta, g[0], 1e-6))
                    o[row] = op.attend(qr, kb, vb, d ** -0.5)[0]
                    row += 1
                stores[l][b] = [kb, vb]
            h = h + om.linear(round_bf16(o).reshape(n, Hq * d), W[l]["wo"])
            y = round_bf16(om.rmsnorm(h, W[l]["norm_ffn"], shape.rms_eps))
            z = round_bf16(silu(om.linear(y, W[l]["wg"])) * om.linear(y, W[l]["wu"]))
            close(hs[l + 1, :n], h + om.linear(z, W[l]["wd"]), f"step {step} layer {l}")


def test_attention_only_layer_over_pages():
    shape = workloads.SHAPES["small_attn"]
    lws = workloads.stack_weights(shape, 21)
    kv, pg = make(shape)
    w = kv.weights(workloads.weights_to(lws, "cuda"))
    W = oracle_weights(shape, lws[0])
    rng = np.random.Generator(np.random.PCG64(9))
    x = torch.from_numpy(rng.standard_normal((50, shape.hidden)).astype(np.float32)).to(torch.bfloat16)
    pg.kvr_page_plan(ints([0]), ints([50]), 50)
    out = workloads.bf16_to_f64(kv.kvr_prefill_pages(pg, x.cuda(), w))
    k, v = (workloads.bf16_to_f64(y).transpose(1, 0, 2) for y in pg.kvr_page_read(0))
    q = round_bf16(om.linear(workloads.bf16_to_f64(x), W["wq"])).reshape(50, -1, shape.head_dim)
    for i in range(50):
        o, _ = op.attend(round_bf16(op.norm_rotate(q[i], i, shape.rope_theta)), k[:, :i + 1], v[:, :i + 1],
                         shape.head_dim ** -0.5)
        close(out[i], om.linear(round_bf16(o).reshape(-1), W["wo"]), f"row {i}")


def test_slots_are_left_alone_and_steps_repeat():
    shape = workloads.SHAPES["small"]
    kv, pg = make(shape)
    w = kv.weights(workloads.weights_to(workloads.stack_weights(shape, 21), "cuda"))
    toks = list(range(20))
    kv.kvr_prefill_suffix(0, toks, workloads.hidden_for_tokens(toks, shape.hidden, 5).cuda(), w)
    arena = kv.arena.clone()
    x = workloads.hidden_for_tokens(list(range(100, 140)), shape.hidden, 5).cuda()
    outs = []
    for _ in range(3):
        pg.kvr_page_plan(ints([0, 0]), ints([33, 7]), 40)
        outs.append(kv.kvr_prefill_pages(pg, x, w))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(kv.arena, arena) and kv.kvr_slot_tokens(0) == toks
    # rows alone give the same as rows in a batch
    pg.kvr_page_plan(ints([0, 0]), ints([33, 0]), 33)
    alone = kv.kvr_prefill_pages(pg, x[:33].contiguous(), w)
    close(workloads.bf16_to_f64(alone), workloads.bf16_to_f64(outs[0][:33]), "alone")


def test_captured_step_of_the_stack():
    """A whole decode step (plan, every layer) captured once and replayed while the sequences grow."""
    shape = workloads.SHAPES["small"]
    w, made = None, []
    for _ in range(2):
        kv, pg = make(shape)
        w = kv.weights(workloads.weights_to(workloads.stack_weights(shape, 21), "cuda"))
        x0 = workloads.hidden_for_tokens(list(range(70)), shape.hidden, 5).cuda()
        pg.kvr_page_plan(ints([0, 0, 0]), ints([60, 3, 7]), 70)
        kv.kvr_prefill_pages(pg, x0, w)
        made.append((kv, pg, w))
    one = ints([1, 1, 1])
    x = torch.empty(3, shape.hidden, dtype=torch.bfloat16, device="cuda")

    def step(kv, pg, w):
        pg.kvr_page_plan(pg.state.lens, one, 3, 1)
        return kv.kvr_prefill_pages(pg, x, w)
    inputs = [workloads.hidden_for_tokens([1000 + 3 * i + j for j in range(3)], shape.hidden, 5) for i in range(8)]
    want = []
    for y in inputs:
        x.copy_(y)
        want.append(step(*made[0]).clone())
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        out = step(*made[1])
    for i, y in enumerate(inputs):
        x.copy_(y)
        g.replay()
        assert torch.equal(out, want[i]), i
    made[1][0].kvr_sync_status()
    made[1][1].kvr_pages_sync()


def test_refusals():
    from prefix_reused_prefill_gb300 import KvrError
    shape = workloads.SHAPES["small"]
    kv, pg = make(shape, max_rows=64)
    w = kv.weights(workloads.weights_to(workloads.stack_weights(shape, 21), "cuda"))
    x = torch.zeros(4, shape.hidden, dtype=torch.bfloat16, device="cuda")
    pg.kvr_page_plan(ints([0]), ints([4]), 4)
    others = [make(shape, n_layers=None, act="fp16")[1], make(shape, n_q_heads=4)[1]]
    for other in others:
        other.kvr_page_plan(ints([0]), ints([4]), 4)
    wide = make(shape, max_rows=200)[1]
    wide.kvr_page_plan(ints([0]), ints([100]), 100)
    big = torch.zeros(100, shape.hidden, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    refused = [
        (lambda: kv.kvr_prefill_pages(others[0], x, w), -1), (lambda: kv.kvr_prefill_pages(others[1], x, w), -1),
        (lambda: kv.kvr_prefill_pages(pg, x[:3].contiguous(), w), -1), (lambda: kv.kvr_prefill_pages(wide, big, w), -2),
        (lambda: kv.kvr_prefill_pages(pg, x.float(), w), -1), (lambda: kv.kvr_prefill_pages(pg, x[:, ::2], w), -1),
        (lambda: kv.kvr_prefill_pages(pg, x, w, [g]), -1), (lambda: kv.kvr_prefill_pages(pg, x, w, None, [g[:32]] * 2), -1),
        (lambda: kv.kvr_prefill_pages(pg, x, w, out=x[:2]), -1),
    ]
    pool = pg.pool.clone()
    for i, (call, code) in enumerate(refused):
        with pytest.raises(KvrError) as e:
            call()
        assert e.value.code == code, i
    assert torch.equal(pg.pool, pool)
    kv.kvr_prefill_pages(pg, x, w)
    kv.kvr_sync_status()
    pg.kvr_pages_sync()
