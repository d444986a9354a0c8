"""Memory of sampling and adapters: what shares bytes is refused, what lies between one another is not, and what another
stream reads outlives its work (GB300)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_results_that_share_memory_are_refused():
    from prefix_reused_prefill_gb300 import KvrError, kvr_sample
    x, u = torch.randn(4, 64, device=DEV), torch.rand(4, device=DEV)
    before = x.clone()
    wide = torch.randn(4, 96, device=DEV)
    for logits, dist in ((x, x), (wide[:, :64], wide[:, 32:]), (wide[:, 32:], wide[:, :64]), (x[:1], x[:1])):
        with pytest.raises(KvrError):
            kvr_sample(logits, u[:len(logits)], dist=dist)
    torch.cuda.synchronize()
    assert torch.equal(x, before)


def test_c_entries_refuse_what_shares_memory():
    from prefix_reused_prefill_gb300 import load_library
    lib = load_library()
    x, f = torch.randn(4, 64, device=DEV), torch.zeros(64, device=DEV)
    i = torch.zeros(64, dtype=torch.int32, device=DEV)
    w = torch.zeros(64, dtype=torch.int32, device=DEV)
    p = lambda t, at=0: t.data_ptr() + 4 * at
    sample = lambda **k: lib.kvr_sample(*{**dict(x=p(x), type=2, stride=64, rows=4, vocab=64, s=None, u=p(f), token=p(i),
                                                 prob=p(f, 8), dist=None, ds=0, st=None), **k}.values())
    assert sample() == 0
    for k in (dict(token=p(f, 3)), dict(prob=p(f, 3)), dict(prob=p(i, 3)), dict(token=p(x, 255)), dict(dist=p(x), ds=64),
              dict(dist=p(x, 32), ds=64)):
        assert sample(**k) == -1, k
    accept = lambda **k: lib.kvr_accept(*{**dict(x=p(x), type=2, stride=64, rows=4, vocab=64, s=None, n=2, cu=p(i),
                                                 tokens=p(i, 8), q=None, qs=0, u=p(f), un=p(f, 8), acc=p(i, 16), nxt=p(i, 24),
                                                 work=p(w), wb=16, st=None), **k}.values())
    assert accept() == 0
    for k in (dict(acc=p(i, 2)), dict(nxt=p(i, 17)), dict(acc=p(i, 11)), dict(work=p(i, 8)), dict(nxt=p(f, 9)), dict(acc=p(w, 3)),
              dict(work=p(x)), dict(nxt=p(x, 200))):
        assert accept(**k) == -1, k
    torch.cuda.synchronize()


def test_rows_between_one_another():
    """Logits and their distribution, inputs and outputs, side by side in rows of one buffer."""
    from prefix_reused_prefill_gb300 import Adapters, KvrError, kvr_sample
    both = torch.randn(6, 200, device=DEV)
    u = torch.rand(6, device=DEV)
    want = kvr_sample(both[:, :100].contiguous(), u, top_p=0.9, dist=True)
    got = kvr_sample(both[:, :100], u, top_p=0.9, dist=both[:, 100:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.Generator().manual_seed(3)
    site = Adapters([((torch.randn(16, 64, generator=g) / 8).to(BF).cuda(), torch.randn(32, 16, generator=g).to(BF).cuda(), 1.0)],
                    [32])
    buf = torch.randn(40, 96, generator=g).to(BF).cuda()
    cu, which = torch.tensor([0, 40], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    want = site.kvr_adapt(buf[:, :64].contiguous(), cu, which)
    assert torch.equal(site.kvr_adapt(buf[:, :64], cu, which, out=buf[:, 64:]), want)
    with pytest.raises(KvrError):
        site.kvr_adapt(buf[:, :64], cu, which, out=buf[:, 56:88])


def test_draft_probabilities_below_zero_and_nan():
    """They take nothing from what is left."""
    from prefix_reused_prefill_gb300 import kvr_accept
    g = torch.Generator().manual_seed(5)
    rows, vocab = 6, 3000
    logits = torch.randn(rows, vocab, generator=g).cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=g).int().cuda()
    q = torch.rand(rows, vocab, generator=g).cuda() * (2.0 / vocab)
    bad = q.clone()
    bad[:, ::3] = -1e30
    bad[:, 1::3] = float("nan")
    q[:, ::3] = 0
    q[:, 1::3] = 0
    for r in range(rows - 1):
        q[r, tokens[r + 1]] = bad[r, tokens[r + 1]] = 1.0
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device=DEV)
    u, u_next = torch.full((rows,), 0.999, device=DEV), torch.rand(3, generator=g).cuda()
    for settings in (dict(), dict(top_k=40), dict(top_p=0.99), dict(top_k=100, top_p=0.5)):
        a, b = (kvr_accept(logits, tokens, cu, u, u_next, draft_probs=x, **settings) for x in (q, bad))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (a[1] >= 0).all()


def test_adapters_given_up_while_another_stream_reads_them():
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator().manual_seed(9)
    make = lambda: Adapters([((torch.randn(64, 4096, generator=g) / 64).to(BF).cuda(),
                              torch.randn(4096, 64, generator=g).to(BF).cuda(), 1.0)], [4096])
    x = torch.randn(8, 4096, generator=g).to(BF).cuda()
    cu, which = torch.tensor([0, 8], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    site = make()
    want = site.kvr_adapt(x, cu, which)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # (some ten milliseconds of work in front)
    out = site.kvr_adapt(x, cu, which, stream=side)
    del site
    for _ in range(4):   # the sizes that were given up, written at once
        for n in (64 * 4096, 24):
            torch.full((n,), float("nan"), dtype=BF, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_wait_that_gave_up_is_reported_once():
    from prefix_reused_prefill_gb300 import Adapters, KvrError, kvr_batch_sync, load_library
    g = torch.Generator().manual_seed(11)
    site = Adapters([((torch.randn(16, 512, generator=g) / 16).to(BF).cuda(), torch.randn(256, 16, generator=g).to(BF).cuda(), 1.0)],
                    [256])
    x = torch.randn(300, 512, generator=g).to(BF).cuda()
    cu, which = torch.tensor([0, 300], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    want = site.kvr_adapt(x, cu, which)
    kvr_batch_sync()
    side = torch.cuda.Stream()
    assert load_library().kvr_batch_selftest_wait(side.cuda_stream) == 0   # (one second)
    with pytest.raises(KvrError) as e:
        kvr_batch_sync(side)
    assert e.value.code == -4 and "gave up" in str(e.value)
    kvr_batch_sync(side)
    kvr_batch_sync()
    assert torch.equal(site.kvr_adapt(x, cu, which), want)
    kvr_batch_sync()


def test_stack_calls_refuse_what_shares_memory():
    """The logits' buffer in the place of another argument, and the adapters' work area in that of the rows."""
    import ctypes

    import workloads
    from prefix_reused_prefill_gb300 import Adapters, Kvr, KvrError, config_for_shape
    from prefix_reused_prefill_gb300.kvr import KvrAdapters, _i32
    shape, vocab = workloads.SHAPES["small"], 512
    lws = workloads.stack_weights(shape, 21)
    kv = Kvr(config_for_shape(shape, 4, 256, 64, vocab=vocab), device="cuda")
    w = kv.weights(workloads.weights_to(lws, "cuda"))
    hw = workloads.head_weights(shape, 31, "cpu", vocab=vocab)
    head = {"norm": hw["norm"].cuda(), "lm": workloads.Int4Matrix(hw["lm"].packed.cuda(), hw["lm"].scales.cuda(), None)}
    rows, toks = 6, [[1, 2, 3], [4, 5, 6]]
    x = workloads.hidden_for_tokens(sum(toks, []), shape.hidden, 5).cuda()
    buf = torch.zeros(2 * rows, vocab, device=DEV)
    u, un = [0.5] * rows, [0.5] * 2
    step = lambda hid, **k: kv.kvr_verify_sample_batch([0, 1], toks, hid, w, head, u, un, **k)
    # hidden and out in the logits' memory
    words = buf.view(-1).view(BF)
    inside = words[64:64 + rows * shape.hidden].view(rows, shape.hidden)
    assert 64 + rows * shape.hidden <= words.numel()
    for hid, k in ((x, dict(logits=buf[:rows], draft_probs=buf[:rows])), (x, dict(logits=buf[:rows], draft_probs=buf[rows - 1:-1])),
                   (x, dict(logits=buf[:rows], draft_probs=buf[1:1 + rows])), (inside, dict(logits=buf[:rows])),
                   (x, dict(logits=buf[:rows], out=inside)), (x, dict(draft_probs=buf[:rows], out=inside))):
        with pytest.raises(KvrError) as e:
            step(hid, **k)
        assert e.value.code == -1
    assert [kv.kvr_slot_len(s) for s in range(2)] == [0, 0]
    nxt, _ = step(x, logits=buf[:rows], draft_probs=buf[rows:])   # side by side
    assert min(nxt) >= 0
    # the work area over hidden, and over out
    g = torch.Generator().manual_seed(3)
    site = Adapters([((torch.randn(8, shape.hidden, generator=g) / 30).to(BF).cuda(),
                      torch.randn(shape.hidden, 8, generator=g).to(BF).cuda(), 1.0)], [shape.hidden])
    sites, _keep = kv.adapters([{"o": site} if shape.n_q_heads * shape.head_dim == shape.hidden else {}] * shape.n_layers)
    wb = kv.lib.kvr_adapters_work_bytes(ctypes.byref(kv.cfg), sites, 3)
    one = torch.zeros(wb + (1 << 16), dtype=torch.uint8, device=DEV)
    mine = one[:3 * shape.hidden * 2].view(BF).view(3, shape.hidden)
    mine.copy_(x[:3])
    out = torch.empty_like(mine)
    call = lambda hid, to: kv.lib.kvr_prefill_batch_adapted(
        kv.ctx, 1, (ctypes.c_int * 1)(3), (ctypes.c_int * 1)(3), _i32([1, 2, 3]), hid.data_ptr(), w[0],
        ctypes.byref(KvrAdapters(sites, one.data_ptr(), wb)), (ctypes.c_int * 1)(0), to.data_ptr(), None)
    assert call(mine, out) == -1 and call(x[:3], mine) == -1 and kv.kvr_slot_len(3) == 0
    assert call(x[:3], out) == 0 and kv.kvr_slot_len(3) == 3
    kv.kvr_sync_status()


def test_a_stream_of_another_device_is_refused():
    import types

    from prefix_reused_prefill_gb300 import Adapters, KvrError, kvr_accept, kvr_sample
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)   # (this machine may have no such device)
    x, u = torch.randn(4, 64, device=DEV), torch.rand(4, device=DEV)
    i = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    site = Adapters([(torch.zeros(8, 64, dtype=BF, device=DEV), torch.zeros(64, 8, dtype=BF, device=DEV), 1.0)], [64])
    for call in (lambda: kvr_sample(x, u, stream=other),
                 lambda: kvr_accept(x, torch.zeros(4, dtype=torch.int32, device=DEV), i, u, u[:1], stream=other),
                 lambda: site.kvr_adapt(x.to(BF), i, i[:1], stream=other)):
        with pytest.raises(KvrError):
            call()
