"""Conversations of one batch with adapters and sampling of their own, through the layer stack (GB300).

The oracle runs each conversation alone on weights that its adapter is merged into.  Rows and K/V are compared at the
stated bar |gpu - oracle| <= 1e-2 + 2e-2 |oracle|; lengths are exact, and so are tokens, given the logits that the call
itself returns (which meet the same bar, once for the rows and once for the head)."""
import numpy as np
import pytest
import torch

import workloads
from conftest import oracle_dims, oracle_weights
from oracle import formats
from oracle import model as om
from oracle import sampling as so

pytestmark = pytest.mark.gpu
ATOL, RTOL = 1e-2, 2e-2


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def close(got, ref, what, factor=1.0):
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    bad = ~(err <= factor * (ATOL + RTOL * np.abs(ref)))
    assert not bad.any(), f"{what}: {int(bad.sum())}/{bad.size} out of tolerance, max err {err.max():.4g}"


SITES = {"qkv": ("wq", "wk", "wv"), "o": ("wo",), "gate_up": ("wg", "wu"), "down": ("wd",)}


def make_adapters(kv, shape, W, ranks, seed, sites=SITES):
    """(what Kvr.adapters makes, per adapter the oracle's merged weights)."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator().manual_seed(seed)
    layers, merged = [], [[dict(w) for w in W] for _ in ranks]
    for l in range(shape.n_layers):
        here = {}
        for site, names in SITES.items():
            cols = [W[l][n].shape[0] for n in names]
            k = W[l][names[0]].shape[1]
            entries = []
            for i, r in enumerate(ranks):
                a = (torch.randn(len(names) * r, k, generator=g) * k ** -0.5).bfloat16()
                b = (torch.randn(sum(cols), r, generator=g) * 0.3 * r ** -0.5).bfloat16()
                scale = [1.0, 0.5][i % 2]
                entries.append((a.cuda(), b.cuda(), scale))
                if site in sites:
                    at = 0
                    for j, n in enumerate(names):
                        merged[i][l][n] = merged[i][l][n] + scale * (
                            b[at:at + cols[j]].double().numpy() @ a[j * r:(j + 1) * r].double().numpy())
                        at += cols[j]
            if site in sites:
                here[site] = Adapters(entries, cols)
        layers.append(here)
    return kv.adapters(layers), merged


def setup(name, vocab=0, seed=21, max_rows=160):
    from prefix_reused_prefill_gb300 import Kvr, config_for_shape
    shape = workloads.SHAPES[name]
    lws = workloads.stack_weights(shape, seed)
    kv = Kvr(config_for_shape(shape, 4, 256, max_rows, vocab=vocab), device="cuda")
    return shape, kv, kv.weights(workloads.weights_to(lws, "cuda")), [oracle_weights(shape, lw) for lw in lws]


def run_batch(kv, shape, w, ad, order, which, seqs, prefixes, fn):
    """The prefixes into their slots under their adapters, then fn(rows, hidden of them)."""
    xs = [workloads.hidden_for_tokens(s, shape.hidden, 5 + j) for j, s in enumerate(seqs)]
    for j, s in enumerate(order):
        if prefixes[j]:
            kv.kvr_prefill_batch_adapted([s], [seqs[j][:prefixes[j]]], xs[j][:prefixes[j]].cuda(), w, ad, [which[j]])
    rows = [s[p:] for s, p in zip(seqs, prefixes)]
    hid = torch.cat([x[p:] for x, p in zip(xs, prefixes)]).contiguous().cuda()
    return xs, fn(rows, hid)


@pytest.mark.parametrize("name,prefixes,lens,which", [
    ("small", [37, 90, 0, 64], [1, 5, 3, 8], [0, 1, -1, 2]),       # 17 rows: GEMV
    ("small", [20, 0, 130, 45], [30, 1, 40, 7], [2, -1, 0, 0]),    # 78 rows: tcgen05 GEMM
    ("small_d128", [50, 11], [4, 2], [1, 0]),
    ("small_bf16", [33, 70, 5], [2, 9, 1], [0, 5, 2]),
    ("small_q4k", [40, 9], [3, 50], [1, 2]),
])
def test_batch_of_adapted_conversations(name, prefixes, lens, which):
    shape, kv, w, W = setup(name)
    ad, merged = make_adapters(kv, shape, W, [16, 8, 48], 4)
    n = len(lens)
    order = [3, 1, 0, 2][:n]
    seqs = [list(range(1000 * (j + 1), 1000 * (j + 1) + prefixes[j] + lens[j])) for j in range(n)]
    xs, out = run_batch(kv, shape, w, ad, order, which, seqs, prefixes,
                        lambda rows, hid: kv.kvr_prefill_batch_adapted(order, rows, hid, w, ad, which))
    kv.kvr_sync_status()
    dims, at = oracle_dims(shape), 0
    for j in range(n):
        s, P, m = order[j], prefixes[j], lens[j]
        assert kv.kvr_slot_tokens(s) == seqs[j]
        cache = om.SlotKV(shape.n_layers, shape.n_kv_heads, 256, shape.head_dim)
        weights = merged[which[j]] if 0 <= which[j] < 3 else W
        whole = om.prefill(dims, weights, cache, workloads.bf16_to_f64(xs[j]), 0)
        close(workloads.bf16_to_f64(out[at:at + m]), whole[P:], f"conversation {j} rows")
        for l in range(shape.n_layers):
            k, v = kv.kvr_slot_kv(s, l)
            close(workloads.bf16_to_f64(k[:, :P + m]), cache.K[l][:, :P + m], f"conversation {j} K layer {l}")
            close(workloads.bf16_to_f64(v[:, :, :P + m].transpose(1, 2)), cache.V[l][:, :P + m],
                  f"conversation {j} V layer {l}")
        at += m


@pytest.mark.parametrize("site", list(SITES))
@pytest.mark.parametrize("rows", [5, 40])
def test_each_site_alone(site, rows):
    shape, kv, w, W = setup("small")
    ad, merged = make_adapters(kv, shape, W, [24], 9, sites=[site])
    seq = list(range(700, 700 + rows))
    x = workloads.hidden_for_tokens(seq, shape.hidden, 3)
    out = kv.kvr_prefill_batch_adapted([1], [seq], x.cuda(), w, ad, [0])
    cache = om.SlotKV(shape.n_layers, shape.n_kv_heads, 256, shape.head_dim)
    close(workloads.bf16_to_f64(out), om.prefill(oracle_dims(shape), merged[0], cache, workloads.bf16_to_f64(x), 0), site)
    plain = om.prefill(oracle_dims(shape), W, om.SlotKV(shape.n_layers, shape.n_kv_heads, 256, shape.head_dim),
                       workloads.bf16_to_f64(x), 0)
    assert np.abs(workloads.bf16_to_f64(out) - plain).max() > 0.1   # (the adapter shows)


@pytest.mark.parametrize("rows", [7, 50])
def test_conversations_without_an_adapter_are_those_of_the_plain_batch(rows):
    shape, kv, w, W = setup("small")
    ad, _ = make_adapters(kv, shape, W, [16], 2)
    a, b = list(range(rows)), list(range(500, 503))
    x = workloads.hidden_for_tokens(a + b, shape.hidden, 3).cuda()
    one = kv.kvr_prefill_batch([0, 1], [a, b], x, w)
    two = kv.kvr_prefill_batch_adapted([2, 3], [a, b], x, w, ad, [-1, 1])
    assert torch.equal(one, two)


@pytest.mark.parametrize("vocab,lens", [(1000, [1, 4, 6, 2]), (32000, [8, 8]), (4101, [20, 1, 30, 13])])
@pytest.mark.parametrize("drafted", [False, True])
def test_speculative_step_of_sampling_conversations(vocab, lens, drafted):
    """Adapters, the stack, the head and the decision in one call, two steps in a row."""
    shape, kv, w, W = setup("small", vocab=vocab)
    ad, merged = make_adapters(kv, shape, W, [16, 8, 48], 4)
    hw = workloads.head_weights(shape, 31, "cpu", vocab=vocab)
    head = {"norm": hw["norm"].cuda(), "lm": workloads.Int4Matrix(hw["lm"].packed.cuda(), hw["lm"].scales.cuda(), None)}
    gain, lm = hw["norm"].double().numpy(), formats.dequant_int4(hw["lm"].packed.numpy(), hw["lm"].scales.numpy())
    n = len(lens)
    order, which, prefixes = [2, 0, 3, 1][:n], [1, -1, 0, 2][:n], [30, 12, 0, 50][:n]
    g = torch.Generator().manual_seed(vocab)
    seqs = [torch.randint(0, vocab, (p + m,), generator=g).tolist() for p, m in zip(prefixes, lens)]
    settings = dict(temperature=[0.7, 1.0, 0.0, 1.5][:n], top_k=[50, 0, 0, 300][:n], min_p=[0.0, 0.01, 0.0, 0.0][:n],
                    top_p=[0.9, 1.0, 1.0, 0.95][:n])
    total = sum(lens)
    q = torch.softmax(torch.randn(total, vocab, generator=g) * 2, 1) if drafted else None
    u, un = torch.rand(total, generator=g) * 0.3, torch.rand(n, generator=g)
    logits = torch.empty(total, vocab, device="cuda")
    rows_out = torch.empty(total, shape.hidden, dtype=torch.bfloat16, device="cuda")
    step = lambda rows, hid: kv.kvr_verify_sample_batch(
        order, rows, hid, w, head, u, un, adapters=ad, which=which, draft_probs=None if q is None else q.cuda(),
        logits=logits, out=rows_out, **settings)
    xs, (nxt, acc) = run_batch(kv, shape, w, ad, order, which, seqs, prefixes, step)

    def check(nxt, acc, prefixes, toks):
        at = 0
        for j in range(n):
            r = slice(at, at + lens[j])
            s = {k: v[j] if k == "top_k" else float(np.float32(v[j])) for k, v in settings.items()}
            want = so.accept(logits[r].double().cpu().numpy(), toks[j], u.double().numpy()[r], float(un[j]),
                             q=None if q is None else q.double().numpy()[r], **s)
            assert (acc[j], nxt[j]) == want, j
            assert kv.kvr_slot_len(order[j]) == prefixes[j] + 1 + acc[j]
            at += lens[j]

    rows = [s[p:] for s, p in zip(seqs, prefixes)]
    check(nxt, acc, prefixes, rows)
    dims, at = oracle_dims(shape), 0
    for j in range(n):
        cache = om.SlotKV(shape.n_layers, shape.n_kv_heads, 256, shape.head_dim)
        weights = merged[which[j]] if which[j] >= 0 else W
        h = om.forward(dims, weights, cache, workloads.bf16_to_f64(xs[j]), om.plain_rows(0, len(seqs[j])), rounded=False)
        ref = om.head_logits(dims, h[prefixes[j]:], gain, lm)
        close(logits[at:at + lens[j]].double().cpu().numpy(), ref, f"conversation {j} logits", 2.0)
        close(workloads.bf16_to_f64(rows_out[at:at + lens[j]]), om.round_bf16(h[prefixes[j]:]), f"conversation {j} rows")
        at += lens[j]
    # the next step goes on from the kept tokens, its first draft the token that the model finds likeliest
    prefixes2 = [p + 1 + a for p, a in zip(prefixes, acc)]
    toks = [[t] + [int(x) for x in torch.randint(0, vocab, (m - 1,), generator=g)] for t, m in zip(nxt, lens)]
    hid = workloads.hidden_for_tokens([t for ts in toks for t in ts], shape.hidden, 77).cuda()
    probe = kv.kvr_verify_sample_batch(order, toks, hid, w, head, u, un, adapters=ad, which=which, logits=logits,
                                       draft_probs=None if q is None else q.cuda(), **settings)
    check(*probe, prefixes2, toks)
    at = 0
    for j, m in enumerate(lens):
        kv.kvr_slot_truncate(order[j], prefixes2[j])
        if m > 1:
            toks[j][1] = int(logits[at].argmax())
        at += m
    check(*kv.kvr_verify_sample_batch(order, toks, hid, w, head, u, un, adapters=ad, which=which, logits=logits,
                                      draft_probs=None if q is None else q.cuda(), **settings), prefixes2, toks)


def test_greedy_settings_are_the_greedy_call():
    shape, kv, w, W = setup("small", vocab=5000)
    hw = workloads.head_weights(shape, 31, "cpu", vocab=5000)
    head = {"norm": hw["norm"].cuda(), "lm": workloads.Int4Matrix(hw["lm"].packed.cuda(), hw["lm"].scales.cuda(), None)}
    toks = [[5, 6, 7], [9, 9]]
    x = workloads.hidden_for_tokens(sum(toks, []), shape.hidden, 8).cuda()
    nxt, _ = kv.kvr_verify_accept_batch([0, 1], toks, x, w, head)
    toks[0][1], toks[1][1] = nxt[0][0], nxt[1][0]
    a = kv.kvr_verify_accept_batch([2, 3], toks, x, w, head)
    for s in range(4):
        kv.kvr_slot_truncate(s, 0)
    b = kv.kvr_verify_sample_batch([2, 3], toks, x, w, head, [0.9] * 5, [0.5] * 2, temperature=[0.0, 0.0])
    assert b[1] == a[1] and b[0] == [a[0][j][a[1][j]] for j in range(2)]


def test_refusals_change_nothing():
    from prefix_reused_prefill_gb300 import Adapters, KvrError
    shape, kv, w, W = setup("small", vocab=500, max_rows=64)
    ad, _ = make_adapters(kv, shape, W, [8], 2)
    hw = workloads.head_weights(shape, 31, "cpu", vocab=500)
    head = {"norm": hw["norm"].cuda(), "lm": workloads.Int4Matrix(hw["lm"].packed.cuda(), hw["lm"].scales.cuda(), None)}
    x = lambda n: torch.zeros(n, shape.hidden, dtype=torch.bfloat16, device="cuda")
    half = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    other = Adapters([(half(8, shape.hidden), half(shape.hidden, 8), 1.0)], [shape.hidden])
    cases = [lambda: kv.kvr_prefill_batch_adapted([0], [[1, 2]], x(2), w, ad, [0, 0]),
             lambda: kv.kvr_prefill_batch_adapted([0, 0], [[1], [2]], x(2), w, ad, [0, 0]),
             lambda: kv.kvr_prefill_batch_adapted([0], [list(range(65))], x(65), w, ad, [0]),
             lambda: kv.kvr_prefill_batch_adapted([0], [[1]], x(2), w, ad, [0]),
             lambda: kv.kvr_prefill_batch_adapted([0], [[1]], x(1), w, kv.adapters([{"o": other}] * shape.n_layers), [0]),
             lambda: kv.adapters([{}]), lambda: kv.adapters([{"up": other}] * shape.n_layers),
             lambda: kv.kvr_verify_sample_batch([0], [[1, 2]], x(2), w, head, [0.5], [0.5]),
             lambda: kv.kvr_verify_sample_batch([0], [[1, 2]], x(2), w, head, [0.5] * 2, [0.5] * 2),
             lambda: kv.kvr_verify_sample_batch([0], [[1, 2]], x(2), w, head, [0.5] * 2, [0.5], top_k=[1, 2]),
             lambda: kv.kvr_verify_sample_batch([9], [[1, 2]], x(2), w, head, [0.5] * 2, [0.5]),
             lambda: kv.kvr_verify_sample_batch([0], [[1, 2]], x(2), w, head, [0.5] * 2, [0.5],
                                                draft_probs=torch.zeros(2, 499, device="cuda")),
             lambda: kv.kvr_verify_sample_batch([0], [[1, 2]], x(2), w, head, [0.5] * 2, [0.5],
                                                logits=torch.zeros(1, 500, device="cuda"))]
    for bad in cases:
        with pytest.raises(KvrError):
            bad()
    assert [kv.kvr_slot_len(s) for s in range(4)] == [0] * 4
    # a head that has no distribution: the token is -1, the slot keeps the row
    head["norm"].fill_(float("nan"))
    nxt, acc = kv.kvr_verify_sample_batch([0], [[1, 2]], workloads.hidden_for_tokens([1, 2], shape.hidden, 1).cuda(), w, head,
                                          [0.5] * 2, [0.5])
    assert nxt == [-1] and acc == [0] and kv.kvr_slot_len(0) == 1
