"""Sampling and speculative sampling on the GPU against 64-bit arithmetic (GB300).

Tokens and counts are equal.  A probability is w / W rounded once (half a step, 2^-24), and W a sum of whole numbers
of 2^-44 of the largest weight: n of them are off by n 2^-45 at most, 2^-27 of W for the largest vocabulary.  So a
probability is within 2^-23 of its value, and within a step of the least float (2^-149)."""
import numpy as np
import pytest
import torch

from oracle import sampling as so

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SETTINGS = [dict(), dict(temperature=0.7, top_k=50, top_p=0.9), dict(temperature=0.0), dict(min_p=0.05),
            dict(top_k=1), dict(top_p=0.3), dict(temperature=1.7, top_k=1000, min_p=0.001, top_p=0.99),
            dict(temperature=100.0, top_p=0.999), dict(temperature=0.01), dict(top_p=0.0), dict(min_p=3.0),
            dict(temperature=2.0, top_k=100000)]


def ops():
    from prefix_reused_prefill_gb300 import kvr_accept, kvr_sample
    return kvr_sample, kvr_accept


def tensors(settings):
    """Settings of several requests, as columns."""
    default = dict(temperature=1.0, top_k=0, min_p=0.0, top_p=1.0)
    full = [dict(default, **s) for s in settings]
    return {k: torch.tensor([s[k] for s in full], dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV)
            for k in default}


def as_float32(settings):
    """What the device reads of them."""
    return {k: v if k == "top_k" else float(np.float32(v)) for k, v in settings.items()}


def bulk(rows, vocab, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * spread
    likely = torch.randint(0, vocab, (rows, 20), generator=g)
    return x.scatter_add_(1, likely, torch.rand(rows, 20, generator=g) * 10)


def check_rows(logits, u, settings, dist=True):
    """Every row of a call against the oracle."""
    kvr_sample, _ = ops()
    out = kvr_sample(logits, u, dist=dist, **tensors(settings))
    x, uu = logits.double().cpu().numpy(), u.double().cpu().numpy()
    token, prob = out[0].tolist(), out[1].double().tolist()
    for r, s in enumerate(settings):
        want = so.sample(x[r], uu[r], **as_float32(s))
        assert token[r] == want[0], (r, s, token[r], want[:2])
        assert abs(prob[r] - want[1]) <= 2.0 ** -23 * want[1] + 2.0 ** -149, (r, s)
        if dist:
            p = out[2][r].double().cpu().numpy()
            assert (np.abs(p - want[2]) <= 2.0 ** -23 * want[2] + 2.0 ** -149).all(), (r, s)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 17, 255, 1000, 4097, 16384, 50001])
def test_rows_of_every_setting(vocab, dtype):
    logits = bulk(len(SETTINGS), vocab, vocab).to(TYPES[dtype]).to(DEV)
    u = torch.rand(len(SETTINGS), generator=torch.Generator().manual_seed(vocab + 1)).to(DEV)
    check_rows(logits, u, SETTINGS)


@pytest.mark.parametrize("rows,vocab", [(1, 262144), (2, 200001), (5, 100003), (40, 32000), (80, 8191), (160, 3001),
                                        (400, 333)])
def test_calls_of_every_shape(rows, vocab):
    """From one row over several CTAs to many rows in waves."""
    logits = bulk(rows, vocab, rows).to(DEV)
    u = torch.rand(rows, generator=torch.Generator().manual_seed(rows)).to(DEV)
    check_rows(logits, u, [SETTINGS[(r * 5 + 1) % len(SETTINGS)] for r in range(rows)], dist=rows <= 5)


@pytest.mark.parametrize("vocab", [5000, 100000, 262144])
@pytest.mark.parametrize("u", [0.0, 0.25, 0.5, 0.7512345, 1 - 2.0 ** -24])
def test_equal_logits_in_the_order_of_their_index(vocab, u):
    """Far more equal tokens than are put in order at once: the draw is floor(u n)."""
    kvr_sample, _ = ops()
    logits = torch.full((4, vocab), -1.5, device=DEV)
    uu = torch.full((4,), u, device=DEV)
    k = torch.tensor([0, 0, 4321, 0], dtype=torch.int32, device=DEV)
    p = torch.tensor([1.0, 0.5, 1.0, 2.0 ** -12], device=DEV)
    token, prob = kvr_sample(logits, uu, top_k=k, top_p=p)
    exact_u = float(np.float32(u))
    sizes = [vocab, -(-vocab // 2), 4321, -(-vocab // 4096)]
    assert token.tolist() == [int(exact_u * n) for n in sizes]
    want = torch.tensor([1.0 / n for n in sizes], dtype=torch.float64)
    assert ((prob.double().cpu() - want).abs() <= 2.0 ** -23 * want).all()


def test_two_levels_of_many_equal_logits():
    """The run ends among equal logits behind a few larger ones, in rows of 16-bit logits too."""
    x = torch.full((3, 60000), -2.0)
    x[:, 100:200] = 5.0
    x[:, 40000:] = -1.0
    for dtype in TYPES.values():
        logits = x.to(dtype).to(DEV)
        u = torch.tensor([0.999, 0.97, 0.9999999], device=DEV)
        check_rows(logits, u, [dict(temperature=2.0), dict(temperature=2.0, top_k=30000), dict(temperature=3.0, top_p=0.99)])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_masked_tokens(dtype):
    """-infinity, the type's lowest value, infinities and NaN."""
    kvr_sample, _ = ops()
    dt = TYPES[dtype]
    low = torch.finfo(dt).min
    v = 3001
    x = bulk(8, v, 5)
    x[0, 10:] = -np.inf               # few tokens left
    x[1, :] = -np.inf
    x[1, 2999] = -7.0                 # one left
    x[2, :] = -np.inf                 # none
    x[3, 77] = np.nan                 # no distribution
    x[4, [5, 900]] = np.inf           # two share the row
    x = x.to(dt)
    x[5, :] = low                     # all alike
    x[6, :3000] = low                 # one above the lowest
    x[7, ::2] = low                   # half of them at the lowest value
    settings = [dict(top_k=50), dict(top_p=0.5), dict(), dict(), dict(top_p=0.9), dict(), dict(min_p=0.1), dict(temperature=0.5)]
    u = torch.linspace(0.05, 0.95, 8)
    check_rows(x.to(DEV), u.to(DEV), settings)
    assert kvr_sample(x.to(DEV), u.to(DEV))[0].tolist()[1:4] == [2999, -1, -1]


def test_settings_out_of_their_range():
    kvr_sample, _ = ops()
    nan, inf = float("nan"), float("inf")
    bad = [dict(temperature=-1.0), dict(temperature=nan), dict(temperature=inf), dict(temperature=2.0 ** -65),
           dict(min_p=nan), dict(top_p=nan), dict(temperature=2.0 ** 65)]
    logits = bulk(len(bad) + 3, 1000, 3).to(DEV)
    u = torch.tensor([0.5] * len(bad) + [1.0, -0.25, nan], device=DEV)
    token, prob, dist = kvr_sample(logits, u, dist=True, **tensors(bad + [dict()] * 3))
    assert token.tolist() == [-1] * len(token) and not prob.any() and not dist.any()
    check_rows(logits[:3], u[:3], [dict(temperature=2.0 ** -64), dict(temperature=2.0 ** 64), dict(top_k=-5, top_p=7.0)])


def test_largest_and_least_logits():
    """Differences that overflow, denormal ones, both zeros."""
    x = torch.zeros(4, 2000)
    x[0, :1000], x[0, 1000:] = 3e38, -3e38
    x[1] = torch.linspace(-1e-40, 1e-40, 2000)
    x[2, ::2] = -0.0
    x[3] = torch.linspace(-2e38, 3e38, 2000)
    u = torch.tensor([0.6, 0.3, 0.1234, 0.9])
    check_rows(x.to(DEV), u.to(DEV), [dict(), dict(temperature=2.0 ** -64), dict(top_k=500), dict(temperature=2.0 ** 64)])


def test_strides_offsets_and_numbers_as_settings():
    kvr_sample, _ = ops()
    for dtype in TYPES.values():
        for off in (0, 1, 3):
            wide = bulk(6, 1000 + 37, off).to(dtype).to(DEV)
            logits = wide[::2, off:off + 1000]
            u = torch.tensor([0.1, 0.5, 0.9], device=DEV)
            check_rows(logits, u, [SETTINGS[1]] * 3)
            a = kvr_sample(logits, u, temperature=0.7, top_k=50, top_p=0.9)
            b = kvr_sample(logits.contiguous(), u, **tensors([SETTINGS[1]] * 3))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dist = torch.full((3, 1200), 9.0, device=DEV)
    out = kvr_sample(logits, u, dist=dist[:, 100:1100])
    assert (dist[:, :100] == 9).all() and (dist[:, 1100:] == 9).all()
    assert torch.equal(out[2], kvr_sample(logits, u, dist=True)[2])


def test_no_rows():
    kvr_sample, kvr_accept = ops()
    logits = torch.zeros(0, 100, device=DEV)
    f, i = torch.zeros(0, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    token, prob = kvr_sample(logits, f)
    assert token.shape == (0,) and prob.shape == (0,)
    acc, nxt = kvr_accept(logits, i, torch.zeros(3, dtype=torch.int32, device=DEV), f, torch.zeros(2, device=DEV))
    assert acc.tolist() == [0, 0] and nxt.tolist() == [-1, -1]


def test_same_call_same_bits_captured_and_on_another_stream():
    kvr_sample, _ = ops()
    logits = bulk(7, 30000, 9).to(DEV)
    u = torch.rand(7, generator=torch.Generator().manual_seed(4)).to(DEV)
    st = tensors([SETTINGS[r] for r in range(7)])
    want = kvr_sample(logits, u, dist=True, **st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kvr_sample(logits, u, dist=True, stream=side, **st)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kvr_sample(logits, u, dist=True, **st)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, out):
        assert torch.equal(a, b) and torch.equal(a, c)
    new = bulk(7, 30000, 10).to(DEV)
    logits.copy_(new)
    u.copy_(torch.rand(7, generator=torch.Generator().manual_seed(5)))
    graph.replay()
    again = kvr_sample(new, u, dist=True, **st)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


# --------------------------------------------------------------------------- accept
def make_steps(lens, vocab, seed, with_q, dtype=torch.float32, heat=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = sum(lens)
    logits = bulk(rows, vocab, seed + 1).to(dtype)
    q = torch.softmax((logits.float() + torch.randn(rows, vocab, generator=g) * 0.5) / heat, 1)
    q = torch.where(q < 0.01 * q.amax(1, keepdim=True), torch.zeros_like(q), q)
    q /= q.sum(1, keepdim=True)
    tokens = torch.zeros(rows, dtype=torch.int32)
    pick = torch.multinomial(q, 1, generator=g)[:, 0] if with_q else q.argmax(1)
    tokens[1:] = pick[:-1].int()
    cu = np.concatenate([[0], np.cumsum(lens)])
    return logits, tokens, torch.tensor(cu, dtype=torch.int32), q if with_q else None, \
        torch.rand(rows, generator=g), torch.rand(len(lens), generator=g)


def check_accept(lens, logits, tokens, cu, q, u, u_next, settings):
    _, kvr_accept = ops()
    d = lambda x: None if x is None else x.to(DEV)
    acc, nxt = kvr_accept(d(logits), d(tokens), d(cu), d(u), d(u_next), draft_probs=d(q), **tensors(settings))
    x, qq = logits.double().numpy(), None if q is None else q.double().numpy()
    got, want = list(zip(acc.tolist(), nxt.tolist())), []
    for b, s in enumerate(settings):
        r = slice(int(cu[b]), int(cu[b + 1]))
        want.append(so.accept(x[r], tokens[r].tolist(), u.double().numpy()[r], float(u_next[b]),
                              q=None if q is None else qq[r], **as_float32(s)))
    assert got == want
    return got


@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,lens", [(40, [1]), (333, [4, 1, 9, 2, 5, 3, 8, 1, 7, 6, 2, 2]), (8191, [8] * 8),
                                        (100003, [3, 5]), (262144, [2])])
def test_accept_against_the_oracle(vocab, lens, dtype, with_q):
    args = make_steps(lens, vocab, vocab + len(lens), with_q, TYPES[dtype])
    got = check_accept(lens, *args, [SETTINGS[(3 * b + 1) % len(SETTINGS)] for b in range(len(lens))])
    if len(lens) > 5:
        assert any(a > 0 for a, _ in got) and any(a < m - 1 for (a, _), m in zip(got, lens))


def test_accept_of_sequences_without_rows_and_a_padded_batch():
    lens = [0, 3, 0, 2, 0]
    logits, tokens, cu, q, u, u_next = make_steps(lens, 500, 3, True)
    check_accept(lens, logits, tokens, cu, q, u, u_next, [dict()] * 5)
    _, kvr_accept = ops()
    pad = lambda x, v: torch.cat([x, torch.full((4, *x.shape[1:]), v, dtype=x.dtype)]).to(DEV)
    a = kvr_accept(pad(logits, float("nan")), pad(tokens, -9), cu.to(DEV), pad(u, 5.0), u_next.to(DEV), draft_probs=pad(q, float("nan")))
    b = kvr_accept(logits.to(DEV), tokens.to(DEV), cu.to(DEV), u.to(DEV), u_next.to(DEV), draft_probs=q.to(DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_accept_of_drafts_outside_the_vocabulary_and_of_bad_rows():
    lens = [4, 4, 4, 4]
    logits, tokens, cu, q, u, u_next = make_steps(lens, 600, 8, False)
    u[:] = 0.0                        # every possible draft stays
    tokens[2], tokens[6] = -1, 600    # but these are none
    logits[9] = float("nan")          # sequence 2 has no distribution after its first draft
    u[13] = 1.5                       # sequence 3 no random number after its second
    got = check_accept(lens, logits, tokens, cu, q, u, u_next, [dict()] * 4)
    assert [a for a, _ in got] == [1, 1, 1, 1] and [t for _, t in got][2:] == [-1, -1]
    u_next[1] = float("nan")
    assert check_accept(lens, logits, tokens, cu, q, u, u_next, [dict()] * 4)[1] == (0, -1)


def test_accept_where_the_drafter_is_the_model():
    """q = p: every draft stays but where a rounding of q passes p; a draft with nothing left is drawn from p."""
    kvr_sample, kvr_accept = ops()
    lens = [6, 6]
    logits, tokens, cu, _, u, u_next = make_steps(lens, 2000, 12, True)
    x = logits.to(DEV)
    _, _, q = kvr_sample(x, u.to(DEV) * 0, temperature=0.8, top_k=40, dist=True)
    drafts = torch.multinomial(q, 1)[:, 0].int().cpu()
    tokens[1:] = drafts[:-1]
    u.clamp_(max=0.99)
    check_accept(lens, logits, tokens, cu, q.cpu(), u, u_next, [dict(temperature=0.8, top_k=40)] * 2)
    acc, _ = kvr_accept(x, tokens.to(DEV), cu.to(DEV), u.to(DEV), u_next.to(DEV), draft_probs=q, temperature=0.8, top_k=40)
    assert acc.tolist() == [5, 5]
    ones = torch.ones_like(q)         # nothing of p is left beside such a drafter
    u[:] = 0.99
    check_accept(lens, logits, tokens, cu, ones.cpu(), u, u_next, [dict()] * 2)


def test_accept_captured_and_its_refusals():
    from prefix_reused_prefill_gb300 import KvrError
    kvr_sample, kvr_accept = ops()
    lens = [3, 2]
    logits, tokens, cu, q, u, u_next = [None if x is None else x.to(DEV) for x in make_steps(lens, 900, 21, True)]
    want = kvr_accept(logits, tokens, cu, u, u_next, draft_probs=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kvr_accept(logits, tokens, cu, u, u_next, draft_probs=q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    for bad in (lambda: kvr_sample(logits.double(), u), lambda: kvr_sample(logits, u[:2]),
                lambda: kvr_sample(logits.cpu(), u), lambda: kvr_sample(logits.t(), u),
                lambda: kvr_sample(logits, u.double()), lambda: kvr_sample(logits, u, top_k=u),
                lambda: kvr_sample(logits, u, dist=torch.empty(5, 899, device=DEV)),
                lambda: kvr_sample(torch.zeros(1, 262145, device=DEV), u[:1]),
                lambda: kvr_accept(logits, tokens.long(), cu, u, u_next),
                lambda: kvr_accept(logits, tokens, cu, u, u),
                lambda: kvr_accept(logits, tokens, cu, u, u_next, draft_probs=q[:, :899]),
                lambda: kvr_accept(logits, tokens, cu[:1], u, u_next)):
        with pytest.raises(KvrError):
            bad()


def test_refusals_of_the_c_entries():
    import ctypes
    from prefix_reused_prefill_gb300 import load_library
    lib = load_library()
    x = torch.zeros(4, 64, device=DEV)
    u, t = torch.zeros(4, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    p = lambda a: a.data_ptr()
    call = lambda **k: lib.kvr_sample(*{**dict(logits=p(x), type=2, stride=64, rows=4, vocab=64, s=None, u=p(u),
                                               token=p(t), prob=None, dist=None, ds=0, st=None), **k}.values())
    assert call() == 0
    for k in (dict(type=3), dict(stride=63), dict(rows=-1), dict(vocab=0), dict(vocab=262145), dict(logits=None),
              dict(u=None), dict(token=None), dict(logits=p(x) + 2), dict(token=p(t) + 1), dict(dist=p(x), ds=63)):
        assert call(**k) == -1, k
        assert lib.kvr_batch_error()
    assert lib.kvr_accept_work_bytes(-1) == 0
    torch.cuda.synchronize()
