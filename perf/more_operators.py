"""The operators of a batch whose requests differ, as they are measured.

adapt   low-rank adapters of the batch's sequences beside a shared projection
sample  a token of each row's logits: temperature, top-k, min-p and top-p, from given random numbers
accept  speculative sampling: which drafts of each sequence stay, and the token after them

Sampling.  The tokens of a row stand in descending order of their logits, equal ones in that of their index, and weigh
w = exp((x - max) / temperature) (temperature 0: the first one weighs 1, the others nothing).  Kept are the first
top_k, as far as w >= min_p; of these the shortest run from the first that holds top_p of their weight.  The token is
the first kept one with a running weight above u times the kept weight.  Draft d of a row stays when u q(d) < p(d); at
the first that does not, the next token is drawn in the same manner from max(p - q, 0) (from p where that is nothing).
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the next token of one conversation under its adapter: q, k and v of a 7B layer
        dict(name="adapt_token_1", op="adapt", n_seq=1, rows=1, k=3584, parts="3584,512,512", rank=16, n_adapters=4,
             dtype="bf16", base="bf16", pick=0),
        # a token of each of 64 conversations, an adapter each: q, k and v of an 8B layer
        dict(name="adapt_token_64", op="adapt", n_seq=64, rows=1, k=4096, parts="4096,1024,1024", rank=16,
             n_adapters=64, dtype="bf16", base="bf16", pick=0),
        # a speculative step of eight conversations over four adapters: the down projection, into the residual stream
        dict(name="adapt_verify_8", op="adapt", n_seq=8, rows=8, k=18944, parts="3584", rank=32, n_adapters=4,
             dtype="bf16", base="fp32", pick=3),
        # the 254 suffix rows of a turn: q, k and v of a 7B layer
        dict(name="adapt_turn_254", op="adapt", n_seq=1, rows=254, k=3584, parts="3584,512,512", rank=64,
             n_adapters=2, dtype="bf16", base="bf16", pick=0),
        # prompts of four conversations, ragged
        dict(name="adapt_prompts_4", op="adapt", n_seq=4, rows=4095, k=4096, parts="4096,1024,1024", rank=64,
             n_adapters=3, dtype="bf16", base="bf16", pick=4),
        # token, verify and prompt rows in one batch, ranks from 8 up, some without an adapter: gate and up in fp16
        dict(name="adapt_mixed_12", op="adapt", n_seq=12, rows=120, k=2560, parts="9728,9728", rank=32, n_adapters=5,
             dtype="fp16", base="fp16", pick=5),
        # one conversation's next token with the usual settings
        dict(name="sample_token_1", op="sample", rows=1, vocab=32000, dtype="fp32", kind="usual", dist=False, pick=1),
        # the tokens of 64 conversations, each with settings of its own, some words banned
        dict(name="sample_batch_64", op="sample", rows=64, vocab=131072, dtype="fp32", kind="mixed", dist=False, pick=2),
        # open sampling at a high temperature over the largest vocabulary: every token counts
        dict(name="sample_open_16", op="sample", rows=16, vocab=262144, dtype="fp32", kind="open", dist=False, pick=3),
        # draft tokens with their whole distributions, odd vocabulary, 16-bit logits (many of them equal)
        dict(name="sample_dist_8", op="sample", rows=8, vocab=50001, dtype="bf16", kind="usual", dist=True, pick=4),
        # a speculative step of eight conversations, drafts without distributions (looked up, not drawn)
        dict(name="accept_lookup_8", op="accept", n_seq=8, rows=4, vocab=32000, dtype="fp32", kind="usual", draft=False,
             pick=5),
        # sixteen conversations of up to eight rows, drafts drawn from a small model's distributions
        dict(name="accept_draft_16", op="accept", n_seq=16, rows=8, vocab=131072, dtype="fp32", kind="mixed", draft=True,
             pick=6),
    ]


# width of a projection's input, and the columns of what it gives to (q, k and v; gate and up; one alone)
SITES = [(3584, "3584,512,512"), (3584, "3584"), (3584, "18944,18944"), (18944, "3584"), (4096, "4096,1024,1024"),
         (12288, "4096"), (2560, "2048,1024,1024"), (2560, "9728,9728"), (512, "512,128,128"), (1000, "520,72")]


def _parts(case):
    return [int(n) for n in case["parts"].split(",")]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapt", "adapt", "sample", "sample", "accept"])
    pick = rng.randrange(1, 1 << 20)
    dtype = rng.choice(["fp32", "fp32", "bf16", "fp16"])
    kind = rng.choice(["usual", "mixed", "mixed", "open"])
    if op == "adapt":
        k, parts = rng.choice(SITES)
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        rank = 8 * _log(rng, 1, 16)
        widths = [int(n) for n in parts.split(",")]
        most = int(1.5e8 / (2 * k + 8 * sum(widths)))                              # (rows in all)
        many = int(1.5e8 / (2 * rank * (k * len(widths) + sum(widths))))           # (adapters)
        rows = _log(rng, 1, min(2048, most))
        return dict(op=op, n_seq=_log(rng, 1, max(1, min(64, most // rows))), rows=rows, k=k, parts=parts, rank=rank,
                    n_adapters=_log(rng, 1, max(1, min(64, many))), dtype=dtype, base=rng.choice([dtype, "fp32"]),
                    pick=pick)
    vocab = _log(rng, 257, 262144)
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, max(1, min(256, 8000000 // vocab))), vocab=vocab, dtype=dtype, kind=kind,
                    dist=rng.random() < 0.25, pick=pick)
    rows = rng.randint(1, 9)
    return dict(op=op, n_seq=_log(rng, 1, max(1, min(32, 8000000 // (vocab * rows)))), rows=rows, vocab=vocab,
                dtype=dtype, kind=kind, draft=rng.random() < 0.5, pick=pick)


def _lengths(case):
    """Rows of each sequence.  pick = 0: all as many as the case says; otherwise ragged, the first one the longest."""
    n = case["n_seq"]
    if case["pick"] == 0:
        return [case["rows"]] * n
    r = random.Random(case["pick"])
    return [case["rows"]] + [r.randint(1, case["rows"]) for _ in range(n - 1)]


def _adapters(case):
    """(rank of each adapter, adapter of each sequence; -1 for none)."""
    n, most, seqs = case["n_adapters"], case["rank"], case["n_seq"]
    if case["pick"] == 0:
        return [most] * n, [b % n for b in range(seqs)]
    r = random.Random(case["pick"] + 1)
    ranks = [most] + [8 * r.randint(1, most // 8) for _ in range(n - 1)]
    return ranks, [0] + [-1 if r.random() < 0.15 else r.randrange(n) for _ in range(seqs - 1)]


def _settings(case, n):
    """temperature, top_k, min_p and top_p of n requests: the settings that users of such a service have."""
    r = random.Random(case["pick"] + 2)
    usual = (0.7, 50, 0.0, 0.9)
    if case["kind"] == "usual":
        s = [usual] * n
    elif case["kind"] == "open":
        s = [(r.uniform(1.0, 2.0), 0, 0.0, 1.0) for _ in range(n)]
    else:
        choices = [usual, (1.0, 0, 0.0, 0.95), (0.8, 0, 0.05, 1.0), (0.0, 0, 0.0, 1.0), (1.3, 200, 0.02, 0.98),
                   (1.0, 0, 0.0, 1.0), (0.6, 20, 0.0, 0.95), (1.5, 1000, 0.0, 1.0), (1.0, 1, 0.0, 1.0)]
        s = [choices[r.randrange(len(choices))] for _ in range(n)]
    t, k, m, p = zip(*s)
    f32 = lambda v: torch.tensor(v, dtype=torch.float32, device=DEV)
    return dict(temperature=f32(t), top_k=torch.tensor(k, dtype=torch.int32, device=DEV), min_p=f32(m), top_p=f32(p))


# --------------------------------------------------------------------------- inputs
def _logits(case, rows, gen):
    """A bulk of unlikely tokens and a few dozen likely ones in each row; in every third row a tenth is banned."""
    v = case["vocab"]
    x = torch.randn(rows, v, generator=gen, device=DEV) * 2.0
    likely = torch.randint(0, v, (rows, 48), generator=gen, device=DEV)
    x.scatter_add_(1, likely, torch.rand(rows, 48, generator=gen, device=DEV) * 12.0)
    banned = torch.rand(rows, v, generator=gen, device=DEV) < 0.1
    banned &= (torch.arange(rows, device=DEV) % 3 == 2)[:, None]
    return x.masked_fill_(banned, -math.inf)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "adapt":
        lens = _lengths(case)
        ranks, which = _adapters(case)
        dt, k, n = DTYPES[case["dtype"]], case["k"], sum(_parts(case))
        rows = sum(lens)
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
        adapters = [((normal(len(_parts(case)) * r, k) * k ** -0.5).to(dt), (normal(n, r) * 0.3).to(dt),
                     2.0 if r > 16 else 1.0) for r in ranks]
        return dict(x=normal(rows, k).to(dt), base=normal(rows, n).to(DTYPES[case["base"]]), adapters=adapters,
                    lens=lens, which=which, cu=torch.tensor(cu, dtype=torch.int32, device=DEV),
                    which_t=torch.tensor(which, dtype=torch.int32, device=DEV))
    dt = DTYPES[case["dtype"]]
    if case["op"] == "sample":
        rows = case["rows"]
        return dict(logits=_logits(case, rows, gen).to(dt), u=torch.rand(rows, generator=gen, device=DEV),
                    settings=_settings(case, rows))
    lens = _lengths(case)
    rows, n = sum(lens), len(lens)
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    logits = _logits(case, rows, gen)
    settings = _settings(case, n)
    # the drafter's view of the same rows, its distribution, and a token of it: the draft of the row after
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), torch.tensor(lens, device=DEV))
    heat = settings["temperature"][seq].clamp_min(0.3)[:, None]
    near = logits + torch.randn(rows, case["vocab"], generator=gen, device=DEV) * 0.5
    q = torch.softmax(near / heat, dim=1)
    top = q.amax(1, keepdim=True)
    q = torch.where(q < 0.02 * top, torch.zeros_like(q), q)   # (it drops the unlikely ones)
    q = q / q.sum(1, keepdim=True)
    drawn = torch.multinomial(q, 1, generator=gen)[:, 0] if case["draft"] else q.argmax(1)
    tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    tokens[1:] = drawn[:-1].to(torch.int32)
    tokens[torch.tensor(cu[:-1], device=DEV)] = 7
    return dict(logits=logits.to(dt), tokens=tokens, lens=lens, cu=torch.tensor(cu, dtype=torch.int32, device=DEV),
                seq=seq, u=torch.rand(rows, generator=gen, device=DEV), u_next=torch.rand(n, generator=gen, device=DEV),
                q=q if case["draft"] else None, settings=settings)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] == "adapt":
        from prefix_reused_prefill_gb300 import Adapters
        s["site"] = Adapters(s["adapters"], _parts(case))
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_adapt(s):
    x, base, case = s["x"], s["base"], s["case"]
    out, at = base.to(torch.float32, copy=True), 0
    for m, a in zip(s["lens"], s["which"]):
        if a >= 0:
            wa, wb, scale = s["adapters"][a]
            r = wb.shape[1]
            low = x[at:at + m].float() @ wa.float().t()
            col = 0
            for j, n in enumerate(_parts(case)):
                out[at:at + m, col:col + n] += scale * (low[:, j * r:(j + 1) * r] @ wb[col:col + n].float().t())
                col += n
        at += m
    return out.to(base.dtype)


def _plain_weights(logits, st):
    """The tokens in order, their weights (64 bits) and which are kept."""
    x, order = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    place = torch.arange(x.shape[1], device=x.device)[None]
    heat = st["temperature"].double()[:, None]
    w = torch.exp((x - x[:, :1]) / heat)
    w = torch.where(heat > 0, w, (place == 0).double())
    k = st["top_k"].long()[:, None]
    keep = (place < torch.where(k > 0, k, x.shape[1])) & (w >= st["min_p"].double()[:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)   # (weight of those in front)
    p = st["top_p"].double()[:, None]
    keep &= (p >= 1) | (before < p * cum[:, -1:])
    return order, torch.where(keep, w, torch.zeros_like(w))


def _plain_draw(order, w, u):
    cum = torch.cumsum(w, 1)
    at = torch.searchsorted(cum, (u.double()[:, None] * cum[:, -1:]), right=True)
    return at, order.gather(1, at)[:, 0].to(torch.int32), cum[:, -1:]


def _plain_sample(s):
    order, w = _plain_weights(s["logits"], s["settings"])
    at, token, total = _plain_draw(order, w, s["u"])
    prob = (w.gather(1, at) / total)[:, 0].float()
    if not s["case"]["dist"]:
        return token, prob
    return token, prob, torch.zeros_like(w).scatter_(1, order, w / total).float()


def _plain_accept(s):
    n, cu, seq, tokens = len(s["lens"]), s["cu"].long(), s["seq"], s["tokens"].long()
    order, w = _plain_weights(s["logits"], {k: v[seq] for k, v in s["settings"].items()})
    p = torch.zeros_like(w).scatter_(1, order, w / w.sum(1, keepdim=True))
    rows = torch.arange(len(seq), device=DEV)
    last = rows == cu[seq + 1] - 1
    draft = torch.roll(tokens, -1)
    q = s["q"].double() if s["q"] is not None else torch.zeros_like(p).scatter_(1, draft[:, None], 1.0)
    stay = s["u"].double() * q.gather(1, draft[:, None])[:, 0] < p.gather(1, draft[:, None])[:, 0]
    # the first row of each sequence whose draft does not stay (its last row has none)
    stop = torch.full((n,), len(seq), device=DEV).scatter_reduce_(
        0, seq, torch.where(last | ~stay, rows, len(seq)), "amin")
    rest = torch.where(last[stop, None], p[stop], (p[stop] - q[stop]).clamp_min(0.0))
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[stop])
    _, token, _ = _plain_draw(order[stop], rest.gather(1, order[stop]), s["u_next"])
    return (stop - cu[:-1]).to(torch.int32), token


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"adapt": _plain_adapt, "sample": _plain_sample, "accept": _plain_accept}[op](state)
    if op == "adapt":
        return state["site"].kvr_adapt(state["x"], state["cu"], state["which_t"], state["base"])
    if op == "sample":
        from prefix_reused_prefill_gb300 import kvr_sample
        return kvr_sample(state["logits"], state["u"], dist=state["case"]["dist"], **state["settings"])
    from prefix_reused_prefill_gb300 import kvr_accept
    return kvr_accept(state["logits"], state["tokens"], state["cu"], state["u"], state["u_next"],
                      draft_probs=state["q"], **state["settings"])


# --------------------------------------------------------------------------- cost and definition
def work(case):
    if case["op"] == "adapt":
        lens, n = _lengths(case), sum(_parts(case))
        ranks, which = _adapters(case)
        size = 4 if case["base"] == "fp32" else 2
        rows = sum(lens)
        per = len(_parts(case)) * case["k"] + n
        adapted = sum(m for m, a in zip(lens, which) if a >= 0)
        return {"bytes": adapted * case["k"] * 2 + 2 * rows * n * size + 2 * per * sum(ranks[a] for a in set(which) if a >= 0),
                "flops": sum(2 * m * ranks[a] * per for m, a in zip(lens, which) if a >= 0)}
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "sample":
        cells = case["rows"] * case["vocab"]
        return {"bytes": cells * (size + (4 if case["dist"] else 0)) + 28 * case["rows"], "flops": 4 * cells}
    rows = sum(_lengths(case))
    # (of a draft's distribution the draft's own share, and the whole of it once for each sequence)
    return {"bytes": rows * (case["vocab"] * size + 12) + case["n_seq"] * (28 + (4 * case["vocab"] if case["draft"] else 0)),
            "flops": 4 * rows * case["vocab"]}


def _exact_row(x, heat, k, floor, p):
    """The kept tokens of one row in order, and their shares."""
    if heat == 0:
        return x.argmax().view(1), torch.ones(1, dtype=torch.float64, device=x.device)
    best = x.max()
    index = torch.argsort(x, descending=True, stable=True)
    if k > 0:
        index = index[:k]
    w = ((x[index] - best) / heat).exp()
    n = int((w >= floor).sum())
    index, w = index[:n], w[:n]
    if p < 1:
        share = torch.cumsum(w, 0)
        n = int((share < p * share[-1]).sum()) + 1
        index, w = index[:n], w[:n]
    return index, w / w.sum()


def _exact_pick(index, share, u):
    run = torch.cumsum(share, 0)
    at = min(int((run <= u * run[-1]).sum()), len(index) - 1)
    return int(index[at]), float(share[at])


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adapt":
        out, at = s["base"].double(), 0
        for m, a in zip(s["lens"], s["which"]):
            if a >= 0:
                wa, wb, scale = s["adapters"][a]
                r, n = wb.shape[1], 0
                for j, cols in enumerate(_parts(case)):
                    low = torch.einsum("mk,jk->mj", s["x"][at:at + m].double(), wa[j * r:(j + 1) * r].double())
                    add = torch.einsum("mj,nj->mn", low, wb[n:n + cols].double())
                    out[at:at + m, n:n + cols] += scale * add
                    n += cols
            at += m
        return out
    st = {k: v.double().tolist() for k, v in s["settings"].items()}
    row = lambda r, i: _exact_row(s["logits"][r].double(), st["temperature"][i], int(st["top_k"][i]), st["min_p"][i],
                                  st["top_p"][i])
    if case["op"] == "sample":
        tokens, probs, dist = [], [], []
        for r, u in enumerate(s["u"].double().tolist()):
            index, share = row(r, r)
            token, prob = _exact_pick(index, share, u)
            tokens.append(token)
            probs.append(prob)
            if case["dist"]:
                dist.append(torch.zeros(case["vocab"], dtype=torch.float64, device=DEV).scatter_(0, index, share))
        out = (torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.tensor(probs, dtype=torch.float64, device=DEV))
        return out + ((torch.stack(dist),) if case["dist"] else ())
    kept, following, at = [], [], 0
    u, draft = s["u"].double().tolist(), s["tokens"].tolist()
    for b, m in enumerate(s["lens"]):
        for i in range(m):
            index, share = row(at + i, b)
            if i == m - 1:
                break
            d = draft[at + i + 1]
            q = s["q"][at + i].double() if s["q"] is not None else None
            q_d = 1.0 if q is None else float(q[d])
            p_d = float(share[index == d].sum())
            if u[at + i] * q_d < p_d:
                continue
            left = share - (q[index] if q is not None else (index == d).double())
            left = left.clamp_min(0.0)
            share = left if float(left.sum()) > 0 else share
            break
        kept.append(i)
        following.append(_exact_pick(index, share, float(s["u_next"][b]))[0])
        at += m
    return (torch.tensor(kept, dtype=torch.int32, device=DEV), torch.tensor(following, dtype=torch.int32, device=DEV))
