"""The operators of the paged 4-bit cache, as they are measured.

plan    the page tables and row maps of a step, built on the GPU from the requests' lengths
append  the step's rows: q and k normed per head and rotated, k and v quantised into the pages
attend  causal grouped-query attention of the step's rows over the 4-bit pages

A page holds 64 tokens.  K and V are held in groups of 32 along the head dimension: s = fp16(max|x| / 7), at most
8188, and a code rint(x / s) in [-8, 7].
"""
import math
import random

import torch

own = False

PAGE = 64
GROUP = 32
DEV = "cuda"
EPS = 1e-6
THETA = 1e6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one speculative step of eight conversations: a few drafts each, two of them new
        dict(name="plan_verify_8", op="plan", n_seq=8, prefix=4096, rows=8, pick=1),
        # continuous batching: 512 conversations, an eighth of them admitted with their prompts
        dict(name="plan_admit_512", op="plan", n_seq=512, prefix=8192, rows=8, pick=2),
        # a token of each of 64 conversations (dense 9B heads, with norms)
        dict(name="append_token_64", op="append", n_seq=64, prefix=8192, rows=1, heads=32, kv_heads=8, d=128,
             dtype="bf16", norm=True, pick=3),
        # the 254 suffix rows of a turn over 1668 cached tokens (7B heads, no norms)
        dict(name="append_turn_254", op="append", n_seq=1, prefix=1668, rows=254, heads=28, kv_heads=4, d=128,
             dtype="bf16", norm=False, pick=0),
        # prompts of three conversations, ragged, from the start of their pages and from inside them
        dict(name="append_prompts_3", op="append", n_seq=3, prefix=1000, rows=4099, heads=32, kv_heads=8, d=128,
             dtype="bf16", norm=True, pick=4),
        # one new token after a short first turn
        dict(name="attend_token_1", op="attend", n_seq=1, prefix=726, rows=1, heads=28, kv_heads=4, d=128,
             dtype="bf16", pick=0),
        # a token of each of 64 conversations of ragged lengths
        dict(name="attend_token_64", op="attend", n_seq=64, prefix=8191, rows=1, heads=32, kv_heads=8, d=128,
             dtype="bf16", pick=5),
        # one token over two long documents
        dict(name="attend_long_2", op="attend", n_seq=2, prefix=131070, rows=1, heads=28, kv_heads=4, d=128,
             dtype="bf16", pick=0),
        # speculative verify: four conversations, eight rows each, over 15360 cached tokens
        dict(name="attend_verify_4", op="attend", n_seq=4, prefix=15360, rows=8, heads=28, kv_heads=4, d=128,
             dtype="bf16", pick=0),
        # the 254 suffix rows of a turn over 1668 cached tokens
        dict(name="attend_turn_254", op="attend", n_seq=1, prefix=1668, rows=254, heads=28, kv_heads=4, d=128,
             dtype="bf16", pick=0),
        # long suffixes of two conversations over long histories
        dict(name="attend_prompts_2", op="attend", n_seq=2, prefix=14001, rows=2047, heads=32, kv_heads=8, d=128,
             dtype="bf16", pick=6),
        # one-token, verify and prompt rows in one batch, 64-wide heads in fp16
        dict(name="attend_mixed_d64", op="attend", n_seq=12, prefix=4000, rows=120, heads=8, kv_heads=2, d=64,
             dtype="fp16", pick=7),
    ]


HEADS = [(28, 4, 128), (32, 8, 128), (16, 8, 128), (8, 2, 64), (6, 2, 128), (8, 2, 128), (4, 1, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    pick = rng.randrange(1, 1 << 20)
    if op == "plan":
        return dict(op=op, n_seq=_log(rng, 2, 512), prefix=_log(rng, 256, 8192), rows=_log(rng, 1, 16), pick=pick)
    heads, kv_heads, d = rng.choice(HEADS)
    c = dict(op=op, heads=heads, kv_heads=kv_heads, d=d, dtype=rng.choice(["bf16", "bf16", "fp16"]), pick=pick)
    if op == "append":
        rows = _log(rng, 1, 4096)
        return dict(c, n_seq=_log(rng, 1, max(1, min(64, 8192 // rows))), prefix=_log(rng, 1, 8192), rows=rows,
                    norm=rng.random() < 0.5)
    kind = rng.choice(["token", "verify", "suffix"])
    if kind == "token":
        prefix = _log(rng, 1, 131072)
        return dict(c, n_seq=_log(rng, 1, max(1, min(64, 500000 // prefix))), prefix=prefix, rows=1)
    if kind == "verify":
        prefix = _log(rng, 1, 16384)
        return dict(c, n_seq=_log(rng, 1, 16), prefix=prefix, rows=rng.randint(2, 8))
    prefix = _log(rng, 1, 8192)
    return dict(c, n_seq=_log(rng, 1, 4), prefix=prefix, rows=_log(rng, 9, 1024))


def _lengths(case):
    """(cached tokens, new rows) of each sequence.  pick = 0: all as long as the case says; otherwise ragged, the
    first one the longest."""
    n = case["n_seq"]
    if case["pick"] == 0:
        return [case["prefix"]] * n, [case["rows"]] * n
    r = random.Random(case["pick"])
    prefix = [case["prefix"]] + [r.randint(0, case["prefix"]) for _ in range(n - 1)]
    rows = [case["rows"]] + [r.randint(1, case["rows"]) for _ in range(n - 1)]
    return prefix, rows


def _plan_steps(case):
    """Two steps of a scheduler, keep and add of each sequence.  First the finished conversations (one in eight)
    leave and the others cut their rejected drafts; then those places take new prompts and the others new rows."""
    prefix, rows = _lengths(case)
    done = [b % 8 == 0 for b in range(len(rows))]
    leave = ([0 if e else p for p, e in zip(prefix, done)], [0] * len(rows))
    admit = (leave[0], [max(1, p // 8) if e else r for p, r, e in zip(prefix, rows, done)])
    return leave, admit


def _pages(n):
    return -(-n // PAGE)


def work(case):
    if case["op"] == "plan":
        (keep0, add0), (keep, add) = _plan_steps(case)
        moved = sum(abs(_pages(k + a) - _pages(k)) for k, a in zip(keep, add))
        n = len(keep)
        # both steps: keep, add and the lengths in, lengths and row offsets out; each moved page leaves and comes back
        # (table and free list); the rows' position, sequence and slot, for the longest rows that the case has
        return {"bytes": 2 * 20 * n + 2 * 8 * moved + 12 * sum(add), "flops": 0}
    prefix, rows = _lengths(case)
    H, Hkv, d = case["heads"], case["kv_heads"], case["d"]
    kv_row = 2 * Hkv * (d // 2 + 2 * d // GROUP)
    if case["op"] == "append":
        n = sum(rows)
        # q, k, v in; rotated q, the 4-bit rows and their values out; the rows' cosines and sines
        return {"bytes": n * ((2 * H + 4 * Hkv) * d * 2 + kv_row + 4 * d), "flops": n * (H + Hkv) * d * 8}
    n = sum(rows)
    seen = sum(m * p + m * (m + 1) // 2 for p, m in zip(prefix, rows))
    return {"bytes": sum(p + m for p, m in zip(prefix, rows)) * kv_row + 2 * n * H * d * 2,
            "flops": 4 * H * d * seen}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _kv_rows(case, g, n):
    """k and v of n tokens as a projection leaves them: a few loud channels in k, quiet v."""
    Hkv, d, T = case["kv_heads"], case["d"], DTYPES[case["dtype"]]
    loud = 0.5 + 1.5 * torch.rand(Hkv, d, device=DEV, generator=g)
    k = torch.randn(n, Hkv, d, device=DEV, generator=g).mul_(loud).to(T)
    v = torch.randn(n, Hkv, d, device=DEV, generator=g).mul_(0.5).to(T)
    return k, v


def _append_inputs(case, seed):
    g = _gen(seed)
    prefix, rows = _lengths(case)
    H, Hkv, d, T = case["heads"], case["kv_heads"], case["d"], DTYPES[case["dtype"]]
    n = sum(rows)
    k, v = _kv_rows(case, g, n)
    q = torch.randn(n, H, d, device=DEV, generator=g).mul_(1.5).to(T)
    # one row of the projection's output holds q, k and v
    qkv = torch.cat([q.view(n, -1), k.view(n, -1), v.view(n, -1)], 1)
    gains = [None, None]
    if case["norm"]:
        gains = [(0.5 + torch.rand(d, device=DEV, generator=g)).to(T) for _ in range(2)]
    return qkv, gains


def _attend_inputs(case, seed):
    g = _gen(seed)
    prefix, rows = _lengths(case)
    k, v = _kv_rows(case, g, sum(prefix) + sum(rows))
    q = torch.randn(sum(rows), case["heads"], case["d"], device=DEV, generator=g).mul_(1.5).to(DTYPES[case["dtype"]])
    return q, k, v


def _handle(case, prefix, rows, pages):
    from prefix_reused_prefill_gb300 import PagedKv, paged_config
    plan = case["op"] == "plan"
    return PagedKv(paged_config(
        n_pages=max(1, pages), n_layers=1, n_q_heads=1 if plan else case["heads"],
        n_kv_heads=1 if plan else case["kv_heads"], head_dim=64 if plan else case["d"],
        max_seqs=len(rows), max_len=max(1, max(p + m for p, m in zip(prefix, rows))),
        max_rows=sum(prefix) + sum(rows) + 8, act="bf16" if plan else case["dtype"], rope_theta=THETA,
        norm_eps=EPS), device=DEV)


def _angles(n, d):
    """cos and sin of each position's angles, in 64 bits."""
    inv = THETA ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cos(a), torch.sin(a)


def prepare(case, seed):
    if case["op"] == "plan":
        steps = _plan_steps(case)
        r = random.Random(seed)
        # the case gives the longest histories and the most rows; the batch is padded to them
        keep = [k - r.randint(0, k // 2) for k in steps[0][0]]
        add = [a - r.randint(0, a // 2) for a in steps[1][1]]
        rows = sum(steps[1][1])
        most = [k + a for k, a in zip(*steps[1])]
        pages, width = sum(_pages(t) for t in most) + 7, _pages(max(most))
        s = dict(op="plan", rows=rows, keep=_ints(keep), none=_ints([0] * len(keep)), add=_ints(add))
        if own:
            s["pg"] = _handle(case, *steps[1], pages)
            s["pg"].kvr_page_plan(s["none"], s["keep"], sum(keep))
            return s
        s["state"] = dict(table=torch.full((len(keep), width), -1, dtype=torch.int32, device=DEV),
                          lens=_ints([0] * len(keep)), count=_ints([pages]),
                          free=torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=DEV))
        _plan(s["state"], s["none"], s["keep"], sum(keep))
        return s
    prefix, rows = _lengths(case)
    pages = sum(_pages(p + m) for p, m in zip(prefix, rows)) + 3
    total = [p + m for p, m in zip(prefix, rows)]
    if case["op"] == "append":
        qkv, gains = _append_inputs(case, seed)
        H, Hkv, d = case["heads"], case["kv_heads"], case["d"]
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([H * d, Hkv * d, Hkv * d], 1))
        s = dict(op="append", q=q, k=k, v=v, norm_q=gains[0], norm_k=gains[1])
        if own:
            s["pg"] = _handle(case, prefix, rows, pages)
            s["pg"].kvr_page_plan(_ints([0] * len(rows)), _ints(prefix), sum(prefix))
            s["pg"].kvr_page_plan(_ints(prefix), _ints(rows), sum(rows))
            return s
        s["cos"], s["sin"] = _angles(max(total), d)
        s["pos"] = torch.cat([torch.arange(p, p + m, device=DEV) for p, m in zip(prefix, rows)])
        return s
    q, k, v = _attend_inputs(case, seed)
    s = dict(op="attend", q=q)
    if own:
        s["pg"] = _handle(case, prefix, rows, pages)
        s["pg"].kvr_page_plan(_ints([0] * len(rows)), _ints(total), sum(total))
        s["pg"].kvr_page_append(0, None, k, v, rotate=False)
        s["pg"].kvr_page_plan(_ints(prefix), _ints(rows), sum(rows), max(rows))
        return s
    n, width = len(rows), max(_pages(t) for t in total)
    order = torch.randperm(pages, device=DEV, generator=_gen(seed))
    count = torch.tensor([_pages(t) for t in total], device=DEV)
    first = count.cumsum(0) - count
    j = torch.arange(width, device=DEV)
    s["table"] = torch.where(j < count[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], 0)
    at = torch.cat([s["table"][b, torch.arange(t, device=DEV) // PAGE] * PAGE + torch.arange(t, device=DEV) % PAGE
                    for b, t in enumerate(total)])
    for name, x in (("k", k), ("v", v)):
        code, scale = _quantise(x.float())
        code = (code.to(torch.int16) + 8).to(torch.uint8).flatten(-2)
        pool = torch.zeros(pages * PAGE, case["kv_heads"], case["d"] // 2, dtype=torch.uint8, device=DEV)
        pool[at] = code[..., 0::2] | (code[..., 1::2] << 4)
        s[name] = pool.unflatten(0, (pages, PAGE))
        pool = torch.zeros(pages * PAGE, case["kv_heads"], case["d"] // GROUP, dtype=torch.float16, device=DEV)
        pool[at] = scale.to(torch.float16).squeeze(-1)
        s[name + "_scale"] = pool.unflatten(0, (pages, PAGE))
    s["lens"], s["m"] = _ints(total), _ints(rows)
    s["row_seq"] = torch.repeat_interleave(torch.arange(n, device=DEV), s["m"])
    s["row_i"] = torch.cat([torch.arange(m, device=DEV) for m in rows])
    s["m_max"] = max(rows)
    return s


# --------------------------------------------------------------------------- plain forms
def _plan(s, keep, add, rows):
    table, lens, free, count = s["table"], s["lens"], s["free"], s["count"]
    j = torch.arange(table.shape[1], device=DEV)
    held, need = ((x + PAGE - 1) // PAGE for x in (lens, keep + add))
    drop = (j >= need[:, None]) & (j < held[:, None])
    take = (j >= held[:, None]) & (j < need[:, None])
    top = count + drop.sum()
    # the released pages go on the stack, the last of them first; the taken ones come off its top
    rank = drop.flatten().cumsum(0).view_as(drop)
    more = torch.cat([free, free.new_zeros(1)])
    more[torch.where(drop, top - rank, free.numel()).long().flatten()] = table.flatten()
    free = more[:-1]
    rank = take.flatten().cumsum(0).view_as(take)
    table = torch.where(take, free[torch.where(take, top - rank, 0).long()], torch.where(drop, -1, table))
    s["table"], s["free"], s["lens"], s["count"] = table, free, keep + add, (top - take.sum()).to(torch.int32)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)]).to(torch.int32)
    r = torch.arange(rows, dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(cu[1:], r, right=True).clamp(max=add.numel() - 1)
    pos = keep[seq] + r - cu[seq]
    page = (pos // PAGE).clamp(max=table.shape[1] - 1)
    slot = table[seq, page.long()] * PAGE + pos % PAGE
    fill = r >= cu[-1]
    s["cu"] = cu
    s["row_seq"], s["row_pos"], s["row_slot"] = (torch.where(fill, -1, x).to(torch.int32) for x in (seq, pos, slot))


def _quantise(x):
    """codes and scales of groups of 32, x [..., d] in 32 bits."""
    g = x.unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1, keepdim=True) / 7).to(torch.float16).clamp(max=8188).float()
    return torch.where(s > 0, torch.round(g / s), 0).clamp(-8, 7), s


def _values(x):
    """What the cache holds for rows x [..., d] of the model's type."""
    c, s = _quantise(x.float())
    return (c * s).flatten(-2).to(x.dtype)


def _rotated(x, gain, cos, sin, wide):
    """Norm (where there is a gain) and rotation, rounded once to the type of x."""
    y = x.to(wide)
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * gain.to(wide)
    a, b = y.chunk(2, -1)
    c, s = cos.to(wide)[:, None], sin.to(wide)[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


def _dense(codes, scale, table):
    """The pages of each sequence, in order, as 32-bit values [n][kv heads][tokens][d]."""
    c, s = codes[table], scale[table]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() - 8
    x = (c.unflatten(-1, (-1, GROUP)) * s.float()[..., None]).flatten(-2)
    return x.flatten(1, 2).transpose(1, 2)


def _attend(s):
    q = s["q"]
    H, d = q.shape[1:]
    k, v = _dense(s["k"], s["k_scale"], s["table"]), _dense(s["v"], s["v_scale"], s["table"])
    n, Hkv, length = k.shape[:3]
    rows = q.new_zeros(n, s["m_max"], H, d, dtype=torch.float32)
    rows[s["row_seq"], s["row_i"]] = q.float()
    rows = rows.unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4)          # [n][kv heads][group][rows][d]
    p = (rows.flatten(2, 3) @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).unflatten(2, (H // Hkv, s["m_max"]))
    last = (s["lens"] - s["m"])[:, None] + torch.arange(s["m_max"], device=DEV)
    seen = torch.arange(length, device=DEV) <= last[..., None]                # [n][rows][tokens]
    p = p.masked_fill_(~seen[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (H // Hkv, s["m_max"])) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[s["row_seq"], s["row_i"]].to(q.dtype)


def run(s):
    if s["op"] == "plan":
        if own:
            pg = s["pg"]
            pg.kvr_page_plan(s["keep"], s["none"], s["rows"])
            pg.kvr_page_plan(s["keep"], s["add"], s["rows"])
            t = pg.state
            return dict(table=t.table, lens=t.lens, free=t.free, count=t.count, cu=t.cu, row_seq=t.row_seq[:s["rows"]],
                        row_pos=t.row_pos[:s["rows"]], row_slot=t.row_slot[:s["rows"]])
        t = s["state"]
        _plan(t, s["keep"], s["none"], s["rows"])
        _plan(t, s["keep"], s["add"], s["rows"])
        return dict(t)
    if s["op"] == "append":
        if own:
            pg = s["pg"]
            q = pg.kvr_page_append(0, s["q"], s["k"], s["v"], s["norm_q"], s["norm_k"])
            k, v = pg.kvr_page_read(0)
            return dict(q=q, k=k, v=v)
        cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
        # k in 64 bits: a value next to the border of two codes must not fall on the other side
        return dict(q=_rotated(s["q"], s["norm_q"], cos, sin, torch.float32),
                    k=_values(_rotated(s["k"], s["norm_k"], cos, sin, torch.float64)), v=_values(s["v"]))
    if own:
        return s["pg"].kvr_page_attend(0, s["q"])
    return _attend(s)


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_cache(x):
    """What the cache stands for, for one head's tokens x [tokens][d], group by group."""
    x = x.double()
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], GROUP):
        part = x[..., g:g + GROUP]
        top = part.abs().max(-1, keepdim=True).values
        s = (top / 7).half().double().clamp(max=8188.0)
        code = torch.clamp(torch.round(part / torch.where(s == 0, torch.ones_like(s), s)), -8, 7)
        out[..., g:g + GROUP] = torch.where(s == 0, torch.zeros_like(code), code * s)
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    prefix, rows = _lengths(case)
    H, Hkv, d, T = case["heads"], case["kv_heads"], case["d"], DTYPES[case["dtype"]]
    if case["op"] == "append":
        qkv, (gq, gk) = _append_inputs(case, seed)
        x = qkv.double().view(len(qkv), H + 2 * Hkv, d)
        pos = torch.tensor([p + i for p, m in zip(prefix, rows) for i in range(m)], dtype=torch.float64, device=DEV)
        half = d // 2
        freq = torch.tensor([THETA ** (-2.0 * j / d) for j in range(half)], dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.ones(len(pos), half, dtype=torch.float64, device=DEV), pos[:, None] * freq)[:, None]
        out = {}
        for name, y, gain in (("q", x[:, :H], gq), ("k", x[:, H:H + Hkv], gk)):
            if gain is not None:
                y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) / d + EPS) * gain.double()
            z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
            out[name] = torch.cat([z.real, z.imag], -1)
        out["k"] = _exact_cache(out["k"].to(T))
        out["v"] = _exact_cache(qkv.view(len(qkv), H + 2 * Hkv, d)[:, H + Hkv:])
        return out
    q, k, v = _attend_inputs(case, seed)
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    at = row = 0
    for p, m in zip(prefix, rows):
        see = torch.arange(p + m, device=DEV)[None] <= torch.arange(p, p + m, device=DEV)[:, None]
        for h in range(Hkv):
            kk, vv = _exact_cache(k[at:at + p + m, h]), _exact_cache(v[at:at + p + m, h])
            for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                score = q[row:row + m, g].double() @ kk.T / math.sqrt(d)
                out[row:row + m, g] = torch.softmax(score.masked_fill(~see, -math.inf), -1) @ vv
        at, row = at + p + m, row + m
    return out
