"""Sampling and speculative sampling in 64 bits (test infrastructure): the definitions of include/kvr.h, a row at a
time and token by token where that is affordable."""
import math

import numpy as np


def row_distribution(x, temperature=1.0, top_k=0, min_p=0.0, top_p=1.0):
    """(order of the kept tokens, their weights), None for a row without a distribution."""
    x = np.asarray(x, np.float64)
    t = float(temperature)
    if np.isnan(x).any() or x.max() == -np.inf or math.isnan(min_p) or math.isnan(top_p):
        return None
    if not (t == 0 or 2.0 ** -64 <= t <= 2.0 ** 64):
        return None
    order = np.lexsort((np.arange(len(x)), -x))
    s = x[order]
    if t == 0:
        w = np.zeros(len(x))
        w[0] = 1.0
    else:
        with np.errstate(invalid="ignore"):
            w = np.exp(np.where(s == s[0], 0.0, s - s[0]) / t)
    n = len(x)
    if top_k > 0:
        n = min(n, int(top_k))
    n = min(n, max(1, int((w >= min(float(min_p), 1.0)).sum())))
    if top_p < 1:
        run = np.cumsum(w[:n])
        need = float(top_p) * run[-1]
        n = min(n, 1 + int((run < need).sum()))
    return order[:n], w[:n]


def draw(order, w, u):
    run = np.cumsum(w)
    return int(order[min(int((run <= float(u) * run[-1]).sum()), len(order) - 1)])


def sample(x, u, **settings):
    """(token, probability, distribution) of one row."""
    d = row_distribution(x, **settings)
    p = np.zeros(len(x))
    if d is None or not 0 <= u < 1:
        return -1, 0.0, p
    order, w = d
    p[order] = w / w.sum()
    token = draw(order, w, u)
    return token, p[token], p


def accept(rows, tokens, u, u_next, q=None, **settings):
    """(drafts that stay, the token after them) of one sequence: rows [m][vocab], tokens [t0, d1 .. dk]."""
    m = len(rows)
    if m == 0:
        return 0, -1
    for i in range(m):
        d = row_distribution(rows[i], **settings)
        if d is None or not 0 <= u_next < 1:
            return i, -1
        order, w = d
        share = w / w.sum()
        if i == m - 1:
            return i, draw(order, share, u_next)
        if not 0 <= u[i] < 1:
            return i, -1
        draft = int(tokens[i + 1])
        inside = 0 <= draft < len(rows[i])
        here = order == draft
        qd = 1.0 if q is None or not inside else float(q[i][draft])
        if inside and u[i] * qd < share[here].sum():
            continue
        rest = share - (here.astype(np.float64) if q is None else np.asarray(q[i], np.float64)[order])
        rest = np.maximum(rest, 0.0)
        return i, draw(order, rest if rest.sum() > 0 else share, u_next)
