"""The paged 4-bit cache, evaluated plainly in float64.

TEST INFRASTRUCTURE ONLY (see the package header).

* ``Tables``: the page tables and the free stack, one sequence after the other;
* ``quantise``: groups of 32, s = min(fp16(max|x| / 7), 8188), codes rounded to
  even and clamped to [-8, 7];
* ``norm_rotate``: per-head RMSNorm and rotate-half RoPE at one position;
* ``attend``: one row over the tokens that it sees.

Pins (tests/test_oracle_pages.py): hand-worked tables, codes of exact halves,
saturation and tiny groups, rotation by a quarter turn.
"""
from __future__ import annotations

from typing import List, Sequence

import numpy as np

PAGE = 64
GROUP = 32


class Tables:
    def __init__(self, n_pages: int, max_seqs: int, max_len: int):
        self.free = list(range(n_pages - 1, -1, -1))   # top of the stack last
        self.pages: List[List[int]] = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.max_len = max_len
        self.rows: List[tuple] = []                     # (sequence, position, slot)

    def plan(self, keep: Sequence[int], add: Sequence[int], rows: int, max_add: int = 0) -> bool:
        """False: refused, nothing changed and no rows."""
        self.rows = []
        bound = max_add if 0 < max_add <= rows else rows
        need = []
        for b, (k, a) in enumerate(zip(keep, add)):
            if not (0 <= k <= self.lens[b] and 0 <= a <= bound and k + a <= self.max_len):
                return False
            need.append(-(-(k + a) // PAGE))
        if sum(add) > rows:
            return False
        released = sum(max(0, len(self.pages[b]) - n) for b, n in enumerate(need))
        taken = sum(max(0, n - len(self.pages[b])) for b, n in enumerate(need))
        if taken > len(self.free) + released:
            return False
        out = []
        for b, n in enumerate(need):
            out += self.pages[b][n:]
            del self.pages[b][n:]
        self.free += out[::-1]
        for b, n in enumerate(need):
            while len(self.pages[b]) < n:
                self.pages[b].append(self.free.pop())
        for b, (k, a) in enumerate(zip(keep, add)):
            self.lens[b] = k + a
            for pos in range(k, k + a):
                self.rows.append((b, pos, self.pages[b][pos // PAGE] * PAGE + pos % PAGE))
        return True


def quantise(x: np.ndarray):
    """codes [..., d/32, 32] and scales [..., d/32, 1] (float64) of x [..., d]; a
    group that is not finite has the scale NaN."""
    g = np.asarray(x, dtype=np.float64)
    g = g.reshape(*g.shape[:-1], g.shape[-1] // GROUP, GROUP)
    top = np.max(np.abs(g), axis=-1, keepdims=True)
    with np.errstate(all="ignore"):
        s = np.minimum(np.float16(top / 7).astype(np.float64), 8188.0)
        s = np.where(np.isfinite(top), s, np.nan)
        c = np.clip(np.round(np.where(s > 0, g / np.where(s > 0, s, 1.0), 0.0)), -8, 7)
    return c, s


def values(x: np.ndarray) -> np.ndarray:
    """What the cache stands for."""
    c, s = quantise(x)
    return (c * s).reshape(x.shape)


def norm_rotate(x: np.ndarray, pos: int, theta: float, gain=None, eps: float = 0.0, rotate: bool = True) -> np.ndarray:
    """x [heads][d]."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gain
    if not rotate:
        return x
    d = x.shape[-1]
    ang = pos * np.power(float(theta), -2.0 * np.arange(d // 2) / d)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], axis=-1)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """q [heads][d] over k, v [kv heads][tokens][d]: (o [heads][d], sum of weight * |v|)."""
    H, Hkv = q.shape[0], k.shape[0]
    o, mag = np.empty_like(q), np.empty_like(q)
    for h in range(H):
        j = h // (H // Hkv)
        s = scale * (k[j] @ q[h])
        w = np.exp(s - np.max(s))
        w /= np.sum(w)
        o[h], mag[h] = w @ v[j], w @ np.abs(v[j])
    return o, mag
