"""The operators around the paged cache's sparse path, restated in float64 (numpy).

Not source-page operations: the norm and rotation of heads on their way into the cache, the 8-bit
digest of a page's keys, the bound on scores that is made from it and the lists of pages that
follow.  Whole numbers here are exact, so the digests and lists have one answer.
"""
from __future__ import annotations

import numpy as np


def rotate(x, pos, weight, eps, inv_freq, interleaved=False, scale=1.0):
    """x [n, heads, D] at positions pos [n] (float64): (normed and rotated rows, the size that an
    error of a factor is relative to: what each result is the sum of)."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    size = np.abs(x)
    if inv_freq is None or not len(inv_freq):
        return x, size
    R = 2 * len(inv_freq)
    # position times frequency exactly enough anywhere: the product's rounding is taken along
    hi = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    cos, sin = scale * np.cos(hi)[:, None], scale * np.sin(hi)[:, None]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = x.copy()
    with np.errstate(invalid="ignore"):
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
    both = (size[..., a] + size[..., b]) * abs(scale)
    size[..., a] = size[..., b] = both
    return y, size


def exponent127(a):
    """The least e in [-50, 50] with a 2^-e <= 127 (0 where a is 0)."""
    a = np.asarray(a, np.float64)
    m, p = np.frexp(np.where(a > 0, a, 1.0))          # a = m 2^p, 0.5 <= m < 1
    return np.where(a > 0, np.clip(p - 7 + (m > 127 / 128), -50, 50), 0).astype(int)


def digest(k):
    """k [keys, D] of one page and head: (lo, hi [D], e)."""
    e = int(exponent127(np.where(np.isfinite(k), np.abs(k), 0.0).max(initial=0.0)))
    some = ~np.isnan(k).all(0) if len(k) else np.zeros(k.shape[1], bool)
    lo = np.where(some, np.where(np.isnan(k), np.inf, k).min(0, initial=np.inf), 0.0)
    hi = np.where(some, np.where(np.isnan(k), -np.inf, k).max(0, initial=-np.inf), 0.0)
    lo, hi = np.floor(np.ldexp(lo, -e)), np.ceil(np.ldexp(hi, -e))
    return np.clip(lo, -127, 127).astype(int), np.clip(hi, -127, 127).astype(int), e


def whole(q):
    """Rows q [..., D] -> (whole numbers in [-127, 127], exponents)."""
    e = exponent127(np.where(np.isfinite(q), np.abs(q), 0.0).max(-1))
    x = np.ldexp(q, -e[..., None])
    return np.clip(np.rint(np.where(np.isnan(x), 0.0, x)), -127, 127), e


def bound(q, lo, hi, e):
    """Rows q [n, D] against digests lo, hi [pages, D], e [pages]: the largest row's score of each."""
    w, eq = whole(q)
    s = np.maximum(w, 0) @ hi.T.astype(np.float64) + np.minimum(w, 0) @ lo.T.astype(np.float64)
    return np.ldexp(np.ldexp(s, eq[:, None]).max(0), e)


def span(p0, n, page_size, n_sink, n_local):
    """Pages of a block of n queries from position p0 on: (end of the sinks, first local page, first
    own page, last own page), None if it sees nothing."""
    p1, pc = p0 + n - 1, max(p0, 0)
    if n < 1 or p1 < 0:
        return None
    own0, own1 = pc // page_size, p1 // page_size
    first = max(0, own0 - n_local)
    return min(n_sink, first), first, own0, own1


def choose(score, s0, first, keep):
    """The `keep` best of pages s0 .. first - 1 (score: all pages'), ties to the earlier, ascending."""
    order = sorted(range(s0, first), key=lambda p: (-score[p], p))
    return sorted(order[:keep])


def select(q, p0, page_size, score_of, keep, n_sink, n_local, q_block):
    """The blocks of one sequence's chunk q [n, H_q, D] from position p0 on; score_of(rows, head)
    gives the scores of the pages: [(first row, rows, [list of each KV head], keys)]."""
    out = []
    for i in range(0, len(q), q_block):
        n = min(q_block, len(q) - i)
        at = span(p0 + i, n, page_size, n_sink, n_local)
        if at is None:
            out.append((i, n, None, 0))
            continue
        s0, first, own0, own1 = at
        lists = []
        for h in range(score_of.heads):
            picked = range(s0, first) if keep >= first - s0 else choose(score_of(q[i:i + n], h), s0, first, keep)
            lists.append(list(range(s0)) + list(picked) + list(range(first, own1 + 1)))
        pc = max(p0 + i, 0)
        before = s0 + min(keep, first - s0) + own0 - first
        out.append((i, n, lists, before * page_size + pc % page_size + (p0 + i + n - pc)))
    return out
