"""The paged key/value cache and its attention, restated in float64 (numpy).

Not a source-page operation.  Rows are quantised to FP8 E4M3 with one power of two per
(token, head); a chunk's row at position p attends the keys j <= p with j > p - n_stream (any,
when n_stream is None) or j < n_sink.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
E_MIN, E_MAX, E_NAN = -116, 119, 128


def e4m3_grid() -> np.ndarray:
    """The magnitudes of the codes 0 .. 126, ascending."""
    sub = [m / 512.0 for m in range(8)]
    norm = [(1.0 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array((sub + norm)[:127])


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """float64 -> E4M3 codes: nearest, ties to the even code, saturating; NaN -> 0x7F."""
    g = e4m3_grid()
    a = np.minimum(np.abs(y), E4M3_MAX)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.searchsorted(g, a, side="left")           # g[hi - 1] < a <= g[hi]
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - g[lo], g[hi] - a
    c = np.where(d_lo < d_hi, lo, hi)
    c = np.where((d_lo == d_hi) & (lo != hi), np.where(lo % 2 == 0, lo, hi), c)
    c = np.where(np.isnan(y), 0x7F, c + np.where(np.signbit(y), 128, 0))
    return c.astype(np.uint8)


def quantise(x: np.ndarray):
    """Rows x [..., D] (float64 values of bf16 elements) -> (codes [..., D], exponents e; E_NAN
    for a row that holds a NaN)."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    m, p = np.frexp(np.where(a > 0, a, 1.0))          # a = m 2^p, 0.5 <= m < 1
    e = p - 9 + (m > 0.875)                           # smallest e with a <= 448 * 2^e
    e = np.where(a > 0, np.clip(e, E_MIN, E_MAX), 0)
    nan = np.isnan(x).any(-1)
    e = np.where(nan, 0, e)
    with np.errstate(invalid="ignore"):
        return e4m3_codes(np.ldexp(x, -e[..., None])), np.where(nan, E_NAN, e)


def dequantise(codes: np.ndarray, e: np.ndarray) -> np.ndarray:
    g = np.append(e4m3_grid(), np.nan)
    x = np.ldexp(g[codes & 127] * np.where(codes > 127, -1.0, 1.0), e[..., None])
    return np.where(e[..., None] == E_NAN, np.nan, x)


def attend(q, k, v, p0: int, n_sink: int, n_stream, scale: float, lost=None):
    """q [n, H_q, D] at positions p0 .. over k, v [T, H_kv, D] (all float64): (out, lse, spread,
    size), where spread = sum_j w_j |v_j| (what a relative error of the weights can move) and
    size = the largest scale * sum_d |q_d k_d| of a head (what a rounding of the dot product is
    relative to).  lost [T] marks keys that are not there (their page is no page).  A score that is
    NaN or plus infinity (a NaN in the query or in a key that it sees, say) makes its row NaN, out
    and lse; one of minus infinity has weight 0.  Infinities and NaN of values reach only who sees
    them."""
    n, H_q, D = q.shape
    T, H_kv, _ = k.shape
    G = H_q // H_kv
    p = p0 + np.arange(n)[:, None]
    j = np.arange(T)[None]
    see = (j <= p) if n_stream is None else (j <= p) & ((j > p - n_stream) | (j < n_sink))
    if lost is not None:
        see = see & ~lost[None]
    out, spread = np.zeros((n, H_q, D)), np.zeros((n, H_q, D))
    lse, size = np.full((n, H_q), -np.inf), np.zeros((n, H_q))
    for h in range(H_q):
        kk, vv = k[:, h // G], v[:, h // G]
        with np.errstate(invalid="ignore"):
            s = scale * (q[:, h] @ kk.T)
        nan = (see & ~(s < np.inf)).any(1)
        s = np.where(see & (s < np.inf), s, -np.inf)
        m = s.max(1, initial=-np.inf)
        some = m > -np.inf
        w = np.exp(s - np.where(some, m, 0.0)[:, None])
        l = w.sum(1)
        w /= np.where(some, l, 1.0)[:, None]
        lse[some, h] = m[some] + np.log(l[some])
        bad = ~np.isfinite(vv)
        vz = np.where(bad, 0.0, vv)
        out[:, h], spread[:, h] = w @ vz, w @ np.abs(vz)
        for x in np.flatnonzero(bad.any(1)):          # only the rows that see the key
            out[see[:, x] & some, h] += np.where(bad[x], vv[x], 0.0)
        out[nan, h], lse[nan, h] = np.nan, np.nan
        ab = scale * (np.abs(np.nan_to_num(q[:, h], posinf=0, neginf=0)) @
                      np.abs(np.nan_to_num(kk, posinf=0, neginf=0)).T)
        size[:, h] = np.where(see, ab, 0.0).max(1, initial=0.0)
    return out, lse, spread, size
