"""Plain CPU reference of a decoder layer's attention: heads normalised,
rotated and appended to a paged cache, and causal attention.  NumPy in fp64,
token by token and row by row from the definitions; shares no code with the HIP
path."""
from __future__ import annotations

import numpy as np

from .step import E4M3_MAX, e4m3_nearest


def rope_heads(x, positions=None, inv_freq=None, norm=None, eps=1e-6, interleaved=False):
    """fp64 [T, H, D] of heads x: normalised by `norm` (None: not), pairs turned
    by positions[t] * inv_freq[i]."""
    h = np.array(x, np.float64)
    if norm is not None:
        h = np.asarray(norm, np.float64) * h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if inv_freq is None:
        return h
    half = len(inv_freq)
    out = h.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        f = (np.asarray(positions, np.float64) * float(inv_freq[i]))[:, None]
        out[..., a] = h[..., a] * np.cos(f) - h[..., b] * np.sin(f)
        out[..., b] = h[..., b] * np.cos(f) + h[..., a] * np.sin(f)
    return out


def e4m3_heads(h):
    """(code values fp64, scale fp64 [...] before its rounding) of heads [..., D]."""
    h = np.where(np.isfinite(h), h, np.nan)
    top = np.max(np.where(np.isnan(h), 0.0, np.abs(h)), axis=-1)
    return e4m3_nearest(h * E4M3_MAX / np.where(top > 0, top, 1.0)[..., None]), top / E4M3_MAX


def attend(q, k, v, end, scale, window=0):
    """One key head: rows q [r, D] over keys k and values v [n, D], row i seeing
    keys [max(0, end[i] - window), end[i]) (window 0: from the first).  Returns
    (y, sum of p |v|, largest sum of |q k| scale of a seen key), all fp64; rows
    that see nothing are 0."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    y, mass, score = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1])), np.zeros(len(q))
    for i in range(len(q)):
        hi = min(max(int(end[i]), 0), len(k))
        lo = max(0, int(end[i]) - window) if window else 0
        if lo >= hi:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            z = (k[lo:hi] @ q[i]) * scale
            score[i] = (np.abs(k[lo:hi]) @ np.abs(q[i])).max() * scale
            if z.max() == -np.inf:
                continue
            p = np.exp(z - z.max())
            p /= p.sum()
            y[i] = p @ v[lo:hi]
            mass[i] = p @ np.abs(v[lo:hi])
    return y, mass, score


def paged(cache, table, length, head):
    """Keys (or values, or their scales) of one sequence and head in the cache
    [pages, Hk, page_size, ...]; the mask of those whose page there is."""
    pages, _, P = cache.shape[:3]
    n = max(0, min(int(length), len(table) * P))
    out = np.zeros((n,) + cache.shape[3:], np.float64)
    held = np.zeros(n, bool)
    for j in range(n):
        page = int(table[j // P])
        if 0 <= page < pages:
            out[j], held[j] = cache[page, head, j % P], True
    return out, held
