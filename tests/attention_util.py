"""Checks of the attention operators against the fp64 oracle, and the bounds
they use.

Heads (rope_cache).  h = x w / sqrt(mean x^2 + eps) in fp32: the mean of D
squares is off by at most (D / 8 + 5) 2^-23 (a lane adds 8, then lanes meet in
pairs; each square and each sum rounds once), the root's reciprocal by 2^-22,
two products by 2^-24 each: under 2^-18 in all.  sin and cos are off by 2^-22 and
by the angle's own error: positions' turns are fp64, with two roundings of
2^-53 of their number.  The turned pair adds two products: within
    (2^-18 + 2^-21 + 2 pi |turns| 2^-51) (|a| + |b|)
of its value, which is rounded to bf16 once (2^-8 of it).  e4m3 codes are half a
step off, 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it, and the
scale as the head's largest value.

Attention.  A score's D products are exact and added in fp32: it is off by
D 2^-23 of the sum of their magnitudes (2^-23, not 2^-24, for the matrix cores
may truncate), and by 4 2^-23 of its own for the scales; a weight by that (times
1, e^x = 1 + x) and 2^-21 for the exponential.  A weight is rounded to bf16 (2^-8)
before it multiplies its value, with an 8-bit value's scale before that (2^-23);
sums of n weights and products are off by n 2^-23 of their magnitudes, and
joined parts by a few more: with P = sum p |v|,
    |y - y_ref| <= (2^-8 + 2 (D + 4) 2^-23 max_j scale sum |q k_j| + 2^-20 + n 2^-22) P + 2^-8 |y_ref|.
The middle term counts twice: in the weight and in their sum.
"""
import numpy as np
import torch

import oracle

F = 2.0 ** -23


def values(t):
    return t.detach().cpu().to(torch.float64).numpy()


def within(got, want, bound, what):
    got = values(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    bad = ~(np.abs(got - want) <= bound) & ~nan & ~(got == want)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first {i}: {got[i]!r}, not {want[i]!r} within {np.broadcast_to(bound, got.shape)[i]!r}")


def attention_bound(y, mass, score, n, D):
    return (2.0 ** -8 + 2 * (D + 4) * F * score[..., None] + 2.0 ** -20 + n * 2 * F) * mass + 2.0 ** -8 * np.abs(y) + 1e-37


def rope_bound(x, positions, inv_freq, norm, eps, interleaved):
    """The bound of rope_heads before the rounding, as an array."""
    h = np.abs(oracle.rope_heads(x, None, None, norm, eps))
    if inv_freq is None:
        return 2.0 ** -18 * h
    half = len(inv_freq)
    both = h.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        turns = np.abs(np.asarray(positions, np.float64) * float(inv_freq[i]))[:, None]
        both[..., a] = both[..., b] = (h[..., a] + h[..., b]) * (1 + (2.0 ** -21 + turns * 2.0 ** -51) / 2.0 ** -18)
    return 2.0 ** -18 * both


def check_decode(got, q, cache, table, lengths, n_new, scale, window):
    """got [B, T, Hq, D] of CPU inputs."""
    B, T, Hq, D = q.shape
    Hk = cache[0].shape[1]
    G = Hq // Hk
    got, q = values(got), values(q)
    parts = [values(t) for t in cache]
    for b in range(B):
        n = T if n_new is None else min(max(int(n_new[b]), 0), T)
        length = min(max(int(lengths[b]), 0), table.shape[1] * parts[0].shape[2])
        end = np.repeat(length - n + 1 + np.arange(n), G)
        for h in range(Hk):
            (k, held), (v, _) = (oracle.paged(parts[i], table[b], length, h) for i in (0, 1))
            if len(parts) == 4:
                k = k * oracle.paged(parts[2], table[b], length, h)[0][:, None]
                v = v * oracle.paged(parts[3], table[b], length, h)[0][:, None]
            rows = q[b, :n, h * G:(h + 1) * G].reshape(n * G, D)
            y, mass, score = _attend_held(rows, k, v, held, end, scale, window)
            what = f"sequence {b} head {h}"
            within(got[b, :n, h * G:(h + 1) * G].reshape(n * G, D), y, attention_bound(y, mass, score, len(k), D), what)
        assert not got[b, n:].any() and not np.isnan(got[b, n:]).any(), f"sequence {b}: rows behind its tokens"


def _attend_held(rows, k, v, held, end, scale, window):
    if held.all():
        return oracle.attend(rows, k, v, end, scale, window)
    # keys without a page take no part: row by row, over those that it sees
    out = [np.zeros((len(rows), v.shape[1] if v.ndim > 1 else rows.shape[1])) for _ in range(2)] + [np.zeros(len(rows))]
    at = np.arange(len(k))
    for i in range(len(rows)):
        see = held & (at < end[i]) & ((at >= end[i] - window) if window else True)
        r = oracle.attend(rows[i:i + 1], k[see], v[see], [int(see.sum())], scale)
        for o, x in zip(out, r):
            o[i] = x[0]
    return out


def check_prefill(got, q, k, v, starts, key_starts, scale, window):
    T, Hq, D = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    got, q, k, v = (values(t) for t in (got, q, k, v))
    key_starts = starts if key_starts is None else key_starts
    for b in range(len(starts) - 1):
        (q0, q1), (k0, k1) = (int(starts[b]), int(starts[b + 1])), (int(key_starts[b]), int(key_starts[b + 1]))
        end = k1 - k0 - (q1 - q0) + 1 + np.arange(q1 - q0)
        for h in range(Hq):
            y, mass, score = oracle.attend(q[q0:q1, h], k[k0:k1, h // G], v[k0:k1, h // G], end, scale, window)
            within(got[q0:q1, h], y, attention_bound(y, mass, score, k1 - k0, D), f"sequence {b} head {h}")
