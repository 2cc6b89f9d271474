"""Plain CPU reference of the draft-and-verify operators: 8-bit block-scaled
quantisation and products, and the verification of drafted tokens.  NumPy in
fp64, row by row from the definitions; shares no code with the HIP path."""
from __future__ import annotations

import numpy as np

from .reference import bf16_value, e4m3fn_value

BLOCK = 128
E4M3_MAX = 448.0


def e4m3_nearest(t) -> np.ndarray:
    """fp64 -> the nearest finite e4m3 value, ties to the even code (|t| <= 448;
    NaN stays): from 2^e on steps of 2^(e-3), below 2^-6 of 2^-9."""
    t = np.asarray(t, np.float64)
    a = np.abs(t)
    with np.errstate(invalid="ignore"):
        e = np.clip(np.frexp(np.where(np.isfinite(a), a, 1.0))[1] - 1, -6, 8)
    step = np.ldexp(1.0, e - 3)
    return np.rint(t / step) * step


def fp8_quantize(x_bits, up_bits=None):
    """(code values fp64 [M, K] (NaN where x, or x * up in fp32, is not finite), scale fp64
    [M, ceil(K / 128)] before its rounding)."""
    h = bf16_value(x_bits).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if up_bits is not None:
            top = h * bf16_value(up_bits).astype(np.float64)
            h = np.where(np.abs(top) < 2.0 ** 128, top, np.nan) / (1.0 + np.exp(-h))
        h = np.where(np.isfinite(h), h, np.nan)
    M, K = h.shape
    codes = np.empty_like(h)
    scale = np.zeros((M, -(-K // BLOCK)))
    for g in range(scale.shape[1]):
        part = h[:, g * BLOCK:(g + 1) * BLOCK]
        top = np.max(np.where(np.isnan(part), 0.0, np.abs(part)), axis=1)
        scale[:, g] = top / E4M3_MAX
        safe = np.where(top > 0, top, 1.0)[:, None]
        codes[:, g * BLOCK:(g + 1) * BLOCK] = e4m3_nearest(part * E4M3_MAX / safe)
    return codes, scale


def fp8_gemm(x_codes, x_scale, w_codes, w_scale, residual_bits=None):
    """y fp64 [M, N] of e4m3 bytes [M, K], [N, K] and fp32 scales."""
    xv, wv = e4m3fn_value(x_codes).astype(np.float64), e4m3fn_value(w_codes).astype(np.float64)
    xs, ws = np.asarray(x_scale, np.float64), np.asarray(w_scale, np.float64)
    M, N = xv.shape[0], wv.shape[0]
    rows = np.arange(N) // BLOCK
    y = np.zeros((M, N))
    for g in range(xs.shape[1]):
        cols = slice(g * BLOCK, (g + 1) * BLOCK)
        y += (xv[:, cols] @ wv[:, cols].T) * xs[:, g:g + 1] * ws[rows, g][None, :]
    if residual_bits is not None:
        y = y + bf16_value(residual_bits)
    return y


def _distribution(logits, temperature):
    """Probabilities of fp64 logits; zeros if the largest is not finite."""
    z = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    top = z.max()
    if not np.isfinite(top):
        return np.zeros_like(z)
    e = np.exp((z - top) / temperature)
    return e / e.sum()


def _draw(weights, order, u):
    """First entry of `order` whose running weight exceeds u * total; -1 without
    any weight."""
    w = weights[order]
    total = w.sum()
    if not total > 0:
        return -1
    c = np.cumsum(w)
    over = np.flatnonzero((c > u * c[-1]) & (w > 0))
    return int(order[over[0]] if len(over) else order[np.flatnonzero(w > 0)[-1]])


def _verify(p_of, q_of, order_of, draft, n, u, D):
    """One sequence.  p_of(i), q_of(i): probabilities over the vocabulary."""
    n = min(max(int(n), 0), D)
    prob = np.zeros(D)
    ok = []
    for i in range(n):
        p, q, d = p_of(i), q_of(i), int(draft[i])
        pd = p[d] if 0 <= d < len(p) else 0.0
        qd = q[d] if 0 <= d < len(p) else 0.0
        prob[i] = min(1.0, pd / qd) if qd > 0 else float(pd > 0)
        ok.append(float(u[i]) * qd < pd)
    a = 0
    while a < n and ok[a]:
        a += 1
    p = p_of(a)
    rest = np.maximum(p - q_of(a), 0.0) if a < n else p
    if not rest.sum() > 0:
        rest = p
    token = np.full(D + 1, -1, np.int64)
    token[:a] = draft[:a]
    token[a] = _draw(rest, order_of(a), float(u[D]))
    return token, a, prob


def verify_topk(logit_bits, draft, u, draft_index, draft_prob, n_draft, temperature, top_k):
    """(token [B, D+1], count [B], accept probability fp64 [B, D])."""
    lg = bf16_value(logit_bits).astype(np.float64)
    lg = np.where(np.isnan(lg), -np.inf, lg)
    B, D1, V = lg.shape
    D = D1 - 1
    T = float(np.float32(temperature))
    outs = []
    for b in range(B):
        orders = {}

        def order_of(i):
            if i not in orders:
                orders[i] = np.lexsort((np.arange(V), -lg[b, i]))[:top_k]
            return orders[i]

        def p_of(i):
            p = np.zeros(V)
            p[order_of(i)] = _distribution(lg[b, i, order_of(i)], T)
            return p

        def q_of(i):
            q = np.zeros(V)
            if draft_index is None:
                if 0 <= draft[b, i] < V:
                    q[draft[b, i]] = 1.0
            else:
                for v, w in zip(draft_index[b, i], draft_prob[b, i]):
                    if 0 <= v < V:
                        q[v] += float(w)
            return q

        outs.append(_verify(p_of, q_of, order_of, draft[b], D if n_draft is None else n_draft[b], u[b], D))
    return tuple(np.stack([o[i] for o in outs]) for i in range(3))


def verify_full(logit_bits, draft, u, draft_logit_bits, n_draft, temperature):
    """(token [B, D+1], count [B], accept probability fp64 [B, D])."""
    lg = bf16_value(logit_bits).astype(np.float64)
    B, D1, V = lg.shape
    D = D1 - 1
    T = float(np.float32(temperature))
    dl = None if draft_logit_bits is None else bf16_value(draft_logit_bits).astype(np.float64)
    order = np.arange(V)
    outs = []
    for b in range(B):
        def q_of(i):
            if dl is not None:
                return _distribution(dl[b, i], T)
            q = np.zeros(V)
            if 0 <= draft[b, i] < V:
                q[draft[b, i]] = 1.0
            return q

        outs.append(_verify(lambda i: _distribution(lg[b, i], T), q_of, lambda i: order, draft[b],
                            D if n_draft is None else n_draft[b], u[b], D))
    return tuple(np.stack([o[i] for o in outs]) for i in range(3))
