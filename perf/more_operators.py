"""Measured cases of a decoder layer's attention: what lies between its q, k, v
projections and its o projection, for prompts and for decode steps.

  rope       q and k heads normalised and rotated to their positions, k and v
             appended to a paged cache (bf16, or e4m3 codes with one fp32
             scale for each token and head)
  decode     attention of one new token per sequence, or of the few rows that
             verify drafted tokens, over such a cache
  prefill    causal attention over packed prompts of different lengths, keys
             of a cached prefix before them

`run` computes a case in elementary torch operations, or, with `own`, through
this repository's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
WORKSPACE = 64 << 20      # one zero-filled scratch buffer, as a serving program keeps for all its calls
EPS = 1e-6
BASE = 10000.0            # of the rotation's frequencies


def listed():
    return [
        # one stream's new token: latency alone
        {"name": "rope one token", "op": "rope", "T": 1, "Hq": 16, "Hk": 4, "D": 128, "rot": 128, "interleaved": False,
         "norm": True, "e4m3": False, "P": 16, "strided": False, "far": False, "k_out": False},
        # 48 streams that verify 4 drafted tokens each, into an 8-bit cache
        {"name": "rope verify step e4m3", "op": "rope", "T": 240, "Hq": 16, "Hk": 4, "D": 128, "rot": 128, "interleaved": True,
         "norm": False, "e4m3": True, "P": 32, "strided": False, "far": False, "k_out": False},
        # a long document's tokens out of one fused q, k, v product, far positions, rotated k wanted beside the cache
        {"name": "rope prompt", "op": "rope", "T": 16385, "Hq": 16, "Hk": 4, "D": 128, "rot": 128, "interleaved": False,
         "norm": True, "e4m3": False, "P": 64, "strided": True, "far": True, "k_out": True},
        # one stream at the longest prompt and answer of the decode step's model
        {"name": "decode one stream", "op": "decode", "B": 1, "T": 1, "L": 2304, "Hq": 16, "Hk": 4, "D": 128, "P": 16, "e4m3": False,
         "window": 0, "ragged": False},
        # 48 streams at all stages of their answers
        {"name": "decode B=48", "op": "decode", "B": 48, "T": 1, "L": 2304, "Hq": 16, "Hk": 4, "D": 128, "P": 16, "e4m3": False,
         "window": 0, "ragged": True},
        # the same streams verifying 4 drafted tokens each, 8-bit cache, an odd longest length
        {"name": "decode verify step e4m3", "op": "decode", "B": 48, "T": 5, "L": 4099, "Hq": 16, "Hk": 4, "D": 128, "P": 32,
         "e4m3": True, "window": 0, "ragged": True},
        # one stream over a very long context
        {"name": "decode long context", "op": "decode", "B": 1, "T": 1, "L": 131071, "Hq": 16, "Hk": 4, "D": 128, "P": 64,
         "e4m3": False, "window": 0, "ragged": False},
        # a batch over long contexts
        {"name": "decode B=32 long", "op": "decode", "B": 32, "T": 1, "L": 32768, "Hq": 16, "Hk": 4, "D": 128, "P": 64,
         "e4m3": False, "window": 0, "ragged": False},
        # one sentence
        {"name": "prefill one sentence", "op": "prefill", "B": 1, "L": 77, "prefix": 0, "Hq": 16, "Hk": 4, "D": 128, "window": 0,
         "ragged": False},
        # the prompts of a batch of requests, packed
        {"name": "prefill packed prompts", "op": "prefill", "B": 48, "L": 2304, "prefix": 0, "Hq": 16, "Hk": 4, "D": 128, "window": 0,
         "ragged": True},
        # later chunks of long documents through a layer with a sliding window, small heads
        {"name": "prefill window, prefix", "op": "prefill", "B": 5, "L": 1999, "prefix": 2048, "Hq": 16, "Hk": 8, "D": 64,
         "window": 1024, "ragged": True},
        # a long document
        {"name": "prefill long prompt", "op": "prefill", "B": 1, "L": 16384, "prefix": 0, "Hq": 16, "Hk": 4, "D": 128, "window": 0,
         "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "prefill", "prefill"])
    Hq, Hk = rng.choice([(16, 4), (16, 4), (16, 8), (32, 8), (8, 8), (14, 2), (12, 1)])
    D = rng.choice([128, 128, 64])
    if op == "rope":
        T = _log_int(rng, 1, 8192)
        return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rng.choice([D, D, D // 2, 0]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.6, "e4m3": rng.random() < 0.4, "P": rng.choice([16, 32, 64, 128]),
                "strided": rng.random() < 0.4, "far": rng.random() < 0.4, "k_out": rng.random() < 0.4}
    if op == "decode":
        B = _log_int(rng, 1, 64)
        L = _log_int(rng, 1, min(131072, (1 << 19) // B))
        return {"op": op, "B": B, "T": rng.choice([1, 1, 1, 2, 3, 5, 8]), "L": L, "Hq": Hq, "Hk": Hk, "D": D,
                "P": rng.choice([16, 32, 64, 128]), "e4m3": rng.random() < 0.4,
                "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), "ragged": rng.random() < 0.6}
    B = _log_int(rng, 1, 64)
    L = _log_int(rng, 1, min(8192, 32768 // B))
    return {"op": op, "B": B, "L": L, "prefix": rng.choice([0, 0, _log_int(rng, 1, 1024)]), "Hq": Hq, "Hk": Hk, "D": D,
            "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), "ragged": rng.random() < 0.6}


def _lengths(case):
    """Lengths spread over 1 .. L (the first is L), the same for every seed."""
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    return [max(1, round(case["L"] * (1 - (0.6180339887498949 * b) % 1.0))) for b in range(case["B"])]


def _seen(n, keys, window):
    """Pairs of a query and a key that it sees: n queries, the last of them at the last key."""
    first = keys - n + 1
    if window and window < keys:
        short = max(0, min(n, window - first + 1))          # queries that see all keys before them
        return sum(range(first, first + short)) + (n - short) * window
    return n * (first + keys) // 2


def work(case):
    op, Hq, Hk, D = case["op"], case["Hq"], case["Hk"], case["D"]
    if op == "rope":
        T = case["T"]
        b = T * (Hq + 2 * Hk) * D * 2 + T * Hq * D * 2 + T * 12 + (2 * D * 2 if case["norm"] else 0) + case["rot"] * 2
        b += T * 2 * Hk * (D + 4 if case["e4m3"] else 2 * D) + (T * Hk * D * 2 if case["k_out"] else 0)
        return {"bytes": b, "flops": T * (Hq + Hk) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    lengths = _lengths(case)
    if op == "decode":
        T, window = case["T"], case["window"]
        row = D + 4 if case["e4m3"] else 2 * D
        b = 2 * case["B"] * T * Hq * D * 2
        f = 0
        for n in lengths:
            t = min(T, n)
            keys = min(n, window + t - 1) if window else n
            b += keys * Hk * row * 2 + 4 * -(-keys // case["P"]) + 4
            f += 4 * D * Hq * _seen(t, n, window)
        return {"bytes": b, "flops": f}
    tokens = sum(lengths)
    b = 2 * tokens * Hq * D * 2 + 2 * (tokens + case["B"] * case["prefix"]) * Hk * D * 2 + 8 * (case["B"] + 1)
    return {"bytes": b, "flops": sum(4 * D * Hq * _seen(n, n + case["prefix"], case["window"]) for n in lengths)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=g, device="cuda")  # noqa: E731
    op, Hq, Hk, D = case["op"], case["Hq"], case["Hk"], case["D"]
    state = {"op": op, "workspace": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if op == "rope":
        T, P, rot = case["T"], case["P"], case["rot"]
        # a head's channels differ in size, as projections' outputs do
        loud = torch.exp(0.5 * randn(Hq + 2 * Hk, D))
        qkv = (randn(T, Hq + 2 * Hk, D) * loud).to(torch.bfloat16)
        parts = (qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:])
        state["q"], state["k"], state["v"] = parts if case["strided"] else [t.contiguous() for t in parts]
        state["q_norm"] = state["k_norm"] = None
        if case["norm"]:
            state["q_norm"], state["k_norm"] = (1 + 0.2 * randn(D)).to(torch.bfloat16), (1 + 0.2 * randn(D)).to(torch.bfloat16)
        state["inv_freq"] = None
        if rot:
            state["inv_freq"] = (BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        start = 1000000 if case["far"] else 0
        state["positions"] = (torch.arange(T, device="cuda") % 4096 + start).to(torch.int32)
        # tokens fill slots of a cache that holds other sequences too; one in 32 is not kept
        pages = -(-T // P) + 3
        slots = perm(pages * P)[:T]
        state["slots"] = torch.where(rand(T) < 1 / 32, -1, slots).to(torch.int64)
        state["interleaved"], state["k_out"] = case["interleaved"], case["k_out"]
        k, v = randn(pages, Hk, P, D), randn(pages, Hk, P, D)
        if case["e4m3"]:
            state["cache"] = (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), rand(pages, Hk, P), rand(pages, Hk, P))
        else:
            state["cache"] = (k.to(torch.bfloat16), v.to(torch.bfloat16))
        return state
    lengths = _lengths(case)
    state["window"] = case["window"]
    state["scale"] = torch.tensor(D ** -0.5, dtype=torch.float32).item()
    if op == "decode":
        B, T, P = case["B"], case["T"], case["P"]
        # normalised heads: scores of a few units, some keys louder
        state["q"] = (randn(B, T, Hq, D) * 1.5).to(torch.bfloat16)
        need = [-(-n // P) for n in lengths]
        pages = sum(need) + 2
        k = torch.empty(pages, Hk, P, D, dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        for at in range(0, pages, 4096):
            part = k[at:at + 4096]
            part.copy_(randn(*part.shape) * torch.exp(0.3 * randn(part.shape[0], Hk, P, 1)))
            v[at:at + 4096].copy_(randn(*part.shape))
        if case["e4m3"]:
            ks, vs = (t.abs().amax(-1).float() / E4M3_MAX for t in (k, v))
            state["cache"] = tuple((t.float() / s[..., None]).to(torch.float8_e4m3fn) for t, s in ((k, ks), (v, vs))) + (ks, vs)
        else:
            state["cache"] = (k, v)
        width = -(-max(lengths) // P)
        taken = torch.tensor(need, device="cuda")
        at = torch.arange(width, device="cuda")
        first = torch.nn.functional.pad(taken.cumsum(0)[:-1], (1, 0))
        order = perm(pages)
        held = at < taken[:, None]
        state["table"] = torch.where(held, order[(first[:, None] + at).clamp_max(pages - 1)], -1).to(torch.int32).contiguous()
        state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        # rows that a sequence has no draft for, or no token yet
        state["n_new"] = torch.tensor([min(T, n) for n in lengths], dtype=torch.int32, device="cuda") if T > 1 else None
        if T > 1:
            some = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            state["n_new"] = torch.where(rand(B) < 0.3, torch.minimum(some, state["n_new"]), state["n_new"])
        return state
    tokens, keys = sum(lengths), sum(lengths) + case["B"] * case["prefix"]
    state["q"] = (randn(tokens, Hq, D) * 1.5).to(torch.bfloat16)
    state["k"] = (randn(keys, Hk, D) * torch.exp(0.3 * randn(keys, Hk, 1))).to(torch.bfloat16)
    state["v"] = randn(keys, Hk, D).to(torch.bfloat16)
    state["lengths"] = lengths
    state["prefix"] = case["prefix"]
    state["starts"] = _offsets(lengths)
    state["key_starts"] = _offsets([n + case["prefix"] for n in lengths]) if case["prefix"] else None
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _heads(x, norm, s):
    """Normalised and rotated heads of x, in float32."""
    h = x.float()
    if norm is not None:
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * norm.float()
    if s["inv_freq"] is None:
        return h
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    rot = 2 * s["inv_freq"].shape[0]
    part = h[..., :rot]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, h[..., rot:]), -1)


def _rope(s):
    q = _heads(s["q"], s["q_norm"], s).to(torch.bfloat16)
    k, v = _heads(s["k"], s["k_norm"], s), s["v"].float()
    cache = s["cache"]
    P = cache[0].shape[2]
    kept = s["slots"] >= 0
    slot = s["slots"][kept]
    page, at = slot // P, slot % P
    for i, h in enumerate((k[kept], v[kept])):
        if len(cache) == 4:
            top = h.abs().amax(-1)
            codes = h * E4M3_MAX / torch.where(top > 0, top, 1.0)[..., None]
            cache[i].view(torch.uint8)[page, :, at] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            cache[i + 2][page, :, at] = top / E4M3_MAX
        else:
            cache[i][page, :, at] = h.to(torch.bfloat16)
    return (q, *cache, k.to(torch.bfloat16)) if s["k_out"] else (q, *cache)


def _decode(s):
    q, table, lengths = s["q"], s["table"].long(), s["lengths"].long()
    B, T, Hq, D = q.shape
    Hk, P = s["cache"][0].shape[1:3]
    G, L = Hq // Hk, table.shape[1] * P
    at = table.clamp_min(0)
    k, v = (t[at].float() for t in s["cache"][:2])                      # [B, pages, Hk, P, D]
    if len(s["cache"]) == 4:
        k, v = (t * w[at][..., None] for t, w in zip((k, v), s["cache"][2:]))
    k, v = (t.transpose(1, 2).reshape(B, Hk, L, D) for t in (k, v))
    rows = q.float().view(B, T, Hk, G, D).transpose(1, 2).reshape(B, Hk, T * G, D)
    score = torch.matmul(rows, k.transpose(2, 3).contiguous()).view(B, Hk, T, G, L) * s["scale"]
    new = s["n_new"].long() if s["n_new"] is not None else torch.full_like(lengths, T)
    i, j = torch.arange(T, device=q.device), torch.arange(L, device=q.device)
    end = lengths[:, None] - new[:, None] + i + 1                       # keys that row i sees end here
    seen = (j < end[..., None]) & (i < new[:, None])[..., None] & (table >= 0).repeat_interleave(P, 1)[:, None]
    if s["window"]:
        seen = seen & (j >= end[..., None] - s["window"])
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    y = torch.matmul(p.view(B, Hk, T * G, L), v).view(B, Hk, T, G, D)
    return y.transpose(1, 2).reshape(B, T, Hq, D).to(torch.bfloat16)


_ROWS = 2048      # queries whose scores are held at a time


def _prefill(s):
    q, window = s["q"], s["window"]
    Hq, D = q.shape[1:]
    Hk = s["k"].shape[1]
    G = Hq // Hk
    out = torch.empty_like(q)
    q0 = k0 = 0
    for n in s["lengths"]:
        m = n + s["prefix"]
        k = s["k"][k0:k0 + m].float().permute(1, 2, 0).contiguous()     # [Hk, D, m]
        v = s["v"][k0:k0 + m].float().transpose(0, 1).contiguous()      # [Hk, m, D]
        for r0 in range(0, n, _ROWS):
            r = min(_ROWS, n - r0)
            end = s["prefix"] + r0 + r                                  # keys that these rows see
            rows = q[q0 + r0:q0 + r0 + r].float().view(r, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * r, D)
            score = torch.matmul(rows, k[:, :, :end].contiguous()).view(Hk, G, r, end) * s["scale"]
            i = torch.arange(end - r, end, device=q.device)[:, None]
            j = torch.arange(end, device=q.device)
            seen = j <= i
            if window:
                seen = seen & (j > i - window)
            score = torch.where(seen, score, -math.inf)
            e = torch.exp(score - score.amax(-1, keepdim=True))
            p = e / e.sum(-1, keepdim=True)
            y = torch.matmul(p.view(Hk, G * r, end), v[:, :end]).view(Hk, G, r, D)
            out[q0 + r0:q0 + r0 + r] = y.permute(2, 0, 1, 3).reshape(r, Hq, D).to(torch.bfloat16)
        q0, k0 = q0 + n, k0 + m
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        import bit_weight_only_q4g128_amd as q4
        if op == "rope":
            q, k = q4.rope_cache(state["q"], state["k"], state["v"], positions=state["positions"], inv_freq=state["inv_freq"],
                                 q_norm=state["q_norm"], k_norm=state["k_norm"], eps=EPS, interleaved=state["interleaved"],
                                 cache=state["cache"], slots=state["slots"], k_out=True if state["k_out"] else None)
            return (q, *state["cache"], k) if state["k_out"] else (q, *state["cache"])
        if op == "decode":
            return q4.attention_decode(state["q"], state["cache"], state["table"], state["lengths"], n_new=state["n_new"],
                                       scale=state["scale"], window=state["window"], workspace=state["workspace"])
        return q4.attention_prefill(state["q"], state["k"], state["v"], state["starts"], key_starts=state["key_starts"],
                                    scale=state["scale"], window=state["window"])
    return {"rope": _rope, "decode": _decode, "prefill": _prefill}[op](state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_nearest(t):
    """The nearest e4m3 value, ties to even: steps of 2^(e - 3) from 2^e on, of
    2^-9 below 2^-6."""
    m, _ = torch.frexp(t)      # t / m is a power of two, exactly
    step = (torch.where(m == 0, 1.0, t) / torch.where(m == 0, 1.0, m) / 16).abs().clamp_min(2.0 ** -9)
    return torch.round(t / step) * step


def _exact_heads(x, norm, s):
    h = x.double()
    if norm is not None:
        h = norm.double() * h / torch.sqrt(h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS)
    if s["inv_freq"] is None:
        return h
    out = h.clone()
    half = s["inv_freq"].shape[0]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        angle = (s["positions"].double() * s["inv_freq"][i].double())[:, None]
        out[..., a] = h[..., a] * torch.cos(angle) - h[..., b] * torch.sin(angle)
        out[..., b] = h[..., a] * torch.sin(angle) + h[..., b] * torch.cos(angle)
    return out


def _exact_rope(s):
    q, k, v = _exact_heads(s["q"], s["q_norm"], s), _exact_heads(s["k"], s["k_norm"], s), s["v"].double()
    cache = [t.double() for t in s["cache"]]
    pages, Hk, P = cache[0].shape[:3]
    # the tokens' rows behind the cache's, one row per slot picked from both
    slots = torch.arange(pages * P, device=q.device)
    source = torch.full((pages * P + 1,), -1, dtype=torch.int64, device=q.device)
    T = q.shape[0]
    source[torch.where(s["slots"] < 0, pages * P, s["slots"])] = torch.arange(T, device=q.device)
    source = source[:-1]
    for i, h in enumerate((k, v)):
        if len(cache) == 4:
            top = h.abs().max(-1).values
            scale = top / E4M3_MAX
            h = torch.where(top[..., None] > 0, _e4m3_nearest(h / top[..., None] * E4M3_MAX), 0.0)
            flat = cache[i + 2].transpose(1, 2).reshape(pages * P, Hk)
            cache[i + 2] = torch.where((source < 0)[:, None], flat[slots], scale[source.clamp_min(0)]).view(pages, P, Hk).transpose(1, 2)
        flat = cache[i].transpose(1, 2).reshape(pages * P, Hk, -1)
        cache[i] = torch.where((source < 0)[:, None, None], flat, h[source.clamp_min(0)]).view(pages, P, Hk, -1).transpose(1, 2)
    cache = [t.contiguous() for t in cache]
    return (q, *cache, k) if s["k_out"] else (q, *cache)


def _exact_rows(q, k, v, end, scale, window):
    """softmax(q k^T scale) v of one key head: rows q [r, D], row i of them sees keys [end_i - window, end_i)."""
    z = torch.mm(q, k.t().contiguous()) * scale
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    hidden = j >= end[:, None]
    if window:
        hidden |= j < (end - window)[:, None]
    z.masked_fill_(hidden, -math.inf)
    return torch.mm(torch.exp(z - torch.logsumexp(z, 1, keepdim=True)), v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    Hq, Hk, D, window = case["Hq"], case["Hk"], case["D"], case["window"]
    G = Hq // Hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        for b, n in enumerate(_lengths(case)):
            new = int(s["n_new"][b]) if s["n_new"] is not None else case["T"]
            pages = s["table"][b, :-(-n // case["P"])].long()
            row = [t[pages].transpose(0, 1).flatten(1, 2)[:, :n].double() for t in s["cache"]]
            if case["e4m3"]:
                row = [row[0] * row[2][..., None], row[1] * row[3][..., None]]
            end = (n - new + 1 + torch.arange(new, device="cuda")).repeat_interleave(G)
            for h in range(Hk):
                rows = s["q"][b, :new, h * G:(h + 1) * G].double().reshape(new * G, D)
                y[b, :new, h * G:(h + 1) * G] = _exact_rows(rows, row[0][h], row[1][h], end, s["scale"], window).view(new, G, D)
        return y
    q0 = k0 = 0
    for n in s["lengths"]:
        m = n + case["prefix"]
        for h in range(Hq):
            k, v = s["k"][k0:k0 + m, h // G].double(), s["v"][k0:k0 + m, h // G].double()
            for r0 in range(0, n, 4096):
                r = min(4096, n - r0)
                end = case["prefix"] + r0 + 1 + torch.arange(r, device="cuda")
                top = case["prefix"] + r0 + r
                y[q0 + r0:q0 + r0 + r, h] = _exact_rows(s["q"][q0 + r0:q0 + r0 + r, h].double(), k[:top], v[:top], end, s["scale"], window)
        q0, k0 = q0 + n, k0 + m
    return y
