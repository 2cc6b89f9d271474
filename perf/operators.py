"""Measured cases of the operators of a draft-and-verify decode step.

A step that verifies drafted tokens runs the target model on several rows per
sequence at once (every drafted position and the one after it), so its
projections leave the few-row regime of plain decoding: activations are
quantised to 8 bits and multiplied with 8-bit weights, and the head's logits
then decide which drafted tokens stand.

  quantize      bf16 activations, or silu(gate) * up, to e4m3 codes with one
                fp32 scale for each 128 columns of a row
  gemm          y = RN_bf16(sum over 128-column blocks g of
                xs[m, g] * ws[n / 128, g] * sum_k x[m, k] w[n, k]  (+ residual)),
                one product or a group of products of one batch
  verify_topk   rejection sampling of drafted tokens against the target's
                top-k distribution, the draft's given as top-k lists
  verify_full   the same against the whole row's softmax, the draft's given as
                logits

`run` computes a case in elementary torch operations, or, with `own`, through
this repository's entry points.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
WORKSPACE = 64 << 20      # one zero-filled scratch buffer, as a serving program keeps for all its calls


def listed():
    return [
        # one decode row's hidden state before its projections: latency alone
        {"name": "quantize one row", "op": "quantize", "M": 1, "K": 2048, "gated": False},
        # the MLP activation of 48 sequences with 4 drafted tokens each
        {"name": "quantize gated M=240", "op": "quantize", "M": 240, "K": 8192, "gated": True},
        # a ragged prompt's hidden states, a column count that ends inside a block
        {"name": "quantize ragged prompt", "op": "quantize", "M": 4099, "K": 2000, "gated": False},
        # the MLP activation of a long prompt
        {"name": "quantize gated prompt", "op": "quantize", "M": 8192, "K": 8192, "gated": True},
        # one sequence, down projection into the residual stream
        {"name": "gemm one row down", "op": "gemm", "M": 1, "K": 8192, "Ns": "2048", "residual": True},
        # a layer's input projections (q, k, v, gate, up) of 48 sequences, one token each
        {"name": "gemm layer M=48", "op": "gemm", "M": 48, "K": 2048, "Ns": "2048,512,512,8192,8192", "residual": False},
        # the head over 48 sequences with 4 drafted tokens each: an odd row count
        {"name": "gemm head M=240", "op": "gemm", "M": 240, "K": 2048, "Ns": "16385", "residual": False},
        # a long prompt through a wide layer
        {"name": "gemm prompt", "op": "gemm", "M": 8192, "K": 8192, "Ns": "8192", "residual": False},
        # one stream, 4 drafted audio tokens of the 2049-row codebook
        {"name": "verify top-k one stream", "op": "verify_topk", "B": 1, "D": 4, "V": 2049, "k": 30, "temperature": 0.8,
         "lists": True},
        # 48 streams over the full head
        {"name": "verify top-k B=48", "op": "verify_topk", "B": 48, "D": 4, "V": 16385, "k": 30, "temperature": 0.8,
         "lists": True},
        # one stream over the full head, whole distributions
        {"name": "verify full one stream", "op": "verify_full", "B": 1, "D": 4, "V": 16385, "temperature": 0.8, "lists": True},
        # a batch over a text-sized vocabulary, 7 drafted tokens each
        {"name": "verify full B=32", "op": "verify_full", "B": 32, "D": 7, "V": 131072, "temperature": 1.0, "lists": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "verify_topk", "verify_full"])
    if op == "quantize":
        return {"op": op, "M": _log_int(rng, 1, 8192), "K": 16 * _log_int(rng, 8, 512), "gated": rng.random() < 0.5}
    if op == "gemm":
        M = _log_int(rng, 1, 8192)
        K = 16 * rng.randint(8, 512) if rng.random() < 0.3 else 128 * _log_int(rng, 1, 64)
        count = rng.choice([1, 1, 2, 3, 5]) if M <= 256 else 1
        Ns = [_log_int(rng, 16, 8192) for _ in range(count)]
        return {"op": op, "M": M, "K": K, "Ns": ",".join(str(n) for n in Ns), "residual": rng.random() < 0.3}
    B, D = _log_int(rng, 1, 32), rng.randint(1, 7)
    t = rng.choice([0.5, 0.8, 1.0, 1.3])
    lists = rng.random() < 0.75
    if op == "verify_topk":
        V = _log_int(rng, 64, 30720)
        return {"op": op, "B": B, "D": D, "V": V, "k": rng.randint(1, 64), "temperature": t, "lists": lists}
    return {"op": op, "B": B, "D": D, "V": _log_int(rng, 512, 131072), "temperature": t, "lists": lists}


def _ns(case):
    return [int(n) for n in case["Ns"].split(",")]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * (5 if case["gated"] else 3) + 4 * case["M"] * _blocks(case["K"]), "flops": 4 * n}
    if op == "gemm":
        M, K, Ns = case["M"], case["K"], _ns(case)
        G = _blocks(K)
        b = M * K + 4 * M * G
        for N in Ns:
            b += N * K + 4 * _blocks(N) * G + M * N * (4 if case["residual"] else 2)
        return {"bytes": b, "flops": 2 * M * K * sum(Ns)}
    B, D, V = case["B"], case["D"], case["V"]
    rows = B * (D + 1) + (B * D if op == "verify_full" and case["lists"] else 0)
    b = rows * V * 2 + B * (12 * D + 8 * (D + 1))
    if op == "verify_topk" and case["lists"]:
        b += 8 * B * D * case["k"]
    return {"bytes": b, "flops": 4 * rows * V}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _fp32(value):
    """The value as the fp32 argument that the entry points take."""
    return torch.tensor(value, dtype=torch.float32).item()


def _quantised(t, rows):
    """e4m3 codes and fp32 scales of blocks of `rows` x 128 of a float32 matrix."""
    n, k = t.shape
    pad = torch.nn.functional.pad(t, (0, -k % BLOCK, 0, -n % rows))
    b = pad.view(-1, rows, _blocks(k), BLOCK)
    amax = b.abs().amax((1, 3)).clamp_min(1e-30)
    q = (b * (E4M3_MAX / amax)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(pad.shape)[:n, :k].contiguous(), (amax / E4M3_MAX).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    op = case["op"]
    state = {"op": op, "workspace": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")}
    if op in ("quantize", "gemm"):
        M, K = case["M"], case["K"]
        # hidden states: normal values, one column in 64 a few times larger, as
        # trained activations have
        loud = torch.where(rand(K) < 1 / 64, 8.0, 1.0)
        if op == "quantize":
            state["x"] = (randn(M, K) * loud).to(torch.bfloat16)
            state["up"] = randn(M, K).to(torch.bfloat16) if case["gated"] else None
            return state
        x, xs = _quantised((randn(M, K) * loud).to(torch.bfloat16).float(), 1)
        state["tasks"] = []
        for N in _ns(case):
            w, ws = _quantised(randn(N, K) * 0.02 * torch.exp(0.5 * randn(N, 1)), BLOCK)
            r = randn(M, N).to(torch.bfloat16) if case["residual"] else None
            state["tasks"].append((x, xs, w, ws, r))
        return state
    B, D, V = case["B"], case["D"], case["V"]
    T = _fp32(case["temperature"])
    state["temperature"] = T
    # the draft's logits are the target's with noise; the drafted tokens are
    # drawn from the draft's distribution (its largest for drafts without one)
    target = randn(B, D + 1, V) * 2.5
    draft = (target[:, :D] + randn(B, D, V) * 0.7).to(torch.bfloat16)
    state["logits"] = target.to(torch.bfloat16)
    del target
    state["n_draft"] = torch.randint(0, D + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    state["n_draft"][rand(B) < 0.6] = D
    state["u"] = rand(B, D + 1).clamp_max(1 - 2.0 ** -24)
    state["draft_index"] = state["draft_prob"] = state["draft_logits"] = None
    if op == "verify_topk":
        k = state["top_k"] = case["k"]
        v, i = torch.sort(draft.float(), dim=-1, descending=True, stable=True)
        v, i = v[..., :k], i[..., :k]
        p = torch.softmax(v / T, -1)
        if case["lists"]:
            at = torch.multinomial(p.view(B * D, k), 1, generator=g).view(B, D, 1)
            state["draft_index"], state["draft_prob"] = i.to(torch.int32).contiguous(), p.contiguous()
        else:
            at = torch.zeros(B, D, 1, dtype=torch.int64, device="cuda")
        state["draft"] = i.gather(2, at)[..., 0].to(torch.int32).contiguous()
        return state
    if case["lists"]:
        noise = -torch.log(-torch.log(rand(B, D, V).clamp(1e-7, 1 - 1e-7)))
        state["draft"] = (draft.float() / T + noise).argmax(-1).to(torch.int32)
        state["draft_logits"] = draft
    else:
        state["draft"] = draft.float().argmax(-1).to(torch.int32)
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _quantize(x, up):
    h = x.float()
    if up is not None:
        h = h / (1 + torch.exp(-h)) * up.float()
    M, K = h.shape
    b = torch.nn.functional.pad(h, (0, -K % BLOCK)).view(M, -1, BLOCK)
    amax = b.abs().amax(-1)
    q = b * E4M3_MAX / torch.where(amax > 0, amax, 1.0)[..., None]
    return q.to(torch.float8_e4m3fn).view(M, -1)[:, :K].contiguous(), amax / E4M3_MAX


def _gemm(x, xs, w, ws, residual):
    M, K = x.shape
    N = w.shape[0]
    xf = x.float() * xs.repeat_interleave(BLOCK, 1)[:, :K]
    wf = w.float() * ws.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    y = xf @ wf.t()
    if residual is not None:
        y = y + residual.float()
    return y.to(torch.bfloat16)


def _decide(pd, qd, draft, n_draft, u):
    """Acceptance of the drafted tokens with target and draft probabilities pd,
    qd: (accepted count, min(1, p / q) of every drafted position)."""
    D = draft.shape[1]
    live = torch.arange(D, device=draft.device) < n_draft[:, None]
    ok = (u[:, :D].double() * qd < pd) & live
    count = ok.long().cumprod(1).sum(1)
    ratio = torch.where(qd > 0, pd / qd, (pd > 0).double()).clamp_max(1.0)
    return count, torch.where(live, ratio, 0.0).float()


def _drawn(p, q, u):
    """Position of the draw from max(p - q, 0), or from p where that is empty."""
    r = (p - q).clamp_min(0)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, p)
    c = r.cumsum(-1)
    return (c <= u.double()[:, None] * c[:, -1:]).sum(-1)


def _tokens(draft, count, new):
    at = torch.arange(draft.shape[1] + 1, device=draft.device)
    padded = torch.nn.functional.pad(draft.long(), (0, 1))
    t = torch.where(at < count[:, None], padded, torch.where(at == count[:, None], new[:, None], -1))
    return t.to(torch.int32), count.to(torch.int32)


def _verify_topk(s):
    B, D = s["draft"].shape
    v, i = torch.sort(s["logits"].float() + 0.0, dim=-1, descending=True, stable=True)
    v, i = v[..., : s["top_k"]].double(), i[..., : s["top_k"]]
    e = torch.exp((v - v[..., :1]) / s["temperature"])
    p = e / e.sum(-1, keepdim=True)
    d = s["draft"].long()
    if s["draft_index"] is not None:
        qi, qp = s["draft_index"].long(), s["draft_prob"].double()
    else:
        qi, qp = d[..., None], torch.ones(B, D, 1, dtype=torch.float64, device=d.device)
    pd = (p[:, :D] * (i[:, :D] == d[..., None])).sum(-1)
    qd = (qp * (qi == d[..., None])).sum(-1)
    count, ratio = _decide(pd, qd, s["draft"], s["n_draft"], s["u"])
    b, at = torch.arange(B, device=d.device), count.clamp_max(D - 1)
    ia, pa = i[b, count], p[b, count]
    qa = ((qi[b, at][:, None, :] == ia[:, :, None]) * qp[b, at][:, None, :]).sum(-1)
    qa = torch.where((count < s["n_draft"])[:, None], qa, 0.0)
    new = ia.gather(1, _drawn(pa, qa, s["u"][:, D])[:, None])[:, 0]
    return *_tokens(s["draft"], count, new), ratio


def _softmax64(logits, temperature):
    z = logits.double()
    e = torch.exp((z - z.amax(-1, keepdim=True)) / temperature)
    return e / e.sum(-1, keepdim=True)


def _verify_full(s):
    B, D = s["draft"].shape
    d = s["draft"].long()
    b = torch.arange(B, device=d.device)
    p = _softmax64(s["logits"], s["temperature"])
    pd = p[:, :D].gather(2, d[..., None])[..., 0]
    if s["draft_logits"] is not None:
        q = _softmax64(s["draft_logits"], s["temperature"])
        qd = q.gather(2, d[..., None])[..., 0]
    else:
        qd = torch.ones_like(pd)
    count, ratio = _decide(pd, qd, s["draft"], s["n_draft"], s["u"])
    at = count.clamp_max(D - 1)
    qa = q[b, at] if s["draft_logits"] is not None else (torch.arange(p.shape[2], device=d.device) == d[b, at][:, None]).double()
    qa = torch.where((count < s["n_draft"])[:, None], qa, 0.0)
    new = _drawn(p[b, count], qa, s["u"][:, D])
    return *_tokens(s["draft"], count, new), ratio


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        import bit_weight_only_q4g128_amd as q4
        if op == "quantize":
            return q4.fp8b128_quantize(state["x"], up=state["up"])
        if op == "gemm":
            return q4.fp8b128_gemm_grouped([(*t, None) for t in state["tasks"]], workspace=state["workspace"])
        if op == "verify_topk":
            return q4.verify_topk(state["logits"], state["draft"], state["u"], draft_index=state["draft_index"],
                                  draft_prob=state["draft_prob"], n_draft=state["n_draft"], temperature=state["temperature"],
                                  top_k=state["top_k"], workspace=state["workspace"])
        return q4.verify_full(state["logits"], state["draft"], state["u"], draft_logits=state["draft_logits"],
                              n_draft=state["n_draft"], temperature=state["temperature"], workspace=state["workspace"])
    if op == "quantize":
        return _quantize(state["x"], state["up"])
    if op == "gemm":
        return [_gemm(*t) for t in state["tasks"]]
    return _verify_topk(state) if op == "verify_topk" else _verify_full(state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_nearest(t):
    """The nearest e4m3 value, ties to even: steps of 2^(e - 3) from 2^e on, of
    2^-9 below 2^-6."""
    m, _ = torch.frexp(t)      # t / m is a power of two, exactly
    step = (torch.where(m == 0, 1.0, t) / torch.where(m == 0, 1.0, m) / 16).clamp_min(2.0 ** -9)
    return torch.round(t / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        h = s["x"].double()
        if s["up"] is not None:
            h = h * torch.sigmoid(h) * s["up"].double()
        M, K = h.shape
        codes = torch.empty_like(h)
        scale = torch.empty(M, _blocks(K), dtype=torch.float64, device=h.device)
        for g in range(_blocks(K)):
            cols = slice(g * BLOCK, min(K, g * BLOCK + BLOCK))
            top = h[:, cols].abs().max(1, keepdim=True).values
            scale[:, g] = top[:, 0] / E4M3_MAX
            codes[:, cols] = torch.where(top > 0, _e4m3_nearest(h[:, cols] * E4M3_MAX / top), 0.0)
        return codes, scale
    if op == "gemm":
        outs = []
        for x, xs, w, ws, r in s["tasks"]:
            y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
            rows = torch.arange(w.shape[0], device=x.device) // BLOCK
            for g in range(xs.shape[1]):
                cols = slice(g * BLOCK, min(x.shape[1], g * BLOCK + BLOCK))
                part = torch.mm(x[:, cols].double(), w[:, cols].double().t().contiguous())
                y += part * (xs[:, g].double()[:, None] * ws[rows, g].double()[None, :])
            outs.append(y if r is None else y + r.double())
        return outs
    B, D, V = case["B"], case["D"], case["V"]
    ratio = torch.zeros(B, D, dtype=torch.float64, device="cuda")
    T = s["temperature"]

    def log_mass(row):
        z = row.double() / T
        return z, torch.logsumexp(z, -1)

    for j in range(D):
        d = s["draft"][:, j].long()
        row = s["logits"][:, j]
        z, _ = log_mass(row)
        zd = z.gather(1, d[:, None])
        if op == "verify_topk":
            lower = torch.arange(V, device=d.device)[None, :] < d[:, None]
            before = ((z > zd) | ((z == zd) & lower)).sum(1)
            top = z.topk(case["k"], 1).values
            p = torch.where(before < case["k"], torch.exp(zd[:, 0] - torch.logsumexp(top, 1)), 0.0)
            q = torch.ones_like(p)
            if s["draft_index"] is not None:
                q = torch.where(s["draft_index"][:, j].long() == d[:, None], s["draft_prob"][:, j].double(), 0.0).sum(1)
        else:
            p = torch.exp(zd[:, 0] - log_mass(row)[1])
            q = torch.ones_like(p)
            if s["draft_logits"] is not None:
                y, lse = log_mass(s["draft_logits"][:, j])
                q = torch.exp(y.gather(1, d[:, None])[:, 0] - lse)
        ratio[:, j] = torch.where(j < s["n_draft"], torch.where(q > 0, p / q, (p > 0).double()).clamp_max(1.0), 0.0)
    return None, None, ratio
