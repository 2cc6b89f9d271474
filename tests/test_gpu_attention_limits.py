"""The attention calls at the ends of what the C header allows: tokens 2^24
elements apart, 2^22 tokens, 256 heads.  What is compared is bit for bit the same
call on contiguous or fewer rows, or the fp64 oracle (bounds: attention_util)."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import attention_bound, check_decode, check_prefill, values, within
from test_gpu_decode_attention import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


@pytest.fixture(scope="module")
def ws():
    return torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")


def rnd(*s, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
def test_tokens_far_apart(q4, ws, D):
    """q, k and v as parts of rows of 2^24 elements (and none farther)."""
    T, Hq, Hk = 130, 4, 2
    base = torch.empty(T, 1 << 24, dtype=torch.bfloat16, device="cuda")
    at = [0, 1 << 20, (1 << 24) - Hk * D]
    parts = [base[:, a:a + h * D].view(T, h, D) for a, h in zip(at, (Hq, Hk, Hk))]
    for i, p in enumerate(parts):
        p.copy_(rnd(*p.shape, seed=i))
    near = [p.contiguous() for p in parts]
    starts = torch.tensor([0, 1, 70, T], dtype=torch.int32, device="cuda")
    for window in (0, 20):
        assert torch.equal(q4.attention_prefill(*parts, starts, window=window), q4.attention_prefill(*near, starts, window=window))
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), 0.1 ** torch.arange(D // 2, device="cuda").float()
    slots = torch.randperm(T, device="cuda")
    caches = [tuple(torch.zeros(9, Hk, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)) for _ in range(2)]
    got = q4.rope_cache(*parts, pos, freq, cache=caches[0], slots=slots, k_out=True)
    want = q4.rope_cache(*near, pos, freq, cache=caches[1], slots=slots, k_out=True)
    assert all(torch.equal(a, b) for a, b in zip((*got, *caches[0]), (*want, *caches[1])))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([64, 33], dtype=torch.int32, device="cuda")
    rows = parts[0][:128].view(2, 64, Hq, D)
    y = q4.attention_decode(rows, caches[0], table, lens, workspace=ws)
    assert torch.equal(y, q4.attention_decode(near[0][:128].view(2, 64, Hq, D), caches[0], table, lens, workspace=ws))
    q4.rope_cache(*parts, pos, freq, cache=caches[1], slots=slots, q_out=parts[0], k_out=parts[1])
    assert torch.equal(parts[0], got[0]) and torch.equal(parts[1], got[1]) and torch.equal(parts[2], near[2])
    with pytest.raises(q4.Q4GemvError):
        wide = torch.empty(2, (1 << 24) + 8, dtype=torch.bfloat16, device="cuda")
        q4.rope_cache(wide[:, :Hq * D].view(2, Hq, D), near[1][:2])


def test_most_tokens(q4):
    """2^22 tokens: one prompt with a window, many of all lengths; their rotation."""
    T, D, window = 1 << 22, 64, 50
    q, k, v = rnd(T, 2, D, seed=3), rnd(T, 1, D, seed=4), rnd(T, 1, D, seed=5)
    y = q4.attention_prefill(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), window=window)
    for t in (0, 1, 49, 50, 63, 64, 1 << 20, (1 << 21) + 77, T - 2, T - 1):
        lo = max(0, t + 1 - window)
        for h in range(2):
            want, mass, score = oracle.attend(values(q[t:t + 1, h]), values(k[lo:t + 1, 0]), values(v[lo:t + 1, 0]), [t + 1 - lo], D ** -0.5)
            within(y[t:t + 1, h], want, attention_bound(want, mass, score, window, D), f"token {t}")
    # the same tokens as 4096 prompts: the last of them alone is the same, bit for bit
    starts = torch.arange(4097, dtype=torch.int32, device="cuda") * 1024
    y = q4.attention_prefill(q, k, v, starts)
    for b in (0, 1, 2047, 4095):
        part = slice(1024 * b, 1024 * b + 1024)
        one = q4.attention_prefill(q[part], k[part], v[part], torch.tensor([0, 1024], dtype=torch.int32, device="cuda"))
        assert torch.equal(y[part], one), b
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    w = rnd(D, seed=6)
    P = 256
    cache = tuple(torch.zeros(T // P, 1, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(T - 1, -1, -1, device="cuda")
    qo, ko = q4.rope_cache(q, k, v, pos, freq, w, w, cache=cache, slots=slots, k_out=True)
    for part in (slice(0, 300), slice(T // 2 - 1, T // 2 + 300), slice(T - 300, T)):
        one = q4.rope_cache(q[part], k[part], positions=pos[part], inv_freq=freq, q_norm=w, k_norm=w)
        assert torch.equal(qo[part], one[0]) and torch.equal(ko[part], one[1])
    assert torch.equal(cache[0].view(T, D).flip(0), ko[:, 0]) and torch.equal(cache[1].view(T, D).flip(0), v[:, 0])


@pytest.mark.parametrize("Hq,Hk", [(256, 256), (256, 1), (255, 5), (256, 128)])
@pytest.mark.parametrize("D", [64, 128])
def test_most_heads(q4, ws, Hq, Hk, D):
    n = 70
    q, k, v = rnd(n, Hq, D, seed=7), rnd(n, Hk, D, seed=8), rnd(n, Hk, D, seed=9)
    starts = torch.tensor([0, 3, n], dtype=torch.int32)
    check_prefill(q4.attention_prefill(q, k, v, starts.cuda()), q, k, v, starts, None, D ** -0.5, 0)
    for e4m3, T in ((False, 1), (True, 3)):
        p = problem([5, 40], T, Hq, Hk, D, 16, 40, e4m3)
        y = q4.attention_decode(p[0].cuda(), tuple(t.cuda() for t in p[1]), p[2].cuda(), p[3].cuda(), workspace=ws)
        check_decode(y, *p, None, D ** -0.5, 0)


@pytest.mark.parametrize("D,e4m3", [(64, True), (128, False)])
def test_most_rows_of_a_head(q4, ws, D, e4m3):
    """64 tokens of 256 heads over one: 512 units of 32 rows for a sequence."""
    p = problem([64, 77], 64, 256, 1, D, 16, 41, e4m3)
    q, cache, table, lens = p[0].cuda(), tuple(t.cuda() for t in p[1]), p[2].cuda(), p[3].cuda()
    y = q4.attention_decode(q, cache, table, lens, workspace=ws)
    # (a token at a time: as a sequence that ends with it)
    some = [0, 1, 31, 32, 62, 63]
    for b, n in enumerate((64, 77)):
        for i in some:
            at = slice(b, b + 1)
            one = (p[0][at, i:i + 1], p[1], p[2][at], torch.tensor([n - 63 + i], dtype=torch.int32))
            check_decode(y[at, i:i + 1], *one, None, D ** -0.5, 0)


def test_one_workspace_for_a_step(q4, ws):
    """Decode attention in turns with the other calls that take a workspace of
    this kind, all of them in one, eager and as two captured graphs that are
    replayed one after the other: each gives what it gives in its own."""
    p = problem([5000, 77, 1234], 3, 8, 2, 128, 32, 42)
    dev = [p[0].cuda(), tuple(t.cuda() for t in p[1]), p[2].cuda(), p[3].cuda()]
    x, w = rnd(15, 4096, seed=10), rnd(512, 4096, seed=11)
    xc, xs = q4.fp8b128_quantize(x)
    wc, wsc = q4.fp8b128_quantize(w)[0], torch.full((4, 32), 0.01, device="cuda")
    logits, draft = rnd(3, 5, 5000, seed=12), torch.randint(0, 5000, (3, 4), dtype=torch.int32, device="cuda")
    u = torch.rand(3, 5, device="cuda")
    qw = torch.randint(0, 256, (2048, 2048), dtype=torch.uint8, device="cuda")
    sc, mn = (torch.rand(2048, 32, device="cuda").half() * 0.01 for _ in range(2))
    calls = [lambda m: q4.attention_decode(*dev, workspace=m), lambda m: q4.fp8b128_gemm(xc, xs, wc, wsc, workspace=m),
             lambda m: q4.attention_decode(*dev, window=900, workspace=m), lambda m: q4.verify_full(logits, draft, u, workspace=m)[1],
             lambda m: q4.verify_topk(logits, draft, u, top_k=20, workspace=m)[0],
             lambda m: q4.q4g128_gemv_grouped([(x, qw, sc, mn, None)], workspace=m)[0]]
    fresh = lambda: torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")  # noqa: E731
    want = [c(fresh()) for c in calls]
    assert q4.fp8b128_workspace_bytes([(xc, xs, wc, wsc, None, None)]) > 0 and q4.q4g128_workspace_bytes([(x, qw, sc, mn, None)]) > 0
    torch.cuda.synchronize()
    order = [0, 1, 0, 3, 2, 5, 0, 4, 1, 2, 5, 3, 0]
    for i in order:
        assert torch.equal(calls[i](ws), want[i]), i
        assert not ws[:65536].any()
    graphs, outs = [], []
    for part in (order[:7], order[7:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([(i, calls[i](ws)) for i in part])
        graphs.append(g)
    for turn in (0, 1, 1, 0, 1):
        for _, y in outs[turn]:
            y.zero_()
        graphs[turn].replay()
        assert torch.equal(calls[0](ws), want[0])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i]) for i, y in outs[turn])
