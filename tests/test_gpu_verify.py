"""GPU parity of the verification of drafted tokens (verify_topk, verify_full)
against the fp64 oracle.  Tokens and counts are whole numbers and have to be
equal: the kernels hold what decides them in fp64 to about 1e-11, and a uniform
within that of a boundary has a probability of about 1e-9 per case.
accept_prob is such a value rounded to fp32 (2^-24, taken as 1.2e-7)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def inputs(B, D, V, seed, sigma=2.5, noise=0.7, ties=False):
    g = synth.make_gen(("verify", B, D, V, seed))
    target = torch.randn(B, D + 1, V, generator=g) * sigma
    draft = target[:, :D] + torch.randn(B, D, V, generator=g) * noise
    if ties:
        target, draft = torch.round(target * 2) / 2, torch.round(draft * 2) / 2
    u = torch.rand(B, D + 1, generator=g).clamp_max(1 - 2.0 ** -24)
    n = torch.randint(0, D + 1, (B,), generator=g, dtype=torch.int32)
    n[torch.rand(B, generator=g) < 0.6] = D
    return target.to(torch.bfloat16), draft.to(torch.bfloat16), u, n, g


def lists_of(draft, T, k, g):
    """The draft's top-k lists and tokens drawn from them."""
    B, D, V = draft.shape
    v, i = torch.sort(draft.float(), dim=-1, descending=True, stable=True)
    p = torch.softmax(v[..., :k] / T, -1)
    at = torch.multinomial(p.view(B * D, k), 1, generator=g).view(B, D, 1)
    i = i[..., :k]
    return i.to(torch.int32).contiguous(), p.contiguous(), i.gather(2, at)[..., 0].to(torch.int32).contiguous()


def drawn_of(draft, T, g):
    B, D, V = draft.shape
    return torch.multinomial(torch.softmax(draft.float() / T, -1).view(B * D, V), 1, generator=g).view(B, D).to(torch.int32)


def check(got, want, what=""):
    token, count, prob = (t.cpu().numpy() for t in got)
    assert np.array_equal(count, want[1]), what
    assert np.array_equal(token, want[0]), what
    assert np.allclose(prob, want[2], rtol=1.2e-7, atol=1e-37), what


def run_topk(q4, lg, d, u, qi, qp, n, T, k, ws=None):
    opt = lambda t: None if t is None else gpu(t)  # noqa: E731
    return q4.verify_topk(gpu(lg), gpu(d), gpu(u), draft_index=opt(qi), draft_prob=opt(qp), n_draft=opt(n), temperature=T, top_k=k,
                          workspace=ws)


def want_topk(lg, d, u, qi, qp, n, T, k):
    opt = lambda t: None if t is None else t.numpy()  # noqa: E731
    return oracle.verify_topk(synth.bits16(lg), d.numpy(), u.numpy(), opt(qi), opt(qp), opt(n), T, k)


TOPK = [(1, 1, 1, 1, 0.8), (1, 4, 2049, 30, 0.8), (3, 2, 64, 64, 1.3), (5, 7, 513, 17, 0.5), (2, 63, 600, 30, 0.8), (4, 3, 2560, 64, 1.0),
        (4, 3, 2561, 64, 1.0), (7, 5, 4097, 1, 0.8), (6, 4, 16385, 30, 0.8), (2, 7, 30720, 64, 0.8), (40, 8, 1025, 5, 1.0), (60, 4, 4097, 64, 0.8),
        (30, 3, 16385, 30, 0.8)]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("B,D,V,k,T", TOPK)
def test_topk_lists(q4, B, D, V, k, T, ties):
    print(f"verify_topk B={B} D={D} V={V} k={k} T={T} ties={ties}", flush=True)
    lg, dl, u, n, g = inputs(B, D, V, 0, ties=ties)
    qi, qp, d = lists_of(dl, T, k, g)
    for cut in (n, None):
        check(run_topk(q4, lg, d, u, qi, qp, cut, T, k), want_topk(lg, d, u, qi, qp, cut, T, k))


@pytest.mark.parametrize("B,D,V,k,T", TOPK)
def test_topk_certain_drafts(q4, B, D, V, k, T):
    lg, dl, u, n, g = inputs(B, D, V, 1)
    d = dl.float().argmax(-1).to(torch.int32)
    check(run_topk(q4, lg, d, u, None, None, n, T, k), want_topk(lg, d, u, None, None, n, T, k))


def test_topk_agrees_with_the_sampler(q4):
    """Without drafted tokens the draw is the sampler's; drafts that the target
    would draw itself, with its own lists, all stand."""
    B, D, V, k = 16, 3, 2049, 30
    lg, _, u, _, _ = inputs(B, D, V, 2)
    none = torch.zeros(B, dtype=torch.int32)
    d = torch.zeros(B, D, dtype=torch.int32)
    token, count, _ = run_topk(q4, lg, d, u, None, None, none, 0.8, k)
    want = q4.sample_topk(gpu(lg[:, 0].contiguous()), gpu(u[:, D].contiguous()), temperature=0.8, top_k=k)
    assert torch.equal(token[:, 0], want) and int(count.sum()) == 0
    rows = gpu(lg[:, :D].reshape(B * D, V).contiguous())
    tok, ti, tp = q4.sample_topk(rows, gpu(u[:, :D].reshape(-1).contiguous()), temperature=0.8, top_k=k, return_topk=True)
    out = q4.verify_topk(gpu(lg), tok.view(B, D), gpu(u * 0.999), draft_index=ti.view(B, D, k), draft_prob=tp.view(B, D, k), top_k=k)
    assert torch.equal(out[1].cpu(), torch.full((B,), D, dtype=torch.int32))


@pytest.mark.parametrize("k", [2, 30])
def test_topk_odd_inputs(q4, k):
    """-inf and NaN logits, rows without a distribution, drafts outside the
    vocabulary, lists that repeat an index or are padded, lists equal to the
    target (nothing left over), uniforms at the ends."""
    B, D, V, T = 9, 4, 300, 0.8
    lg, dl, u, _, g = inputs(B, D, V, 3)
    qi, qp, d = lists_of(dl, T, k, g)
    lg[0, :, 1::2] = float("-inf")
    lg[1, :, ::3] = float("nan")
    lg[2, 1] = float("-inf")
    lg[3, 0, 5] = float("inf")
    lg[4, 2] = float("nan")
    d[5, 0], d[5, 1] = -1, V
    d[6] = 2 ** 31 - 1
    qi[7, 0, :] = qi[7, 0, 0]
    qp[7, 0, :] = 0.5 / k
    qi[7, 1, k // 2:] = -1
    _, ti, tp = oracle.sample_topk(synth.bits16(lg[8, :D]), float(np.float32(T)), k, np.zeros(D))
    qi[8], qp[8] = torch.from_numpy(ti).to(torch.int32), torch.from_numpy(tp).float()
    d[8] = qi[8, :, k - 1]
    u[0, 0], u[1, D], u[8] = 0.0, 0.0, 1 - 2.0 ** -24
    n = torch.tensor([D, D, D, D, D, D, D, D + 5, -3], dtype=torch.int32)
    n[8] = D
    want = want_topk(lg, d, u, qi, qp, n, T, k)
    check(run_topk(q4, lg, d, u, qi, qp, n, T, k), want)
    n[8] = -3
    check(run_topk(q4, lg, d, u, qi, qp, n, T, k), want_topk(lg, d, u, qi, qp, n, T, k))


def run_full(q4, lg, d, u, dl, n, T, ws=None):
    opt = lambda t: None if t is None else gpu(t)  # noqa: E731
    return q4.verify_full(gpu(lg), gpu(d), gpu(u), draft_logits=opt(dl), n_draft=opt(n), temperature=T, workspace=ws)


def want_full(lg, d, u, dl, n, T):
    return oracle.verify_full(synth.bits16(lg), d.numpy(), u.numpy(), None if dl is None else synth.bits16(dl),
                              None if n is None else n.numpy(), T)


FULL = [(1, 1, 1, 0.8), (1, 1, 7, 1.0), (2, 63, 33, 0.8), (1, 4, 2049, 0.8), (5, 3, 4095, 1.3), (3, 4, 8193, 0.5), (4, 2, 16385, 0.8),
        (2, 7, 50000, 1.0), (3, 1, 131072, 1.0), (1, 2, 200001, 0.8), (1, 1, 1 << 20, 1.0), (520, 1, 40, 0.8), (100, 4, 2056, 0.8)]


@pytest.mark.parametrize("B,D,V,T", FULL)
def test_full(q4, B, D, V, T):
    print(f"verify_full B={B} D={D} V={V} T={T}", flush=True)
    lg, dl, u, n, g = inputs(B, D, V, 0)
    d = drawn_of(dl, T, g)
    for cut in (n, None):
        check(run_full(q4, lg, d, u, dl, cut, T), want_full(lg, d, u, dl, cut, T), "logits")
    d = dl.float().argmax(-1).to(torch.int32)
    check(run_full(q4, lg, d, u, None, n, T), want_full(lg, d, u, None, n, T), "certain")


def test_full_flat_distributions(q4):
    """Nearly uniform rows: every vocabulary entry is a boundary of the draw."""
    B, D, V = 64, 2, 3001
    lg, dl, u, n, g = inputs(B, D, V, 5, sigma=0.01, noise=0.01)
    d = drawn_of(dl, 1.0, g)
    check(run_full(q4, lg, d, u, dl, n, 1.0), want_full(lg, d, u, dl, n, 1.0))


def test_full_odd_inputs(q4):
    B, D, V, T = 10, 3, 5001, 0.8
    lg, dl, u, _, g = inputs(B, D, V, 6)
    d = drawn_of(dl, T, g)
    lg[0, :, 1::2] = float("-inf")
    lg[1, :, ::3] = float("nan")
    lg[2, 1] = float("-inf")
    lg[3, 0, 5] = float("inf")
    dl[4] = float("-inf")
    dl[5, 0, 3], dl[5, 1, ::2] = float("nan"), float("nan")
    d[6, 0], d[6, 1] = -1, V
    dl[7] = lg[7, :D]
    u[7] = 1 - 2.0 ** -24
    lg[8] = float("-inf")
    lg[8, :, V - 1] = -3.0
    u[9] = 0.0
    n = torch.full((B,), D, dtype=torch.int32)
    n[1], n[9] = D + 9, -1
    check(run_full(q4, lg, d, u, dl, n, T), want_full(lg, d, u, dl, n, T))


@pytest.mark.parametrize("V", [32768, 33001, 40003, 70001])
def test_full_long_rows_of_many_sequences(q4, V):
    """Rows whose logits are counted by value: ordinary ones, and values outside
    the counted range (zeros, tiny and large ones, masks of the lowest value,
    -inf, NaN), rows of one value, rows without a distribution."""
    B, D, T = 80, 3, 0.8
    print(f"verify_full B={B} D={D} V={V}", flush=True)
    lg, dl, u, n, g = inputs(B, D, V, 11)
    d = drawn_of(dl, T, g)
    low = float(torch.finfo(torch.bfloat16).min)
    for k, value in enumerate((0.0, -0.0, 1e-6, -2e-5, low, float("-inf"), float("nan"))):
        at = torch.rand(V, generator=g) < (0.5 if k % 2 else 0.98)
        lg[k, :, at] = value
        dl[k, :, at] = value
    lg[7], dl[7] = low, low
    lg[8], dl[8] = 0.0, 0.0
    lg[9], dl[9] = 1.5, 1.5
    lg[10], dl[10] = -0.0, 3e-5
    lg[11] *= 60
    lg[12], dl[12] = lg[12] * 1e-4, dl[12] * 1e-4
    lg[13] += 60
    lg[14] -= 100
    lg[15, 0] = float("-inf")
    lg[16, 1] = float("nan")
    lg[17, 0, V - 1] = float("inf")
    dl[18, 0] = float("-inf")
    lg[19, :, V - 1] = 300.0
    lg[20], dl[20] = low, low
    lg[20, :, 7] = -1e38
    n[:24] = D
    check(run_full(q4, lg, d, u, dl, n, T), want_full(lg, d, u, dl, n, T))


@pytest.mark.parametrize("form,B,V", [("full", 8, 301), ("full", 8, 5001), ("full", 24, 16384), ("full", 80, 33001), ("topk", 8, 301),
                                      ("topk", 8, 2049), ("topk", 8, 16385), ("topk", 300, 5001)])
@pytest.mark.parametrize("T", [0.7, 1.3])
def test_masked_rows(q4, form, B, V, T):
    """Rows whose logits are all, or all but a few, a mask's value: the type's
    lowest, the largest and other far values."""
    D, k = 3, 30
    print(f"{form} B={B} V={V} T={T}", flush=True)
    lg, dl, u, n, g = inputs(B, D, V, 12)
    n[:8] = D
    for b, value in enumerate((torch.finfo(torch.bfloat16).min, -1e30, -65504.0, torch.finfo(torch.bfloat16).max)):
        lg[b], dl[b] = value, value
        keep = torch.rand(V, generator=g) < 0.02
        lg[4 + b, :, ~keep], dl[4 + b, :, ~keep] = value, value
    p, i = torch.softmax(dl.double() / T, -1), None
    if form == "topk":
        p, i = torch.sort(p, dim=-1, descending=True, stable=True)
        p, i = (p[..., :k] / p[..., :k].sum(-1, keepdim=True)).float(), i[..., :k].to(torch.int32).contiguous()
    d = torch.multinomial(p.view(B * D, -1), 1, generator=g).view(B, D, 1)
    if form == "full":
        d = d[..., 0].to(torch.int32).contiguous()
        check(run_full(q4, lg, d, u, dl, n, T), want_full(lg, d, u, dl, n, T))
        check(run_full(q4, lg, d, u, None, n, T), want_full(lg, d, u, None, n, T))
    else:
        d = i.gather(2, d)[..., 0].contiguous()
        check(run_topk(q4, lg, d, u, i, p, n, T, k), want_topk(lg, d, u, i, p, n, T, k))


def test_dirty_shared_workspace(q4):
    """One workspace for both forms and for products, its scratch full of
    rubbish, its first 64 KiB left as they are."""
    ws = torch.full((32 << 20,), 0xAB, dtype=torch.uint8, device="cuda")
    ws[:65536] = 0
    lg, dl, u, n, g = inputs(6, 4, 16385, 7)
    T, k = 0.8, 30
    qi, qp, d = lists_of(dl, T, k, g)
    for rep in range(2):
        check(run_full(q4, lg, d, u, dl, n, T, ws), want_full(lg, d, u, dl, n, T))
        check(run_topk(q4, lg, d, u, qi, qp, n, T, k, ws), want_topk(lg, d, u, qi, qp, n, T, k))
    assert int(ws[:65536].count_nonzero()) == 0


@pytest.mark.parametrize("form", ["topk", "full"])
def test_stream_and_graph(q4, form):
    """A side stream, and a graph replayed with other logits and uniforms."""
    B, D, V, T, k = 5, 4, 16385, 0.8, 30
    sets = []
    for seed in range(3):
        lg, dl, u, n, g = inputs(B, D, V, 20 + seed)
        qi, qp, d = lists_of(dl, T, k, g)
        sets.append([gpu(t) for t in (lg, dl, u, n, qi, qp, d)])
    cur = [t.clone() for t in sets[0]]
    size = q4.verify_topk_workspace_bytes(B, D, V, k) if form == "topk" else q4.verify_full_workspace_bytes(B, D, V)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def step():
        lg, dl, u, n, qi, qp, d = cur
        if form == "topk":
            return q4.verify_topk(lg, d, u, draft_index=qi, draft_prob=qp, n_draft=n, temperature=T, top_k=k, workspace=ws)
        return q4.verify_full(lg, d, u, draft_logits=dl, n_draft=n, temperature=T, workspace=ws)

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(6):
        for t, s in zip(cur, sets[rep % 3]):
            t.copy_(s)
        for t in out:
            t.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), f"replay {rep}"
    del graph


def test_calls_at_once_on_their_own_workspaces(q4):
    """Both forms and a second batch of one of them on three streams at a time."""
    T, k = 0.8, 30
    cases = []
    for seed, (B, D, V) in enumerate(((6, 4, 16385), (90, 3, 33001), (20, 4, 16385))):
        lg, dl, u, n, g = inputs(B, D, V, 40 + seed)
        full = seed < 2
        qi, qp, d = (None, None, drawn_of(dl, T, g)) if full else lists_of(dl, T, k, g)
        ws = torch.zeros(q4.verify_full_workspace_bytes(B, D, V) if full else q4.verify_topk_workspace_bytes(B, D, V, k),
                         dtype=torch.uint8, device="cuda")
        a = [None if t is None else gpu(t) for t in (lg, d, u, qi, qp, dl, n)]

        def call(a=a, ws=ws, full=full):
            if full:
                return q4.verify_full(a[0], a[1], a[2], draft_logits=a[5], n_draft=a[6], temperature=T, workspace=ws)
            return q4.verify_topk(a[0], a[1], a[2], draft_index=a[3], draft_prob=a[4], n_draft=a[6], temperature=T, top_k=k, workspace=ws)

        cases.append((call, [t.clone() for t in call()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for rep in range(8):
        outs = []
        for call, _, stream in cases:
            with torch.cuda.stream(stream):
                outs.append(call())
        torch.cuda.synchronize()
        for got, (_, want, _) in zip(outs, cases):
            assert all(torch.equal(x, y) for x, y in zip(got, want)), f"repetition {rep}"


def test_draft_and_verify_step(q4):
    """The operators as a step uses them: hidden states of every drafted
    position quantised, the head's 8-bit product, the draft's tokens from the
    sampler, the verification of both forms on the logits that came out; and
    the gated activation through the down projection with its residual."""
    B, D, H, F, V, k, T = 3, 4, 512, 1024, 2049, 30, 0.8
    g = synth.make_gen("step")
    M = B * (D + 1)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731

    def weights(n, kk):
        w = rnd(n, kk) * 0.05
        G = -(-kk // 128)
        pad = torch.nn.functional.pad(w, (0, -kk % 128, 0, -n % 128)).view(-1, 128, G, 128)
        s = pad.abs().amax((1, 3)) / 448
        c = (pad / s[:, None, :, None]).view(-1, G * 128)[:n, :kk].clamp(-448, 448)
        return c.to(torch.float8_e4m3fn).cuda().contiguous(), s.cuda().contiguous()

    gate, up, down, head = weights(F, H), weights(F, H), weights(H, F), weights(V, H)
    x = gpu(rnd(M, H).to(torch.bfloat16))
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    xc, xs = q4.fp8b128_quantize(x)
    gy, uy = q4.fp8b128_gemm_grouped([(xc, xs, *gate, None, None), (xc, xs, *up, None, None)], workspace=ws)
    hc, hs = q4.fp8b128_quantize(gy, up=uy)
    y = q4.fp8b128_gemm(hc, hs, *down, residual=x, workspace=ws)
    yc, ys = q4.fp8b128_quantize(y)
    logits = q4.fp8b128_gemm(yc, ys, *head, workspace=ws).view(B, D + 1, V)
    # every stage from its own inputs
    from test_gpu_fp8 import check_gemm, check_plain
    cpu = lambda *t: tuple(v.cpu() for v in t)  # noqa: E731
    check_plain(xc, xs, synth.bits16(x.cpu()))
    check_gemm(gy, cpu(xc, xs, *gate))
    check_gemm(y, cpu(hc, hs, *down), x.cpu())
    check_plain(yc, ys, synth.bits16(y.cpu()))
    check_gemm(logits.view(M, V), cpu(yc, ys, *head))
    # a draft near the target
    dl = (logits[:, :D].float() + gpu(rnd(B, D, V)) * 0.3).to(torch.bfloat16).contiguous()
    u = torch.rand(B, D + 1, generator=g)
    tok, ti, tp = q4.sample_topk(dl.view(B * D, V), gpu(torch.rand(B * D, generator=g)), temperature=T, top_k=k, return_topk=True)
    d, ti, tp = tok.view(B, D), ti.view(B, D, k), tp.view(B, D, k)
    lg = logits.cpu()
    check(q4.verify_topk(logits, d, gpu(u), draft_index=ti, draft_prob=tp, temperature=T, top_k=k, workspace=ws),
          want_topk(lg, d.cpu(), u, ti.cpu(), tp.cpu(), None, T, k))
    check(q4.verify_full(logits, d, gpu(u), draft_logits=dl, temperature=T, workspace=ws),
          want_full(lg, d.cpu(), u, dl.cpu(), None, T))


def test_binding_refusals(q4):
    lg, dl, u, n, g = inputs(2, 3, 100, 9)
    lg, dl, u, n = gpu(lg), gpu(dl), gpu(u), gpu(n)
    d = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        q4.verify_full(lg, d[:, :2].contiguous(), u)
    with pytest.raises(TypeError):
        q4.verify_full(lg, d.long(), u)
    with pytest.raises(ValueError):
        q4.verify_full(lg, d, u[:, :3].contiguous())
    with pytest.raises(ValueError):
        q4.verify_full(lg, d, u, draft_logits=lg)
    with pytest.raises(ValueError):
        q4.verify_full(lg, d, u, n_draft=n[:1].contiguous())
    with pytest.raises(ValueError):
        q4.verify_full(lg.transpose(0, 1), d, u)
    with pytest.raises(q4.Q4GemvError):
        q4.verify_full(lg, d, u, temperature=0.0)
    with pytest.raises(q4.Q4GemvError):
        q4.verify_full(lg, d, u, workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(q4.Q4GemvError):
        q4.verify_topk(lg, d, u, top_k=65)
    with pytest.raises(q4.Q4GemvError):
        q4.verify_topk(lg, d, u, draft_index=torch.zeros(2, 3, 4, dtype=torch.int32, device="cuda"), top_k=4)
    with pytest.raises(q4.Q4GemvError):
        q4.verify_topk(lg[:, :1].contiguous(), d[:, :0].contiguous(), u[:, :1].contiguous(), top_k=4)
