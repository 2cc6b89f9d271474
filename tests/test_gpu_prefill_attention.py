"""GPU parity of attention_prefill against the fp64 oracle, through the
binding; and a layer's attention as a user runs it.  Bounds: attention_util."""
import numpy as np
import pytest
import torch

import oracle
import synth
from attention_util import check_decode, check_prefill, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)


def problem(lengths, keys, Hq, Hk, D, seed, behind=0):
    g = synth.make_gen(("prefill", tuple(lengths), tuple(keys), Hq, Hk, D, seed))
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    T, S = sum(lengths) + behind, sum(keys) + behind
    return rnd(T, Hq, D) * 1.5, rnd(S, Hk, D), rnd(S, Hk, D), offsets(lengths), None if lengths == keys else offsets(keys)


def run(q4, q, k, v, starts, key_starts, **kw):
    return q4.attention_prefill(q, k, v, starts.cuda(), None if key_starts is None else key_starts.cuda(), **kw)


def check(q4, p, window=0, scale=None):
    y = run(q4, *p, window=window, scale=scale)
    check_prefill(y, *p, p[0].shape[2] ** -0.5 if scale is None else scale, window)
    return y


HEADS = [(16, 4, 128), (4, 4, 64), (7, 1, 128), (8, 2, 64), (3, 3, 128), (24, 1, 64),
         (72, 72, 64), (144, 72, 128)]     # of so many heads: more workgroups than CUs


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [63], [64], [65], [130], [300], [0, 1, 0, 77, 5, 129, 0]])
def test_lengths(q4, Hq, Hk, D, lengths):
    check(q4, problem(lengths, lengths, Hq, Hk, D, 0))


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("window", [1, 5, 64, 100])
def test_windows(q4, Hq, Hk, D, window):
    check(q4, problem([1, 70, 250], [1, 70, 250], Hq, Hk, D, 1), window)


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("window", [0, 3, 90])
def test_prefixes(q4, Hq, Hk, D, window):
    """More keys than tokens, and fewer (the first tokens see nothing), none."""
    check(q4, problem([5, 100, 70, 33, 0, 1], [205, 101, 40, 0, 9, 64], Hq, Hk, D, 2), window)


@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (6, 2, 64)])
@pytest.mark.parametrize("window", [0, 200])
def test_many_rows(q4, Hq, Hk, D, window):
    """Enough rows for the larger workgroups."""
    T = 65536 // Hq * 2
    lengths = [600, T - 1300, 1, 699]
    q, k, v, st, _ = problem(lengths, lengths, Hq, Hk, D, 3)
    y = run(q4, q, k, v, st, None, window=window)
    # a long one by a few of its tokens
    for b, at in [(0, range(0, 600, 7)), (1, [0, 63, 64, 511, 5000, lengths[1] - 1]), (2, [0]), (3, range(690))]:
        q0 = int(st[b])
        rows = [q0 + i for i in at]
        for h in range(Hq):
            ke, ve = (values(t[q0:q0 + lengths[b], h // (Hq // Hk)]) for t in (k, v))
            y0, mass, score = oracle.attend(values(q[rows, h]), ke, ve, np.array(list(at)) + 1, D ** -0.5, window)
            from attention_util import attention_bound, within
            within(y[rows, h], y0, attention_bound(y0, mass, score, lengths[b], D), f"{b} {h}")


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("window", [0, 70])
def test_unseen_values_have_no_effect(q4, big, window):
    """Infinities and NaNs in keys and values of later tokens, of tokens before
    the window and of other prompts: rows that do not see them are what they are
    without."""
    Hq, Hk, D = (64, 8, 128) if big else (4, 2, 128)
    lengths = [300, 190, 700]
    q, k, v, st, _ = problem(lengths, lengths, Hq, Hk, D, 4)
    clean = run(q4, q, k, v, st, None, window=window)
    bad = [120, 299, 300 + 64, 490 + 333, 490 + 699]
    kb, vb = k.clone(), v.clone()
    kb[bad], vb[bad] = float("nan"), float("inf")
    vb[bad[1]], kb[bad[3]] = float("nan"), k[bad[3]]
    y = run(q4, q, kb, vb, st, None, window=window)
    for b in range(3):
        for t in range(int(st[b]), int(st[b + 1])):
            sees = any(int(st[b]) <= j <= t and (not window or j > t - window) for j in bad)
            if sees:
                assert not torch.isfinite(y[t]).all(-1).any(), t
            else:
                assert torch.equal(y[t], clean[t]), t


def test_infinite_values_that_are_seen(q4):
    q, k, v, st, _ = problem([100], [100], 4, 2, 64, 5)
    spots = [(70, 3, float("inf")), (75, 5, float("-inf")), (2, 9, float("inf"))]
    for j, c, x in spots:
        v[j, :, c] = x
    y = values(run(q4, q, k, v, st, None))
    for t in range(100):
        for j, c, x in spots:
            assert (y[t, :, c] == x).all() if t >= j else np.isfinite(y[t, :, c]).all(), (t, c)
        assert np.isfinite(np.delete(y[t], [3, 5, 9], axis=1)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_meet(q4, bad):
    """A head of q that is no number is that head's row alone."""
    q, k, v, st, ks = problem([150, 33], [150, 33], 8, 2, 64, 12)
    clean = check(q4, (q, k, v, st, ks))
    odd = q.clone()
    odd[70, 2], odd[160, 5] = bad, bad
    y = run(q4, odd, k, v, st, ks)
    for at in ((70, 2), (160, 5)):
        assert torch.isnan(y[at]).all()
        y[at] = clean[at]
    check_prefill(y, q, k, v, st, ks, 64 ** -0.5, 0)


def test_scores_of_any_size(q4):
    p = problem([150, 40], [150, 40], 4, 2, 128, 6)
    for scale in (1.0, 1e-3):
        check(q4, p, scale=scale)
    p[0].mul_(30)
    check(q4, p, scale=1.0)


def test_strided_parts(q4):
    """q, k and v as parts of one product's rows."""
    lengths = [90, 65]
    q, k, v, st, _ = problem(lengths, lengths, 6, 2, 64, 7)
    y = run(q4, q, k, v, st, None)
    qkv = torch.cat((q, k, v), 1)
    assert torch.equal(run(q4, qkv[:, :6], qkv[:, 6:8], qkv[:, 8:], st, None), y)


def test_rows_of_no_sequence_are_left(q4):
    """Before the first, between, and behind the last; sequences taken within
    the arrays."""
    q, k, v, st, _ = problem([50, 70], [50, 70], 4, 2, 64, 8, behind=30)
    out = torch.full_like(q, 7.0)
    y = run(q4, q, k, v, st + 10, None, out=out)
    assert y is out and (out[:10] == 7).all() and (out[130:] == 7).all()
    check_prefill(out[10:130], q[10:130], k[10:130], v[10:130], st, None, 64 ** -0.5, 0)
    for starts in ([-5, 40, 1000], [0, 150, 150], [150, 150, 150], [100, 50, 60]):
        starts = torch.tensor(starts, dtype=torch.int32)
        out.fill_(7.0)
        run(q4, q, k, v, starts, None, out=out)
        within = starts.clamp(0, 150)
        inside = torch.zeros(150, dtype=torch.bool)
        for b in range(2):
            lo, hi = int(within[b]), max(int(within[b]), int(within[b + 1]))
            inside[lo:hi] = True
            if hi > lo:
                check_prefill(out[lo:hi], q[lo:hi], k[lo:hi], v[lo:hi], torch.tensor([0, hi - lo]), None, 64 ** -0.5, 0)
        assert (out[~inside.cuda()] == 7).all()


@pytest.mark.parametrize("B", [64, 65, 1000, 4096])
def test_many_sequences(q4, B):
    lengths = [(5 * b * b) % 9 for b in range(B)]
    check(q4, problem(lengths, lengths, 2, 1, 64, 9))


def test_repeats_streams_and_graph(q4):
    lengths = [333, 20, 1, 150]
    q, k, v, st, _ = problem(lengths, lengths, 8, 2, 128, 10)
    st = st.cuda()
    y = q4.attention_prefill(q, k, v, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = q4.attention_prefill(q, k, v, st)
    torch.cuda.synchronize()
    assert torch.equal(other, y)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4.attention_prefill(q, k, v, st, out=out)
    for i in range(3):
        q.copy_(torch.randn_like(q))
        st[1:4].add_(1)                 # other lengths, the same tokens in all
        eager = q4.attention_prefill(q, k, v, st)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_as_it_is_used(q4, e4m3):
    """Prompts through projections, heads into the cache, attention over the
    prompts; then steps of three tokens (two of them drafted) that append and
    attend over the cache: each stage against the oracle on its own inputs, and
    what the steps give against attention over the whole sequences."""
    Hq, Hk, D, P, H = 8, 2, 128, 16, 512
    g = synth.make_gen(("layer", e4m3))
    lengths, T, steps = [37, 5, 130], 3, 2
    B = len(lengths)
    tokens = [n + T * steps for n in lengths]
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = {n: (rnd(h * D, H) / H ** 0.5).to(torch.bfloat16).cuda() for n, h in (("q", Hq), ("k", Hk), ("v", Hk))}
    qn, kn = ((1 + 0.2 * rnd(D)).to(torch.bfloat16).cuda() for _ in range(2))
    f = torch.tensor(10000.0 ** (-np.arange(0, D, 2) / D), dtype=torch.float32).cuda()
    width = -(-max(tokens) // P)
    pages = B * width + 1
    table = torch.randperm(pages, generator=g)[:B * width].view(B, width).to(torch.int32)
    shape = (pages, Hk, P, D)
    cache = tuple(torch.zeros(shape, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda") for _ in range(2))
    if e4m3:
        cache += tuple(torch.zeros(shape[:3], device="cuda") for _ in range(2))
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    xs = [rnd(n, H).to(torch.bfloat16).cuda() for n in tokens]

    def projected(x):
        rows = []
        for i in range(0, len(x), 64):
            part = x[i:i + 64].contiguous()
            rows.append(torch.cat(q4.bf16_gemv_grouped([(part, w[n], None) for n in "qkv"]), 1))
        qkv = torch.cat(rows).view(len(x), Hq + 2 * Hk, D)
        return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]

    def slots_of(pos):
        return torch.tensor([int(table[b, p // P]) * P + p % P for b, p in pos], dtype=torch.int64).cuda()

    def append(x, pos, k_out=None):
        q, k, v = projected(x)
        positions = torch.tensor([p for _, p in pos], dtype=torch.int32).cuda()
        return (*q4.rope_cache(q, k, v, positions, f, qn, kn, 1e-6, False, cache, slots_of(pos), k_out=k_out), v)

    prompt = torch.cat([x[:n] for x, n in zip(xs, lengths)])
    q, k, v = append(prompt, [(b, p) for b, n in enumerate(lengths) for p in range(n)], True)
    st = offsets(lengths)
    check_prefill(q4.attention_prefill(q, k, v, st.cuda()), q, k, v, st, None, D ** -0.5, 0)
    last = []
    for s in range(steps):
        at = [n + s * T for n in lengths]
        x = torch.cat([x[a:a + T] for x, a in zip(xs, at)])
        q, _, _ = append(x, [(b, a + i) for b, a in enumerate(at) for i in range(T)])
        lens = torch.tensor([a + T for a in at], dtype=torch.int32)
        y = q4.attention_decode(q.view(B, T, Hq, D), cache, table.cuda(), lens.cuda(), workspace=ws)
        check_decode(y, q.view(B, T, Hq, D), cache, table, lens, None, D ** -0.5, 0)
        last.append(y)
    # the whole sequences at once (a bf16 cache holds the same keys and values)
    if not e4m3:
        q, k, v = projected(torch.cat(xs))
        positions = torch.cat([torch.arange(n) for n in tokens]).to(torch.int32).cuda()
        q, k = q4.rope_cache(q, k, positions=positions, inv_freq=f, q_norm=qn, k_norm=kn)
        st = offsets(tokens)
        whole = q4.attention_prefill(q, k, v, st.cuda()).float()
        for b, n in enumerate(lengths):
            for s in range(steps):
                a = int(st[b]) + n + s * T
                assert torch.allclose(last[s][b].float(), whole[a:a + T], rtol=0.05, atol=0.05)


def test_binding_refusals(q4):
    q, k, v, st, _ = problem([20], [20], 4, 2, 64, 11)
    st = st.cuda()
    call = lambda **kw: q4.attention_prefill(**{**dict(q=q, k=k, v=v, starts=st), **kw})  # noqa: E731
    call()
    for kw in (dict(k=k[:-1]), dict(v=v[:-1]), dict(k=k[:, :, :32]), dict(starts=st[None]), dict(key_starts=st[:1]), dict(out=q[:-1]),
               dict(q=q[:, 0]), dict(q=q.transpose(0, 1)), dict(starts=st.cpu()), dict(k=k.cpu()), dict(window=2 ** 32 + 5),
               dict(window=1 - 2 ** 32)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(starts=st.long()), dict(q=q.half()), dict(v=v.float()), dict(q=3)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(scale=-1.0), dict(window=-1), dict(out=q), dict(q=q[:, :3]), dict(starts=st[:1])):
        with pytest.raises(q4.Q4GemvError):
            call(**kw)
