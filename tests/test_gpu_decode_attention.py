"""GPU parity of attention_decode against the fp64 oracle, through the binding.
Bounds: attention_util."""
import numpy as np
import pytest
import torch

import oracle
import synth
from attention_util import attention_bound, check_decode, values, within

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


def problem(lengths, T, Hq, Hk, D, P, seed, e4m3=False, spare=2):
    """CPU inputs; pages in no order, table entries behind a length -1, slots
    behind it filled with what must not count."""
    g = synth.make_gen(("decode", tuple(lengths), T, Hq, Hk, D, P, seed))
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    B = len(lengths)
    need = [-(-max(0, n) // P) for n in lengths]
    pages, width = sum(need) + spare, max(1, max(need))
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    k, v = rnd(pages, Hk, P, D), rnd(pages, Hk, P, D)
    used = torch.zeros(pages, P, dtype=torch.bool)
    for b, n in enumerate(lengths):
        for j in range(need[b]):
            table[b, j] = order.pop()
            used[table[b, j], :max(0, min(P, n - j * P))] = True
    q = (rnd(B, T, Hq, D) * 1.5).to(torch.bfloat16)
    if e4m3:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        scales = [(torch.rand(pages, Hk, P, generator=g) + 0.2) for _ in range(2)]
        for t in (k, v):
            t.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)       # NaN
        for s in scales:
            s.masked_fill_(~used[:, None], float("inf"))
        cache = (k, v, *scales)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        k.masked_fill_(~used[:, None, :, None], float("nan"))
        v.masked_fill_(~used[:, None, :, None], float("inf"))
        cache = (k, v)
    return q, cache, table, torch.tensor(lengths, dtype=torch.int32)


def run(q4, ws, q, cache, table, lengths, n_new=None, window=0, scale=None, out=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = q4.attention_decode(dev(q), tuple(dev(t) for t in cache), dev(table), dev(lengths), dev(n_new), scale, window, out, ws)
    assert not ws[:65536].any()
    return y


def check(q4, ws, p, n_new=None, window=0, scale=None):
    y = run(q4, ws, *p, n_new, window, scale)
    check_decode(y, *p, n_new, p[0].shape[3] ** -0.5 if scale is None else scale, window)
    return y


HEADS = [(16, 4, 128), (4, 4, 128), (8, 1, 64), (14, 2, 64), (3, 1, 128), (32, 2, 64)]


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_lengths(q4, ws, Hq, Hk, D, P, e4m3):
    """From no key to several blocks, at the edges of tiles, pages and blocks."""
    check(q4, ws, problem([0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 513], 1, Hq, Hk, D, P, 0, e4m3))


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("T", [2, 5, 8])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 3, 130])
def test_several_rows(q4, ws, Hq, Hk, D, T, e4m3, window):
    """Drafted rows: fewer than T, none, more than there are keys; windows."""
    lengths = [0, 1, 3, T, 33, 127, 131, 260, 395]
    p = problem(lengths, T, Hq, Hk, D, 32, 1, e4m3)
    n = torch.tensor([T, 1, T, 0, T, 1, T - 1, T, 2], dtype=torch.int32)
    check(q4, ws, p, n, window)


@pytest.mark.parametrize("T,Hq,Hk", [(64, 4, 4), (33, 8, 1), (64, 16, 1), (17, 3, 1)])
def test_many_rows(q4, ws, T, Hq, Hk):
    """More rows than a workgroup holds at a time, up to the most."""
    check(q4, ws, problem([64, 70, 200], T, Hq, Hk, 128, 16, 2))
    check(q4, ws, problem([90, 5, 200], T, Hq, Hk, 64, 16, 3, True), torch.tensor([T, 70, -3], dtype=torch.int32), 40)


@pytest.mark.parametrize("lengths,P", [([20000], 16), ([9000, 1, 4097, 300], 128), ([1] * 700, 16), ([40] * 130 + [5000], 32)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_split_and_joined(q4, ws, lengths, P, e4m3):
    """One long sequence over all workgroups, ragged ones, more sequences than
    workgroups, a long one among short ones."""
    check(q4, ws, problem(lengths, 1, 4, 2, 128, P, 4, e4m3))


@pytest.mark.parametrize("T,Hq,Hk", [(1, 2, 2), (1, 12, 1), (8, 2, 1), (8, 6, 2), (40, 1, 1)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_parts(q4, ws, T, Hq, Hk, e4m3):
    """Long sequences after each other, each over many workgroups, the first and
    the last of them shared: parts joined in groups.  Twice in one workspace."""
    p = problem([9000, 14000, 33, 16000, 4500], T, Hq, Hk, 64, 64, 11, e4m3)
    y = check(q4, ws, p)
    assert torch.equal(check(q4, ws, p).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("T,G", [(1, 1), (3, 2), (2, 6), (8, 4), (16, 4)])
def test_one_unit_over_all_workgroups(q4, ws, T, G):
    """One sequence and key head: hundreds of parts of 1 to 32 rows (or two units of them)."""
    p = problem([70001], T, G, 1, 64, 64, 23)
    y = check(q4, ws, p)
    assert torch.equal(run(q4, ws, *p).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk", [(70, 40, 2, 1), (64, 9, 8, 2), (200, 2, 32, 2)])
def test_many_rows_of_many_sequences(q4, ws, B, T, Hq, Hk, e4m3):
    """A padded batch: sequences of no tokens and of fewer new ones than T."""
    p = problem([(11 * b * b) % 170 if b % 9 else 0 for b in range(B)], T, Hq, Hk, 64, 16, 21, e4m3)
    n = torch.tensor([(5 * b) % (T + 1) if b % 9 else 0 for b in range(B)], dtype=torch.int32)
    check(q4, ws, p, n)
    check(q4, ws, p, n, 37)


@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_meet(q4, ws, T, bad):
    """A head of q that is no number is that head's row alone."""
    q, cache, table, lens = problem([150, 33], T, 8, 2, 64, 16, 22)
    clean = check(q4, ws, (q, cache, table, lens))
    odd = q.clone()
    odd[0, T - 1, 2], odd[1, 0, 5] = bad, bad
    y = run(q4, ws, odd, cache, table, lens)
    for at in ((0, T - 1, 2), (1, 0, 5)):
        assert torch.isnan(y[at]).all()
        y[at] = clean[at]
    check_decode(y, q, cache, table, lens, None, 64 ** -0.5, 0)


@pytest.mark.parametrize("B", [64, 65, 129, 4096])
def test_many_sequences(q4, ws, B):
    """The search for a workgroup's place among sequences."""
    lengths = [(7 * b * b) % 90 for b in range(B)]
    check(q4, ws, problem(lengths, 1, 2, 1, 64, 16, 5))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 4])
def test_pages_that_hold_nothing(q4, ws, e4m3, T):
    """Entries that are no page of the cache: their keys take no part; a
    sequence of only such is 0.  Values that are not finite elsewhere count."""
    p = problem([100, 300, 64, 700], T, 8, 2, 128, 16, 6, e4m3)
    q, cache, table, lengths = p
    pages = cache[0].shape[0]
    table[0, 2], table[0, 6] = -1, pages
    table[1, 5:14] = torch.tensor([-7, pages, 2 ** 31 - 1, -2 ** 31, pages + 5, -1, -1, -1, -1], dtype=torch.int32)
    table[2, :] = -1
    table[3, 1::2] = -1
    y = check(q4, ws, p)
    assert not y[2].any()


def test_same_page_twice(q4, ws):
    """A page shared by sequences, and twice in one."""
    p = problem([48, 100, 100], 1, 4, 2, 64, 16, 7)
    p[2][1, :3] = p[2][0, :3]
    p[2][2, :4] = p[2][1, 2]
    check(q4, ws, p)


@pytest.mark.parametrize("T,window", [(1, 0), (1, 50), (4, 0), (4, 50), (64, 0), (40, 20)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_unseen_values_have_no_effect(q4, ws, T, window, e4m3):
    """Infinities and NaNs in keys and values that a row does not see, among
    the keys that rows beside it do see: it is what it is without them."""
    lengths = [200, 161, 300]
    q, cache, table, lens = problem(lengths, T, 4, 1, 128, 16, 8, e4m3)
    clean = run(q4, ws, q, cache, table, lens, window=window)
    check_decode(clean, q, cache, table, lens, None, 128 ** -0.5, window)
    bad = [t.clone() for t in cache]
    for b, n in enumerate(lengths):
        # the last token's own key and value, and, with a window, those before the last row's
        for j in [n - 1] + ([n - window - 1] if window else []):
            page, at = int(table[b, j // 16]), j % 16
            if e4m3:
                bad[0].view(torch.uint8)[page, :, at], bad[1].view(torch.uint8)[page, :, at] = 0x7F, 0xFF
                bad[3][page, :, at] = float("nan")
            else:
                bad[0][page, :, at], bad[1][page, :, at] = float("nan"), float("inf")
    y = run(q4, ws, q, bad, table, lens, window=window)
    hit = lambda i: i == T - 1 or (bool(window) and i < T - 1 and T > 1)  # noqa: E731
    for i in range(T):
        end = 1 + i - T       # of row i, from the length
        sees = end == 0 or (window and end - window <= -window - 1 < end)
        if not sees:
            assert torch.equal(y[:, i], clean[:, i]), i
        else:
            assert torch.isnan(y[:, i]).any(), (i, hit(i))


def test_infinite_values_that_are_seen(q4, ws):
    """An infinite value goes to the rows that see it, with its sign, and to no
    other; in the last step, where rows see different keys, too."""
    T = 4
    q, cache, table, lens = problem([130], T, 4, 1, 64, 16, 9)
    for j, col, x in [(127, 3, float("inf")), (128, 5, float("-inf")), (129, 7, float("inf")), (10, 9, float("-inf"))]:
        cache[1][int(table[0, j // 16]), 0, j % 16, col] = x
    y = values(run(q4, ws, q, cache, table, lens))[0]
    inf = np.inf
    for i in range(T):      # row i sees keys below 127 + i
        for j, col, x in [(127, 3, inf), (128, 5, -inf), (129, 7, inf), (10, 9, -inf)]:
            want = x if j < 127 + i else None
            assert (y[i, :, col] == x).all() if want else np.isfinite(y[i, :, col]).all(), (i, col)
        rest = [c for c in range(64) if c not in (3, 5, 7, 9)]
        assert np.isfinite(y[i][:, rest]).all()


def test_scores_of_any_size(q4, ws):
    """Large scores, a scale of its own; a key with a score of +-infinity."""
    p = problem([77, 140], 1, 4, 2, 128, 16, 10)
    check(q4, ws, p, scale=1.0)
    check(q4, ws, p, scale=1e-3)
    q, cache, table, lens = p
    q.mul_(30)
    check(q4, ws, p, scale=1.0)
    cache[0][int(table[0, 1]), 0, 3] = 0
    cache[0][int(table[0, 1]), 0, 3, 0] = float("inf")
    y = values(run(q4, ws, *p, scale=1.0))
    sign = values(q)[0, 0, :2, 0] > 0
    assert np.isnan(y[0, 0, :2][sign]).all() and np.isfinite(y[0, 0, :2][~sign]).all() and np.isfinite(y[0, 0, 2:]).all()


def test_window_of_all_keys(q4, ws):
    p = problem([40, 300, 1000], 2, 4, 2, 64, 16, 11)
    y = run(q4, ws, *p)
    for window in (1000, 2 ** 24, 2 ** 31 - 1):
        assert torch.equal(run(q4, ws, *p, window=window), y)


def test_lengths_out_of_range(q4, ws):
    """Lengths below 0 and past the table are taken at its ends."""
    p = problem([0, 64, 64], 2, 4, 2, 64, 16, 12)
    y = run(q4, ws, *p)
    p[3][0], p[3][1], p[3][2] = -9, 2 ** 31 - 1, 65
    assert torch.equal(run(q4, ws, *p), y)


def test_strided_queries(q4, ws):
    q, cache, table, lens = problem([50, 129], 3, 8, 2, 64, 16, 13)
    y = run(q4, ws, q, cache, table, lens)
    wide = torch.zeros(2, 3, 12, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 2:10] = q.cuda()
    dev = tuple(t.cuda() for t in cache)
    got = q4.attention_decode(wide[:, :, 2:10], dev, table.cuda(), lens.cuda(), workspace=ws)
    assert torch.equal(got, y)
    for b in (slice(0, 1), slice(1, 2)):
        one = q4.attention_decode(wide[b, :, 2:10], dev, table[b].cuda(), lens[b].cuda(), workspace=ws)
        check_decode(one, q[b], cache, table[b], lens[b], None, 64 ** -0.5, 0)
    one = q4.attention_decode(wide[:, 1:2, 2:10], dev, table.cuda(), lens.cuda(), workspace=ws)
    check_decode(one, q[:, 1:2], cache, table, lens, None, 64 ** -0.5, 0)


def test_repeats_are_equal(q4, ws):
    """Same inputs, same bits, with or without a workspace of its own, into a
    given output and on another stream."""
    p = problem([5000, 77, 1234], 3, 8, 2, 128, 32, 14)
    y = run(q4, ws, *p)
    dev = [p[0].cuda(), tuple(t.cuda() for t in p[1]), p[2].cuda(), p[3].cuda()]
    for _ in range(5):
        out = torch.full_like(dev[0], 7.0)
        assert q4.attention_decode(*dev, out=out, workspace=ws) is out and torch.equal(out, y)
    assert torch.equal(q4.attention_decode(*dev), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = q4.attention_decode(*dev)
    torch.cuda.synchronize()
    assert torch.equal(other, y)


def test_calls_at_once(q4):
    """Calls on several streams, each with a workspace of its own."""
    cases = []
    for i, lengths in enumerate([[3000], [40] * 90, [1000, 2000, 5]]):
        p = problem(lengths, 1, 8, 2, 128, 16, 15 + i)
        dev = [p[0].cuda(), tuple(t.cuda() for t in p[1]), p[2].cuda(), p[3].cuda()]
        cases.append((dev, torch.zeros(16 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    want = [q4.attention_decode(*d, workspace=w) for d, w, _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for d, w, s in cases:
            with torch.cuda.stream(s):
                outs.append(q4.attention_decode(*d, workspace=w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_graph(q4, ws):
    """Captured once, replayed as the sequences grow: two calls that share the
    workspace, with eager work between the replays."""
    lengths = [100, 600, 31]
    q, cache, table, lens = problem([n + 60 for n in lengths], 2, 8, 2, 128, 16, 18)
    q, cache, table = q.cuda(), tuple(torch.nan_to_num(t, 0, 0, 0).cuda() for t in cache), table.cuda()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def step(a, b):
        q4.attention_decode(q, cache, table, lens, out=a, workspace=ws)
        q4.attention_decode(a, cache, table, lens, out=b, window=70, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*outs)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*outs)
    for i in range(4):
        eager = [torch.empty_like(q) for _ in range(2)]
        step(*eager)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        lens.add_(13)
        q.copy_(torch.randn_like(q))


def test_long_cache_offsets(q4, ws):
    """Pages that lie past 2^32 bytes of the cache."""
    Hk, D, P = 4, 128, 256
    pages = (1 << 32) // (Hk * P * D * 2) + 8
    q, small, table, lens = problem([600, 300], 1, 8, Hk, D, P, 19, spare=0)
    cache = tuple(torch.zeros(pages, Hk, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = small[0].shape[0]
    for big, s in zip(cache, small):
        big[pages - n:] = s.cuda()
    far = torch.where(table >= 0, table + (pages - n), -1)
    y = q4.attention_decode(q.cuda(), cache, far.cuda(), lens.cuda(), workspace=ws)
    assert torch.equal(y, run(q4, ws, q, small, table, lens))


@pytest.mark.parametrize("D,T", [(64, 1), (128, 8)])
def test_table_in_parts(q4, ws, D, T):
    """So many keys that a workgroup takes its pages in parts: a table that goes
    over a few pages again and again, 2^24 keys less the new ones' last page.  All
    keys weigh alike in every round, so the result is attention over one round (a
    whole number of rounds for the last row's; the rows before it miss keys among
    2^24).  A lane adds 2^24 * Hk / 512 / 16 weights at most, and 512 parts meet."""
    Hk, P, n = 4, 16, 64
    rounds = (1 << 20) // n
    q, cache, _, _ = problem([n * P], T, 8, Hk, D, P, 21, spare=0)
    table = torch.arange(n, dtype=torch.int32).repeat(rounds)[None]
    lens = torch.tensor([1 << 24], dtype=torch.int32)
    y = values(run(q4, ws, q, cache, table, lens))[0]
    k, v = (values(t).transpose(1, 0, 2, 3).reshape(Hk, n * P, D) for t in cache)
    for h in range(Hk):
        rows = values(q)[0, :, 2 * h:2 * h + 2].reshape(2 * T, D)
        want, mass, score = oracle.attend(rows, k[h], v[h], [n * P] * (2 * T), D ** -0.5)
        bound = attention_bound(want, mass, score, (1 << 24) * Hk // 512 // 16 + 512, D) + T * 2.0 ** -14
        within(y[:, 2 * h:2 * h + 2].reshape(2 * T, D), want, bound, f"head {h}")


def test_binding_refusals(q4, ws):
    q, cache, table, lens = (x for x in problem([40, 50], 2, 4, 2, 64, 16, 20))
    q, cache, table, lens = q.cuda(), tuple(t.cuda() for t in cache), table.cuda(), lens.cuda()
    ok = dict(q=q, cache=cache, table=table, lengths=lens, workspace=ws)
    call = lambda **kw: q4.attention_decode(**{**ok, **kw})  # noqa: E731
    call()
    for kw in (dict(q=q[0]), dict(q=q[:1]), dict(table=table[:1]), dict(lengths=lens[:1]), dict(cache=cache[:1]), dict(table=table[0]),
               dict(cache=tuple(t.transpose(1, 2) for t in cache)), dict(out=q[:, :1]), dict(n_new=lens[:1]), dict(q=q.transpose(2, 3)),
               dict(table=table.cpu()), dict(q=q.transpose(0, 1)), dict(cache=(cache[0], cache[1][:-1])), dict(window=2 ** 32 + 5),
               dict(window=1 - 2 ** 32)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=q.float()), dict(table=table.long()), dict(lengths=lens.long()), dict(cache=tuple(t.float() for t in cache)),
               dict(workspace=1 << 20), dict(n_new=lens.float()), dict(q=None), dict(cache=(*cache, *cache))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(scale=0.0), dict(window=-1), dict(workspace=ws[:70000]), dict(out=q)):
        with pytest.raises(q4.Q4GemvError):
            call(**kw)
