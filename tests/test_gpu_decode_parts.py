"""attention_decode's parts one by one, through the binding: that each tile of
keys, each workgroup's part, each group of a join and each list of pages arrives
once and where it belongs.  Inputs and tolerances: attention_parts; that they show
what they are meant to: test_attention_parts.  And infinities and NaNs, row by row
of every sequence and head."""
import numpy as np
import pytest
import torch

from attention_parts import Planted, counted, counted_check, counted_want, list_pages, marked, marked_check, marked_want, places, segments
from attention_util import values
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


def on_gpu(q, cache, table, lens):
    return q.cuda(), tuple(t.cuda() for t in cache), table.cuda(), lens.cuda()


# one unit over all workgroups, with joins in one to four turns (1 to 32 rows, or
# two units of them); units that share workgroups; ragged ones
LENGTHS = [([70001], 1, 1, 1), ([70001], 3, 2, 1), ([70001], 2, 6, 1), ([70001], 8, 4, 1), ([70001], 16, 4, 1), ([20000], 1, 2, 2),
           ([9000, 14000, 33, 16000, 4500], 1, 12, 1), ([9000, 14000, 70, 16000, 4500], 8, 6, 2), ([9000, 1100, 4097, 300], 1, 4, 2),
           ([1300] * 3 + [40] * 70 + [5000, 700], 1, 4, 2), ([3000] * 64 + [40000], 5, 4, 1)]


@pytest.mark.parametrize("lengths,T,G,Hk", LENGTHS)
@pytest.mark.parametrize("D,P", [(64, 64), (128, 16)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_every_tile_counts(q4, ws, lengths, T, G, Hk, D, P, e4m3):
    q, cache, table, lens = on_gpu(*counted(lengths, T, G * Hk, Hk, D, P, e4m3))
    n_new = [1 + (3 * b) % T for b in range(len(lengths))]
    for new, window in ((None, 0), (n_new, 0), (None, 1000)):
        dev = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        y = q4.attention_decode(q, cache, table, lens, dev, 1.0, window, workspace=ws)
        assert not ws[:65536].any()
        counted_check(values(y), counted_want(lengths, new, T, G * Hk, Hk, D, window))


@pytest.mark.parametrize("lengths,T,G,Hk", [c for c in LENGTHS if min(c[0]) > 32 * c[1] * c[2] + c[1]])
@pytest.mark.parametrize("e4m3", [False, True])
def test_every_tile_decides(q4, ws, lengths, T, G, Hk, e4m3):
    p = Planted(lengths, T, G * Hk, Hk, 64, 64, e4m3, "cuda")
    q, table, lens = p.q.cuda(), p.table.cuda(), p.lens.cuda()
    for s in range(p.turns):
        p.plant(s)
        y = q4.attention_decode(q, p.cache, table, lens, workspace=ws)
        p.check(y, f"turn {s}")
        p.lift()
    assert not ws[:65536].any()


@pytest.mark.parametrize("D,Hk,G,T,P,e4m3", [(64, 3, 1, 1, 16, False), (128, 8, 1, 1, 16, False), (64, 8, 2, 9, 16, False),
                                             (64, 8, 1, 1, 32, False), (64, 4, 1, 1, 16, True), (128, 8, 1, 1, 16, True)])
def test_every_list_of_pages(q4, ws, D, Hk, G, T, P, e4m3):
    """More pages to a workgroup than its list holds: those at the ends of its
    lists and of its part, each with keys and values of its own."""
    n = (1 << 24) - 5
    assert min(t for _, t in segments(n, Hk, G * T)[:8]) * 32 > list_pages(D, G * T) * P
    at, ends = places(n, Hk, G * T, D, P, 8 * D // 5)
    assert ends > D
    y = q4.attention_decode(*on_gpu(*marked(n, T, G * Hk, Hk, D, P, e4m3, at)), scale=1.0, workspace=ws)
    want = marked_want(n, T, D, P, at)
    for h in range(G * Hk):
        marked_check(values(y)[0, :, h], want)


@pytest.mark.parametrize("T,window", [(1, 0), (1, 50), (4, 0), (4, 50), (64, 0), (40, 20)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(4, 1), (6, 2)])
def test_keys_that_are_no_numbers(q4, ws, T, window, e4m3, Hq, Hk):
    """NaNs in keys at the ends of what rows see: every head of every row that
    sees one is NaN, every other row what it is without."""
    lengths, P = [200, 161, 300, 75], 16
    p = problem(lengths, T, Hq, Hk, 128, P, 30, e4m3)
    q, cache, table, lens = on_gpu(*p)
    call = lambda: q4.attention_decode(q, cache, table, lens, window=window, workspace=ws)  # noqa: E731
    clean = call()
    spots = {b: [n - 1] + ([n - window - 1] if window else [n - 40]) for b, n in enumerate(lengths)}
    for b, js in spots.items():
        for j in js:
            page, at = int(p[2][b, j // P]), j % P
            if e4m3:
                cache[0].view(torch.uint8)[page, :, at, 7] = 0x7F
            else:
                cache[0][page, :, at, 7] = float("nan")
    y = call()
    for b, n in enumerate(lengths):
        for i in range(T):
            end = n - T + i + 1
            if any(max(0, end - window if window else 0) <= j < end for j in spots[b]):
                assert torch.isnan(y[b, i]).all(), (b, i)
            else:
                assert torch.equal(y[b, i], clean[b, i]), (b, i)


@pytest.mark.parametrize("T,window", [(1, 0), (4, 0), (4, 50), (64, 0), (40, 20)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,Hq,Hk", [(128, 4, 1), (64, 6, 2)])
def test_values_that_are_no_numbers(q4, ws, T, window, e4m3, D, Hq, Hk):
    """An infinity or NaN in one column of a value, each sequence and head with
    columns of its own: that column of the rows that see it, and nothing else."""
    lengths, P, G = [200, 161, 300, 75], 16, Hq // Hk
    p = problem(lengths, T, Hq, Hk, D, P, 31, e4m3)
    q, cache, table, lens = on_gpu(*p)
    call = lambda: q4.attention_decode(q, cache, table, lens, window=window, workspace=ws)  # noqa: E731
    clean = call()
    want = clean.clone()
    for b, n in enumerate(lengths):
        js = sorted({n - 1, n - 2, max(n - T - 1, 0), max(n - T - (window or 35), 0), max(n - (window or 50) - 2, 0)})
        for h in range(Hk):
            for x, j in enumerate(js):
                page, at, col = int(p[2][b, j // P]), j % P, (11 * b + 5 * h + 3 * x) % D
                odd = [float("inf"), float("nan"), float("-inf")][(b + h + x) % 3]
                if e4m3:
                    odd = float("nan")
                    cache[1].view(torch.uint8)[page, h, at, col] = 0x7F
                else:
                    cache[1][page, h, at, col] = odd
                for i in range(T):
                    end = n - T + i + 1
                    if max(0, end - window if window else 0) <= j < end:
                        want[b, i, h * G:(h + 1) * G, col] = odd
    y = call()
    same = (y == want) | (torch.isnan(y) & torch.isnan(want))
    assert same.all(), (~same).nonzero()[:4].tolist()


@pytest.mark.parametrize("T,Hq,Hk,D", [(1, 16, 4, 128), (5, 8, 2, 64), (8, 6, 1, 128)])
@pytest.mark.parametrize("window", [0, 45])
@pytest.mark.parametrize("part", [0.95, -0.95])
def test_equal_values(q4, ws, T, Hq, Hk, D, window, part):
    """A row's rounded weights are divided by their own sum: where all values that
    it sees are one, that is the row.  The weights are 1 (the first key that a row
    sees, the first of all, or none) and the one whose rounding to bf16 is off by
    0.95 of the most, all to one side; the value's last step is 2^-8 of it.  The sum
    and the products of 9000 weights in fp32 are at most 2 9000 2^-23 apart, less
    than half of that step."""
    q, cache, table, lens = on_gpu(*problem([9000, 77, 8, 700], T, Hq, Hk, D, 16, 32))
    q.zero_()[..., 0] = 1.0
    cache[0].zero_()[..., 0] = -1.0
    for b in range(4):
        cache[0][table[b, 0].item(), :, 0, 0] = 0.0
    weight = 0.75 * (1 + part * 2.0 ** -8 / 1.5)
    cache[1].fill_(1.9921875)
    y = q4.attention_decode(q, cache, table, lens, scale=-np.log(weight), window=window, workspace=ws)
    assert (y == 1.9921875).all()
