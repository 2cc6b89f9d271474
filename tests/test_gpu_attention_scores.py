"""Attention where scores are large, infinite, or leave fp32's range, through
the binding.  Heads differ from 0 in their first column alone, so that a score
is one product, known exactly, and what a row has to give is known without a
softmax:

- scores of seen keys that lie 128 and more apart leave the largest's key alone:
  the others weigh below 2^-184, which fp32 does not hold, and the largest 2^0
  to 2^8 times its own sum of weights, so that the row is that key's value, bit
  for bit;
- a score that is +infinity, or leaves fp32's range that way, makes its row NaN
  (infinity minus infinity); -infinity weighs 0, and a row of nothing else is 0;
- keys of score 0 weigh alike, exactly, beside others that weigh 0: the row is
  the mean of n values, off by n 2^-22 of their magnitudes and one rounding.
"""
import numpy as np
import pytest
import torch

import synth
from attention_util import values, within

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def along(numbers, heads, D):
    """bf16 [n, heads, D]: numbers [n, heads] in the first column."""
    t = torch.zeros(len(numbers), heads, D, dtype=torch.float64)
    t[:, :, 0] = torch.as_tensor(numbers, dtype=torch.float64)
    out = t.to(torch.bfloat16)
    assert torch.equal(out.double(), t)
    return out.cuda()


def prefill(q4, q, k, v, scale, window):
    n, m = len(q), len(k)
    at = lambda x: torch.tensor([0, x], dtype=torch.int32, device="cuda")  # noqa: E731
    return q4.attention_prefill(q, k, v, at(n), at(m) if m != n else None, scale, window)


def decode(q4, q, k, v, scale, window):
    """The same rows over a paged cache, up to 64 at a time, as sequences of one
    cache: each call's last row sees the keys up to its own."""
    n, m, Hk, D, P = len(q), len(k), k.shape[1], k.shape[2], 16
    pages = -(-m // P)
    pad = lambda t: torch.cat((t, t.new_zeros(pages * P - m, Hk, D))).view(pages, P, Hk, D).transpose(1, 2).contiguous()  # noqa: E731
    cache = (pad(k), pad(v))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = []
    for r0 in range(0, n, 7):
        rows = q[r0:r0 + 7]
        lens = torch.tensor([m - n + r0 + len(rows)], dtype=torch.int32, device="cuda")
        out.append(q4.attention_decode(rows[None], cache, table, lens, scale=scale, window=window)[0])
    return torch.cat(out)


CALLS = {"prefill": prefill, "decode": decode}
SIZES = [7, 11, 12, 13, 20, 24, 28, 31, 32, 40, 64, 100, 118]      # 100 * 2^118 log2 e is below 2^126


def problem(n, m, Hq, Hk, D, seed):
    g = synth.make_gen(("scores", n, m, Hq, Hk, D, seed))
    place = torch.stack([torch.randperm(m, generator=g) - m // 2 for _ in range(Hk)], 1).numpy()       # [m, Hk], all different
    v = torch.randn(m, Hk, D, generator=g).to(torch.bfloat16).cuda()
    return place, v


def seen(t, more, window):
    end = t + 1 + more
    return (max(0, end - window) if window else 0), end


def best(place, sign, n, more, window):
    """Key of the largest score of each row and head: [n, Hq]."""
    Hq, G = len(sign), len(sign) // place.shape[1]
    out = np.zeros((n, Hq), np.int64)
    for t in range(n):
        lo, hi = seen(t, more, window)
        for h in range(Hq):
            out[t, h] = lo + int(np.argmax(sign[h] * place[lo:hi, h // G]))
    return out


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D,more,window", [(128, 0, 0), (64, 0, 0), (128, 50, 70), (64, 3, 100)])
def test_largest_score_alone(q4, call, size, D, more, window):
    """Scores (-100 .. 100) 2^size: the largest key's value, whichever sign."""
    n, Hq, Hk = 150, 4, 2
    place, v = problem(n, n + more, Hq, Hk, D, 0)
    sign = np.array([1, -1, -1, 1])
    q = along(np.tile(sign * 2.0 ** size, (n, 1)), Hq, D)
    y = CALLS[call](q4, q, along(place, Hk, D), v, 1.0, window)
    at = torch.from_numpy(best(place, sign, n, more, window)).cuda()
    want = torch.stack([v[at[:, h], h // 2] for h in range(Hq)], 1)
    assert torch.equal(y, want), f"rows {sorted(set((y != want).any(-1).nonzero()[:, 0].tolist()))[:8]}"


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [10, 40, 100])
def test_largest_score_with_an_infinite_value(q4, call, D, size):
    """The largest score's own value is infinite in one column: rows that see it
    have it, with the key's other values; rows before it are what they were."""
    n = 150
    for j in (149, 140, 100, 20):
        place, v = problem(n, n, 1, 1, D, 1)
        place = place.copy()
        place[place == place.max()], place[j] = place[j], place.max()
        q, k = along(np.full((n, 1), 2.0 ** size), 1, D), along(place, 1, D)
        clean = CALLS[call](q4, q, k, v, 1.0, 0)
        v = v.clone()
        v[j, 0, 5] = -INF
        y = CALLS[call](q4, q, k, v, 1.0, 0)
        assert torch.equal(y[:j], clean[:j]), j
        assert torch.equal(y[j:, 0], v[j:j + 1, 0].expand(n - j, D)), j


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("key,scale", [(2.0 ** 20, 2.0 ** 10), (2.0 ** 27, 2.0), (INF, 1.0), (2.0 ** 20, 2.0 ** 126)])
def test_infinite_scores(q4, call, D, window, key, scale):
    """Keys of scores -infinity, then 0, one of +infinity, then 0 again: infinite
    before the scale or only after it."""
    n = 200
    kind = np.array([-1.0] * 70 + [0.0] * 80 + [1.0] + [0.0] * 49)
    k = np.array([x * key if x else 0.0 for x in kind])
    v = problem(n, n, 1, 1, D, 2)[1]
    y = values(CALLS[call](q4, along(np.full((n, 1), 2.0 ** 100), 1, D), along(k[:, None], 1, D), v, scale, window))
    ve = values(v)[:, 0]
    for t in range(n):
        lo, hi = seen(t, 0, window)
        if (kind[lo:hi] > 0).any():
            assert np.isnan(y[t]).all(), t
            continue
        even = [j for j in range(lo, hi) if kind[j] == 0]
        if not even:
            assert not y[t].any(), t
            continue
        want = ve[even].mean(0)
        within(y[t, 0], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * len(even) * np.abs(ve[even]).mean(0), f"row {t}")


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -126, 2.0 ** -149])
def test_scale_at_its_limits(q4, call, scale):
    """Queries of 0 give every key the score 0, whatever the scale."""
    n, D = 70, 64
    v = problem(n, n, 1, 1, D, 3)[1]
    k = torch.randn(n, 1, D, device="cuda").to(torch.bfloat16)
    y = values(CALLS[call](q4, torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda"), k, v, scale, 0))
    ve = values(v)[:, 0]
    for t in range(n):
        want = ve[:t + 1].mean(0)
        within(y[t, 0], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * (t + 1) * np.abs(ve[:t + 1]).mean(0), f"row {t}")


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("D,Hq,Hk", [(64, 2, 1), (128, 4, 2), (128, 2, 2)])
@pytest.mark.parametrize("window", [0, 90])
def test_rows_stand_alone(q4, call, D, Hq, Hk, window):
    """What a row gives is its own keys' and its own query's, to the last bit:
    neither a key that only later rows see, however large its score, nor the
    other heads' queries beside it change it."""
    n, g = 210, synth.make_gen(("alone", D, Hq, Hk))
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v = rnd(n, Hq, D), rnd(n, Hk, D), rnd(n, Hk, D)
    clean = CALLS[call](q4, q, k, v, D ** -0.5, window)
    for j in (40, 75, 150, 170, 209):
        loud = k.clone()
        loud[j] *= 30
        y = CALLS[call](q4, q, loud, v, D ** -0.5, window)
        other = (y[:j] != clean[:j]).any(-1).any(-1)
        assert not other.any(), f"key {j}: rows {other.nonzero()[:, 0].tolist()[:8]}"
        assert not torch.equal(y[j:], clean[j:])
    for h in range(Hq):
        loud = q * 30
        loud[:, h] = q[:, h]
        y = CALLS[call](q4, loud, k, v, D ** -0.5, window)
        assert torch.equal(y[:, h], clean[:, h]), f"head {h}"


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 45])
@pytest.mark.parametrize("part", [0.95, -0.95])
def test_equal_values(q4, call, D, window, part):
    """A row's rounded weights are divided by their own sum: where all its values
    are one, that is the row.  The weights are 1 (the first key's) and one whose
    rounding to bf16 is off by 0.95 of the most, all to one side; a row's sum and its
    products differ by less than 2 300 2^-23 of them, and the value's step is 2^-8."""
    n = 300
    weight = 0.75 * (1 + part * 2.0 ** -8 / 1.5)
    k = along(np.array([[0.0]] + [[-1.0]] * (n - 1)), 1, D)
    v = torch.full((n, 1, D), 1.9921875, dtype=torch.bfloat16, device="cuda")
    y = CALLS[call](q4, along(np.ones((n, 2)), 2, D), k, v, -float(np.log(weight)), window)
    assert (y == 1.9921875).all()
