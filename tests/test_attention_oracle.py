"""The attention oracle against facts fixed outside it."""
import math

import numpy as np
import pytest

import oracle


def test_rotation_by_a_quarter_turn():
    x = np.arange(1.0, 17.0).reshape(1, 1, 16)
    f = [math.pi / 2] + [0.0] * 7
    y = oracle.rope_heads(x, [1], f)
    assert np.allclose(y[0, 0], [-9, 2, 3, 4, 5, 6, 7, 8, 1, 10, 11, 12, 13, 14, 15, 16])
    y = oracle.rope_heads(x, [1], f, interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1] + list(range(3, 17)))


def test_rotation_keeps_lengths_and_products():
    """Turned by positions m and n, a pair's product depends on m - n alone."""
    g = np.random.default_rng(0)
    q, k = g.standard_normal((2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    for inter in (False, True):
        turn = lambda x, m: oracle.rope_heads(x, [m], f, interleaved=inter)[0, 0]  # noqa: E731
        assert np.isclose(np.linalg.norm(turn(q, 77)), np.linalg.norm(q))
        assert np.isclose(turn(q, 1007) @ turn(k, 1000), turn(q, 7) @ turn(k, 0))


def test_norm():
    x = np.array([[[3.0, 4.0]]])
    y = oracle.rope_heads(x, norm=[1.0, 2.0], eps=0.0)
    assert np.allclose(y, [[[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]])


def test_codes():
    codes, scale = oracle.e4m3_heads(np.array([[448.0, -1.0, 0.3, np.inf], [0.0, 0.0, 0.0, 0.0]]))
    assert scale.tolist() == [1.0, 0.0]
    assert codes[0, :3].tolist() == [448.0, -1.0, 0.3125] and np.isnan(codes[0, 3]) and not codes[1].any()


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attend(window):
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((3, 5, 4))
    end = np.array([0, 1, 2, 5, 5])
    y, _, _ = oracle.attend(q, k, v, end, 0.5, window)
    for i in range(5):
        lo = max(0, end[i] - window) if window else 0
        w = [math.exp(0.5 * float(q[i] @ k[j])) for j in range(lo, end[i])]
        want = sum((x / sum(w) * v[lo + n] for n, x in enumerate(w)), np.zeros(4))
        assert np.allclose(y[i], want)
    assert not y[0].any()


def test_paged():
    cache = np.arange(3 * 2 * 16 * 1.0).reshape(3, 2, 16, 1)
    got, held = oracle.paged(cache, [2, -1, 0], 40, 1)
    assert got.shape == (40, 1) and held.tolist() == [True] * 16 + [False] * 16 + [True] * 8
    assert got[3, 0] == cache[2, 1, 3, 0] and got[33, 0] == cache[0, 1, 1, 0]
    assert len(oracle.paged(cache, [0], 99, 0)[0]) == 16 and len(oracle.paged(cache, [0], -4, 0)[0]) == 0
