"""The CPU oracle of the draft-and-verify operators against facts fixed outside
it: torch's e4m3 conversion, exact rationals, and the law that rejection
sampling has to obey (the token that comes out is distributed as the target's
own sample)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import synth


def _bf16_bits(a):
    return synth.bits16(torch.as_tensor(np.asarray(a, np.float32)).to(torch.bfloat16))


def test_e4m3_nearest_is_the_library_rounding():
    t = np.concatenate([np.linspace(-448, 448, 100001), np.linspace(-0.04, 0.04, 100001)]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oracle.e4m3_nearest(t.astype(np.float64)), want)


def test_e4m3_nearest_ties_to_even():
    v = oracle.e4m3fn_value(np.arange(0, 127, dtype=np.uint8))      # the finite codes from 0, ascending
    mid = (v[:-1] + v[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    assert np.array_equal(oracle.e4m3_nearest(mid), even)
    assert np.array_equal(oracle.e4m3_nearest(-mid), -even)


def test_quantize_exact_rationals():
    rng = np.random.default_rng(0)
    bits = _bf16_bits(rng.normal(size=(3, 160)))
    bits[2, 128:] = 0
    codes, scale = oracle.fp8_quantize(bits)
    x = oracle.bf16_value(bits)
    grid = [Fraction(float(v)) for v in oracle.e4m3fn_value(np.arange(0, 127, dtype=np.uint8))]
    for m in range(3):
        for g in range(2):
            cols = range(128 * g, min(160, 128 * g + 128))
            a = max(abs(Fraction(float(x[m, k]))) for k in cols)
            assert Fraction(float(scale[m, g])) == pytest.approx(a / 448, rel=1e-15)
            for k in cols:
                if a == 0:
                    assert codes[m, k] == 0
                    continue
                t = abs(Fraction(float(x[m, k]))) * 448 / a
                best = min(range(127), key=lambda i: (abs(grid[i] - t), i % 2))
                assert Fraction(abs(float(codes[m, k]))) == grid[best], (m, k)


def test_gemm_exact_rationals():
    rng = np.random.default_rng(1)
    M, N, K = 2, 130, 144
    xc, wc = rng.integers(0, 127, (M, K)).astype(np.uint8), rng.integers(0, 127, (N, K)).astype(np.uint8)
    xc[0] |= 0x80
    xs, ws = rng.uniform(0.5, 2, (M, 2)).astype(np.float32), rng.uniform(0.5, 2, (2, 2)).astype(np.float32)
    r = _bf16_bits(rng.normal(size=(M, N)))
    y = oracle.fp8_gemm(xc, xs, wc, ws, r)
    xv, wv, rv = oracle.e4m3fn_value(xc), oracle.e4m3fn_value(wc), oracle.bf16_value(r)
    for m, n in ((0, 0), (1, 127), (0, 128), (1, 129)):
        want = Fraction(float(rv[m, n]))
        for k in range(K):
            want += Fraction(float(xv[m, k])) * Fraction(float(wv[n, k])) * Fraction(float(xs[m, k // 128])) * \
                Fraction(float(ws[n // 128, k // 128]))
        assert abs(y[m, n] - float(want)) <= 1e-12 * abs(float(want)) + 1e-9


def _law(verify, p, q, V):
    """The distribution of the first token over drafts d ~ q and both uniforms,
    by a grid of draws."""
    grid = (np.arange(4000) + 0.5) / 4000
    got = np.zeros(V)
    for d in np.flatnonzero(q > 0):
        accept = None
        rest = np.zeros(V)
        for x in grid:
            token, count, prob = verify(int(d), 1.0 - 2.0 ** -24, x)
            accept = prob
            if accept < 1.0:
                assert count == 0
                rest[token] += 1 / len(grid)
        got[d] += q[d] * accept
        got += q[d] * (1 - accept) * rest
    return got


def test_the_law_of_rejection_sampling_topk():
    rng = np.random.default_rng(2)
    V, k, T = 9, 5, 0.8
    lg = _bf16_bits(rng.normal(size=(1, 2, V)) * 2)
    dl = _bf16_bits(rng.normal(size=(1, V)) * 2)
    _, qi, qp = oracle.sample_topk(dl, float(np.float32(T)), k, np.zeros(1))
    _, pi, pp = oracle.sample_topk(lg[:, 0], float(np.float32(T)), k, np.zeros(1))
    p, q = np.zeros(V), np.zeros(V)
    p[pi[0]], q[qi[0]] = pp[0], qp[0]

    def run(d, u0, u1):
        t, c, a = oracle.verify_topk(lg, np.array([[d]]), np.array([[u0, u1]]), qi[None], qp[None], None, T, k)
        return int(t[0, int(c[0])]), int(c[0]), float(a[0, 0])

    assert np.allclose(_law(run, p, q, V), p, atol=2e-3)


def test_the_law_of_rejection_sampling_full():
    rng = np.random.default_rng(3)
    V, T = 7, 1.3
    lg = _bf16_bits(rng.normal(size=(1, 2, V)) * 2)
    dl = _bf16_bits(rng.normal(size=(1, 1, V)) * 2)

    def softmax(bits):
        e = np.exp(oracle.bf16_value(bits) / float(np.float32(T)))
        return e / e.sum()

    p, q = softmax(lg[0, 0]), softmax(dl[0, 0])

    def run(d, u0, u1):
        t, c, a = oracle.verify_full(lg, np.array([[d]]), np.array([[u0, u1]]), dl, None, T)
        return int(t[0, int(c[0])]), int(c[0]), float(a[0, 0])

    assert np.allclose(_law(run, p, q, V), p, atol=2e-3)


def test_verify_by_hand():
    """p = (1/2, 1/4, 1/4) at every row; the draft was certain of its tokens."""
    bits = _bf16_bits(np.broadcast_to([1.0, 0.0, 0.0], (1, 3, 3)))
    T = float(1 / np.log(2.0))
    t, c, a = oracle.verify_full(bits, np.array([[0, 1]]), np.array([[0.49, 0.26, 0.3]]), None, None, T)
    # 0 stands (0.49 < 1/2), 1 does not (0.26 >= 1/4): drawn from (1/2, 0, 1/4), 0.3 < 2/3
    assert t.tolist() == [[0, 0, -1]] and c.tolist() == [1]
    assert np.allclose(a, [[0.5, 0.25]], rtol=1e-6)
    t, c, _ = oracle.verify_full(bits, np.array([[0, 1]]), np.array([[0.49, 0.24, 0.9]]), None, None, T)
    assert t.tolist() == [[0, 1, 2]] and c.tolist() == [2]
    t, c, _ = oracle.verify_full(bits, np.array([[0, 1]]), np.array([[0.49, 0.24, 0.6]]), None, np.array([0]), T)
    assert t.tolist() == [[1, -1, -1]] and c.tolist() == [0]
