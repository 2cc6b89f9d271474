"""That the inputs which show each part of a decode call (attention_parts) show
it: mistakes planted in a plain computation are found."""
import numpy as np
import pytest
import torch

import oracle
from attention_parts import TILE, Planted, counted, counted_check, counted_want, list_pages, marked, marked_check, marked_want, places, segments


def rounded(y):
    return torch.from_numpy(y).to(torch.bfloat16).double().numpy()


def gathered(cache, table, n, h):
    """(k, v) fp64 [n, D] of a sequence and key head."""
    P = cache[0].shape[2]
    at = table[:-(-n // P)].long()
    out = []
    for i in (0, 1):
        t = cache[i][at, h].double()
        if len(cache) == 4:
            t = t * cache[2 + i][at, h].double()[..., None]
        out.append(t.reshape(-1, t.shape[-1])[:n].numpy())
    return out


def sums(q, k, v, scale, keys):
    """Sums of weights and of weighted values over the given keys, for rows q."""
    z = q @ k[keys].T * scale
    w = np.exp(z - (q @ k.T * scale).max(1, keepdims=True))
    return w.sum(1), w @ v[keys]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,D", [(70001, 64), (70001, 128), (16000, 64), (20000, 128)])
def test_counted_shows_a_tile(n, D, e4m3):
    q, cache, table, _ = counted([n], 1, 1, 1, D, 64, e4m3)
    k, v = gathered(cache, table[0], n, 0)
    want = counted_want([n], None, 1, 1, 1, D)
    zero = np.zeros((1, D))
    l, o = sums(zero, k, v, 1.0, np.arange(n))
    counted_check(rounded(o / l[:, None])[None, None], want)
    tiles = -(-n // TILE)
    share = max(1, tiles // 512)
    # tiles lost, counted twice, one in place of another; a part of as many as a workgroup has, 16 of them
    for first, count in [(0, 1), (tiles // 2, 1), (tiles - 2, 1), (100, share), (100, 16 * share), (tiles - share, share)]:
        keys = np.arange(first * TILE, min(n, (first + count) * TILE))
        part_l, part_o = sums(zero, k, v, 1.0, keys)
        for sign in (-1, 1):
            with pytest.raises(AssertionError):
                counted_check(rounded((o + sign * part_o) / (l + sign * part_l)[:, None])[None, None], want)
        other_l, other_o = sums(zero, k, v, 1.0, (keys + 37 * TILE * count) % (tiles * TILE - TILE))
        with pytest.raises(AssertionError):
            counted_check(rounded((o - part_o + other_o) / (l - part_l + other_l)[:, None])[None, None], want)


def test_counted_rows_heads_and_windows():
    lengths, T, Hq, Hk, D, P = [0, 5, 300, 1000], 3, 4, 2, 64, 16
    q, cache, table, lens = counted(lengths, T, Hq, Hk, D, P, False)
    for n_new, window in ((None, 0), ([0, 2, 1, 3], 0), (None, 77)):
        want = counted_want(lengths, n_new, T, Hq, Hk, D, window)
        for b, n in enumerate(lengths):
            new = T if n_new is None else n_new[b]
            for h in range(Hk):
                k, v = gathered(cache, table[b], n, h) if n else (np.zeros((0, D)), np.zeros((0, D)))
                y, _, _ = oracle.attend(np.zeros((new, D)), k, v, n - new + 1 + np.arange(new), 1.0, window)
                assert np.allclose(want[b, :new, 2 * h], y, rtol=1e-12) and np.array_equal(want[b, :, 2 * h], want[b, :, 2 * h + 1])
            assert not want[b, new:].any()


@pytest.mark.parametrize("e4m3", [False, True])
def test_planted_shows_a_part(e4m3):
    n, T, Hq, Hk, D = 3001, 2, 4, 2, 64
    p = Planted([n], T, Hq, Hk, D, 16, e4m3, "cpu")
    seen = set()
    before = [t.clone() for t in p.cache]
    for s in range(p.turns):
        p.plant(s)
        seen |= set((p.at // TILE).flatten().tolist())
        if s % 8 == 0:
            y = np.zeros((1, T, Hq, D))
            lost = y.copy()
            for h in range(Hk):
                k, v = gathered(p.cache, p.table[0], n, h)
                rows = p.rows[0, h].double().numpy()
                l, o = sums(rows, k, v, D ** -0.5, np.arange(n))
                y[0, :, 2 * h:2 * h + 2] = (o / l[:, None]).reshape(T, 2, D)
                # the tile of the first row's key, of key head 1, is lost
                at = int(p.at[0, 0]) // TILE * TILE
                kept = np.array([j for j in range(n) if h == 0 or not at <= j < at + TILE])
                l, o = sums(rows, k, v, D ** -0.5, kept)
                lost[0, :, 2 * h:2 * h + 2] = (o / l[:, None]).reshape(T, 2, D)
            p.check(torch.from_numpy(y).to(torch.bfloat16))
            for wrong in (lost, y[:, ::-1].copy(), y[:, :, ::-1].copy(), y[:, :, [0, 1, 3, 2]].copy()):
                with pytest.raises(AssertionError):
                    p.check(torch.from_numpy(wrong).to(torch.bfloat16))
        p.lift()
    assert len(seen) >= (n - T) // TILE
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, p.cache))


REFILLED = [(64, 3, 1, 1, 16), (128, 8, 1, 1, 16), (64, 8, 2, 9, 16), (64, 8, 1, 1, 32)]


@pytest.mark.parametrize("D,Hk,G,T,P", REFILLED)
def test_marked_shows_a_list(D, Hk, G, T, P):
    n = (1 << 24) - 5
    at, ends = places(n, Hk, G * T, D, P, 8 * D // 5)
    assert ends > D and 4 * D < len(at) <= 16 * D
    parts = segments(n, Hk, G * T)
    assert sum(t for _, t in parts) == Hk * -(-G * T // 32) * -(-n // TILE)
    want = marked_want(n, T, D, P, at)
    marked_check(rounded(want), want)
    at = np.array(at)
    # one marked page lost or taken twice; a list of pages lost, or the one before it in its place
    first, tiles = max(parts, key=lambda s: s[1])
    page, hold = first * TILE // P, list_pages(D, G * T)
    for keep in [np.where(at == at[len(at) // 2], x, 1.0) for x in (0.0, 2.0)] + [np.where((at >= page + hold) & (at < page + 2 * hold), 0.0, 1.0),
                                                                                 np.where((at >= page) & (at < page + hold), 2.0, 1.0)]:
        assert (keep != 1).any()
        with pytest.raises(AssertionError):
            marked_check(rounded(marked_want(n, T, D, P, at, keep)), want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_marked_inputs(e4m3):
    """The inputs give what is wanted of them."""
    n, T, Hq, Hk, D, P = 40000 - 5, 2, 4, 2, 64, 16
    at = [0, 3, 4, 900] + list(range(1000, 1140))
    q, cache, table, _ = marked(n, T, Hq, Hk, D, P, e4m3, at)
    for h in range(Hk):
        k, v = gathered(cache, table[0], n, h)
        y, _, _ = oracle.attend(q[0, :, 2 * h].double().numpy(), k, v, n - T + 1 + np.arange(T), 1.0)
        assert np.allclose(y, marked_want(n, T, D, P, at), rtol=1e-12)
