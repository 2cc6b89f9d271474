"""Inputs that show each part of a decode call's work by itself, what has to come
out, and how far it may be off.  Over random keys a lost part of some hundred
among 70000 is inside any bound of a softmax's rounding.

Counted.  Queries of 0: every key weighs 1, exactly.  Value j is 2^h (of key head
h) in one column: the sequence's tiles of 32 keys are split over the D columns,
each a run of them, so that a column counts its keys, and a row is those counts
2^h / n.  Sums of up to 2^24 ones are exact in fp32 in any order, and so are the
factors that join them (2^0): what is left is the quotient's rounding, below
2^-22, and the one to bf16, 2^-8.  With 34 tiles to a column (70001 keys, 64
columns) a lost, doubled or misplaced tile is 2.9 % of its column; larger parts
are whole columns.

Planted.  Key j of a row is 8 times its query: it outweighs all others by e^40 (a
condition that is checked), and the row is value j, which bf16 holds.  Every tile
of 32 keys has its turn.  A part that is lost or joined into another row is
another value altogether.

Marked.  A table of 2^24 keys that names one page of zeros everywhere but at
chosen places, each of which has a page of its own, of keys that outweigh those
zeros by e^14, and values of 1, 2 or 4 in one column: a column counts its marked
pages, up to 16 of them, so that one that is lost, doubled or read with another
page's keys, values or scales is 2.7 % of its column or more.  Marked keys weigh 1,
exactly, and the others have no value; the sum of up to 2^24 weights is off by the
weights a lane adds, some thousand of 2^-24 each, below 2^-10.
"""
import numpy as np
import torch

import synth

TILE = 32


def pages_of(lengths, P, g, spare=2):
    """(table [B, width], pages): every sequence's pages, in no order."""
    need = [-(-n // P) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


# ---------------------------------------------------------------------------
# counted
# ---------------------------------------------------------------------------
def column_of(n, D):
    """The columns that n keys count in."""
    tiles = -(-n // TILE)
    return np.arange(n) // TILE // max(1, -(-tiles // D))


def counted(lengths, T, Hq, Hk, D, P, e4m3):
    """(q, cache, table, lengths) on the CPU."""
    g = synth.make_gen(("counted", tuple(lengths), T, Hq, Hk, D, P))
    table, pages = pages_of(lengths, P, g)
    k = torch.randn(pages, Hk, P, D, generator=g)
    v = torch.full((pages, Hk, P, D), float("nan"))
    top = 2.0 ** torch.arange(Hk)
    for b, n in enumerate(lengths):
        j = torch.arange(n)
        one = torch.zeros(n, D)
        one[j, torch.from_numpy(column_of(n, D))] = 1.0
        v[table[b, j // P].long(), :, j % P] = one[:, None] * (1.0 if e4m3 else top[:, None])
    q = torch.zeros(len(lengths), T, Hq, D, dtype=torch.bfloat16)
    if not e4m3:
        return q, (k.to(torch.bfloat16), v.to(torch.bfloat16)), table, torch.tensor(lengths, dtype=torch.int32)
    cache = (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.rand(pages, Hk, P, generator=g),
             top[:, None].expand(pages, Hk, P).contiguous())
    return q, cache, table, torch.tensor(lengths, dtype=torch.int32)


def counted_want(lengths, n_new, T, Hq, Hk, D, window=0):
    """fp64 [B, T, Hq, D]."""
    y = np.zeros((len(lengths), T, Hk, Hq // Hk, D))
    for b, n in enumerate(lengths):
        new = T if n_new is None else int(n_new[b])
        for i in range(new):
            end = n - new + i + 1
            lo = max(0, end - window) if window else 0
            if end > lo:
                count = np.bincount(column_of(n, D)[lo:end], minlength=D) / (end - lo)
                y[b, i] = count * 2.0 ** np.arange(Hk)[:, None, None]
    return y.reshape(len(lengths), T, Hq, D)


def counted_check(y, want):
    assert y.shape == want.shape
    bad = ~(np.abs(y - want) <= (2.0 ** -8 + 2.0 ** -20) * want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first {tuple(np.argwhere(bad)[0])}: {y[bad][0]!r}, not {want[bad][0]!r}"


# ---------------------------------------------------------------------------
# planted
# ---------------------------------------------------------------------------
class Planted:
    """A cache on `device` and its queries; `plant(s)` puts turn s's keys in,
    `lift()` takes them out, `check(y)` compares a call's outputs."""
    def __init__(self, lengths, T, Hq, Hk, D, P, e4m3, device):
        g = synth.make_gen(("planted", tuple(lengths), T, Hq, Hk, D, P))
        self.lengths, self.T, self.Hk, self.D, self.P, self.e4m3 = lengths, T, Hk, D, P, e4m3
        self.R = T * (Hq // Hk)
        table, pages = pages_of(lengths, P, g)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q = (rnd(len(lengths), T, Hq, D) * 1.5).to(torch.float8_e4m3fn).to(torch.bfloat16)
        kv = [rnd(pages, Hk, P, D).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2)]
        if e4m3:
            kv += [torch.ones(pages, Hk, P), 2.0 ** torch.randint(-2, 3, (pages, Hk, P), generator=g)]
        self.cache = tuple(t.to(device) for t in kv)
        self.v = kv[1].float() * (kv[3][..., None] if e4m3 else 1.0)         # what a row that sees one key gives
        self.table = table
        self.lens = torch.tensor(lengths, dtype=torch.int32)
        # rows of a key head [B, Hk, R, D], in the order of tokens, then heads
        G = Hq // Hk
        self.rows = self.q.view(len(lengths), T, Hk, G, D).transpose(1, 2).reshape(len(lengths), Hk, self.R, D)
        self._margin(kv)
        self.turns = max(-(-(-(-n // TILE)) // self.R) for n in lengths)

    def _margin(self, kv):
        scale = self.D ** -0.5
        k = kv[0].float()
        for b, n in enumerate(self.lengths):
            at = self.table[b, :-(-n // self.P)].long()
            for h in range(self.Hk):
                r = self.rows[b, h].float()
                z = r @ r.T * 8 * scale
                own = z.diagonal().clone()
                z.fill_diagonal_(-np.inf)
                other = torch.maximum(z.amax(1), (r @ k[at, h].reshape(-1, self.D).T * scale).amax(1))
                assert (own - other).min() > 40, "a planted key does not outweigh the others"

    def spots(self, s):
        """Keys [B, R] of turn s: every tile in turn, at changing places of it; all rows see them."""
        out = np.zeros((len(self.lengths), self.R), np.int64)
        for b, n in enumerate(self.lengths):
            last = n - self.T                    # the last key that the first row sees
            tiles = last // TILE + 1
            assert tiles >= self.R, "as many tiles as rows, each row's key in its own"
            for r in range(self.R):
                tile = (s * self.R + r) % tiles
                out[b, r] = min(last, tile * TILE + (7 * s + 5 * r) % TILE)
        return out

    def plant(self, s):
        self.at = torch.from_numpy(self.spots(s))
        b = torch.arange(len(self.lengths))[:, None]
        self.page, self.slot = self.table[b, self.at // self.P].long(), self.at % self.P
        h = torch.arange(self.Hk)[None, :, None]
        self.index = (self.page[:, None].expand(-1, self.Hk, -1), h.expand(len(self.lengths), -1, self.R),
                      self.slot[:, None].expand(-1, self.Hk, -1))
        where = tuple(t.to(self.cache[0].device) for t in self.index)
        k = self.cache[0].view(torch.uint8) if self.e4m3 else self.cache[0]
        self.kept = (where, k[where].clone())
        rows = self.rows.to(k.device)
        k[where] = rows.to(torch.float8_e4m3fn).view(torch.uint8) if self.e4m3 else rows * 8
        if self.e4m3:
            self.cache[2][where] = 8.0

    def lift(self):
        where, k = self.kept
        (self.cache[0].view(torch.uint8) if self.e4m3 else self.cache[0])[where] = k
        if self.e4m3:
            self.cache[2][where] = 1.0

    def want(self):
        """fp32 [B, T, Hq, D]: the planted keys' values."""
        B, T = len(self.lengths), self.T
        v = self.v[self.index]                                                # [B, Hk, R, D]
        return v.view(B, self.Hk, T, self.R // T, self.D).transpose(1, 2).reshape(B, T, -1, self.D)

    def check(self, y, what=""):
        want = self.want()
        y = y.float().cpu()
        # the others together are below n e^-40 4; the value is a bf16 number
        bad = ~((y - want).abs() <= 2.0 ** -10 * want.abs() + 1e-10)
        assert not bad.any(), f"{what}: {int(bad.any(-1).sum())} rows off, first {bad.any(-1).nonzero()[0].tolist()}"


# ---------------------------------------------------------------------------
# marked
# ---------------------------------------------------------------------------
WORKGROUPS, OWN = 512, 8         # of a decode call of many tiles; places that a unit takes beside its tiles


def list_pages(D, R):
    """Pages that a workgroup's list holds: 4 waves' outputs of 16 or 32 rows, in whole steps of 128 keys."""
    return 4 * (16 if R <= 16 else 32) * (D + 4) // 8 * 8


def segments(n, Hk, R):
    """(first tile, tiles) of every workgroup's part of a unit, one sequence of n keys."""
    Z = -(-R // 32)
    tiles = -(-n // TILE)
    unit = tiles + OWN
    total = Hk * Z * unit
    share = -(-total // WORKGROUPS)
    out = []
    for start in range(0, total, share):
        pos, stop = start, min(total, start + share)
        while pos < stop:
            at = pos % unit
            first, last = max(at, OWN), min(unit, at + stop - pos)
            if last > first:
                out.append((first - OWN, last - first))
            pos += min(unit - at, stop - pos)
    return out


def places(n, Hk, R, D, P, most):
    """Page numbers of the sequence where a workgroup's part or a list of its
    pages begins or ends, those of up to `most` segments; how many lists end
    inside a segment."""
    parts = segments(n, Hk, R)
    hold, ends, found = list_pages(D, R), 0, set()
    chosen = parts if len(parts) <= most else [parts[i * (len(parts) - 1) // (most - 1)] for i in range(most)]
    whole = n // P
    for first, tiles in chosen:
        page, last = first * TILE // P, ((first + tiles) * TILE - 1) // P
        found |= {page, last}
        while (page := page + hold) <= last:
            found |= {page - 1, page, page + 1}
            ends += 1
    return sorted(x for x in found if x < whole), ends


LOUD = 14.0                      # of a marked key's score, 3.5 * 4 (e4m3 and bf16 numbers)


def marked(n, T, Hq, Hk, D, P, e4m3, at):
    """(q, cache, table, lengths) on the CPU, pages `at` of the table marked."""
    pages = 1 + len(at)
    value = 2.0 ** (torch.arange(len(at)) // D % 3)
    q = torch.zeros(1, T, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = 4.0
    k, v = torch.zeros(pages, Hk, P, D), torch.zeros(pages, Hk, P, D)
    k[1:, :, :, 0] = 3.5
    m = torch.arange(len(at))
    v[1 + m, :, :, m % D] = 1.0 if e4m3 else value[:, None, None]
    table = torch.zeros(1, -(-n // P), dtype=torch.int32)
    table[0, torch.tensor(at)] = (1 + m).to(torch.int32)
    lens = torch.tensor([n], dtype=torch.int32)
    if not e4m3:
        return q, (k.to(torch.bfloat16), v.to(torch.bfloat16)), table, lens
    ks, vs = torch.full((pages, Hk, P), 0.25), torch.full((pages, Hk, P), 16.0)
    ks[1:], vs[1:] = 1.0, value[:, None, None]
    return q, (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), ks, vs), table, lens


def marked_want(n, T, D, P, at, counts=None):
    """fp64 [T, D]; counts: how often each marked page is taken (1)."""
    m = np.arange(len(at))
    counts = np.ones(len(at)) if counts is None else counts
    loud = np.exp(LOUD)
    y = np.zeros((T, D))
    for i in range(T):
        end = n - T + i + 1
        l = loud * P * counts.sum() + (end - P * len(at))
        np.add.at(y[i], m % D, loud * P * counts * 2.0 ** (m // D % 3) / l)
    return y


def marked_check(y, want):
    assert y.shape == want.shape
    bad = ~(np.abs(y - want) <= (2.0 ** -8 + 2.0 ** -9) * want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first {tuple(np.argwhere(bad)[0])}: {y[bad][0]!r}, not {want[bad][0]!r}"
