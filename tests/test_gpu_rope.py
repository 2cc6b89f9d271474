"""GPU parity of rope_cache against the fp64 oracle, through the binding.
Bounds: attention_util."""
import numpy as np
import pytest
import torch

import oracle
import synth
from attention_util import rope_bound, values, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def freqs(rot, base=10000.0):
    return torch.tensor(base ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32)


def problem(T, Hq, Hk, D, P, seed, e4m3=False, strided=False, far=0):
    g = synth.make_gen(("rope", T, Hq, Hk, D, P, seed))
    loud = torch.exp(torch.randn(Hq + 2 * Hk, D, generator=g))
    qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=g) * loud).to(torch.bfloat16).cuda()
    parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    q, k, v = parts if strided else [t.contiguous() for t in parts]
    pos = (torch.randint(0, 5000, (T,), generator=g) + far).to(torch.int32)
    pages = -(-T // P) + 2
    slots = torch.randperm(pages * P, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16)  # noqa: E731
    shape = (pages, Hk, P, D)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cache = [rnd(*shape).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2)]
    if e4m3:
        cache += [torch.rand(shape[:3], generator=g) for _ in range(2)]
    return q, k, v, pos, slots, w(), w(), tuple(t.cuda() for t in cache)


def check_heads(got, x, pos, freq, norm, eps, inter, what):
    x, norm = values(x), None if norm is None else values(norm)
    freq = None if freq is None else values(freq)
    want = oracle.rope_heads(x, pos.numpy(), freq, norm, eps, inter)
    within(got, want, rope_bound(x, pos.numpy(), freq, norm, eps, inter) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 1e-40, what)
    return want


def check_cache(cache, before, k_want, k_bound, v, slots):
    """Slots of tokens hold them, the others what they held."""
    after, before = [values(t) for t in cache], [values(t) for t in before]
    pages, Hk, P, D = after[0].shape
    kept = {int(s): t for t, s in enumerate(slots) if 0 <= int(s) < pages * P}
    other = np.array([s for s in range(pages * P) if s not in kept])
    for a, b in zip(after, before):
        flat = lambda t: np.moveaxis(t, 1, 2).reshape((pages * P, Hk) + t.shape[3:])  # noqa: E731
        assert np.array_equal(flat(a)[other], flat(b)[other], equal_nan=True)
    at = list(kept)
    t = [kept[s] for s in at]
    rows = [np.moveaxis(a, 1, 2).reshape((pages * P, Hk) + a.shape[3:])[at] for a in after]
    v = values(v)[t]
    if len(after) == 2:
        within(rows[0], k_want[t], k_bound[t] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(k_want[t]) + 1e-40, "cache k")
        assert np.array_equal(rows[1], v, equal_nan=True)
        return
    codes, scale = oracle.e4m3_heads(v)                 # one rounding each of what fp32 holds: exact
    assert np.array_equal(rows[1], codes, equal_nan=True)
    assert np.array_equal(rows[3].astype(np.float32), scale.astype(np.float32))
    codes, scale = oracle.e4m3_heads(k_want[t])
    top = (k_bound[t].max(-1) + np.abs(k_want[t]).max(-1) * 2.0 ** -22) / 448
    within(rows[2], scale, top + 1e-40, "cache k scale")
    err = k_bound[t] + 2.0 ** -22 * np.abs(k_want[t])
    within(rows[0] * rows[2][..., None], k_want[t], err + 2.0 ** -4 * (np.abs(k_want[t]) + err) + 2.0 ** -10 * rows[2][..., None] + 1e-40, "cache k codes")


@pytest.mark.parametrize("T,Hq,Hk,D,P", [(1, 16, 4, 128, 16), (3, 14, 2, 64, 32), (5, 1, 1, 128, 16), (48, 16, 4, 128, 64), (1, 8, 8, 64, 256),
                                         (1030, 5, 3, 64, 16), (1027, 12, 1, 128, 128), (2570, 5, 3, 64, 16), (2563, 12, 1, 128, 128)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_norm_rotate_append(q4, T, Hq, Hk, D, P, inter, e4m3, strided):
    q, k, v, pos, slots, qw, kw, cache = problem(T, Hq, Hk, D, P, 0, e4m3, strided)
    before = [t.clone() for t in cache]
    f, eps = freqs(D), 1e-5
    kept = [t.clone() for t in (q, k, v)]
    qo, ko = q4.rope_cache(q, k, v, pos.cuda(), f.cuda(), qw.cuda(), kw.cuda(), eps, inter, cache, slots.cuda(), k_out=True)
    check_heads(qo, q, pos, f, qw, eps, inter, "q")
    want = check_heads(ko, k, pos, f, kw, eps, inter, "k")
    check_cache(cache, before, want, rope_bound(values(k), pos.numpy(), values(f), values(kw), eps, inter), v, slots)
    assert all(torch.equal(a, b) for a, b in zip(kept, (q, k, v)))


@pytest.mark.parametrize("D,rot", [(128, 0), (128, 16), (128, 64), (128, 112), (64, 32), (64, 48), (64, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norms", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("T", [37, 2569])
def test_parts_of_it(q4, T, D, rot, inter, norms):
    """Partial rotations, none, either norm; without a cache; in place."""
    Hq, Hk = 6, 2
    q, k, v, pos, slots, qw, kw, cache = problem(T, Hq, Hk, D, 16, 1, strided=True)
    f = freqs(rot) if rot else None
    args = dict(positions=pos.cuda() if rot else None, inv_freq=f.cuda() if rot else None, q_norm=qw.cuda() if norms[0] else None,
                k_norm=kw.cuda() if norms[1] else None, eps=1e-6, interleaved=inter)
    qo, ko = q4.rope_cache(q, k, **args)
    check_heads(qo, q, pos, f, qw if norms[0] else None, 1e-6, inter, "q")
    check_heads(ko, k, pos, f, kw if norms[1] else None, 1e-6, inter, "k")
    q4.rope_cache(q, k, v, **args, cache=cache, slots=slots.cuda(), q_out=q, k_out=k)      # parts of one array, in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    kept = slots >= 0
    at = slots[kept]
    assert torch.equal(cache[0].cpu()[at // 16, :, at % 16], ko.cpu()[kept]) and torch.equal(cache[1].cpu()[at // 16, :, at % 16], v.cpu()[kept])


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 6000, -2 ** 31])
def test_far_positions(q4, far):
    q, k, v, pos, slots, *_ = problem(50, 2, 1, 128, 16, 2)
    pos = (pos.long() + far).to(torch.int32)
    f = freqs(128)
    qo, ko = q4.rope_cache(q, k, positions=pos.cuda(), inv_freq=f.cuda())
    check_heads(qo, q, pos, f, None, 1e-6, False, "q")
    check_heads(ko, k, pos, f, None, 1e-6, False, "k")


def test_sizes_of_values(q4):
    """Rows of zeros, of very large and very small values, infinities and NaNs:
    the norm is the formula's, and a row's codes leave out what is not finite."""
    T, D, P = 8, 128, 16
    q, k, v, pos, slots, qw, kw, cache = problem(T, 2, 1, D, P, 3, True)
    k[0], k[1], v[1] = 0, 3e38, 0
    k[2] *= 1e-38
    k[3] *= 1e30
    k[4, 0, 5], v[4, 0, 7] = float("inf"), float("-inf")
    k[5, 0, 3], v[5, 0, 9] = float("nan"), float("nan")
    v[6] = 3e38
    v[7] *= 1e-38
    slots = torch.arange(T)
    qo, ko = q4.rope_cache(q, k, v, None, None, qw.cuda(), kw.cuda(), 1e-6, False, cache, slots.cuda(), k_out=True)
    with np.errstate(invalid="ignore"):
        want = check_heads(ko, k, pos, None, kw, 1e-6, False, "k")
        fine = np.isfinite(want).all(-1)[:, 0]
    codes, scale = oracle.e4m3_heads(values(v))
    assert np.array_equal(values(cache[1])[0, 0, :T], codes[:, 0], equal_nan=True)
    assert np.array_equal(values(cache[3])[0, 0, :T].astype(np.float32), scale[:, 0].astype(np.float32))
    got = values(cache[0])[0, 0, :T] * values(cache[2])[0, 0, :T, None]
    for t in range(T):
        if fine[t]:
            within(got[t], want[t, 0], 2.0 ** -4 * np.abs(want[t, 0]) * 1.01 + values(cache[2])[0, 0, t] * 2.0 ** -9 + 1e-40, f"row {t}")
    assert np.isnan(got[5]).all()        # a NaN is in every value's norm


def test_slots_outside_and_others_left(q4):
    T, P = 20, 16
    q, k, v, pos, _, qw, kw, cache = problem(T, 2, 2, 64, P, 4)
    pages = cache[0].shape[0]
    slots = torch.tensor([pages * P, -5, 2 ** 40, -2 ** 62, pages * P + 3] + list(range(15)))
    before = [t.clone() for t in cache]
    q4.rope_cache(q, k, v, cache=cache, slots=slots.cuda())
    check_cache(cache, before, values(k), np.zeros(k.shape), v, slots)


def test_streams_graph_and_devices(q4):
    """On another stream than the default, captured and replayed with new
    inputs, with its own eager work between the replays."""
    T = 48
    q, k, v, pos, slots, qw, kw, cache = problem(T, 16, 4, 128, 16, 5, True)
    f, pos_d, slots_d, qw, kw = freqs(128).cuda(), pos.cuda(), slots.cuda(), qw.cuda(), kw.cuda()
    call = lambda c, qo, ko: q4.rope_cache(q, k, v, pos_d, f, qw, kw, 1e-6, True, c, slots_d, qo, ko)  # noqa: E731
    fresh = lambda: (tuple(t.clone() for t in cache), torch.empty_like(q), torch.empty_like(k))  # noqa: E731
    static = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*static)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*static)
    for i in range(3):
        q.copy_(torch.randn_like(q))
        v.copy_(torch.randn_like(v))
        pos_d.add_(17)
        eager = fresh()
        call(*eager)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*static[0], *static[1:]), (*eager[0], *eager[1:])))


def test_long_cache_offsets(q4):
    """Slots whose values lie past 2^32 bytes of the cache."""
    T, Hk, D, P = 4, 8, 128, 256
    pages = (1 << 32) // (Hk * P * D * 2) + 40
    q, k, v, *_ = problem(T, 8, Hk, D, P, 6)
    cache = tuple(torch.zeros(pages, Hk, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([pages * P - 1, 0, (pages - 3) * P + 7, pages * P // 2])
    q4.rope_cache(q, k, v, cache=cache, slots=slots.cuda())
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(cache[0][s // P, :, s % P], k[t]) and torch.equal(cache[1][s // P, :, s % P], v[t])
    assert sum(int((c != 0).any(-1).sum()) for c in cache) == 2 * T * Hk


def test_binding_refusals(q4):
    q, k, v, pos, slots, qw, kw, cache = problem(4, 4, 2, 64, 16, 7)
    f, pos, slots = freqs(64).cuda(), pos.cuda(), slots.cuda()
    with pytest.raises(ValueError):
        q4.rope_cache(q, k[:3], v, cache=cache, slots=slots)
    with pytest.raises(TypeError):
        q4.rope_cache(q.float(), k)
    with pytest.raises(ValueError):
        q4.rope_cache(q.transpose(0, 1), k)
    with pytest.raises(ValueError):
        q4.rope_cache(q, k, v)
    with pytest.raises(TypeError):
        q4.rope_cache(q, k, v, cache=cache, slots=slots.int())
    with pytest.raises(TypeError):
        q4.rope_cache(q, k, v, cache=cache)
    with pytest.raises(ValueError):
        q4.rope_cache(q, k, v, cache=cache[:1], slots=slots)
    with pytest.raises(ValueError):
        q4.rope_cache(q, k, v, cache=tuple(t.transpose(1, 2) for t in cache), slots=slots)
    with pytest.raises(TypeError):
        q4.rope_cache(q, k, inv_freq=f)
    with pytest.raises(TypeError):
        q4.rope_cache(q, k, positions=pos.long(), inv_freq=f)
    with pytest.raises(q4.Q4GemvError):
        q4.rope_cache(q, k, positions=pos, inv_freq=torch.ones(4, device="cuda"))
    with pytest.raises(q4.Q4GemvError):
        q4.rope_cache(q, k, q_norm=qw.cuda(), eps=0.0)
    with pytest.raises(q4.Q4GemvError):
        q4.rope_cache(q, k, q_out=k.new_empty(4, 4, 64), k_out=v, v=v, cache=cache, slots=slots)
    with pytest.raises(ValueError):
        q4.rope_cache(q, k, q_norm=torch.ones(32, dtype=torch.bfloat16, device="cuda"))
