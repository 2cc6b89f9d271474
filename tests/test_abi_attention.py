"""Refusals of the attention entry points, on the host (only invalid argument
sets and size queries are passed, so nothing is launched)."""
import ctypes
import math

import pytest
import torch

q4 = pytest.importorskip("bit_weight_only_q4g128_amd")
lib = q4.lib

OK, EPTR, ESHAPE, EALIGN, EALIAS, ESCRATCH = 0, -1, -2, -3, -4, -7
STEP = 1 << 40       # between made-up device addresses; never dereferenced


def at(i):
    return STEP * (i + 1)


def kv(k=at(20), v=at(21), ks=None, vs=None, pages=8, page_size=16):
    return q4.KvCache(k, v, ks, vs, pages, page_size)


def rope(q=at(0), k=at(1), v=at(2), T=4, Hq=16, Hk=4, D=128, qs=2048, ks=512, vs=512, qn=at(3), kn=at(4), eps=1e-6, pos=at(5), freq=at(6),
         rot=128, inter=0, q_out=at(7), k_out=at(8), cache=kv(), slots=at(9)):
    return lib.q4_rope_cache(q, k, v, T, Hq, Hk, D, qs, ks, vs, qn, kn, eps, pos, freq, rot, inter, q_out, k_out,
                             None if cache is None else ctypes.byref(cache), slots, None)


CACHE = [
    (dict(pages=0), ESHAPE), (dict(page_size=8), ESHAPE), (dict(page_size=24), ESHAPE), (dict(page_size=512), ESHAPE),
    (dict(page_size=0), ESHAPE), (dict(page_size=-16), ESHAPE), (dict(pages=-1), ESHAPE), (dict(pages=1 << 25), ESHAPE),
]


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), EPTR), (dict(k=None), EPTR), (dict(v=None), EPTR), (dict(q_out=None), EPTR), (dict(slots=None), EPTR),
    (dict(pos=None), EPTR), (dict(freq=None), EPTR), (dict(cache=None, k_out=None), EPTR),
    (dict(T=0), ESHAPE), (dict(T=(1 << 22) + 1), ESHAPE), (dict(Hq=0), ESHAPE), (dict(Hq=257, qs=1 << 17), ESHAPE), (dict(Hk=0), ESHAPE),
    (dict(D=96), ESHAPE), (dict(D=256), ESHAPE), (dict(rot=-16), ESHAPE), (dict(rot=8), ESHAPE), (dict(rot=144), ESHAPE),
    (dict(D=64, rot=128), ESHAPE), (dict(eps=0.0), ESHAPE), (dict(eps=-1.0), ESHAPE), (dict(eps=math.nan), ESHAPE), (dict(eps=math.inf), ESHAPE),
    (dict(qs=2047), ESHAPE), (dict(qs=2040), ESHAPE), (dict(qs=2052), ESHAPE), (dict(ks=504), ESHAPE), (dict(vs=504), ESHAPE), (dict(vs=-512), ESHAPE),
    (dict(q=at(0) + 8), EALIGN), (dict(k=at(1) + 2), EALIGN), (dict(v=at(2) + 8), EALIGN), (dict(qn=at(3) + 2), EALIGN),
    (dict(kn=at(4) + 8), EALIGN), (dict(pos=at(5) + 2), EALIGN), (dict(freq=at(6) + 1), EALIGN), (dict(q_out=at(7) + 8), EALIGN),
    (dict(k_out=at(8) + 8), EALIGN), (dict(slots=at(9) + 4), EALIGN),
    (dict(q_out=at(0) + 16), EALIAS), (dict(q_out=at(1)), EALIAS), (dict(k_out=at(2)), EALIAS), (dict(k_out=at(7)), EALIAS),
    (dict(q_out=at(3)), EALIAS), (dict(q_out=at(9) - 64), EALIAS), (dict(k_out=at(5)), EALIAS), (dict(k_out=at(6)), EALIAS),
    (dict(k_out=at(0)), EALIAS),
])
def test_rope_refusals(kw, rc):
    assert rope(**kw) == rc


@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(k=None), EPTR), (dict(v=None), EPTR), (dict(ks=at(22)), EPTR), (dict(vs=at(23)), EPTR),
    (dict(k=at(20) + 8), EALIGN), (dict(v=at(21) + 4), EALIGN), (dict(ks=at(22) + 4, vs=at(23)), EALIGN), (dict(ks=at(22), vs=at(23) + 8), EALIGN),
    (dict(k=at(21) + 64), EALIAS), (dict(k=at(0)), EALIAS), (dict(v=at(7) - 64), EALIAS), (dict(ks=at(20), vs=at(23)), EALIAS),
    (dict(ks=at(22), vs=at(9)), EALIAS), (dict(k=at(6)), EALIAS), (dict(v=at(3)), EALIAS),
])
def test_rope_cache_refusals(kw, rc):
    assert rope(cache=kv(**kw)) == rc


def test_rope_parts_of_one_array():
    """q, k and v between each other in one product's rows: an output in another
    part's place overlaps it."""
    base, row = at(0), 24 * 128
    parts = dict(q=base, k=base + 2 * 2048, v=base + 2 * 2560, qs=row, ks=row, vs=row, cache=None)
    assert rope(**parts, q_out=base + 2 * 2048, k_out=at(8)) == EALIAS
    assert rope(**parts, q_out=at(7), k_out=base) == EALIAS
    assert rope(**{**parts, "k": base + 2 * 2040}, q_out=base, k_out=at(8)) == EALIAS


def decode(q=at(0), B=3, T=2, Hq=16, Hk=4, D=128, qs=2048, table=at(1), width=8, lengths=at(2), n_new=at(3), scale=0.1, window=0, y=at(4),
           ws=at(5), nb=1 << 30, **c):
    return lib.q4_attention_decode(q, B, T, Hq, Hk, D, qs, ctypes.byref(kv(**c)), table, width, lengths, n_new, scale, window, y, ws, nb, None)


@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(q=None), EPTR), (dict(table=None), EPTR), (dict(lengths=None), EPTR), (dict(y=None), EPTR), (dict(ws=None), EPTR),
    (dict(k=None), EPTR), (dict(v=None), EPTR), (dict(ks=at(22)), EPTR),
    (dict(B=0), ESHAPE), (dict(B=4097), ESHAPE), (dict(T=0), ESHAPE), (dict(T=65), ESHAPE), (dict(Hq=15, qs=1920), ESHAPE), (dict(Hk=0), ESHAPE),
    (dict(Hk=32), ESHAPE), (dict(Hq=512, qs=1 << 16), ESHAPE), (dict(D=32), ESHAPE), (dict(qs=2044), ESHAPE), (dict(qs=2040), ESHAPE),
    (dict(width=0), ESHAPE), (dict(width=(1 << 20) + 1), ESHAPE), (dict(B=4096, width=1 << 20), ESHAPE), (dict(B=4096, T=64, width=1 << 17), ESHAPE), (dict(window=-1), ESHAPE), (dict(scale=0.0), ESHAPE),
    (dict(scale=-1.0), ESHAPE), (dict(scale=math.inf), ESHAPE), (dict(scale=math.nan), ESHAPE),
    (dict(q=at(0) + 8), EALIGN), (dict(table=at(1) + 2), EALIGN), (dict(lengths=at(2) + 1), EALIGN), (dict(n_new=at(3) + 2), EALIGN),
    (dict(y=at(4) + 8), EALIGN), (dict(ws=at(5) + 128), EALIGN), (dict(nb=65536), ESCRATCH), (dict(nb=0), ESCRATCH),
    (dict(y=at(0)), EALIAS), (dict(y=at(1)), EALIAS), (dict(y=at(2)), EALIAS), (dict(y=at(3)), EALIAS), (dict(y=at(20) + 64), EALIAS),
    (dict(y=at(21)), EALIAS), (dict(ws=at(0)), EALIAS), (dict(ws=at(4)), EALIAS), (dict(ws=at(21)), EALIAS), (dict(ws=at(1)), EALIAS),
    (dict(ks=at(22), vs=at(23), y=at(22)), EALIAS), (dict(ks=at(22), vs=at(23), ws=at(23)), EALIAS),
])
def test_decode_refusals(kw, rc):
    assert decode(**kw) == rc


def test_decode_workspace():
    size = q4.attention_decode_workspace_bytes
    assert size(1, 16, 4, 128) > 65536 and size(5, 16, 4, 128) > size(1, 16, 4, 128) > size(1, 16, 4, 64)
    assert size(0, 16, 4, 128) == size(65, 16, 4, 128) == size(1, 15, 4, 128) == size(1, 16, 4, 96) == 0
    need = size(2, 16, 4, 128)
    assert decode(nb=need - 1) == ESCRATCH
    assert decode(nb=need, ws=at(4) - need + 256) == EALIAS      # its last bytes are the output's first


def prefill(q=at(0), T=8, k=at(1), v=at(2), S=8, Hq=16, Hk=4, D=128, qs=2048, ks=512, vs=512, starts=at(3), key_starts=None, B=2, scale=0.1,
            window=0, y=at(5)):
    return lib.q4_attention_prefill(q, T, k, v, S, Hq, Hk, D, qs, ks, vs, starts, key_starts, B, scale, window, y, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), EPTR), (dict(k=None), EPTR), (dict(v=None), EPTR), (dict(starts=None), EPTR), (dict(y=None), EPTR),
    (dict(T=0), ESHAPE), (dict(T=(1 << 22) + 1), ESHAPE), (dict(S=0), ESHAPE), (dict(S=(1 << 22) + 1), ESHAPE), (dict(B=0), ESHAPE),
    (dict(B=4097), ESHAPE), (dict(Hq=14), ESHAPE), (dict(Hk=0), ESHAPE), (dict(D=80), ESHAPE), (dict(qs=2040), ESHAPE), (dict(ks=516), ESHAPE),
    (dict(vs=0), ESHAPE), (dict(scale=0.0), ESHAPE), (dict(scale=math.nan), ESHAPE), (dict(window=-5), ESHAPE),
    (dict(q=at(0) + 2), EALIGN), (dict(k=at(1) + 8), EALIGN), (dict(v=at(2) + 4), EALIGN), (dict(starts=at(3) + 2), EALIGN),
    (dict(key_starts=at(4) + 1), EALIGN), (dict(y=at(5) + 8), EALIGN),
    (dict(y=at(0)), EALIAS), (dict(y=at(1) + 16), EALIAS), (dict(y=at(2)), EALIAS), (dict(y=at(3)), EALIAS), (dict(key_starts=at(5) + 16), EALIAS),
])
def test_prefill_refusals(kw, rc):
    assert prefill(**kw) == rc


def test_binding_refuses_host_tensors():
    h = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        q4.rope_cache(h, h)
    with pytest.raises(ValueError, match="GPU"):
        q4.attention_prefill(h, h, h, i)
    with pytest.raises(ValueError, match="GPU"):
        q4.attention_decode(h[:, None], (h[None], h[None]), i[None], i)
    with pytest.raises(TypeError):
        q4.rope_cache([1.0], h)
    with pytest.raises(TypeError):
        q4.attention_prefill(h.float(), h, h, i)
