"""Refusals of the 8-bit block-scaled and verification entry points, on the
host (only invalid argument sets and size queries are passed, so nothing is
launched)."""
import ctypes

import pytest

q4 = pytest.importorskip("bit_weight_only_q4g128_amd")
lib = q4.lib

OK, EPTR, ESHAPE, EALIGN, EALIAS, ESCRATCH = 0, -1, -2, -3, -4, -7
A = 0x100000000      # aligned, made-up device addresses; never dereferenced
STEP = 1 << 32


def at(i):
    return A + i * STEP


def quantize(x=at(0), up=None, M=4, K=2048, codes=at(1), scale=at(2)):
    return lib.fp8b128_quantize(x, up, M, K, codes, scale, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EPTR), (dict(codes=None), EPTR), (dict(scale=None), EPTR),
    (dict(M=0), ESHAPE), (dict(M=(1 << 19) + 1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=8), ESHAPE), (dict(K=2056), ESHAPE),
    (dict(K=32784), ESHAPE),
    (dict(x=at(0) + 8), EALIGN), (dict(up=at(3) + 2), EALIGN), (dict(codes=at(1) + 8), EALIGN), (dict(scale=at(2) + 2), EALIGN),
    (dict(codes=at(0) + 64), EALIAS), (dict(scale=at(0)), EALIAS), (dict(scale=at(1) + 4096), EALIAS),
    (dict(up=at(3), codes=at(3) + 4 * 2048 * 2 - 16), EALIAS),
])
def test_quantize_refusals(kw, rc):
    assert quantize(**kw) == rc


def task(i=0, **kw):
    base = dict(x=at(8 * i), xscale=at(8 * i + 1), w=at(8 * i + 2), wscale=at(8 * i + 3), residual=None, y=at(8 * i + 4), N=2048,
                K=2048)
    base.update(kw)
    return q4.Fp8Task(**base)


def group(*tasks, M=4, ws=None, nb=0):
    return lib.fp8b128_gemm_grouped_ws((q4.Fp8Task * len(tasks))(*tasks), len(tasks), M, ws, nb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EPTR), (dict(xscale=None), EPTR), (dict(w=None), EPTR), (dict(wscale=None), EPTR), (dict(y=None), EPTR),
    (dict(N=0), ESHAPE), (dict(N=(1 << 24) + 1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=24), ESHAPE), (dict(K=32784), ESHAPE),
    (dict(x=at(0) + 8), EALIGN), (dict(w=at(2) + 4), EALIGN), (dict(xscale=at(1) + 2), EALIGN), (dict(wscale=at(3) + 1), EALIGN),
    (dict(y=at(4) + 1), EALIGN), (dict(residual=at(5) + 1), EALIGN),
    (dict(y=at(0) + 16), EALIAS), (dict(y=at(1)), EALIAS), (dict(y=at(2)), EALIAS), (dict(y=at(3) + 4), EALIAS),
    (dict(residual=at(4) + 2), EALIAS),
])
def test_gemm_refusals(kw, rc):
    assert group(task(**kw)) == rc
    nb = ctypes.c_size_t(5)
    assert lib.fp8b128_workspace_bytes((q4.Fp8Task * 1)(task(**kw)), 1, 4, ctypes.byref(nb)) == rc and nb.value == 5
    t = task(**kw)
    assert lib.fp8b128_gemm(t.x, t.xscale, 4, t.K, t.w, t.wscale, t.N, t.residual, t.y, None) == rc


def test_group_refusals():
    assert lib.fp8b128_gemm_grouped_ws(None, 1, 1, None, 0, None) == EPTR
    one = (q4.Fp8Task * 1)(task())
    assert lib.fp8b128_gemm_grouped_ws(one, 0, 1, None, 0, None) == ESHAPE
    assert lib.fp8b128_gemm_grouped_ws(one, 9, 1, None, 0, None) == ESHAPE
    assert group(task(), M=0) == ESHAPE
    assert group(task(), M=(1 << 19) + 1) == ESHAPE
    assert lib.fp8b128_workspace_bytes(one, 1, 4, None) == EPTR
    assert group(task(0), task(1, y=at(4) + 64)) == EALIAS                  # two tasks share an output
    assert group(task(0), task(1, y=at(2) + 64)) == EALIAS                  # over another task's weights
    assert group(task(0, residual=at(5)), task(1, y=at(5))) == EALIAS       # over another task's residual
    assert group(task(), ws=at(7) + 16, nb=1 << 20) == EALIGN
    assert group(task(), ws=at(4), nb=1 << 20) == EALIAS                    # the workspace over an output
    assert group(task(), ws=at(2) + 4096, nb=1 << 20) == EALIAS             # over the weights
    nb = ctypes.c_size_t(5)
    assert lib.fp8b128_workspace_bytes((q4.Fp8Task * 2)(task(0), task(1, residual=at(12), y=at(12))), 2, 4, ctypes.byref(nb)) == OK


TOPK = dict(logits=at(0), B=4, D=3, V=16385, draft=at(1), di=at(2), dp=at(3), dk=30, nd=at(4), u=at(5), T=0.8, k=30, token=at(6),
            count=at(7), prob=at(8), ws=at(9), nb=1 << 30)


def topk(**kw):
    a = {**TOPK, **kw}
    return lib.q4_verify_topk(a["logits"], a["B"], a["D"], a["V"], a["draft"], a["di"], a["dp"], a["dk"], a["nd"], a["u"], a["T"],
                              a["k"], a["token"], a["count"], a["prob"], a["ws"], a["nb"], None)


def full(**kw):
    a = {**TOPK, **kw}
    return lib.q4_verify_full(a["logits"], a["B"], a["D"], a["V"], a["draft"], a["di"], a["nd"], a["u"], a["T"], a["token"],
                              a["count"], a["prob"], a["ws"], a["nb"], None)


COMMON = [
    (dict(logits=None), EPTR), (dict(draft=None), EPTR), (dict(u=None), EPTR), (dict(token=None), EPTR), (dict(count=None), EPTR),
    (dict(ws=None), EPTR),
    (dict(B=0), ESHAPE), (dict(D=0), ESHAPE), (dict(D=64), ESHAPE), (dict(B=16385), ESHAPE), (dict(V=0, k=1), ESHAPE),
    (dict(T=0.0), ESHAPE), (dict(T=-1.0), ESHAPE), (dict(T=float("inf")), ESHAPE), (dict(T=float("nan")), ESHAPE),
    (dict(logits=at(0) + 1), EALIGN), (dict(draft=at(1) + 2), EALIGN), (dict(nd=at(4) + 1), EALIGN), (dict(u=at(5) + 2), EALIGN),
    (dict(token=at(6) + 2), EALIGN), (dict(count=at(7) + 2), EALIGN), (dict(prob=at(8) + 2), EALIGN), (dict(ws=at(9) + 64), EALIGN),
    (dict(nb=1024), ESCRATCH),
    (dict(token=at(0) + 64), EALIAS), (dict(count=at(1)), EALIAS), (dict(prob=at(5)), EALIAS), (dict(token=at(4)), EALIAS),
    (dict(count=at(6) + 16), EALIAS), (dict(prob=at(6)), EALIAS), (dict(ws=at(0)), EALIAS), (dict(ws=at(8)), EALIAS),
]


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(dp=None), EPTR), (dict(di=None), EPTR), (dict(k=0), ESHAPE), (dict(k=65), ESHAPE), (dict(V=20, k=21), ESHAPE),
    (dict(V=30721), ESHAPE), (dict(dk=0), ESHAPE), (dict(dk=65), ESHAPE), (dict(di=at(2) + 1), EALIGN), (dict(dp=at(3) + 2), EALIGN),
    (dict(token=at(2)), EALIAS), (dict(count=at(3) + 4), EALIAS), (dict(ws=at(3)), EALIAS),
])
def test_verify_topk_refusals(kw, rc):
    assert topk(**kw) == rc


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(V=(1 << 20) + 1), ESHAPE), (dict(di=at(2) + 1), EALIGN), (dict(token=at(2) + 1024), EALIAS), (dict(ws=at(2)), EALIAS),
])
def test_verify_full_refusals(kw, rc):
    assert full(**kw) == rc


def test_verify_workspace_sizes():
    f, t = q4.verify_full_workspace_bytes, q4.verify_topk_workspace_bytes
    assert f(0, 1, 10) == 0 and f(1, 0, 10) == 0 and f(1, 64, 10) == 0 and f(1, 1, 0) == 0 and f(1, 1, (1 << 20) + 1) == 0
    assert t(1, 1, 30721, 30) == 0 and t(1, 1, 20, 21) == 0 and t(1, 1, 20, 0) == 0
    assert t(1, 4, 2049, 30) == 0                      # a row fits one wave: no scratch
    assert t(48, 4, 16385, 30) >= (64 << 10) + 48 * 5 * 17 * 30 * 4
    assert f(1, 1, 1) > 64 << 10                       # the counters of other calls come first
    assert f(32, 7, 131072) > f(32, 7, 16385) > f(1, 7, 16385)


def test_verify_workspace_of_the_largest_batch_serves_smaller_ones():
    for V in (2561, 5000, 16385, 30720):
        sizes = [q4.verify_topk_workspace_bytes(B, 4, V, 30) for B in range(1, 200)]
        assert sizes == sorted(sizes)
    for D in (1, 7):
        for V in (1, 2049, 16384, 16385, 32768, 50001, 131072, 1 << 20):
            sizes = [q4.verify_full_workspace_bytes(B, D, V) for B in range(1, 600)]
            assert sizes == sorted(sizes)


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q4.fp8b128_quantize(x)
    c = torch.zeros(2, 128, dtype=torch.uint8)
    s = torch.zeros(2, 1)
    with pytest.raises(ValueError):
        q4.fp8b128_gemm(c, s, c, s)
    lg, d, u = torch.zeros(1, 2, 8, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2)
    with pytest.raises(ValueError):
        q4.verify_topk(lg, d, u, top_k=2)
    with pytest.raises(ValueError):
        q4.verify_full(lg, d, u)
