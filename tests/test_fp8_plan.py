"""How calls of the 8-bit product are launched, on the host (nothing is
launched): the workspace query and the launch decide alike."""
import ctypes

import pytest

q4 = pytest.importorskip("bit_weight_only_q4g128_amd")
lib = q4.lib

OK, EPTR, ESHAPE = 0, -1, -2
A, STEP = 1 << 40, 1 << 44      # made-up device addresses; never dereferenced
LARGE = 64 << 20


def tasks_of(K, Ns):
    at = lambda i, j: A + (8 * i + j) * STEP  # noqa: E731
    return (q4.Fp8Task * len(Ns))(*[q4.Fp8Task(x=at(0, 0), xscale=at(0, 1), w=at(i, 2), wscale=at(i, 3), residual=None, y=at(i, 4), N=n, K=K)
                                    for i, n in enumerate(Ns)])


def query(M, K, Ns):
    nb = ctypes.c_size_t(0)
    assert lib.fp8b128_workspace_bytes(tasks_of(K, Ns), len(Ns), M, ctypes.byref(nb)) == OK
    return nb.value


def launches(M, K, Ns, ws):
    out, n = (q4.Fp8Launch * 16)(), ctypes.c_int(-1)
    assert lib.fp8b128_launches(tasks_of(K, Ns), len(Ns), M, ws, out, 16, ctypes.byref(n)) == OK
    assert 1 <= n.value <= 16
    return [(v.tile_m, v.tile_n, tuple(v.N[:v.count]), tuple(v.slices[:v.count]), v.workspace_bytes) for v in out[:n.value]]


def check(M, K, Ns):
    """A call with exactly the queried bytes runs as one with more."""
    need = query(M, K, Ns)
    want = launches(M, K, Ns, LARGE)
    what = (M, K, Ns, need, want)
    assert max(v[4] for v in want) == need, what
    for ws in {need, need + 1, 48 << 20, 1 << 40}:
        assert launches(M, K, Ns, ws) == want, what
    for ws in {0, need // 2, max(need - 1, 0), 65536}:
        assert all(v[4] <= ws for v in launches(M, K, Ns, ws)), what
    assert all(s == 1 for v in launches(M, K, Ns, 0) for s in v[3]), what
    # every weight row once, in order
    rows = [n for v in want for n in v[2]]
    assert rows == list(Ns) or (len(Ns) == 1 and len(rows) == 2 and sum(rows) == Ns[0] and rows[0] % 256 == 0), what
    return need, want


@pytest.mark.parametrize("M", [1, 5, 16, 17, 48, 100, 240, 512, 1000, 2048, 4096, 8192, 100000])
def test_queried_bytes_give_the_plan_of_a_large_workspace(M):
    for K in (16, 256, 400, 512, 1040, 2048, 4096, 4208, 7904, 8192, 16400, 32768):
        for N in (1, 64, 255, 256, 257, 513, 1000, 2048, 2049, 4097, 6000, 8193, 8249, 16385, 32769, 50001, 131073):
            check(M, K, (N,))
        check(M, K, (2048, 512, 515, 8192, 8193))
        check(M, K, (1, 300))


@pytest.mark.parametrize("M,N,K", [(512, 8249, 4208), (512, 8249, 7904), (512, 8249, 8192), (512, 8249, 32768)])
def test_split_behind_the_last_whole_tile_is_in_the_query(M, N, K):
    """Weight rows past the last whole 256 in a launch of their own, whose K is
    split: the query has that split's bytes."""
    need, want = check(M, K, (N,))
    assert need > 65536
    assert [v[2] for v in want] == [(N - N % 256,), (N % 256,)]
    assert want[1][3][0] > 1 and want[1][4] > 65536


def test_a_byte_short_splits_less():
    """A workspace smaller than the query's still splits K where a split fits."""
    need = query(48, 32768, (1024,))
    full, = launches(48, 32768, (1024,), need)
    less, = launches(48, 32768, (1024,), need - 1)
    assert full[3][0] > 1 and less[3][0] > 1 and less[4] < need


def test_group_past_one_grid_goes_task_by_task():
    Ns = (1 << 24,) * 8
    assert [v[2] for v in launches(2, 16, Ns, LARGE)] == [(1 << 24,)] * 8
    check(2, 16, Ns)


def test_launches_refusals():
    t, out, n = tasks_of(2048, (64,)), (q4.Fp8Launch * 1)(), ctypes.c_int(7)
    assert lib.fp8b128_launches(t, 1, 4, 0, out, 1, None) == EPTR
    assert lib.fp8b128_launches(t, 1, 4, 0, None, 1, ctypes.byref(n)) == EPTR
    assert lib.fp8b128_launches(None, 1, 4, 0, out, 1, ctypes.byref(n)) == EPTR
    assert lib.fp8b128_launches(t, 0, 4, 0, out, 1, ctypes.byref(n)) == ESHAPE
    assert lib.fp8b128_launches(t, 1, 0, 0, out, 1, ctypes.byref(n)) == ESHAPE
    assert n.value == 7
    assert lib.fp8b128_launches(t, 1, 4, 0, None, 0, ctypes.byref(n)) == OK and n.value == 1
