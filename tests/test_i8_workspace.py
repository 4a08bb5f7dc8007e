"""The 8-bit product's workspace: what is reported for some sizes serves them and all
smaller ones, so that a caller may allocate once for its largest round.  No GPU."""
import ctypes
import random

import pytest

PROJECTIONS = ((4096, 1024), (1024, 2048), (6144, 2560), (2560, 4096), (19456, 2560), (2560, 9728), (6144, 4096),
               (24576, 4096), (4096, 12288), (7168, 5120), (5120, 5120), (34816, 5120), (5120, 17408))


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def used(q3, *sizes):
    """What the operator asks for with exactly these sizes."""
    n = ctypes.c_int64()
    assert q3.lib().q3_i8_matmul_workspace_used(*sizes, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("m,k", PROJECTIONS + ((7, 100), (1, 1), (200, 700), (129, 768), (5003, 769), (1000, 131071), (100000, 3)))
def test_it_serves_every_smaller_round(q3, m, k):
    most = 0
    for t in (*range(2200), *range(2200, 40000, 97), 1 << 20, 1 << 30):
        most = max(most, used(q3, t, m, k))
        reported = q3.i8_matmul_workspace(t, m, k)
        assert reported >= most, t
        most = reported                                   # and so grows with t


def test_it_serves_every_smaller_matrix(q3):
    r = random.Random(1)
    size = lambda most: int(2 ** r.uniform(0, most))  # noqa: E731
    for _ in range(20000):
        t, m, k = size(14), size(17), size(16)
        bound = q3.i8_matmul_workspace(t, m, k)
        less = r.randint(1, t), r.randint(1, m), r.randint(1, k)
        assert q3.i8_matmul_workspace(*less) <= bound and used(q3, *less) <= bound and used(q3, t, m, k) <= bound, (t, m, k, less)


def test_the_operator_takes_it_for_a_smaller_round(q3):
    """The operator asks for no more than it uses (a refusal names a workspace; other arguments are refused before)."""
    L, p = q3.lib(), 1 << 20
    falls = [(t, m, k) for m, k in PROJECTIONS for t in range(33, 2049) if used(q3, t, m, k) and not used(q3, t + 3, m, k)]
    assert falls                                          # there are such sizes: more tokens that need none
    for t, m, k in falls:
        need = used(q3, t, m, k)
        assert q3.i8_matmul_workspace(t + 3, m, k) >= need
        for ws, n in ((None, 0), (p, need - 1), (p + 16, need)):
            assert L.q3_op_i8_matmul(p, k, p, p, k, p, t, m, k, p, 1, m, ws, n, None, None) == -1
            assert b"workspace" in L.q3_last_error()


def test_refusals(q3):
    n = ctypes.c_int64()
    for bad in ((-1, 7, 100), (9, 0, 100), (9, 7, 0), (9, 7, 131072), ((1 << 30) + 1, 7, 100), (9, (1 << 30) + 1, 100)):
        assert q3.lib().q3_i8_matmul_workspace_used(*bad, ctypes.byref(n)) == -1
    assert q3.lib().q3_i8_matmul_workspace_used(9, 7, 100, None) == -1
