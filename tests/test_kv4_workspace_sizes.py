"""q3_kv4_prefill_workspace takes the sizes that q3_op_kv4_prefill_attention
takes and refuses the others, before any of them is multiplied (host only)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3.lib()


# ns, T, n_q, n_kv, max_blocks, n_blocks
TAKEN = [(1, 1, 1, 1, 1, 1), (3, 100, 32768, 4096, 7, 20), (1, (1 << 31) // 8 - 1, 64, 8, 4, 4), (0, 0, 8, 8, 1, 1), (1, 1, 32, 8, 1 << 20, (1 << 31) - 1),
         (4, 1, 32, 8, 1 << 20, 4194303)]
REFUSED = [(1, 1, 4097, 4097, 4, 4), (1, 1, 1 << 30, 1 << 30, 4, 4), (1, 1, 1 << 30, 1 << 27, 4, 4), (1, 1, 64, 1 << 28, 4, 4),
           (1, 1 << 28, 64, 8, 4, 4), (1, (1 << 31) - 1, 2, 2, 4, 4), (4, 1, 32, 8, 1 << 20, 1 << 22),
           (1 << 20, 1, 32, 8, 1 << 20, (1 << 31) - 1)]


def prefill(L, ns, T, n_q, n_kv, max_blocks, n_blocks, P=1 << 20):
    """The operator's answer, which names no buffer that it could launch on: a workspace that is too small."""
    return L.q3_op_kv4_prefill_attention(P, n_q * 128, P, P, None, ns, T, n_q, n_kv, P, max(ns, 1), max_blocks, P, n_blocks, P, None, 0, None, None)


@pytest.mark.parametrize("sizes", TAKEN, ids=str)
def test_taken(L, sizes):
    n = C.c_int64(-1)
    assert L.q3_kv4_prefill_workspace(*sizes, C.byref(n)) == 0
    ns, T, n_q, n_kv, max_blocks, n_blocks = sizes
    blocks = min(n_blocks, ns * max_blocks)
    assert blocks * n_kv * 16384 <= n.value <= blocks * n_kv * 16384 + (64 << 20) + 16 * (T + ns)


@pytest.mark.parametrize("sizes", REFUSED, ids=str)
def test_refused(L, sizes):
    n = C.c_int64(-1)
    assert L.q3_kv4_prefill_workspace(*sizes, C.byref(n)) == -1 and n.value == -1
    if sizes[2] * 128 < 1 << 31:
        assert prefill(L, *sizes) == -1
