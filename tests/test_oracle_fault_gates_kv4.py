"""The mutation gate over the 4-bit K/V cache: the addressing faults of
tests/test_oracle_fault_gates.py planted in the oracle's gather of an
AFFINE4-cache session.  Its rounds over fp16 activations are compared with the
oracle at a bound derived for codes that flip (6.8e-3 a layer,
tests/test_gpu_kv4_model.py) instead of 1e-4: every fault that the identity
layout can show lies beyond it, and the block-table gate is bitwise as ever."""
import shutil

import numpy as np
import pytest

from synthetic import AFFINE4, Shape, make_block_permutation, make_tokens, make_weights
from test_oracle_fault_gates import EXPECTED, N_TOK, _faulty_oracle

KV4 = Shape("oracle-kv4", 2, 128, 4, 2, 32, 128, 256, True, rope_theta=1e4, kv_quant=AFFINE4)
BOUND = 6.8e-3 * KV4.n_layers


@pytest.mark.parametrize("fault", sorted(EXPECTED), ids=["none", "read-block", "read-slot", "rollover", "kv-swap"])
def test_gates_catch_the_planted_fault_over_the_4_bit_cache(tmp_path, orc, fault):
    if not shutil.which("gcc"):
        pytest.skip("gcc is needed to build the planted-fault oracle")
    w, toks = make_weights(KV4, seed=7), make_tokens(N_TOK, KV4.vocab, seed=31)
    honest = orc.Model(KV4, w, n_threads=2).session(max_ctx=128).eval(toks, all_rows=True).astype(np.float64)
    m = _faulty_oracle(tmp_path, fault).Model(KV4, w, n_threads=2)

    def run(table, blocks):
        s = m.session(pool=m.pool(blocks), max_ctx=128) if table is not None else m.session(max_ctx=128)
        if table is not None:
            s.set_block_table(np.asarray(table, np.int32))
        return s.eval(toks, all_rows=True)

    ident = run(range(4), 8).astype(np.float64)
    tolerance = bool(np.all(((ident - honest) ** 2).sum(1) <= BOUND * (honest ** 2).sum(1)))
    contiguous = run(None, 0)
    table = all(np.array_equal(run(make_block_permutation(16, seed)[:4], 16), contiguous) for seed in (1, 2))
    assert (tolerance, table) == EXPECTED[fault], fault
