"""Prefill attention over the 4-bit cache in the layouts of its fp16 copy (by
sequence, or by the pool's block numbers where the tables together exceed the
pool) and with several whole items a CTA.  Tolerances as in test_gpu_kv4.py:
half an fp16 step of the output, 2^-12 of max |V| for the FP32 softmax and
2^-11 for the weights' rounding."""
import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def case(n_q, n_kv, seqs, seed, shared, wide):
    """Sequences (rows, first position) that share their first `shared` blocks; wide: tables of so many entries that they exceed
    the pool."""
    r = np.random.default_rng(seed)
    need = [(n + p + 31) // 32 for n, p in seqs]
    n_blocks = shared + sum(max(n - shared, 0) for n in need) + 2
    ids = list(r.permutation(n_blocks).astype(np.int32))
    per = max(need) + 1 if not wide else max(max(need) + 1, n_blocks // len(seqs) + 1)
    common = [ids.pop() for _ in range(shared)]
    tables = np.empty((len(seqs), per), np.int32)
    tables[:] = n_blocks + 7                                       # entries past a sequence's end are never looked at
    for i, n in enumerate(need):
        tables[i, :n] = (common + [ids.pop() for _ in range(max(n - shared, 0))])[:n]
    at = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
    q = dev(r.normal(size=(int(at[-1]), n_q, D)).astype(np.float16))
    assert (len(seqs) * per >= n_blocks) == wide
    return q, ref.random_pool(n_blocks, n_kv, seed), tables, at, np.array([p for _, p in seqs], np.int32)


def check(q3, q, kv, tables, at, pos, n_kv, stored=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(at), dev(pos), dev(tables), dev(kv)
    got = q3.op_kv4_prefill_attention(q, *args, status=status)
    q3.check_status(status)
    K, V = stored or ref.stored(kv)
    qf, vmax = q.float().cpu().numpy().astype(np.float64), np.abs(V).max()
    g = got.cpu().numpy().astype(np.float64)
    for i in range(len(pos)):
        a, b = at[i], at[i + 1]
        if a == b:
            continue
        want = ref.attend(qf[a:b], K, V, tables[i], pos[i] + np.arange(b - a), n_kv)
        assert np.all(np.abs(g[a:b] - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + (2.0 ** -12 + 2.0 ** -11) * vmax), i
    assert torch.equal(got, q3.op_kv4_prefill_attention(q, *args))
    return got


# n_q, n_kv, sequences: dealt whole, and few on long contexts (cut)
LAYOUTS = [(32, 8, [(37, 0)], 0), (16, 8, [(97, 31), (1, 64), (0, 5), (130, 0)], 0), (40, 8, [(60, 77), (26, 0), (5, 140)], 2),
           (16, 8, [(40, 0), (90, 0), (7, 57), (33, 31)], 2), (8, 2, [(5, 1), (9, 6000), (0, 9), (70, 513)], 1), (1, 1, [(3, 5000)], 0),
           (24, 8, [(10, 3000), (12, 2990), (3, 3007)], 90), (14, 2, [(129, 1000), (40, 1000)], 31)]


@pytest.mark.parametrize("c", LAYOUTS, ids=str)
def test_copies_by_the_pools_numbers_and_by_sequence(q3, c):
    n_q, n_kv, seqs, shared = c
    # a lone sequence's table always fits the pool; wide tables must exceed it
    q, kv, tables, at, pos = case(n_q, n_kv, seqs, 500 + n_q, shared, True)
    stored = ref.stored(kv)
    check(q3, q, kv, tables, at, pos, n_kv, stored)
    room = np.concatenate([kv, np.zeros((1000,) + kv.shape[1:], np.uint8)])      # a pool that the tables do not exceed
    narrow = tables[:, :900 // len(seqs)]
    assert len(seqs) * narrow.shape[1] < len(room)
    check(q3, q, room, np.ascontiguousarray(narrow), at, pos, n_kv, stored)


# n_q, n_kv, sequences: two to five whole items for a CTA of 152
DEALT = [(32, 8, [(1600, 0)]), (64, 8, [(130, 40), (200, 0), (77, 300), (150, 9)]), (16, 16, [(130, 5)] * 20), (40, 8, [(900, 100)]),
         (24, 8, [(411, 134), (195, 134), (300, 134)] * 2), (8, 8, [(700, 10), (1300, 0), (33, 500), (129, 129)])]


@pytest.mark.parametrize("c", DEALT, ids=str)
def test_several_whole_items_for_a_cta(q3, c):
    n_q, n_kv, seqs = c
    R = 128 // (n_q // n_kv)
    assert sum((n + R - 1) // R for n, _ in seqs) * n_kv > 152 or n_q == 8
    q, kv, tables, at, pos = case(n_q, n_kv, seqs, 600 + n_q, 0, True)
    check(q3, q, kv, tables, at, pos, n_kv)


def test_model_round_whose_tables_exceed_the_pool():
    """Mixed and decode rounds of four sessions of 16 table entries over a pool of 40 blocks, against the oracle at the bound of
    test_gpu_kv4_model.py."""
    import synthetic
    from helpers import Pair
    from test_gpu_kv4_model import TINY_KV4, gate4
    pair = Pair(TINY_KV4, seed=1201, max_ctx=512, max_round_tokens=256, n_blocks=40)
    perm = synthetic.make_block_permutation(40, seed=1202)
    lens = [3, 70, 33, 100]
    gs, os_, lists = [], [], []
    for i, n in enumerate(lens):
        g, o = pair.sessions(table=perm[10 * i:10 * i + 8])
        pair.eval(g, o, synthetic.make_tokens(25 * i + 1, TINY_KV4.vocab, seed=1210 + i))
        gs.append(g)
        os_.append(o)
        lists.append(synthetic.make_tokens(n, TINY_KV4.vocab, seed=1220 + i))
    for step in range(3):
        got, want, am = pair.eval_batch(gs, os_, lists)
        for i in range(len(gs)):
            c = gate4(got[i], want[i], 2, ("tables exceed the pool", step, i))
            assert am[i] == c.argmax_gpu
        lists = [[int(np.argmax(r))] for r in want]
    for g in gs:
        g.close()
