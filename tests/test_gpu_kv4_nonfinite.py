"""Prefill attention over a 4-bit cache whose live places hold scales or biases
that are not finite: rows that do not attend such a place are as if it were
clean, bit for bit, and the place is reported."""
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


def spoil(kv, blk, r, which, half=np.float16("nan"), part=None):
    """The parameters of place r of a block (K or V, every head and group) become `half`: the scale, the bias or both."""
    kv = kv.copy()
    word = np.array([half], np.float16).view(np.uint8)
    for grp in range(4):
        s = 2048 + r * 16 + grp * 4 if which == 0 else 2048 + (r // 2) * 32 + grp * 8 + (r % 2) * 2
        b = s + (2 if which == 0 else 4)
        for at in {"scale": (s,), "bias": (b,), None: (s, b)}[part]:
            kv[blk, which, :, at:at + 2] = word
    return kv


def case(n_q, n_kv, seqs, seed):
    r = np.random.default_rng(seed)
    per = max((n + p + 31) // 32 for n, p in seqs) + 1
    n_blocks = len(seqs) * per + 2
    tables = r.permutation(n_blocks)[:len(seqs) * per].reshape(len(seqs), per).astype(np.int32)
    at = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
    q = dev(r.normal(size=(int(at[-1]), n_q, D)).astype(np.float16))
    return q, ref.random_pool(n_blocks, n_kv, seed), tables, at, np.array([p for _, p in seqs], np.int32)


# n_q, n_kv, sequences, the sequence and position that is spoilt: inside a tile, in a tile's first step, before every row, cut items
PREFILL = [(32, 8, [(100, 0)], 0, 50), (16, 8, [(70, 200), (90, 0)], 0, 210), (40, 8, [(60, 77), (26, 0)], 1, 25), (8, 2, [(9, 6000)], 0, 6004)]


@pytest.mark.parametrize("half,part", [(np.nan, None), (np.inf, "scale"), (-np.inf, "bias")], ids=str)
@pytest.mark.parametrize("c", PREFILL, ids=str)
def test_prefill_rows_before_a_v_that_is_not_finite(q3, c, half, part):
    n_q, n_kv, seqs, s, p = c
    q, kv, tables, at, pos = case(n_q, n_kv, seqs, 31 + n_q)
    bad = spoil(kv, tables[s, p // 32], p % 32, 1, half, part)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(at), dev(pos), dev(tables)
    clean = q3.op_kv4_prefill_attention(q, *args, dev(kv), status=status)
    assert status.item() == 0
    got = q3.op_kv4_prefill_attention(q, *args, dev(bad), status=status)
    assert status.item() == 0x8                                    # reported
    rows = np.arange(int(at[-1]))
    sees = (rows >= at[s]) & (rows < at[s + 1]) & (pos[s] + rows - at[s] >= p)
    assert torch.equal(got[dev(~sees)], clean[dev(~sees)])
    # a V value that is not finite counts as zero
    K, V = ref.stored(bad)
    V[~np.isfinite(V)] = 0
    a, b = at[s], at[s + 1]
    want = ref.attend(q[a:b].float().cpu().numpy().astype(np.float64), K, V, tables[s], pos[s] + np.arange(b - a), n_kv)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + (2.0 ** -12 + 2.0 ** -11) * np.abs(V).max()
    assert np.all(np.abs(got[a:b].float().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("c", PREFILL, ids=str)
def test_prefill_rows_before_a_k_that_is_not_a_number(q3, c):
    n_q, n_kv, seqs, s, p = c
    q, kv, tables, at, pos = case(n_q, n_kv, seqs, 47 + n_q)
    bad = spoil(kv, tables[s, p // 32], p % 32, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(at), dev(pos), dev(tables)
    clean = q3.op_kv4_prefill_attention(q, *args, dev(kv))
    got = q3.op_kv4_prefill_attention(q, *args, dev(bad), status=status)
    rows = np.arange(int(at[-1]))
    sees = (rows >= at[s]) & (rows < at[s + 1]) & (pos[s] + rows - at[s] >= p)
    assert torch.equal(got[dev(~sees)], clean[dev(~sees)])
    assert torch.isnan(got[dev(sees)]).all() and status.item() == 0x8


def test_prefill_sequences_that_share_a_block_past_the_end_of_one(q3):
    """Two sequences of one table, one ending before the spoilt place: it counts for the longer one only, and repeats agree."""
    q, kv, tables, _, _ = case(16, 8, [(70, 0)], 61)
    tables = np.concatenate([tables, tables])
    at, pos = np.array([0, 40, 70], np.int32), np.array([0, 40], np.int32)     # positions 0 .. 39, and 40 .. 69
    bad = spoil(kv, tables[0, 1], 50 - 32, 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(kv))
    first = None
    # by the pool's numbers (eight table entries for six blocks), and by sequence
    for pool in (bad, np.concatenate([bad, np.zeros((20,) + bad.shape[1:], np.uint8)])):
        for _ in range(3):
            got = q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(pool), status=status)
            assert status.item() == 0x8
            assert torch.equal(got[:50], clean[:50]) and torch.isfinite(got).all()
            first = got if first is None else first
            assert torch.equal(first, got)


def test_stale_places_behind_every_sequence_are_not_reported(q3):
    q, kv, tables, at, pos = case(32, 8, [(45, 20), (70, 0)], 62)
    bad = kv
    for i in range(2):
        for p in range(pos[i] + at[i + 1] - at[i], tables.shape[1] * 32):
            for which in (0, 1):
                bad = spoil(bad, tables[i, p // 32], p % 32, which)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(at), dev(pos), dev(tables)
    a = q3.op_kv4_prefill_attention(q, *args, dev(kv))
    b = q3.op_kv4_prefill_attention(q, *args, dev(bad), status=status)
    assert status.item() == 0 and torch.equal(a, b)
