"""Attention over the 4-bit cache where one position outweighs a long tail,
and where scores rise slowly.

A position's score is set by one group of K (the other three are zero), so a
score is one product of exact fp16 numbers summed over 32 equal terms: its
error is under 2^-18 and the weights' under 2^-17 of their size.  The softmax
weights enter the second product with 11 bits (prefill) or 22 (decode), none
finer than 2^-32 of the largest weight: n positions may lose n 2^-32, here
2^-15.  FP32 sums of chains of a few hundred terms add 2^-16.  Together that is
2^-14 of max |V|, beside half an fp16 step of the output (2^-11 |ref|, 2^-25
below the normal range); where every weight is of ordinary size, prefill's
rounding of each adds 2^-11 max |V|.
"""
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


def pool_of_scores(unit, n_kv, seed, head_v):
    """A pool in block order whose position p scores `unit[p]` for q = 1 in the first 32 dimensions: K group 0 is the constant
    unit[p] sqrt(128) / 32, V is near 1, and zero at the positions of head_v."""
    n = len(unit)
    assert n % 32 == 0
    r = np.random.default_rng(seed)
    kv = r.integers(0, 256, (n // 32, 2, n_kv, ref.TILE), dtype=np.uint8)
    k = np.zeros((n, 4, 2), np.float16)                            # scale, bias
    k[:, 0, 1] = unit * np.sqrt(128.0) / 32
    kv[:, 0, :, 2048:] = k.reshape(n // 32, 1, 256).view(np.uint8)
    s = r.uniform(0.02, 0.06, (n, 4)).astype(np.float16)
    b = (1.0 - 7.5 * s).astype(np.float16)
    s[head_v], b[head_v] = 0.0, 0.0
    v = np.stack([s.reshape(-1, 16, 2, 4), b.reshape(-1, 16, 2, 4)], 2).transpose(0, 1, 4, 2, 3)     # pair, group, s/b, parity
    kv[:, 1, :, 2048:] = np.ascontiguousarray(v).reshape(n // 32, 1, 256).view(np.uint8)
    return kv


def queries(T, n_q):
    """q of row t and head h: 1 + h / 64 in the first 32 dimensions."""
    q = torch.zeros(T, n_q, D, device="cuda")
    q[:, :, :32] = (1 + torch.arange(n_q, device="cuda") / 64).view(1, -1, 1)
    return q


def check(got, want, vmax, share):
    got = got.float().cpu().numpy().astype(np.float64)
    d = np.abs(got - want) / (2.0 ** -11 * np.abs(want) + 2.0 ** -25 + share * vmax)
    assert np.all(d <= 1), float(d.max())


N = 131072
# the outweighing position's place; the tail lies 18 nats below it
SINKS = [0, 70001]


def sink_case(at, n_kv):
    r = np.random.default_rng(at)
    unit = r.normal(0, 0.1, N)
    unit[at] = 18.0
    kv = pool_of_scores(unit, n_kv, at + 1, [at])
    K, V = ref.stored(kv)
    table = np.arange(N // 32, dtype=np.int32)
    return kv, K, V, table


# rows of one slot: two are split over many warps, of which one has the outweighing position; 320 are not, so a warp with a
# quarter of the tail has it
@pytest.mark.parametrize("T", [2, 320])
@pytest.mark.parametrize("at", SINKS)
@pytest.mark.parametrize("n_q,qt", [(4, torch.float16), (4, torch.float32), (8, torch.float16), (8, torch.float32)])
def test_decode_keeps_a_tail_below_one_position(q3, at, n_q, qt, T):
    kv, K, V, table = sink_case(at, 1)
    q = queries(T, n_q)
    want = ref.attend(q[:1].cpu().numpy().astype(np.float64), K, V, table, np.array([N - 1]), 1)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = q3.op_kv4_decode_attention(q.to(qt), i32([N - 1] * T), i32([0] * T), i32(table).view(1, -1), torch.from_numpy(kv).cuda())
    check(out, want, np.abs(V).max(), 2.0 ** -14)


# 1 row of 1 head, 3 of 8: cut into many pieces; 2,432 of 8: 152 tiles, one for a CTA, whose half with the position has half the tail
@pytest.mark.parametrize("T,n_q", [(1, 1), (3, 8), (2432, 8)])
@pytest.mark.parametrize("at", SINKS)
def test_prefill_keeps_a_tail_below_one_position(q3, at, T, n_q):
    kv, K, V, table = sink_case(at, 1)
    q = queries(T, n_q).half()
    rows = [0, T // 2, T - 1]
    want = ref.attend(q[rows].float().cpu().numpy().astype(np.float64), K, V, table, N - T + np.array(rows), 1)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = q3.op_kv4_prefill_attention(q, i32([0, T]), i32([N - T]), i32(table).view(1, -1), torch.from_numpy(kv).cuda())
    check(out[rows], want, np.abs(V).max(), 2.0 ** -14)


@pytest.mark.parametrize("nats", [2.5, 5.3, 40.0, 700.0])
def test_scores_that_rise_slowly(q3, nats):
    """Maxima that grow by less than what makes a kernel rescale, by just more, and by much: no weight overflows."""
    n, n_q, n_kv = 1600, 8, 2
    kv = pool_of_scores(np.linspace(0, nats, n), n_kv, 11, [n - 1])
    K, V = ref.stored(kv)
    table = np.arange(n // 32, dtype=np.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tab, dkv = torch.from_numpy(table).cuda().view(1, -1), torch.from_numpy(kv).cuda()
    q = queries(200, n_q).half()
    q64 = q.float().cpu().numpy().astype(np.float64)
    want = ref.attend(q64, K, V, table, n - 200 + np.arange(200), n_kv)
    # a score of `nats` is rounded at 2^-18 of itself: its weight at nats 2^-18
    share = 2.0 ** -14 + nats * 2.0 ** -18
    check(q3.op_kv4_prefill_attention(q, i32([0, 200]), i32([n - 200]), tab, dkv), want, np.abs(V).max(), share + 2.0 ** -11)
    out = q3.op_kv4_decode_attention(q[-3:], i32([n - 3, n - 2, n - 1]), i32([0, 0, 0]), tab, dkv)
    check(out, want[-3:], np.abs(V).max(), share)
