"""The 4-bit K/V cache's operators against plain 64-bit readings of their
definitions (tests/kv4_ref.py, the oracle's AFFINE4 packer).

Tolerances, per element, fixed from the operations:
- q_out: half an fp16 step (2^-11 |ref|, 2^-25 below the normal range) and the
  FP32 norm and rotation, under 32 roundings of the row's largest value
  (2^-19 max).
- packed K against the FP32 row y: the code is off by at most half a step, the
  top code by the scale's own rounding over 15 steps, the lowest by the
  bias's, and the stored value by half an fp16 step:
  s / 2 + 15 s 2^-11 + 2^-11 |min| + 2^-11 |value| + 2^-19 max.  V comes
  straight from the input, so its record equals the oracle's bit for bit.
- attention: half an fp16 step of the output (2^-11 |ref|; none for FP32) and
  the FP32 softmax and sums: scores of unit data are under 16 in size with 130
  roundings each, 2^-13 of max |V| in the weights and as much in the sums.
- prefill, besides: each softmax weight rounded to fp16 once, 2^-11 max |V|.
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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def rope_np(n, theta=1e6):
    a = np.arange(n)[:, None] * theta ** (-np.arange(0, 128, 2) / 128.0)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def norm_rope(x, gain, cs, eps):
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    a, b = y[..., :64], y[..., 64:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


# ---------------------------------------------------------------- append

APPEND = [  # n_q, n_kv, rows per slot, first positions, type, row padding
    (16, 8, [1], [0], "f32", 0),
    (32, 8, [1, 1, 1], [31, 32, 700], "f32", 0),
    (40, 8, [67, 33], [0, 30], "bf16", 64),
    (8, 8, [5], [95], "f16", 8),
    (14, 2, [130], [1], "f32", 4),
    (1, 1, [3], [62], "bf16", 0),
    (64, 8, [9, 2], [25, 64], "f16", 0),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(q3, orc, case):
    n_q, n_kv, counts, first, typ, pad = case
    r = np.random.default_rng(sum(counts) + n_q)
    rows = [(i, first[i] + j) for i in range(len(counts)) for j in range(counts[i])]
    rows.insert(len(rows) // 2, (0, -1))                        # a padding row
    T, W = len(rows), (n_q + 2 * n_kv) * D
    slot, pos = np.array(rows, np.int32).T
    per = int(pos.max()) // 32 + 1
    n_blocks = len(counts) * per + 2
    tables = r.permutation(n_blocks)[:len(counts) * per].reshape(len(counts), per).astype(np.int32)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[typ]
    wide = dev(r.normal(0, 1.5, (T, W + pad)).astype(np.float32), dt)
    qkv = wide[:, :W]
    x = qkv.float().cpu().numpy().astype(np.float64).reshape(T, -1, D)
    gq, gk = (dev(1 + 0.2 * r.normal(size=D).astype(np.float32), torch.bfloat16) for _ in range(2))
    rope = rope_np(int(pos.max()) + 1)
    before = r.integers(0, 256, (n_blocks, 2, n_kv, ref.TILE), dtype=np.uint8)
    kv = dev(before)
    kv_out = torch.full((T, 2, n_kv, D), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = q3.op_kv4_append(qkv, gq, gk, dev(rope), dev(pos), dev(slot), dev(tables), kv, n_q, eps=1e-6, kv_out=kv_out, status=status)
    q3.check_status(status)
    q, kv_out, after = (t.cpu().numpy() for t in (q, kv_out, kv))

    live = pos >= 0
    cs = rope[np.maximum(pos, 0)].astype(np.float64)
    g64 = [g.float().cpu().numpy().astype(np.float64) for g in (gq, gk)]
    wq = norm_rope(x[:, :n_q], g64[0], cs, 1e-6)
    wk = norm_rope(x[:, n_q:n_q + n_kv], g64[1], cs, 1e-6)
    wv = x[:, n_q + n_kv:]
    tol = 2.0 ** -11 * np.abs(wq) + 2.0 ** -25 + 2.0 ** -19 * np.abs(wq).max(-1, keepdims=True)
    assert np.all(np.abs(q.astype(np.float64) - wq)[live] <= tol[live])
    assert not q[~live].any() and not kv_out[~live].any()

    parts = ref.read_tiles(after)
    blk, at = tables[slot, np.maximum(pos, 0) // 32], np.maximum(pos, 0) % 32
    for which, name, want in ((0, "k", wk), (1, "v", wv)):
        codes, scale, bias = (p[blk, :, at] for p in parts[name])              # [T, n_kv, ...]
        got = (np.repeat(scale, 32, -1) * codes + np.repeat(bias, 32, -1))
        s, lo = np.repeat(scale, 32, -1), np.repeat(want.reshape(T, n_kv, 4, 32).min(-1), 32, -1)
        big = np.abs(want).max(-1, keepdims=True)
        tol = s * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * (np.abs(lo) + np.abs(got)) + 2.0 ** -19 * big + 2.0 ** -24
        assert np.all(np.abs(got - want)[live] <= tol[live]), name
        np.testing.assert_array_equal(kv_out[live, which], got.astype(np.float16)[live])
        # the oracle's packer on the same FP32 rows
        rec = orc.affine4_pack(want.astype(np.float32).reshape(T * n_kv, D)).reshape(T, n_kv, 4, 20)
        oc = np.stack([rec[..., :16] & 15, rec[..., :16] >> 4], -1).reshape(T, n_kv, D)
        osb = np.ascontiguousarray(rec[..., 16:]).view(np.float16).astype(np.float64)
        if which:
            np.testing.assert_array_equal(codes[live], oc[live])
            np.testing.assert_array_equal(scale[live], osb[live, ..., 0])
            np.testing.assert_array_equal(bias[live], osb[live, ..., 1])
        else:
            assert np.abs(codes - oc)[live].max() <= 1
            assert (codes != oc)[live].mean() <= 1e-3                          # rounding neighbours only

    # every other byte of the pool is as it was
    mine = np.zeros((n_blocks, 2, n_kv, ref.TILE), bool)
    for t in np.flatnonzero(live):
        p = at[t]
        mine[blk[t], 0, :, p * 64:p * 64 + 64] = True
        mine[blk[t], 0, :, 2048 + p * 16:2064 + p * 16] = True
        w = (p // 2) * 128 + (p % 2) * 2 + np.arange(32) * 4
        mine[blk[t], 1][:, np.concatenate([w, w + 1])] = True
        w = 2048 + (p // 2) * 32 + (p % 2) * 2 + np.arange(8) * 4
        mine[blk[t], 1][:, np.concatenate([w, w + 1])] = True
    np.testing.assert_array_equal(after[~mine], before[~mine])


def _small_append(q3, **kw):
    g = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    a = dict(qkv=torch.randn(3, 4 * D, device="cuda"), pos=[0, 1, 2], slot=[0, 0, 0], tables=[[1]], n_q=2)
    a.update(kw)
    kv = torch.zeros(2, 2, 1, ref.TILE, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = q3.op_kv4_append(a["qkv"], g, g, q3.rope_table(8, 1e6), i32(a["pos"]), i32(a["slot"]), i32(a["tables"]), kv, a["n_q"], status=status)
    return q, kv, int(status.item())


def test_append_places_outside_their_range_are_reported_and_not_written(q3):
    for kw in (dict(tables=[[2]]), dict(tables=[[-1]]), dict(slot=[1, 1, 1]), dict(slot=[-1, -1, -1]), dict(pos=[8, 9, 40])):
        q, kv, status = _small_append(q3, **kw)
        assert status == 0x2, kw
        assert not kv.any().item(), kw
    q, kv, status = _small_append(q3)
    assert status == 0 and kv[1].any().item() and not kv[0].any().item()


def test_append_reports_values_beyond_the_format(q3):
    big = torch.randn(3, 4 * D, device="cuda")
    big[1, 3 * D + 5] = 7e4                                      # a V value
    assert _small_append(q3, qkv=big)[2] == 0x8
    big[1, 3 * D + 5] = float("nan")
    assert _small_append(q3, qkv=big)[2] == 0x8
    big[1, 3 * D + 5] = 64000.0
    assert _small_append(q3, qkv=big)[2] == 0


def test_append_constant_and_zero_groups(q3):
    x = torch.zeros(3, 4 * D, device="cuda")
    x[1, 3 * D:] = 2.5
    x[2, 3 * D: 3 * D + 32] = -0.75
    q, kv, status = _small_append(q3, qkv=x)
    assert status == 0 and not q.any().item()                    # zero rows stay zero through the norm
    k, v = ref.stored(kv.cpu().numpy())
    assert not k[1, 0, :3].any() and not v[1, 0, 0].any()
    assert (v[1, 0, 1] == 2.5).all() and (v[1, 0, 2, :32] == -0.75).all() and not v[1, 0, 2, 32:].any()


# ---------------------------------------------------------------- decode attention

def _bound(want, vmax, f16, prefill=False):
    return (2.0 ** -11 * np.abs(want) + 2.0 ** -25 if f16 else 0.0) + 2.0 ** -12 * vmax + (2.0 ** -11 * vmax if prefill else 0.0)


DECODE = [  # n_q, n_kv, contexts, q type, out type
    (32, 8, [1], "f16", "f16"), (32, 8, [31, 32, 33, 0, 64, 65], "f32", "f16"), (40, 8, [700, 2, 1300], "f16", "f32"),
    (16, 8, [97, 513, 0, 0, 40], "f16", "f16"), (8, 8, [257], "f32", "f32"), (24, 8, [1000, 3], "f16", "f16"),
    (64, 8, [200, 1, 129], "f32", "f16"), (14, 2, [3000, 17], "f16", "f16"), (48, 8, [350], "f16", "f16"), (1, 1, [5], "f32", "f16"),
    (32, 8, [int(x) for x in np.linspace(1, 260, 70)], "f16", "f16"), (32, 4, [4100], "f16", "f16"),
]


def _decode_case(n_q, n_kv, lens, qt, seed):
    r = np.random.default_rng(seed)
    per = max(1, (max(lens) + 31) // 32) + 1                     # a table longer than any context
    n_blocks = len(lens) * per + 3
    tables = r.permutation(n_blocks)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
    q = dev(r.normal(size=(len(lens), n_q, D)).astype(np.float32), torch.float32 if qt == "f32" else torch.float16)
    return q, ref.random_pool(n_blocks, n_kv, seed), tables, np.array(lens, np.int32) - 1


def _decode_ref(q, kv, tables, pos, n_kv):
    K, V = ref.stored(kv)
    qf = q.float().cpu().numpy().astype(np.float64)
    return np.concatenate([ref.attend(qf[i:i + 1], K, V, tables[i], pos[i:i + 1], n_kv) for i in range(len(pos))]), np.abs(V).max()


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_attention(q3, case):
    n_q, n_kv, lens, qt, ot = case
    q, kv, tables, pos = _decode_case(n_q, n_kv, lens, qt, 50 + len(lens) + n_q)
    out = torch.full(q.shape, 9.0, dtype=torch.float32 if ot == "f32" else torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = np.arange(len(lens), dtype=np.int32)
    q3.op_kv4_decode_attention(q, dev(pos), dev(slot), dev(tables), dev(kv), max_ctx=max(1, max(lens)), out=out, status=status)
    q3.check_status(status)
    want, vmax = _decode_ref(q, kv, tables, pos, n_kv)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= _bound(want, vmax, ot == "f16"))
    assert not got[pos < 0].any()


def test_decode_attention_masked_bytes_do_not_matter(q3):
    # positions past a row's own hold scales and biases that are not numbers
    lens = [1, 31, 33, 70, 128, 0]
    q, kv, tables, pos = _decode_case(32, 8, lens, "f16", 91)
    dirty = kv.copy()
    for i, n in enumerate(lens):
        for p in range(n, tables.shape[1] * 32):
            b, r = tables[i, p // 32], p % 32
            dirty[b, 0, :, 2048 + r * 16:2064 + r * 16] = 0xff
            w = 2048 + (r // 2) * 32 + (r % 2) * 2 + np.arange(8) * 4
            dirty[b, 1][:, np.concatenate([w, w + 1])] = 0xff
    args = dev(pos), dev(np.arange(len(lens), dtype=np.int32)), dev(tables)
    a = q3.op_kv4_decode_attention(q, *args, dev(kv))
    b = q3.op_kv4_decode_attention(q, *args, dev(dirty))
    assert torch.isfinite(b).all() and torch.equal(a, b)


def test_decode_attention_rows_share_a_slot_and_strides(q3):
    # four rows of one slot at different positions, q a slice of wider rows
    q, kv, tables, _ = _decode_case(32, 8, [200], "f16", 92)
    pos = np.array([199, 3, 64, 199], np.int32)
    wide = torch.randn(4, 48, D, device="cuda").half()
    qq = wide[:, :32]
    out = q3.op_kv4_decode_attention(qq, dev(pos), dev(np.zeros(4, np.int32)), dev(tables), dev(kv))
    K, V = ref.stored(kv)
    want = ref.attend(qq.float().cpu().numpy().astype(np.float64), K, V, tables[0], pos, 8)
    assert np.all(np.abs(out.cpu().numpy() - want) <= _bound(want, np.abs(V).max(), True))


def test_decode_attention_reports_bad_places(q3):
    q, kv, tables, pos = _decode_case(32, 8, [70, 70], "f16", 93)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (dict(t=kv.shape[0]), dict(t=-1), dict(s=2), dict(s=-1), dict(p=tables.shape[1] * 32), dict(p=2 ** 31 - 1)):
        t, s, p = tables.copy(), np.arange(2, dtype=np.int32), pos.copy()
        if "t" in bad:
            t[1, 1] = bad["t"]
        if "s" in bad:
            s[1] = bad["s"]
        if "p" in bad:
            p[1] = bad["p"]
        out = q3.op_kv4_decode_attention(q, dev(p), dev(s), dev(t), dev(kv), status=status)
        with pytest.raises(q3.Q3Error) as e:
            q3.check_status(status)
        assert e.value.code == -7 and "0x2" in str(e.value)
        good, _ = _decode_ref(q[:1], kv, tables, pos[:1], 8)
        assert np.all(np.abs(out[:1].cpu().numpy() - good) <= 0.01)       # the other row is untouched by it
        assert torch.isfinite(out).all()
    q3.check_status(status)                                               # cleared


def test_decode_attention_large_scores(q3):
    # scores in the thousands: the maximum is subtracted before any exponential
    q, kv, tables, pos = _decode_case(32, 8, [150], "f32", 94)
    q = q * 900
    out = q3.op_kv4_decode_attention(q, dev(pos), dev(np.zeros(1, np.int32)), dev(tables), dev(kv))
    want, vmax = _decode_ref(q, kv, tables, pos, 8)
    # scores carry 130 roundings of sum |q k| / sqrt(128) ~ 900 * 7.2: 2^-24 * 130 * 6480 = 0.05 absolute
    assert np.all(np.abs(out.cpu().numpy() - want) <= 0.11 * vmax)


# ---------------------------------------------------------------- prefill attention

PREFILL = [  # n_q, n_kv, (rows, first position) of each sequence
    (32, 8, [(1, 0)]), (32, 8, [(37, 0)]), (32, 8, [(300, 0)]), (32, 8, [(83, 200)]), (16, 8, [(97, 31), (1, 64), (0, 5), (130, 0)]),
    (40, 8, [(60, 77), (26, 0)]), (8, 8, [(200, 0)]), (24, 8, [(50, 3)]), (64, 8, [(33, 129)]), (14, 2, [(129, 1000)]), (1, 1, [(7, 0)]),
    (48, 8, [(22, 0), (22, 41)]), (32, 8, [(5, -3)]),
]


def _prefill_case(n_q, n_kv, seqs, seed, tail=4):
    r = np.random.default_rng(seed)
    per = max(1, max((n + max(p, 0) + 31) // 32 for n, p in seqs)) + 1
    n_blocks = len(seqs) * per + 3
    tables = r.permutation(n_blocks)[:len(seqs) * per].reshape(len(seqs), per).astype(np.int32)
    at = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
    q = dev(r.normal(size=(int(at[-1]) + tail, n_q, D)).astype(np.float32), torch.float16)
    return q, ref.random_pool(n_blocks, n_kv, seed), tables, at, np.array([p for _, p in seqs], np.int32)


def _prefill_ref(q, kv, tables, at, pos, n_kv, slots=None):
    K, V = ref.stored(kv)
    qf = q.float().cpu().numpy().astype(np.float64)
    out = np.full(qf.shape, np.nan)
    for i in range(len(pos)):
        a, b = at[i], at[i + 1]
        out[a:b] = ref.attend(qf[a:b], K, V, tables[i if slots is None else slots[i]], pos[i] + np.arange(b - a), n_kv) if b > a else 0
    return out, np.abs(V).max()


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill_attention(q3, case):
    n_q, n_kv, seqs = case
    q, kv, tables, at, pos = _prefill_case(n_q, n_kv, seqs, 200 + n_q + len(seqs))
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(kv), out=out, status=status)
    q3.check_status(status)
    want, vmax = _prefill_ref(q, kv, tables, at, pos, n_kv)
    got = out.cpu().numpy().astype(np.float64)
    n = at[-1]
    assert np.all(np.abs(got - want)[:n] <= _bound(want, vmax, True, prefill=True)[:n])
    assert (got[n:] == 9.0).all()                                  # rows of no sequence are left alone


# Few tiles on long contexts, which are cut into pieces: (query heads, KV heads, [(rows, first position)])
CUT = [(1, 1, [(3, 5000)]), (40, 8, [(60, 3000), (1, 2047)]), (8, 2, [(5, 1), (9, 6000), (0, 9), (70, 513)]), (16, 16, [(260, 800)])]


@pytest.mark.parametrize("case", CUT, ids=str)
def test_prefill_attention_of_few_tiles_on_long_contexts(q3, case):
    n_q, n_kv, seqs = case
    q, kv, tables, at, pos = _prefill_case(n_q, n_kv, seqs, 700 + n_q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [dev(at), dev(pos), dev(tables), dev(kv)]
    n = at[-1]
    got = q3.op_kv4_prefill_attention(q, *args, status=status)[:n]
    q3.check_status(status)
    want, vmax = _prefill_ref(q, kv, tables, at, pos, n_kv)
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - want[:n]) <= _bound(want, vmax, True, prefill=True)[:n])
    for _ in range(5):                                             # whichever piece is last, the sums' order is one
        assert torch.equal(got, q3.op_kv4_prefill_attention(q, *args)[:n])


def test_prefill_attention_twice_is_the_same(q3):
    """Tiles of equal length are listed in no fixed order: their places in a CTA's work do not show."""
    q, kv, tables, at, pos = _prefill_case(24, 8, [(411, 134), (195, 134), (300, 134)] * 2, 304)
    args = [dev(at), dev(pos), dev(tables), dev(kv)]
    got = q3.op_kv4_prefill_attention(q, *args)[:at[-1]]
    for _ in range(20):
        assert torch.equal(got, q3.op_kv4_prefill_attention(q, *args)[:at[-1]])


def test_prefill_attention_of_rows_in_many_sequences(q3):
    """Sequences that go back to earlier rows have more tiles than the workspace lists: reported, and nothing is written past
    it."""
    T, ns = 256, 40                                                # 20 x 16 tiles for a list of 16 + 40
    q, kv, _, _, _ = _prefill_case(16, 2, [(T, 0)], 303, tail=0)
    tables = torch.arange(8, dtype=torch.int32, device="cuda").repeat(ns, 1)
    at = torch.tensor([0, T] * (ns // 2) + [0], dtype=torch.int32, device="cuda")
    pos = torch.zeros(ns, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = q3.kv4_prefill_workspace(ns, T, 16, 2, 8, kv.shape[0])
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)                                      # what is not listed is left as it was
    q3.op_kv4_prefill_attention(q, at, pos, tables, dev(kv), out=out, workspace=room[:size], status=status)
    with pytest.raises(q3.Q3Error) as e:
        q3.check_status(status)
    assert e.value.code == -7 and (room[size:] == 77).all() and torch.isfinite(out.float()).all()


def test_prefill_attention_masked_bytes_and_slots(q3):
    q, kv, tables, at, pos = _prefill_case(32, 8, [(45, 20), (70, 0)], 301)
    slots = np.array([1, 0], np.int32)
    dirty = kv.copy()
    for i, s in enumerate(slots):
        for p in range(pos[i] + at[i + 1] - at[i], tables.shape[1] * 32):
            b, r = tables[s, p // 32], p % 32
            dirty[b, 0, :, 2048 + r * 16:2064 + r * 16] = 0xff
            w = 2048 + (r // 2) * 32 + (r % 2) * 2 + np.arange(8) * 4
            dirty[b, 1][:, np.concatenate([w, w + 1])] = 0xff
    n = at[-1]
    a = q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(kv), seq_slot=dev(slots))[:n]
    b = q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(dirty), seq_slot=dev(slots))[:n]
    assert torch.isfinite(b).all() and torch.equal(a, b)
    want, vmax = _prefill_ref(q, kv, tables, at, pos, 8, slots)
    assert np.all(np.abs(a.cpu().numpy() - want[:n]) <= _bound(want, vmax, True, prefill=True)[:n])


def test_prefill_attention_reports_bad_places(q3):
    q, kv, tables, at, pos = _prefill_case(32, 8, [(70, 0), (10, 0)], 302)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = q3.op_kv4_prefill_attention(q, dev(at), dev(pos), dev(tables), dev(kv), status=status)
    q3.check_status(status)
    for bad in (dict(t=kv.shape[0]), dict(t=-1), dict(s=5), dict(p=tables.shape[1] * 32)):
        t, s, p = tables.copy(), np.arange(2, dtype=np.int32), pos.copy()
        if "t" in bad:
            t[0, 1] = bad["t"]
        if "s" in bad:
            s[0] = bad["s"]
        if "p" in bad:
            p[0] = bad["p"]
        out = q3.op_kv4_prefill_attention(q, dev(at), dev(p), dev(t), dev(kv), seq_slot=dev(s), status=status)
        with pytest.raises(q3.Q3Error) as e:
            q3.check_status(status)
        assert e.value.code == -7 and "0x2" in str(e.value)
        assert torch.isfinite(out[:80]).all() and torch.equal(out[70:80], good[70:80])


# ---------------------------------------------------------------- together

def test_append_prefill_decode_together_captured_and_on_another_stream(q3):
    """A prompt appended and attended, then three decode steps, eagerly, replayed from a graph and on a side stream: the
    same bits, and the reference's attention over the cache the appends left."""
    n_q, n_kv, T = 32, 8, 75
    g = torch.Generator(device="cuda").manual_seed(5)
    gains = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    rope = q3.rope_table(128, 1e6)
    prompt = torch.randn(T, 48 * D, generator=g, device="cuda")
    steps = torch.randn(3, 1, 48 * D, generator=g, device="cuda")
    tables = torch.tensor([[3, 0, 4, 1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    step_pos = [torch.tensor([T + i], dtype=torch.int32, device="cuda") for i in range(3)]

    def whole(kv, stream=None):
        outs = []
        q = q3.op_kv4_append(prompt, *gains, rope, pos, zero, tables, kv, n_q, stream=stream)
        outs += [q, q3.op_kv4_prefill_attention(q, at, zero[:1], tables, kv, stream=stream)]
        for i in range(3):
            q = q3.op_kv4_append(steps[i], *gains, rope, step_pos[i], zero[:1], tables, kv, n_q, stream=stream)
            outs += [q, q3.op_kv4_decode_attention(q, step_pos[i], zero[:1], tables, kv, stream=stream)]
        return outs

    def fresh():
        return torch.zeros(5, 2, n_kv, ref.TILE, dtype=torch.uint8, device="cuda")

    kv = fresh()
    outs = [o.clone() for o in whole(kv)]
    K, V = ref.stored(kv.cpu().numpy())
    vmax = np.abs(V).max()
    tab = tables[0].cpu().numpy()
    want = ref.attend(outs[0].cpu().numpy().astype(np.float64), K, V, tab, np.arange(T), n_kv)
    assert np.all(np.abs(outs[1].cpu().numpy() - want) <= _bound(want, vmax, True, prefill=True))
    for i in range(3):
        want = ref.attend(outs[2 + 2 * i].cpu().numpy().astype(np.float64), K, V, tab, np.array([T + i]), n_kv)
        assert np.all(np.abs(outs[3 + 2 * i].cpu().numpy() - want) <= _bound(want, vmax, True))

    side = torch.cuda.Stream()
    kv2 = fresh()
    torch.cuda.synchronize()
    got = whole(kv2, stream=side)
    side.synchronize()
    assert torch.equal(kv, kv2) and all(torch.equal(a, b) for a, b in zip(outs, got))

    kv3 = fresh()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = whole(kv3)
    for _ in range(2):
        kv3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kv, kv3) and all(torch.equal(a, b) for a, b in zip(outs, got))


def test_operators_follow_copies_and_other_streams_in_a_graph(q3):
    """Calls captured behind a copy, behind a memset and behind another stream's work read what those wrote."""
    n_q, n_kv, T = 32, 8, 40
    g = torch.Generator(device="cuda").manual_seed(8)
    gains = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    rope = q3.rope_table(64, 1e6)
    source = torch.randn(T, 48 * D, generator=g, device="cuda")
    tables = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    qkv, kv = torch.empty_like(source), torch.empty(3, 2, n_kv, 2560, dtype=torch.uint8, device="cuda")
    logits = torch.empty(T, 1000, device="cuda")
    seed = torch.randn(T, 1000, generator=g, device="cuda")
    side = torch.cuda.Stream()

    def steps():
        kv.zero_()
        qkv.copy_(source)
        q = q3.op_kv4_append(qkv, *gains, rope, pos, zero, tables, kv, n_q)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            logits.copy_(seed)
            logits.mul_(3.0)
            rows = q3.op_kv4_prefill_attention(q, at, zero[:1], tables, kv)
        one = q3.op_kv4_decode_attention(q[-1:], pos[-1:], zero[:1], tables, kv)
        main.wait_stream(side)
        return [q, rows, one, kv, *q3.op_token_logprobs(logits, zero, 3)]

    want = [t.clone() for t in steps()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps()
    for _ in range(3):
        for t in (kv, qkv, logits):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("default", [False, True])
def test_operators_wait_for_events(q3, default):
    """A call behind another call and an event of slow work elsewhere reads what that work wrote."""
    other, here = torch.cuda.Stream(), torch.cuda.default_stream() if default else torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    source, targets = torch.randn(64, 5000, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    late = torch.empty_like(source)
    want = q3.op_token_logprobs(source, targets, 4)
    for _ in range(5):
        late.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            b = a
            for _ in range(6):
                b = b @ a * 1e-2
            late.copy_(source)
            event = other.record_event()
        with torch.cuda.stream(here):
            q3.op_token_logprobs(source, targets, 4)
            here.wait_event(event)
            got = q3.op_token_logprobs(late, targets, 4)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
