"""Refusals of the 4-bit cache and scoring operators that need no GPU: the C
entry points check sizes, strides, types and alignment before any CUDA call,
the binding checks tensors' shapes, types and devices before the library."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3.lib()


P, ODD = 1 << 20, (1 << 20) + 4           # an aligned and a misaligned address (never read)


def _append(L, **kw):
    a = dict(qkv=P, type=0, stride=48 * 128, qg=P, kg=P, eps=1e-6, rope=P, rope_len=64, pos=P, slot=P, T=4, n_q=32, n_kv=8,
             tables=P, n_slots=2, max_blocks=2, kv=P, n_blocks=8, q_out=P, kv_out=None, status=None)
    a.update(kw)
    return L.q3_op_kv4_append(*a.values(), None)


def _decode(L, **kw):
    a = dict(q=P, type=1, stride=32 * 128, pos=P, slot=P, T=4, n_q=32, n_kv=8, tables=P, n_slots=2, max_blocks=2, max_ctx=0, kv=P,
             n_blocks=8, out=P, out_type=1, status=None)
    a.update(kw)
    return L.q3_op_kv4_decode_attention(*a.values(), None)


def _prefill(L, **kw):
    a = dict(q=P, stride=32 * 128, rows=P, pos=P, slot=None, ns=1, T=4, n_q=32, n_kv=8, tables=P, n_slots=2, max_blocks=2, kv=P,
             n_blocks=8, out=P, ws=P, ws_bytes=1 << 40, status=None)
    a.update(kw)
    return L.q3_op_kv4_prefill_attention(*a.values(), None)


def _logprobs(L, **kw):
    a = dict(x=P, type=0, stride=100, N=4, V=100, targets=P, top=5, lp=P, H=P, ids=P, tlp=P, status=None)
    a.update(kw)
    return L.q3_op_token_logprobs(*a.values(), None)


SIZES = [dict(n_kv=0), dict(n_q=31), dict(n_q=72), dict(T=-1), dict(tables=None), dict(n_slots=0), dict(max_blocks=0),
         dict(max_blocks=(1 << 20) + 1), dict(kv=None), dict(kv=ODD), dict(n_blocks=0), dict(T=1 << 28)]


@pytest.mark.parametrize("bad", SIZES + [
    dict(qkv=None), dict(qkv=ODD), dict(type=3), dict(type=-1), dict(stride=48 * 128 - 4), dict(stride=48 * 128 + 2),
    dict(type=1, stride=48 * 128 + 4), dict(qg=None), dict(kg=ODD), dict(rope=None), dict(rope=ODD), dict(rope_len=0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(slot=None), dict(q_out=ODD), dict(kv_out=ODD)], ids=str)
def test_append_refuses(L, bad):
    assert _append(L, **bad) == -1


@pytest.mark.parametrize("bad", SIZES + [
    dict(q=None), dict(q=ODD), dict(type=2), dict(out_type=2), dict(stride=32 * 128 - 8), dict(stride=32 * 128 + 4),
    dict(pos=None), dict(slot=None), dict(out=None), dict(out=ODD), dict(max_ctx=-1), dict(max_ctx=65)], ids=str)
def test_decode_refuses(L, bad):
    assert _decode(L, **bad) == -1


@pytest.mark.parametrize("bad", SIZES + [
    dict(q=None), dict(q=ODD), dict(stride=32 * 128 + 4), dict(rows=None), dict(pos=None), dict(ns=-1), dict(ns=3),
    dict(out=None), dict(out=ODD)], ids=str)
def test_prefill_refuses(L, bad):
    assert _prefill(L, **bad) == -1


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 2), dict(type=1, x=P + 1), dict(type=7), dict(stride=99), dict(N=-1), dict(V=0, stride=0),
    dict(targets=None), dict(top=-1), dict(top=33), dict(V=4, top=5)], ids=str)
def test_logprobs_refuses(L, bad):
    assert _logprobs(L, **bad) == -1


def test_nothing_to_do_is_no_error(L):
    # zero rows need no GPU
    assert _append(L, T=0) == 0
    assert _decode(L, T=0) == 0
    assert _prefill(L, T=0) == 0 and _prefill(L, ns=0) == 0
    assert _logprobs(L, N=0) == 0


def test_binding_refuses_before_the_library():
    import qwen3_dense_decoder_gb300 as q3
    kv = torch.zeros(4, 2, 8, 2560, dtype=torch.uint8)
    tab = torch.zeros(1, 2, dtype=torch.int32)
    row = torch.zeros(3, dtype=torch.int32)
    gain = torch.ones(128, dtype=torch.bfloat16)
    rope = torch.zeros(64, 64, 2)
    qkv = torch.zeros(3, 48 * 128)
    q = torch.zeros(3, 32, 128, dtype=torch.float16)
    bad = [
        lambda: q3.op_kv4_append(qkv[:, :-128], gain, gain, rope, row, row, tab, kv, 32),
        lambda: q3.op_kv4_append(qkv, gain.float(), gain, rope, row, row, tab, kv, 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope[:, :32], row, row, tab, kv, 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row[:2], row, tab, kv, 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row.long(), row, tab, kv, 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row, row, tab[0], kv, 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row, row, tab, kv[..., :-1], 32),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row, row, tab, kv, 32, kv_out=torch.zeros(3, 2, 8, 128)),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row, row, tab, kv, 32, status=torch.zeros(2, dtype=torch.int32)),
        lambda: q3.op_kv4_append(qkv, gain, gain, rope, row, row, tab, kv, 32),                     # CPU tensors
        lambda: q3.op_kv4_decode_attention(q.bfloat16(), row, row, tab, kv),
        lambda: q3.op_kv4_decode_attention(q.transpose(0, 1), row, row, tab, kv),
        lambda: q3.op_kv4_decode_attention(q, row, row, tab, kv, out=torch.zeros(2, 32, 128, dtype=torch.float16)),
        lambda: q3.op_kv4_decode_attention(q, row, row, tab, kv),                                    # CPU tensors
        lambda: q3.op_kv4_prefill_attention(q.float(), row[:2], row[:1], tab, kv),
        lambda: q3.op_kv4_prefill_attention(q, row, row[:1], tab, kv),
        lambda: q3.op_kv4_prefill_attention(q, row[:2], row[:1], tab, kv),                           # CPU tensors
        lambda: q3.op_token_logprobs(qkv.double()),
        lambda: q3.op_token_logprobs(qkv.t()),
        lambda: q3.op_token_logprobs(qkv, row[:2]),
        lambda: q3.op_token_logprobs(qkv, row),                                                      # CPU tensors
        lambda: q3.op_token_logprobs([1.0, 2.0]),
        lambda: q3.op_token_logprobs(qkv, top_k=1 << 40),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")


def test_prefill_workspace_is_planned_on_the_host(L):
    import qwen3_dense_decoder_gb300 as q3
    copy = 8 * 16384                                    # one block of eight KV heads in fp16, K and V
    rest = 2 * 152 * 128 * (128 + 4) * 4 + (1 << 16)    # two pieces of a cut tile a CTA: output, maximum and sum of 128 rows; lists
    # the pool's blocks, or the sequences' tables where those are fewer
    assert q3.kv4_prefill_workspace(1, 2048, 32, 8, 64, 40) - 40 * copy < rest
    assert q3.kv4_prefill_workspace(2, 100, 32, 8, 4, 100000) - 8 * copy < rest
    sizes = [q3.kv4_prefill_workspace(n, 300, 32, 8, 16, 64) for n in (0, 1, 2, 4, 5, 9)]
    assert sizes == sorted(sizes)
    for bad in ((-1, 1, 32, 8, 4, 4), (1, -1, 32, 8, 4, 4), (1, 1, 31, 8, 4, 4), (1, 1, 72, 8, 4, 4), (1, 1, 32, 0, 4, 4), (1, 1, 32, 8, 0, 4),
                (1, 1, 32, 8, 4, 0)):
        with pytest.raises(q3.Q3Error):
            q3.kv4_prefill_workspace(*bad)
    assert _prefill(L, ws=None) == -1 and _prefill(L, ws=P + 16) == -1 and _prefill(L, ws_bytes=2 * copy) == -1


def test_score_refuses_without_a_session(L):
    assert L.q3_session_score(None, None, 1, 1, None, 0, None, None, None, None) == -1


def test_oracle_cache_scheme(orc):
    """The oracle's 4-bit cache: its size, and a forward near the BF16 one without equalling it."""
    import numpy as np
    import synthetic
    s = synthetic.SHAPES["4b"]
    assert orc.kv_bytes_per_position(s.replace(kv_quant=synthetic.AFFINE4)) == 2 * 8 * 80
    small = synthetic.Shape("kv4-small", 2, 128, 4, 2, 32, 128, 256, True)
    w = synthetic.make_weights(small, seed=3)
    toks = synthetic.make_tokens(40, small.vocab, seed=4)
    bf, q4 = (orc.Model(small.replace(kv_quant=k), w, n_threads=2).session(max_ctx=64).eval(toks, all_rows=True)
              for k in (synthetic.BF16, synthetic.AFFINE4))
    e = float(((q4 - bf) ** 2).sum() / (bf ** 2).sum())
    assert 0 < e < 0.05, e
    assert np.isfinite(q4).all()
    with pytest.raises(ValueError):                     # whole groups of 32 values a head row
        orc.Model(small.replace(head_dim=16, kv_quant=synthetic.AFFINE4), w, n_threads=1)
