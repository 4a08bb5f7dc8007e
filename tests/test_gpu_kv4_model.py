"""A model over the 4-bit K/V cache, and scored rounds.

- A position's K and V take 2 * n_kv * 80 bytes a layer: 3.2x under BF16.
- The forward against the oracle's AFFINE4-cache forward.  Token by token (FP32
  projections) the usual gate holds: NMSE <= 1e-4, identical argmax.  Prompt
  rounds, mixed rounds and batched decode round their activations to fp16
  before the projections, and a 4-bit cache turns that into code changes:
  gate4() below, a wiring fault being an NMSE near 1.
- A permuted block table gives the identity table's logits bit for bit;
  truncate and a shared prefix give the same logits as a fresh evaluation.
- q3_session_score equals the log probabilities of q3_session_eval_n's logits
  (the same logits: only the way of summing differs, tolerances as in
  test_gpu_logprobs.py), over every cache, in chunks, and for one token on the
  fused and the per-operation step.

The bound of rounds over fp16 activations.  A K or V row of spread sigma
carries a rounding of 2^-11 sigma from them.  Packed, the group's bias (|min|
<= 4 sigma) and its scale over 15 steps (a range <= 8 sigma) may each land on
the next fp16 number, moving every value of the group by up to (4 + 8) 2^-11
sigma against its code boundaries: Delta <= 13 * 2^-11 sigma in all.  A value
changes its code with probability Delta / step and then moves by one step (<= 8
sigma / 15): Delta * step <= 3.4e-3 sigma^2 a value, an NMSE of 3.4e-3 of K and
of V.  V's error passes through the average; K's moves scores of unit spread by
sqrt(3.4e-3), as much again: 6.8e-3 a layer, added over the layers.
"""
import numpy as np
import pytest
import torch

import synthetic
from helpers import Pair, check_row, make_shape
from test_gpu_logprobs import close, reference

pytestmark = pytest.mark.gpu

TINY_KV4 = make_shape("tiny", kv_quant=synthetic.AFFINE4, name="tiny-kv-affine4")


@pytest.fixture(scope="module")
def pair():
    return Pair(TINY_KV4, seed=901, max_ctx=512, max_round_tokens=256, n_blocks=96)


def gate4(got, ref, n_layers, what):
    c = check_row(got, ref)
    assert c.nmse <= 6.8e-3 * n_layers, (what, c)
    return c


def _run(pair, g, o, rounds, n_decode, tag):
    for r in rounds:
        got, ref, am = pair.eval(g, o, r)
        c = gate4(got, ref, 2, (tag, len(r)))
    tok = c.argmax_ref
    for step in range(n_decode):
        got, ref, am = pair.eval(g, o, [tok])
        c = gate4(got, ref, 2, (tag, step))
        assert am == c.argmax_gpu
        tok = c.argmax_ref


def test_token_by_token_meets_the_usual_gate(pair):
    perm = synthetic.make_block_permutation(96, seed=899)
    g, o = pair.sessions(table=perm[60:63])
    for step, tok in enumerate(synthetic.make_tokens(70, TINY_KV4.vocab, seed=898)):
        got, ref, am = pair.eval(g, o, [tok])
        c = check_row(got, ref, "kv4/tiny/one")
        assert c.ok, (step, c)
        assert am == c.argmax_gpu
    g.close()


def test_paths_and_bytes(pair, orc):
    q3 = pair.q3
    assert not pair.model.fused_decode and pair.model.prefill_tc
    with pytest.raises(q3.Q3Error):
        pair.model.set_prefill_tc(False)
    assert pair.model.kv_bytes_per_position == orc.kv_bytes_per_position(TINY_KV4) == 2 * 8 * 80
    assert 2 * 8 * 128 * 2 / pair.model.kv_bytes_per_position == 3.2


def test_prompt_then_greedy_decode_permuted_table(pair):
    perm = synthetic.make_block_permutation(96, seed=902)
    g, o = pair.sessions(table=perm[:4])
    _run(pair, g, o, [synthetic.make_tokens(8, TINY_KV4.vocab, seed=903)], 8, "kv4/tiny")
    g.close()


def test_chunked_prompt_across_block_edges(pair):
    perm = synthetic.make_block_permutation(96, seed=904)
    g, o = pair.sessions(table=perm[20:32])
    toks = synthetic.make_tokens(280, TINY_KV4.vocab, seed=905)
    _run(pair, g, o, [toks[:256], toks[256:]], 20, "kv4/tiny-300")
    g.close()


def test_paged_equals_identity_table_bitwise_and_truncate(pair):
    prompt = synthetic.make_tokens(70, TINY_KV4.vocab, seed=906)
    outs = []
    for table in (np.arange(40, 43), synthetic.make_block_permutation(96, seed=907)[50:53]):
        g = pair.pool.session()
        g.set_block_table(table)
        rows = []
        for toks in (prompt[:45], prompt[45:], [5], [6], [7]):
            g.eval(torch.tensor(np.asarray(toks, np.int32), device="cuda"), pair.logits[0])
            pair.model.sync()
            rows.append(pair.logits[0].cpu().numpy().copy())
        g.truncate(70)                                          # the decode steps again
        for i, tok in enumerate((5, 6, 7)):
            g.eval(torch.tensor([tok], dtype=torch.int32, device="cuda"), pair.logits[0])
            pair.model.sync()
            np.testing.assert_array_equal(pair.logits[0].cpu().numpy(), rows[2 + i])
        outs.append(np.stack(rows))
        g.close()
    np.testing.assert_array_equal(outs[0], outs[1])


def test_mixed_rounds_and_batched_decode(pair):
    lens = [1, 40, 100, 33]
    gs, os_, lists = [], [], []
    for i, n in enumerate(lens):
        g, o = pair.sessions()
        first = synthetic.make_tokens(30 * i + 1, TINY_KV4.vocab, seed=910 + i)
        pair.eval(g, o, first)
        gs.append(g)
        os_.append(o)
        lists.append(synthetic.make_tokens(n, TINY_KV4.vocab, seed=920 + i))
    for step in range(4):                                      # a mixed round, then decode rounds
        got, ref, am = pair.eval_batch(gs, os_, lists)
        for i in range(len(gs)):
            c = gate4(got[i], ref[i], 2, ("mixed", step, i))
            assert am[i] == c.argmax_gpu
        lists = [[int(np.argmax(r))] for r in ref]
    for g in gs:
        g.close()


def test_prefix_sharing(pair):
    pool = pair.model.pool(40, 4)
    pool.enable_prefix()
    toks = synthetic.make_tokens(150, TINY_KV4.vocab, seed=931)
    dev = torch.tensor(toks, device="cuda")
    a = pool.session()
    a.eval(dev[:128].contiguous(), pair.logits[0])
    a.eval(dev[128:].contiguous(), pair.logits[0])
    assert a.publish(toks) == 4
    b = pool.session()
    n = b.attach_prefix(toks)
    assert n == 128
    b.eval(dev[n:].contiguous(), pair.logits[1])
    c = pair.pool.session()
    c.eval(dev[:n].contiguous(), pair.logits[2])
    c.eval(dev[n:].contiguous(), pair.logits[2])
    pair.model.sync()
    assert torch.equal(pair.logits[1], pair.logits[2])          # the same rounds over the same stored values
    for s in (a, b, c):
        s.close()


def test_qwen3_4b_heads_batched_decode_at_2000_positions():
    shape = make_shape("4b", n_layers=1, kv_quant=synthetic.AFFINE4, name="qwen3-4b-kv-affine4")
    B, n = 4, 2000
    pair = Pair(shape, seed=940, max_ctx=n + 64, max_round_tokens=2048, n_blocks=B * 66 + 8, max_sessions=B + 2)
    gs, os_ = [], []
    for i in range(B):
        g, o = pair.sessions()
        toks = synthetic.make_tokens(n - 37 * i, shape.vocab, seed=941 + i)
        g.eval(torch.tensor(toks, device="cuda"), pair.logits[0])
        o.append(toks)
        gs.append(g)
        os_.append(o)
    pair.model.sync()
    nxt = [[int(t)] for t in synthetic.make_tokens(B, shape.vocab, seed=950)]
    for step in range(3):
        got, ref, am = pair.eval_batch(gs, os_, nxt)
        for i in range(B):
            gate4(got[i], ref[i], 1, ("4b", step, i))
        nxt = [[int(np.argmax(r))] for r in ref]
    for g in gs:
        g.close()


# ---------------------------------------------------------------- scored rounds

def _scored(model, pool, toks, targets, k, vocab, split=None):
    """(score's outputs, eval_n's logits) of the same round, each in a session of its own."""
    dev = torch.tensor(toks, device="cuda")
    t = torch.tensor(targets, dtype=torch.int32, device="cuda")
    n = len(targets)
    a, b = pool.session(), pool.session()
    if split:
        warm = torch.empty(vocab, device="cuda")
        a.eval(dev[:split].contiguous(), warm)
        b.eval(dev[:split].contiguous(), warm)
        dev = dev[split:].contiguous()
    got = a.score(dev, t, top_k=k)
    logits = torch.empty(n, vocab, device="cuda")
    b.eval_n(dev, n, logits)
    model.sync()
    assert a.pos == b.pos == len(toks)
    a.close()
    b.close()
    return [o.cpu().numpy() for o in got], logits.cpu().numpy().astype(np.float64)


def _check_scores(got, logits, targets, k):
    targets = np.asarray(targets)
    lp, H, ids, tlp, m = reference(logits, np.maximum(targets, 0), k)
    np.testing.assert_array_equal(got[2], ids)
    close(got[0], np.where(targets < 0, 0.0, lp), np.abs(m) + np.abs(logits).max(1))
    close(got[1], H, np.abs(m))
    close(got[3], tlp, 2 * np.abs(m)[:, None])


@pytest.mark.parametrize("kv", [synthetic.BF16, synthetic.Q8_0, synthetic.AFFINE4])
def test_scores_equal_the_logits_of_the_round(kv):
    shape = make_shape("tiny", kv_quant=kv, name=f"tiny-{kv}")
    pair = Pair(shape, seed=960, max_ctx=512, max_round_tokens=128, n_blocks=64)
    r = np.random.default_rng(961)
    toks = synthetic.make_tokens(300, shape.vocab, seed=962)
    for n, k, split in ((300, 5, None), (299, 0, None), (130, 20, None), (1, 32, 299), (40, 3, 260), (128, 1, 100)):
        targets = r.integers(0, shape.vocab, n).astype(np.int32)
        targets[0] = -1 if n > 1 else targets[0]
        got, logits = _scored(pair.model, pair.pool, toks, targets, k, shape.vocab, split)
        _check_scores(got, logits, targets, k)


def test_one_token_scores_on_both_steps_and_in_chunks():
    shape = make_shape("tiny")
    pair = Pair(shape, seed=970, max_ctx=2048, max_round_tokens=1200, n_blocks=160)
    toks = synthetic.make_tokens(1500, shape.vocab, seed=971)
    for fused in (True, False):
        pair.model.set_fused_decode(fused)
        got, logits = _scored(pair.model, pair.pool, toks[:65], [7], 4, shape.vocab, 64)
        _check_scores(got, logits, [7], 4)
    # 1,100 rows of logits pass through the 512-row scratch in three parts
    targets = np.concatenate([toks[1:1100], [-1]]).astype(np.int32)
    got, logits = _scored(pair.model, pair.pool, toks[:1100], targets, 6, shape.vocab)
    _check_scores(got, logits, targets, 6)


def test_score_refusals_and_bad_targets():
    shape = make_shape("tiny")
    pair = Pair(shape, seed=980, max_ctx=64, max_round_tokens=32, n_blocks=8)
    q3 = pair.q3
    s = pair.pool.session()
    toks = torch.tensor(synthetic.make_tokens(20, shape.vocab, seed=981), device="cuda")
    t = torch.zeros(20, dtype=torch.int32, device="cuda")
    for bad in (lambda: s.score(toks.long()), lambda: s.score(toks, t.long()), lambda: s.score(toks, t, n_score=19),
                lambda: s.score(toks, n_score=21), lambda: s.score(toks, n_score=0), lambda: s.score(toks, top_k=-1),
                lambda: s.score(toks, t.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q3.Q3Error) as e:
        s.score(toks, top_k=33)
    assert e.value.code == -1
    with pytest.raises(q3.Q3Error) as e:
        s.score(torch.zeros(65, dtype=torch.int32, device="cuda"))
    assert e.value.code == -5
    assert s.pos == 0
    s.score(toks[:1])
    assert q3.lib().q3_session_score(s.h, toks.data_ptr(), 2 ** 31 - 1, 1, None, 0, None, None, None, None) == -5
    t[3] = shape.vocab
    s.score(toks, t)
    with pytest.raises(q3.Q3Error) as e:
        pair.model.sync()
    assert e.value.code == -7 and "0x1" in str(e.value)
