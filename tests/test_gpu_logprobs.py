"""Token log probabilities, entropy and top alternatives against 64 bits.

Ranks are exact: by value, the lowest index first among equals.  The sums run
over at most 600 terms a chain in FP32, a random walk of sqrt(600) roundings
of 2^-24 (1.5e-6 relative; six of them 9e-6), the exponentials are within
2^-21, and m + log s and x - lse round at 2^-24 of |x| + |m| + |log s|:
1e-5 (1 + |value|) + 2^-22 (|x| + |m|) holds each output.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def reference(x, targets, k):
    """x f64 [N, V] without NaN or +inf."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(1, keepdims=True)
        none = np.isneginf(m)
        d = np.where(np.isneginf(x), -np.inf, x - np.where(none, 0, m))
        e = np.exp(d)
        s = e.sum(1, keepdims=True)
        lse = np.where(none, -np.inf, m + np.log(s))
        lp = np.where(none | np.isneginf(x), -np.inf, x - np.where(none, 0, lse))
        H = np.where(none[:, 0], 0.0, (np.log(s) - (np.where(e > 0, d, 0) * e).sum(1, keepdims=True) / s)[:, 0])
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    return lp[np.arange(len(x)), targets], H, order, np.take_along_axis(lp, order, 1), m[:, 0]


def close(got, want, size):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    d = np.abs(got - want)[~inf]
    tol = (1e-5 * (1 + np.abs(want)) + 2.0 ** -22 * size)[~inf]
    assert np.all(d <= tol), float((d / tol).max())


def check(q3, x, k, seed=0, targets=None):
    N, V = x.shape
    t = np.random.default_rng(seed).integers(0, V, N).astype(np.int32) if targets is None else targets
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp, H, ids, tlp = (o.cpu().numpy() for o in q3.op_token_logprobs(x, torch.from_numpy(t).cuda(), k, status=status))
    q3.check_status(status)
    xf = x.float().cpu().numpy().astype(np.float64)
    wlp, wH, wids, wtlp, m = reference(xf, t, k)
    size = np.where(np.isinf(m), 0, np.abs(m))
    xt = xf[np.arange(N), t]
    np.testing.assert_array_equal(ids, wids)
    close(lp, wlp, size + np.abs(np.where(np.isinf(xt), 0, xt)))
    close(H, wH, size)
    close(tlp, wtlp, 2 * size[:, None])


CASES = [(1, 1, 1), (3, 2, 2), (1, 40, 20), (5, 1000, 32), (2, 4096, 1), (7, 32003, 20), (1, 151936, 20), (9, 151936, 5), (300, 1537, 8),
         (33, 50257, 0), (700, 257, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,V,k", CASES)
def test_logprobs(q3, N, V, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(N * 31 + V)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3 + 5).to(dtype)      # the 16-bit types tie often
    check(q3, x, k, seed=V)


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two", "zigzag"])
@pytest.mark.parametrize("V", [33, 5000, 151936])
def test_orders_that_fill_the_alternatives(q3, order, V):
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    x = {"rising": i / V * 20, "falling": -i / V * 20, "equal": torch.full_like(i, 3.25), "two": (i % 2) * 1.5,
         "zigzag": torch.where(i % 2 == 0, i, -i) / V * 20}[order]
    check(q3, torch.stack([x, x.flip(0)]), 32)


def test_infinities(q3):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(6, 3001, generator=g, device="cuda") * 2
    x[0, 1:] = -float("inf")                                      # one token possible
    x[1, :] = -float("inf")                                       # none
    x[2, 100:2900] = -float("inf")
    x[3, :3000] = -float("inf")
    x[4] = 1e30 * torch.randn(3001, generator=g, device="cuda")   # a certain token among huge logits
    x[5] = torch.finfo(torch.float32).min                         # the mask value of the type in every place
    check(q3, x, 20, targets=np.array([0, 7, 100, 3000, int(x[4].argmax()), 9], np.int32))


def test_nan_and_plus_infinity_rows_give_nan_and_others_do_not(q3):
    x = torch.randn(4, 500, device="cuda")
    x[1, 77] = float("nan")
    x[2, 5] = float("inf")
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    lp, H, ids, tlp = q3.op_token_logprobs(x, t, 32)
    bad = torch.tensor([False, True, True, False], device="cuda")
    assert torch.equal(torch.isnan(lp), bad) and torch.equal(torch.isnan(H), bad)
    assert torch.equal(torch.isnan(tlp).all(1), bad) and torch.equal(torch.isnan(tlp).any(1), bad)
    assert ids[2, 0].item() == 5 and not (ids[1] == 77).any()
    check(q3, x[[0, 3]], 32)
    y = torch.full((1, 3), float("nan"), device="cuda")
    y[0, 1] = 2.0
    assert q3.op_token_logprobs(y, None, 3)[2].tolist() == [[1, 0, 2]]


def test_strided_rows_odd_offsets_and_missing_targets(q3):
    wide = torch.randn(11, 2050, device="cuda")
    for view in (wide[:, 1:2002], wide[::2, 3:1000], wide[4:5, 7:]):
        check(q3, view, 7)
        check(q3, wide.half()[:, 1:2002], 7)
    lp, H, ids, tlp = q3.op_token_logprobs(wide, None, 0)
    assert lp is None and ids.shape == (11, 0) and tlp.shape == (11, 0)
    t = torch.full((11,), -1, dtype=torch.int32, device="cuda")
    t[3] = 9
    lp = q3.op_token_logprobs(wide, t)[0]
    assert (lp[t < 0] == 0).all() and lp[3] < 0


def test_bad_targets_are_reported(q3):
    x = torch.randn(3, 50, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp = q3.op_token_logprobs(x, torch.tensor([50, 49, -2], dtype=torch.int32, device="cuda"), status=status)[0]
    assert torch.isnan(lp).tolist() == [True, False, True]
    with pytest.raises(q3.Q3Error) as e:
        q3.check_status(status)
    assert "0x1" in str(e.value)


def test_captured_and_on_another_stream(q3):
    x = torch.randn(5, 20011, device="cuda")
    t = torch.arange(5, dtype=torch.int32, device="cuda")
    want = q3.op_token_logprobs(x, t, 9)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = q3.op_token_logprobs(x, t, 9, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    buf = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q3.op_token_logprobs(buf, t, 9)
    buf.copy_(x)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
