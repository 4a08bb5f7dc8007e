"""Token log probabilities of logits far from zero: x - m - log s rounds at
the size of x - m and of the result, never at that of m, so the bound is the
sums' alone, 1e-5 (1 + |value|), however far the row is shifted."""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def check(q3, x, targets, k):
    lp, H, ids, tlp = (o.cpu().numpy().astype(np.float64) for o in q3.op_token_logprobs(x, torch.from_numpy(targets).cuda(), k))
    wlp, wH, wids, wtlp, _ = reference(x.float().cpu().numpy().astype(np.float64), targets, k)
    np.testing.assert_array_equal(ids, wids)
    for got, want in ((lp, wlp), (H, wH), (tlp, wtlp)):
        assert np.all(np.abs(got - want) <= 1e-5 * (1 + np.abs(want))), float(np.abs(got - want).max())


@pytest.mark.parametrize("offset", [0.0, 3000.0, -3000.0, 60000.0, -60000.0])
@pytest.mark.parametrize("V", [700, 50257])
def test_rows_shifted_by_a_constant(q3, offset, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(6, V, generator=g, device="cuda") * 2 + offset
    check(q3, x, np.arange(6, dtype=np.int32) * 97, 16)


def test_a_nearly_certain_token_far_from_zero(q3):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(4, 4096, generator=g, device="cuda") + 3000
    x[:, 123] = torch.tensor([3018.0, 3022.5, 3030.0, 3012.0], device="cuda")
    check(q3, x, np.full(4, 123, np.int32), 4)
    for dt, at in ((torch.float16, 30000.0), (torch.bfloat16, 1e6)):
        y = (torch.randn(3, 1000, generator=g, device="cuda") * 40 + at).to(dt)
        check(q3, y, np.array([0, 10, 999], np.int32), 5)
