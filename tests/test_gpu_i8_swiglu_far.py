"""SwiGLU in 8-bit integers at gates as far out as their type holds: z / (1 + e^-z)
is z, or zero, there, and the row has the codes and the scale that 64 bits give.

The bounds are those of the other tests of the row writers: a code within 0.5 + 2^-13
of y / scale, a scale within 2^-17.  Here e is exactly 0, silu(z) exactly z or zero,
and y a single product; both bounds hold with room."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def check(q3, x):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = q3.op_i8_swiglu(x, status=status)
    g, u = np.split(x.double().cpu().numpy(), 2, axis=1)
    with np.errstate(over="ignore"):
        y = g / (1 + np.exp(-g)) * u
    want = np.abs(y).max(1) / 127
    c, s = codes.double().cpu().numpy(), scales.double().cpu().numpy()
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want)
    assert np.all(np.abs(c - y / np.where(want > 0, want, 1)[:, None]) <= 0.5 + 2.0 ** -13)
    assert status.item() == 0


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("k", [1, 8, 333, 20500])
@pytest.mark.parametrize("up", [1e-30, 0.5, -0.25])
@pytest.mark.parametrize("dtype", TYPES)
def test_gates_up_to_the_largest(q3, dtype, up, k, at):
    most = torch.finfo(TYPES[dtype]).max
    for far in (90.0, 199.0, 201.0, 263.0, 265.0, 1e30, 2.3e38, 2.4e38, most):
        for gate in (far, -far):
            buf = torch.zeros(3 * 2 * k + at, device="cuda")
            x = buf[at:].view(3, 2 * k)
            x[:, :k] = torch.randn(3, k, device="cuda")
            x[:, k:] = up
            x[0, 0], x[2, k - 1] = gate, gate
            if k == 1 and gate < 0 and far < 1e30:
                continue                             # the row is one y below what FP32 holds
            wide = torch.zeros(buf.numel(), dtype=TYPES[dtype], device="cuda")
            wide.copy_(buf)
            check(q3, wide[at:].view(3, 2 * k))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", [float("inf"), -float("inf"), float("nan")])
def test_gates_that_are_no_numbers_stay_such(q3, dtype, gate):
    x = torch.ones(3, 80, dtype=TYPES[dtype], device="cuda")
    x[1, 7] = gate
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = q3.op_i8_swiglu(x, status=status)
    assert status.item() == 8
    assert torch.isnan(scales).tolist() == [False, True, False] and not codes[1].any()
