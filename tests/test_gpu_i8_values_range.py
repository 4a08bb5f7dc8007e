"""Values that 8-bit rows stand for, in a type that does not hold them: infinities, and
the status says so.  A row's largest code is 127, so its largest value is 127 * scale,
rounded to FP32 and then to the values' type; torch rounds alike."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def run(f, t, k, dtype):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    values = torch.empty(t, k, dtype=dtype, device="cuda")
    codes, scales = f(values, status)[:2]
    want = (codes.float() * scales.unsqueeze(1)).to(dtype)
    assert torch.equal(values, want)
    finite = bool(torch.isfinite(want).all())
    assert status.item() == (0 if finite else 8)
    return finite


@pytest.mark.parametrize("k", [1, 333, 2560, 20000, 20500, 20501])
@pytest.mark.parametrize("values", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(q3, dtype, values, k):
    x = torch.randn(300, k, device="cuda").clamp(-3, 3).to(TYPES[dtype])
    assert run(lambda v, s: q3.op_i8_quantize(x, values=v, status=s), 300, k, TYPES[values])
    seen = set()
    for top in (65504.0, 65519.0, 65520.0, 65536.0, 1e30, 3.3895e38, 3.3961e38, 3.3962e38, MOST):
        if not torch.isfinite(torch.tensor(top, dtype=TYPES[dtype])):
            continue
        y = x.clone()
        y[299, k - 1] = -top
        seen.add(run(lambda v, s: q3.op_i8_quantize(y, values=v, status=s), 300, k, TYPES[values]))
    if dtype == "f16":
        assert seen == {True}                                     # 65,504 at most
    if (dtype, values) in (("f32", "f16"), ("f32", "bf16")):
        assert seen == {True, False}


@pytest.mark.parametrize("k", [8, 333, 9728, 20501])
@pytest.mark.parametrize("dtype", TYPES)
def test_swiglu_and_norm(q3, dtype, k):
    x = torch.ones(5, 2 * k, dtype=TYPES[dtype], device="cuda")
    assert run(lambda v, s: q3.op_i8_swiglu(x, values=v, status=s), 5, k, torch.float16)
    x[3, 0] = x[3, k] = 300.0                                     # 300 * 300 = 90,000
    assert not run(lambda v, s: q3.op_i8_swiglu(x, values=v, status=s), 5, k, torch.float16)
    assert run(lambda v, s: q3.op_i8_swiglu(x, values=v, status=s), 5, k, torch.bfloat16)
    gain = torch.full((2 * k,), 60000.0, device="cuda").bfloat16()
    y = torch.ones(5, 2 * k, dtype=TYPES[dtype], device="cuda")
    for delta in (None, y):
        assert run(lambda v, s: q3.op_i8_norm(y, gain, delta=delta, values=v, status=s), 5, 2 * k, torch.float16)
        assert not run(lambda v, s: q3.op_i8_norm(y, gain * 2, delta=delta, values=v, status=s), 5, 2 * k, torch.float16)


def test_a_call_without_values_or_status_is_as_before(q3):
    x = torch.full((3, 40), 1e6, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = q3.op_i8_quantize(x, status=status)
    assert status.item() == 0 and bool((codes == 127).all())
    values = torch.empty(3, 40, dtype=torch.float16, device="cuda")
    assert torch.equal(q3.op_i8_quantize(x, values=values)[0], codes) and torch.isinf(values).all()
