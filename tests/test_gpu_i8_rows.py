"""Rows in 8-bit integers -- as they are, after the norm, as SwiGLU -- against
64 bits.

With z = y / scale of the definition in 64 bits a code lies within 0.5 + 2^-13
of z: FP32 leaves 3 roundings of 2^-24 in s * gain, its maximum and the
reciprocal, and expf (2 ulp), a sum, a quotient and a product in SwiGLU, under
2^-21 for y and for the maximum, times 127.  Scales are within 2^-17: the
squares are summed in chains of at most 128 + 10 roundings of 2^-24, halved by
the root, the rest is a few roundings.  The sum with the residual and the values
that codes stand for are single roundings and equal bit for bit.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def wide(t, k, dtype, gap, seed, scale=1.0, at=0):
    """Rows k wide, k + gap apart, beginning at element `at` of a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(t * (k + gap) + at + gap, generator=g, device="cuda") * scale
    return buf.to(dtype)[at: at + t * (k + gap)].view(t, k + gap)[:, :k]


def f64(t):
    return t.double().cpu().numpy()


def check(y, codes, scales, values):
    """codes, scales and values against the rows y (f64 numpy)."""
    c, s = f64(codes), f64(scales)
    want = np.abs(y).max(1) / 127
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want), float((np.abs(s - want) / want).max())
    z = y / np.where(want > 0, want, 1)[:, None]
    off = np.abs(c - z)
    assert np.all(off <= 0.5 + 2.0 ** -13), float(off.max())
    assert np.all(np.abs(c) <= 127)
    if values is not None:
        assert torch.equal(values, (codes.float() * scales.unsqueeze(1)).to(values.dtype))


def norm64(s, gain, eps):
    return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * gain


def swiglu64(x):
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


SIZES = [(1, 1, 0), (3, 2, 0), (1, 16, 0), (5, 31, 1), (2, 255, 1), (7, 256, 0), (4, 1000, 24), (33, 2047, 33), (1, 2560, 0), (300, 1024, 8),
         (2, 8192, 0), (2, 8193, 0), (3, 9728, 16), (2, 16384, 0), (2, 16385, 3), (2, 17408, 0), (1, 40001, 0), (1, 131071, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k,gap", SIZES)
def test_quantize(q3, t, k, gap, dtype):
    x = wide(t, k, TYPES[dtype], gap, k + t)
    values = torch.full((t, k), 7.0, dtype=TYPES[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = q3.op_i8_quantize(x, values=values, status=status)
    q3.check_status(status)
    check(f64(x), codes, scales, values)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("delta", ["", "f32", "f16", "bf16"])
@pytest.mark.parametrize("t,k,gap", SIZES)
def test_norm(q3, t, k, gap, delta, dtype):
    x = wide(t, k, TYPES[dtype], gap, k + t)
    d = wide(t, k, TYPES[delta], gap // 2, k + t + 1, 0.5) if delta else None
    gain = (1 + 0.1 * torch.randn(k, device="cuda")).bfloat16()
    want = (x.float() + d.float()).to(x.dtype) if delta else x
    keep = x.clone()
    values = torch.empty(t, k, dtype=torch.float16, device="cuda")
    codes, scales, total = q3.op_i8_norm(x, gain, 1e-6, delta=d, values=values)
    assert torch.equal(total, want) and torch.equal(x, keep)
    check(norm64(f64(want), f64(gain), 1e-6), codes, scales, values)
    if delta:                                                     # in place
        again = q3.op_i8_norm(x, gain, 1e-6, delta=d, sum_out=x)
        assert again[2].data_ptr() == x.data_ptr() and torch.equal(x, want)
        assert torch.equal(again[0], codes) and torch.equal(again[1], scales)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k,gap", SIZES)
def test_swiglu(q3, t, k, gap, dtype):
    x = wide(t, 2 * k, TYPES[dtype], gap, k + t, 3.0)
    values = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
    codes, scales = q3.op_i8_swiglu(x, values=values)
    check(swiglu64(f64(x)), codes, scales, values)


@pytest.mark.parametrize("at", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_any_alignment(q3, dtype, at):
    x = wide(9, 2 * 333, TYPES[dtype], 7, at, at=at)
    check(f64(x), *q3.op_i8_quantize(x), None)
    check(swiglu64(f64(x)), *q3.op_i8_swiglu(x), None)
    d = wide(9, 2 * 333, torch.float16, 0, at, at=at)
    gain = torch.ones(2 * 333 + at, device="cuda").bfloat16()[at:]
    for out in (None, wide(9, 2 * 333, TYPES[dtype], 2, 1, at=1)):
        codes, scales, total = q3.op_i8_norm(x, gain, delta=d, sum_out=out)
        assert torch.equal(total, (x.float() + d.float()).to(x.dtype))
        check(norm64(f64(total), f64(gain), 1e-6), codes, scales, None)


@pytest.mark.parametrize("k", [40, 100, 2560])
def test_halves_go_to_even_and_columns_beside_stay(q3, k):
    # scale 1/2: every value is a multiple of a quarter, z a multiple of 1/2, exact in FP32
    x = torch.arange(k, device="cuda").remainder(255).sub(127).float().unsqueeze(0).repeat(3, 1) / 4
    x[:, 0] = 63.5
    base = torch.full((3, (k + 15) // 16 * 16 + 32), 99, dtype=torch.int8, device="cuda")
    scales = torch.empty(3, device="cuda")
    codes, _ = q3.op_i8_quantize(x, codes=base[:, 16: 16 + k], scales=scales)
    assert codes.data_ptr() == base.data_ptr() + 16
    assert torch.equal(codes.float(), torch.round(x * 2)) and torch.equal(scales, torch.full((3,), 0.5, device="cuda"))
    assert bool((base[:, :16] == 99).all()) and bool((base[:, 16 + k:] == 99).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t,k,gap", [(700, 256, 0), (50, 5120, 0), (9, 333, 1), (3, 17408, 0), (2, 40001, 1)])
def test_codes_of_16_bit_values_are_the_definitions(q3, t, k, gap, dtype):
    """127 x and code * max are whole multiples of one power of two below 2^53: the remainder is exact, and a half goes to even."""
    x = wide(t, k, TYPES[dtype], gap, t + k)
    codes, _ = q3.op_i8_quantize(x)
    v, c = f64(x), f64(codes)
    top = np.abs(v).max(1, keepdims=True)
    d = 2 * np.abs(127 * v - c * top)
    assert np.all(d <= top)
    half = d == top
    assert half.any() or k < 1000
    assert np.all(c[half] % 2 == 0)


@pytest.mark.parametrize("k", [24, 1000, 5120, 16389])
def test_rows_of_zeros_and_of_what_is_no_number(q3, k):
    x = torch.randn(8, k, device="cuda")
    x[1] = 0
    x[2] = -0.0
    x[3, k - 1] = float("nan")
    x[4, 0] = float("inf")
    x[5, k // 2] = -float("inf")
    x[6] = float("nan")
    gain = torch.ones(k, device="cuda", dtype=torch.bfloat16)
    for f in (lambda s: q3.op_i8_quantize(x, status=s), lambda s: q3.op_i8_norm(x, gain, status=s),
              lambda s: q3.op_i8_norm(x, gain, delta=torch.zeros_like(x), status=s),
              lambda s: q3.op_i8_norm(x, gain, 0.0, status=s),
              lambda s: q3.op_i8_swiglu(torch.cat([torch.ones_like(x), x], 1), status=s)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        codes, scales = f(status)[:2]
        assert status.item() == 8
        bad = [3, 4, 5, 6]
        assert bool(torch.isnan(scales[bad]).all()) and not codes[bad].any()
        assert not codes[1:3].any() and not scales[1:3].any()
        assert bool((scales[[0, 7]] > 0).all()) and bool((codes[[0, 7]].abs().amax(1) == 127).all())


@pytest.mark.parametrize("size", [1e-42, 1e-38, 1e-33, 1e-25, 1e-18, 1e18, 1e25, 1e36])
@pytest.mark.parametrize("k", [100, 20000])
def test_values_near_the_ends_of_fp32(q3, k, size):
    """Squares, products with the gain or the reciprocal leave FP32's range; the outputs are its numbers."""
    x = (torch.randn(3, k, device="cuda").double() * size).float()
    gain = (1 + 0.3 * torch.randn(k, device="cuda")).bfloat16()
    gain[0] = 16.0
    values = torch.empty(3, k, device="cuda")
    codes, scales = q3.op_i8_quantize(x, values=values)
    if size > 1e-36:                                              # below, scales are rounded as subnormal numbers
        check(f64(x), codes, scales, values)
    for eps in (0.0, 1e-6):
        y = norm64(f64(x), f64(gain), eps)
        codes, scales, _ = q3.op_i8_norm(x, gain, eps)
        if np.abs(y).max() > 1e-34:
            check(y, codes, scales, None)
        else:
            assert np.all(np.abs(f64(codes) * f64(scales)[:, None] - y) <= np.abs(y).max(1, keepdims=True) / 127 + 1e-44)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [2047, 2560, 5120, 20000])
def test_rare_rows_among_others_and_in_place(q3, k, dtype):
    """Enough rows that a CTA takes several: some near the ends of FP32, of zeros or no numbers; the sum in x's place."""
    t = 1000
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn(t, k, generator=g, device="cuda")
    delta = torch.randn(t, k, generator=g, device="cuda")
    if dtype != "f16":
        for rows in (x, delta):
            rows[::3] *= 1e-25
            rows[1::7] *= 1e20
    x[5::11] = delta[5::11] = 0
    x[9::50, k - 1] = float("nan")
    x, delta = x.to(TYPES[dtype]), delta.to(TYPES[dtype])
    gain = (1 + 0.3 * torch.randn(k, generator=g, device="cuda")).bfloat16()
    codes, scales, total = q3.op_i8_norm(x, gain, delta=delta)
    assert torch.equal(total.nan_to_num(7.0), (x + delta).nan_to_num(7.0))
    good = ~torch.isnan(total).any(1)
    assert torch.equal(torch.isnan(scales), ~good)
    check(norm64(f64(total[good]), f64(gain), 1e-6), codes[good], scales[good], None)
    c, s = q3.op_i8_quantize(x)
    check(f64(x[good]), c[good], s[good], None)
    assert torch.equal(torch.isnan(s), ~good) and not c[~good].any()
    c, s, same = q3.op_i8_norm(x, gain, delta=delta, sum_out=x)
    assert same is x or same.data_ptr() == x.data_ptr()
    assert torch.equal(c, codes) and torch.equal(s.nan_to_num(7.0), scales.nan_to_num(7.0))
    assert torch.equal(x.nan_to_num(7.0), total.nan_to_num(7.0))


def test_swiglu_of_gates_far_out(q3):
    g = torch.tensor([[-1e4, -90.0, -88.0, -1.0, 0.0, 1.0, 88.0, 1e4]], device="cuda").repeat_interleave(5, 1)
    x = torch.cat([g, torch.full_like(g, 0.5)], 1)
    check(swiglu64(f64(x)), *q3.op_i8_swiglu(x), None)
    x = torch.cat([g[:, :10], torch.full_like(g[:, :10], 3e38)], 1)           # exp(-90) times a large number is one of FP32's
    check(swiglu64(f64(x)), *q3.op_i8_swiglu(x), None)


def test_massive_activations(q3):
    """A few channels a thousand times the others' size, as deep layers have them."""
    x = torch.randn(64, 2560, device="cuda")
    x[:, [7, 1111]] *= 1000
    check(f64(x.bfloat16()), *q3.op_i8_quantize(x.bfloat16()), None)
    gain = torch.full((2560,), 0.02, device="cuda").bfloat16()
    codes, scales, _ = q3.op_i8_norm(x, gain)
    check(norm64(f64(x), f64(gain), 1e-6), codes, scales, None)


def test_another_stream_and_a_captured_call(q3):
    x, d = torch.randn(17, 2560, device="cuda"), torch.randn(17, 2560, device="cuda").half()
    gain = torch.ones(2560, device="cuda", dtype=torch.bfloat16)
    want = q3.op_i8_norm(x, gain, delta=d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q3.op_i8_norm(x, gain, delta=d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q3.op_i8_norm(x, gain, delta=d)
        act = q3.op_i8_swiglu(got[2])
    x.mul_(2)
    graph.replay()
    want = q3.op_i8_norm(x, gain, delta=d)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(act, q3.op_i8_swiglu(want[2])))


def test_rows_beyond_2_31_elements(q3):
    x = torch.empty(300000, 8192, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 262143, 262144, 262145, 299999]
    x.zero_()
    x[at] = torch.randn(len(at), 8192, device="cuda").bfloat16()
    codes, scales = q3.op_i8_quantize(x)
    check(f64(x[at]), codes[at], scales[at], None)
    assert int((scales != 0).sum()) == len(at)
    codes, scales = q3.op_i8_swiglu(x, codes=codes[:, :4096], scales=scales)
    check(swiglu64(f64(x[at])), codes[at], scales[at], None)
