"""The product of 8-bit integer rows.  The sum over k is a whole number below
2^31 and has to be that number; what follows are three roundings of FP32 and one
to the output's type, done here by the same operations: results are equal bit
for bit.  64-bit floating point holds every sum exactly."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def rows(n, k, seed, gap=0, lo=-127, hi=127):
    """Codes whose rows begin on 16-byte boundaries, `gap` 16-byte pieces further apart than they need; junk between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, (n, (k + 15) // 16 * 16 + 16 * gap), generator=g, device="cuda", dtype=torch.int8)[:, :k]


def scales(n, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(n, generator=g, device="cuda") + 0.5) * size


def reference(x, xs, w, ws, dtype):
    acc = torch.matmul(x.double(), w.double().t()).to(torch.int64)
    return (acc.float() * xs.unsqueeze(1) * ws).to(dtype)


def check(q3, x, w, dtype, seed=1, **kw):
    # results of ordinary size: sums of K products reach 128^2 K
    xs, ws = scales(x.shape[0], seed, 2.0 ** -7), scales(w.shape[0], seed + 1, 2.0 ** -9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = q3.op_i8_matmul(x, xs, w, ws, dtype=dtype, status=status, **kw)
    q3.check_status(status)
    want = reference(x, xs, w, ws, dtype)
    assert got.dtype == dtype and got.shape == want.shape
    assert torch.equal(got, want), (got.float() - want.float()).abs().max().item()


SIZES = [(1, 1, 1), (1, 16, 16), (2, 3, 5), (8, 17, 15), (9, 17, 17), (1, 257, 63), (3, 128, 64), (16, 129, 65), (15, 1000, 1111), (5, 5003, 130),
         (17, 128, 128), (31, 640, 127), (32, 2560, 2560), (33, 300, 4099), (61, 1003, 1040), (64, 4096, 1024), (65, 128, 2049), (100, 6144, 256),
         (127, 200, 9728), (128, 1024, 1025), (129, 1000, 3000), (200, 4099, 511), (255, 256, 700), (256, 2560, 1024), (257, 33, 5000),
         (511, 777, 1234), (701, 2560, 4096), (1024, 1024, 2048), (2048, 2560, 128), (2049, 515, 1100), (1, 19456, 2560), (7, 5120, 17408)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,m,k", SIZES)
def test_matmul(q3, t, m, k, dtype):
    check(q3, rows(t, k, t + k), rows(m, k, m), TYPES[dtype])


@pytest.mark.parametrize("k", [1024, 1040, 1041, 2049, 131071])
@pytest.mark.parametrize("t", [1, 8, 12, 40, 130, 300])
@pytest.mark.parametrize("lo,hi", [(127, 127), (-128, -128), (-127, -126), (-128, 127)])
def test_largest_codes(q3, t, k, lo, hi):
    """Every partial sum at the largest it can be: whole numbers throughout."""
    x, w = rows(t, k, 1, lo=lo, hi=hi), rows(150, k, 2, lo=lo, hi=hi)
    check(q3, x, w, torch.float32)
    check(q3, x, -w.clamp(-127, 127)[:, :k] if k % 16 == 0 else w, torch.bfloat16)


@pytest.mark.parametrize("t", [1, 5, 9, 24, 70, 140, 400])
def test_strides_and_what_lies_between(q3, t):
    x, w = rows(t, 333, 3, gap=2), rows(259, 333, 4, gap=1)
    xs, ws = scales(t, 5, 2.0 ** -7), scales(259, 6, 2.0 ** -9)
    for dtype in TYPES.values():
        wide = torch.full((t + 2, 300), 3.0, dtype=dtype, device="cuda")
        got = q3.op_i8_matmul(x, xs, w, ws, out=wide[1: t + 1, 7: 266])
        assert got.data_ptr() == wide[1, 7:].data_ptr()
        assert torch.equal(got, reference(x, xs, w, ws, dtype))
        wide[1: t + 1, 7: 266] = 3.0
        assert bool((wide == 3.0).all())


@pytest.mark.parametrize("m,k", [(2560, 4096), (5003, 1111), (19456, 2560)])
def test_a_row_does_not_depend_on_its_neighbours(q3, m, k):
    x, w = rows(300, k, 7), rows(m, k, 8)
    xs, ws = scales(300, 9, 2.0 ** -7), scales(m, 10, 2.0 ** -9)
    whole = q3.op_i8_matmul(x, xs, w, ws, dtype=torch.float32)
    for n in (1, 2, 7, 8, 9, 16, 31, 33, 64, 65, 128, 129, 200, 256):
        assert torch.equal(q3.op_i8_matmul(x[:n], xs[:n], w, ws, dtype=torch.float32), whole[:n]), n


@pytest.mark.parametrize("t", [1, 3, 20, 90, 300])
def test_scales_that_are_no_numbers_stay_in_their_row(q3, t):
    x, w = rows(t, 200, 11), rows(100, 200, 12)
    xs, ws = scales(t, 13), scales(100, 14)
    xs[t // 2], ws[5] = float("nan"), float("inf")
    x[t // 2] = 0                                                 # as the quantisers leave such a row
    got = q3.op_i8_matmul(x, xs, w, ws, dtype=torch.float32)
    assert bool(torch.isnan(got[t // 2]).all())
    keep = [i for i in range(t) if i != t // 2]
    cols = [i for i in range(100) if i != 5]
    want = reference(x, xs, w, ws, torch.float32)
    assert torch.equal(got[keep][:, cols], want[keep][:, cols])
    xs[t // 2] = 0.0
    assert not q3.op_i8_matmul(x, xs, w, scales(100, 14), dtype=torch.float16)[t // 2].any()


@pytest.mark.parametrize("t", [1, 3, 20, 90, 300])
def test_fp16_results_beyond_its_range_are_reported(q3, t):
    x, w = rows(t, 160, 15, lo=100, hi=127), rows(130, 160, 16, lo=100, hi=127)
    one = torch.ones(t, device="cuda"), torch.ones(130, device="cuda")
    for dtype, bit in ((torch.float16, 8), (torch.bfloat16, 0), (torch.float32, 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = q3.op_i8_matmul(x, one[0], w, one[1], dtype=dtype, status=status)
        assert status.item() == bit
        assert torch.equal(got, reference(x, *one[:1], w, one[1], dtype))


def test_out_decides_the_type(q3):
    x, w = rows(3, 64, 1), rows(20, 64, 2)
    xs, ws = scales(3, 1), scales(20, 2, 2.0 ** -9)
    assert q3.op_i8_matmul(x, xs, w, ws).dtype == torch.float16
    out = torch.empty(3, 20, device="cuda")
    assert q3.op_i8_matmul(x, xs, w, ws, out=out) is not None and torch.equal(out, reference(x, xs, w, ws, torch.float32))


@pytest.mark.parametrize("t", [1, 20, 90, 300])
def test_another_stream_a_captured_call_and_two_at_once(q3, t):
    x, w = rows(t, 2049, 17), rows(1500, 2049, 18)
    xs, ws = scales(t, 19, 2.0 ** -7), scales(1500, 20, 2.0 ** -9)
    want = reference(x, xs, w, ws, torch.bfloat16)
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):                                            # on two streams at once
        got.append(q3.op_i8_matmul(x, xs, w, ws, dtype=torch.bfloat16, stream=sides[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q3.op_i8_matmul(x, xs, w, ws, dtype=torch.bfloat16)
    x.copy_(rows(t, 2049, 21))
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, reference(x, xs, w, ws, torch.bfloat16))


def test_calls_in_a_row_that_feed_one_another(q3):
    """Writers and products launched behind one another with nothing between: each sees the one before."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(1024, 1024, generator=g, device="cuda").half()
    wc, ws = q3.op_i8_quantize(w)
    for t in (1, 6, 30, 100, 300):
        x = torch.randn(t, 1024, generator=g, device="cuda").half()
        want = x
        for _ in range(5):
            c, s = q3.op_i8_quantize(want)
            torch.cuda.synchronize()
            want = q3.op_i8_matmul(c, s, wc, ws) * 0.03125
            torch.cuda.synchronize()
        got = x
        for _ in range(5):
            got = q3.op_i8_matmul(*q3.op_i8_quantize(got), wc, ws) * 0.03125
        assert torch.equal(got, want), t


@pytest.mark.parametrize("k", [1024, 2048, 2049, 32768, 33 * 1024 + 5, 131071])
@pytest.mark.parametrize("size", [1, 8, 33, 127])
def test_sums_of_tokens_of_different_sizes(q3, k, size):
    """Long sums where the codes are small, short ones where some tokens' are not; the weights all of one sign and largest."""
    x = rows(400, k, size, lo=-size, hi=size)
    x[7] = 127
    x[199, : k // 2] = -128
    x[200:210, k // 3:] = 127
    w = rows(260, k, 5, lo=100, hi=127)
    w[::2] = -128
    check(q3, x, w, torch.float32)


def test_sums_at_the_largest_that_fp32_holds(q3):
    """sum |x| of 1,024 inputs at 2^17 / n: n chunks in one sum reach 2^24 exactly, one more code would pass it."""
    for n in (1, 2, 4, 32, 33, 64):
        k = 70 * 1024
        x = torch.zeros(300, k, dtype=torch.int8, device="cuda")
        full = 131072 // n // 128                                # codes of -128 in each 1,024
        x.view(300, 70, 1024)[:, :, :full] = -128
        x[::3].view(100, 70, 1024)[:, ::2, 1023] = 1
        w = torch.full((260, k), -128, dtype=torch.int8, device="cuda")
        w[1::2] = 127
        check(q3, x, w, torch.float32)


def test_outputs_and_codes_beyond_2_31_elements(q3):
    t, m, k = 70000, 32768, 64
    x, w = rows(t, k, 1), rows(m, k, 2)
    xs, ws = scales(t, 3, 2.0 ** -7), scales(m, 4, 2.0 ** -9)
    out = q3.op_i8_matmul(x, xs, w, ws, dtype=torch.bfloat16)
    at = torch.tensor([0, 1, 191, 192, 65535, 65536, 69900, t - 1], device="cuda")
    assert torch.equal(out[at], reference(x[at], xs[at], w, ws, torch.bfloat16))
    del out
    # the channels' rows lie beyond 2^31 bytes
    wide = torch.empty(m * 8, 16384, dtype=torch.int8, device="cuda")[:, :k]
    wide[-300:] = w[:300]
    wide[:300] = w[300:600]
    for n in (9, 40, 300):
        x, xs = rows(n, k, 6), scales(n, 7, 2.0 ** -7)
        big = scales(m * 8, 8, 2.0 ** -9)
        got = q3.op_i8_matmul(x, xs, wide, big, dtype=torch.float32)
        assert torch.equal(got[:, -300:], reference(x, xs, w[:300], big[-300:], torch.float32))
        assert torch.equal(got[:, :300], reference(x, xs, w[300:600], big[:300], torch.float32))


@pytest.mark.parametrize("t", [1, 40, 300])
def test_the_first_call_of_a_process_may_be_captured(t):
    import os
    import subprocess
    import sys
    code = f"""
import torch, qwen3_dense_decoder_gb300 as q3
x = torch.randn({t}, 512, device="cuda").half(); w = torch.randint(-127, 128, (700, 512), device="cuda", dtype=torch.int8)
ws = torch.rand(700, device="cuda"); g = torch.ones(512, device="cuda").bfloat16()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    c, s, _ = q3.op_i8_norm(x, g)
    y = q3.op_i8_matmul(c, s, w, ws, dtype=torch.float32)
    z = q3.op_i8_swiglu(y)
graph.replay()
torch.cuda.synchronize()
want = (c.double() @ w.double().T).float() * s.unsqueeze(1) * ws
assert torch.equal(y, want) and z[0].abs().amax() == 127
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
