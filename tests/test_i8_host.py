"""Refusals of the 8-bit integer operators that need no GPU: the C entry points
check sizes, strides, types and alignment before any CUDA call, the binding
checks tensors' shapes, types and devices before the library."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3.lib()


P, ODD = 1 << 20, (1 << 20) + 4           # an aligned and a misaligned address (never read)


def _quantize(L, **kw):
    a = dict(x=P, type=0, stride=100, T=4, K=100, codes=P, code_stride=112, scales=P, values=None, values_type=0, status=None)
    a.update(kw)
    return L.q3_op_i8_quantize(*a.values(), None)


def _norm(L, **kw):
    a = dict(x=P, type=0, stride=100, delta=P, delta_type=1, delta_stride=100, sum=P, sum_stride=100, gain=P, eps=1e-6, T=4, K=100, codes=P,
             code_stride=112, scales=P, values=None, values_type=0, status=None)
    a.update(kw)
    return L.q3_op_i8_norm(*a.values(), None)


def _swiglu(L, **kw):
    a = dict(x=P, type=0, stride=200, T=4, K=100, codes=P, code_stride=112, scales=P, values=None, values_type=0, status=None)
    a.update(kw)
    return L.q3_op_i8_swiglu(*a.values(), None)


def _matmul(L, **kw):
    a = dict(x=P, x_stride=112, xs=P, w=P, w_stride=112, ws=P, T=4, M=7, K=100, out=P, out_type=1, out_stride=7, ws_dev=None, ws_bytes=0,
             status=None)
    a.update(kw)
    return L.q3_op_i8_matmul(*a.values(), None)


ROWS = [dict(x=None), dict(x=P + 2), dict(type=1, x=P + 1), dict(type=3), dict(type=-1), dict(stride=99), dict(T=-1), dict(T=(1 << 30) + 1), dict(K=0),
        dict(K=131072, stride=1 << 20, code_stride=1 << 20), dict(codes=None), dict(codes=ODD), dict(code_stride=96), dict(code_stride=108),
        dict(scales=None), dict(scales=P + 2), dict(values=P + 2), dict(values=P + 1, values_type=1), dict(values=P, values_type=3)]


@pytest.mark.parametrize("bad", ROWS, ids=str)
def test_quantize_refuses(L, bad):
    assert _quantize(L, **bad) == -1


@pytest.mark.parametrize("bad", ROWS + [
    dict(delta=P + 2, delta_type=0), dict(delta=P + 1), dict(delta_type=3), dict(delta_stride=99), dict(sum=None), dict(sum=P + 2),
    dict(sum_stride=99), dict(delta=None), dict(gain=None), dict(gain=P + 1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(sum=P, sum_stride=104)], ids=str)
def test_norm_refuses(L, bad):
    assert _norm(L, **bad) == -1


@pytest.mark.parametrize("bad", ROWS + [dict(stride=199)], ids=str)
def test_swiglu_refuses(L, bad):
    assert _swiglu(L, **bad) == -1


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=ODD), dict(x_stride=96), dict(x_stride=104), dict(xs=None), dict(xs=P + 2), dict(w=None), dict(w=ODD),
    dict(w_stride=96), dict(w_stride=104), dict(ws=None), dict(ws=P + 1), dict(T=-1), dict(T=(1 << 30) + 1), dict(M=0), dict(M=(1 << 30) + 1, out_stride=1 << 31), dict(K=0),
    dict(K=131072, x_stride=1 << 20, w_stride=1 << 20), dict(out=None), dict(out=P + 1), dict(out=P + 2, out_type=0), dict(out_type=3),
    dict(out_stride=6)], ids=str)
def test_matmul_refuses(L, bad):
    assert _matmul(L, **bad) == -1
    assert L.q3_last_error()


def test_matmul_workspace(L):
    import qwen3_dense_decoder_gb300 as q3
    assert [q3.i8_matmul_workspace(t, 7, 100) for t in (0, 1, 8, 9, 64)] == [0] * 5
    need = q3.i8_matmul_workspace(4096, 4096, 1000)
    assert need >= 4096 * 1000 * 2
    big = dict(T=4096, M=4096, K=1000, x_stride=1008, w_stride=1008, out_stride=4096)
    for bad in (dict(), dict(ws_dev=P, ws_bytes=need - 1), dict(ws_dev=P + 16, ws_bytes=need)):
        assert _matmul(L, **big, **bad) == -1
    for bad in ((-1, 7, 100), (9, 0, 100), (9, 7, 0), (9, 7, 131072)):
        with pytest.raises(q3.Q3Error):
            q3.i8_matmul_workspace(*bad)


def test_nothing_to_do_is_no_error(L):
    # zero rows need no GPU
    assert _quantize(L, T=0) == 0 and _norm(L, T=0) == 0 and _swiglu(L, T=0) == 0 and _matmul(L, T=0) == 0


def test_binding_refuses_before_the_library():
    import qwen3_dense_decoder_gb300 as q3
    x = torch.zeros(3, 100)
    gain = torch.ones(100, dtype=torch.bfloat16)
    codes = torch.zeros(3, 112, dtype=torch.int8)[:, :100]
    w = torch.zeros(7, 112, dtype=torch.int8)[:, :100]
    s3, s7 = torch.zeros(3), torch.zeros(7)
    status = torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: q3.op_i8_quantize(x.double()),
        lambda: q3.op_i8_quantize(x[0]),
        lambda: q3.op_i8_quantize(x.t()),
        lambda: q3.op_i8_quantize(x[:, :0]),
        lambda: q3.op_i8_quantize([1.0]),
        lambda: q3.op_i8_quantize(x, codes=codes.float()),
        lambda: q3.op_i8_quantize(x, codes=codes[:2]),
        lambda: q3.op_i8_quantize(x, codes=torch.zeros(3, 100, dtype=torch.int8)),                   # rows 100 bytes apart
        lambda: q3.op_i8_quantize(x, codes=torch.zeros(3, 128, dtype=torch.int8)[:, 4:104]),         # begins in between
        lambda: q3.op_i8_quantize(x, scales=s7),
        lambda: q3.op_i8_quantize(x, scales=s3.half()),
        lambda: q3.op_i8_quantize(x, values=x.double()),
        lambda: q3.op_i8_quantize(x, values=torch.zeros(3, 101)[:, :100]),
        lambda: q3.op_i8_quantize(x, status=status),
        lambda: q3.op_i8_quantize(x),                                                                # CPU tensors
        lambda: q3.op_i8_swiglu(x[:, :99]),
        lambda: q3.op_i8_swiglu(x, codes=codes),                                                     # 50 wide
        lambda: q3.op_i8_swiglu(x),
        lambda: q3.op_i8_norm(x, gain.float()),
        lambda: q3.op_i8_norm(x, gain[:99]),
        lambda: q3.op_i8_norm(x, gain, delta=x[:2]),
        lambda: q3.op_i8_norm(x, gain, delta=x.double()),
        lambda: q3.op_i8_norm(x, gain, sum_out=x),                                                   # nothing is added
        lambda: q3.op_i8_norm(x, gain, delta=x, sum_out=x.half()),
        lambda: q3.op_i8_norm(x, gain, delta=x),                                                     # CPU tensors
        lambda: q3.op_i8_matmul(codes.to(torch.uint8), s3, w, s7),
        lambda: q3.op_i8_matmul(codes, s7, w, s7),
        lambda: q3.op_i8_matmul(codes, s3, w[:, :96], s7),
        lambda: q3.op_i8_matmul(codes, s3, w.contiguous(), s7),                                      # rows 100 bytes apart
        lambda: q3.op_i8_matmul(codes, s3, w, s3),
        lambda: q3.op_i8_matmul(codes, s3, w, s7, dtype=torch.float64),
        lambda: q3.op_i8_matmul(codes, s3, w, s7, dtype=16),
        lambda: q3.op_i8_matmul(codes, s3, w, s7, out=torch.zeros(7, 3)),
        lambda: q3.op_i8_matmul(codes, s3, w, s7, out=torch.zeros(3, 7), dtype=torch.float16),
        lambda: q3.op_i8_matmul(codes, s3, w, s7),                                                   # CPU tensors
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")


def test_no_rows_give_empty_outputs():
    import qwen3_dense_decoder_gb300 as q3
    none = torch.zeros(0, 40)
    codes, scales = q3.op_i8_quantize(none)
    assert codes.shape == (0, 40) and codes.dtype == torch.int8 and scales.shape == (0,)
    codes, scales, total = q3.op_i8_norm(none, torch.ones(40, dtype=torch.bfloat16), delta=none.half())
    assert codes.shape == (0, 40) and total.shape == (0, 40) and total.dtype == torch.float32
    assert q3.op_i8_swiglu(none)[0].shape == (0, 20)
    out = q3.op_i8_matmul(codes, scales, torch.zeros(5, 48, dtype=torch.int8)[:, :40], torch.zeros(5), dtype=torch.bfloat16)
    assert out.shape == (0, 5) and out.dtype == torch.bfloat16
