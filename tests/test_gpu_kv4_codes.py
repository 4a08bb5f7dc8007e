"""Every code that the 4-bit append writes.

V comes straight from the input: its record equals the oracle packer's bit for
bit, also where quotients lie on a half or next to one.  K passes the FP32
norm and rotation: its quotient (y - bias) / scale, with the stored scale and
bias, carries the row's error, 2^-19 of its largest value (under 32 roundings
of 2^-24), over the scale, and a rounding each of the difference and the quotient (2^-20 below 16);
further than that from a half, the code is the quotient's nearest whole
number."""
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


def append(q3, x, n_q, n_kv, gains, rope, dtype=torch.float32):
    """Rows x [T, heads, 128] at positions 0 .. T of one slot in block order: the pool."""
    T = len(x)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    blocks = (T + 31) // 32
    kv = torch.zeros(blocks, 2, n_kv, ref.TILE, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv = torch.from_numpy(np.ascontiguousarray(x.reshape(T, -1))).cuda().to(dtype)
    q3.op_kv4_append(qkv, *gains, rope, i32(np.arange(T)), i32(np.zeros(T)), i32(np.arange(blocks)).view(1, -1), kv, n_q, status=status)
    q3.check_status(status)
    return kv.cpu().numpy(), qkv.float().cpu().numpy().reshape(x.shape)


def places(part, T):
    """A part [blocks, n_kv, 32, m] as rows [T, n_kv, m]."""
    return part.transpose(0, 2, 1, 3).reshape(-1, part.shape[1], part.shape[3])[:T]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_k_codes_away_from_borders_are_exact(q3, dtype):
    r = np.random.default_rng(17)
    T, n_q, n_kv = 2000, 1, 1
    x = r.normal(0, 1.5, (T, n_q + 2 * n_kv, D)).astype(np.float32)
    gains = [torch.from_numpy((1 + 0.2 * r.normal(size=D)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]
    rope = q3.rope_table(T, 1e6)
    kv, x = append(q3, x, n_q, n_kv, gains, rope, dtype)
    k = x[:, n_q:n_q + n_kv].astype(np.float64)
    cs = rope.cpu().numpy().astype(np.float64)
    y = k / np.sqrt((k * k).mean(-1, keepdims=True) + 1e-6) * gains[1].float().cpu().numpy().astype(np.float64)
    a, b = y[..., :64], y[..., 64:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    codes, scale, bias = (places(p, T) for p in ref.read_tiles(kv)["k"])
    quot = (y - np.repeat(bias, 32, -1)) / np.repeat(scale, 32, -1)
    band = 2.0 ** -19 * np.abs(y).max(-1, keepdims=True) / np.repeat(scale, 32, -1) + 2.0 ** -19
    want = np.clip(np.rint(quot), 0, 15)
    clear = np.abs(quot - np.floor(quot) - 0.5) > band
    assert clear.mean() > 0.999
    np.testing.assert_array_equal(codes[clear], want[clear])
    assert np.abs(codes - want).max() <= 1
    # the parameters: fp16 of the row's least value and of its range over 15, or the next number where the row's error decides
    g = y.reshape(T, n_kv, 4, 32)
    for got, exact in ((bias, g.min(-1)), (scale, (g.max(-1) - g.min(-1)) / 15)):
        off = 2.0 ** -11 * np.abs(exact) + 2.0 ** -25 + 2.0 ** -18 * np.abs(y).max(-1, keepdims=True)
        assert np.all(np.abs(got - exact) <= off)


def test_v_codes_on_and_next_to_halves(q3, orc):
    """Groups from 0 to 15 s with values s (c + 1/2) and their neighbours up to three ulps, for scales of any fp16 bits; and the
    same above a bias."""
    r = np.random.default_rng(18)
    T, n_kv = 4096, 1
    s = (2.0 ** r.uniform(-13, 9, (T, 4))).astype(np.float16).astype(np.float32)
    c = r.integers(0, 15, (T, 4, 32)).astype(np.float32)
    v = s[..., None] * (c + np.float32(0.5))
    for step in range(3):
        more = r.integers(-1, 2, v.shape)
        v = np.where(more > 0, np.nextafter(v, np.float32(np.inf)), np.where(more < 0, np.nextafter(v, np.float32(-np.inf)), v)).astype(np.float32)
    v[..., 0], v[..., 31] = 0.0, s * np.float32(15)
    lift = np.where(r.random((T, 4)) < 0.5, 0, s * r.integers(-40, 40, (T, 4))).astype(np.float16).astype(np.float32)
    v = (v + lift[..., None]).astype(np.float32).reshape(T, 1, D)
    x = np.concatenate([r.normal(size=(T, 2, D)).astype(np.float32), v], 1)
    gains = [torch.ones(D, dtype=torch.bfloat16, device="cuda")] * 2
    kv, _ = append(q3, x, 1, n_kv, gains, q3.rope_table(T, 1e6))
    codes, scale, bias = (places(p, T) for p in ref.read_tiles(kv)["v"])
    rec = orc.affine4_pack(v.reshape(T, D)).reshape(T, 1, 4, 20)
    oc = np.stack([rec[..., :16] & 15, rec[..., :16] >> 4], -1).reshape(T, 1, D)
    osb = np.ascontiguousarray(rec[..., 16:]).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(scale, osb[..., 0])
    np.testing.assert_array_equal(bias, osb[..., 1])
    np.testing.assert_array_equal(codes, oc)
