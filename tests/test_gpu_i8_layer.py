"""Decoder layers run from the operators alone: norms, projections and SwiGLU in
8-bit integers around the 4-bit cache's append and attention, as a program that
owns its layers calls them.

Every operator's output is checked against 64 bits on the very inputs that it got
(the bounds are those of the operators' own tests): products equal bit for bit,
codes lie within 0.5 + 2^-13 of y / scale.  A row's way through the projections does
not depend on the rows beside it, so the first layer's cache holds the same bytes
whether its rows come as one prompt or one by one.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
HIDDEN, N_Q, N_KV, D, FFN, EPS = 1024, 16, 8, 128, 2816, 1e-6


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def near_codes(codes, scales, y):
    c, s, y = (t.double().cpu().numpy() for t in (codes, scales, y))
    want = np.abs(y).max(1) / 127
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want)
    assert np.all(np.abs(c - y / np.where(want > 0, want, 1)[:, None]) <= 0.5 + 2.0 ** -13)


def product(x, xs, w, ws, dtype):
    return (torch.matmul(x.double(), w.double().t()).float() * xs.unsqueeze(1) * ws).to(dtype)


class Layers:
    def __init__(self, q3, n, n_blocks, max_blocks, seed):
        self.q3 = q3
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        gain = lambda k: (1 + 0.05 * rand(k)).bfloat16()  # noqa: E731
        self.layers = []
        for _ in range(n):
            w = {name: q3.op_i8_quantize(rand(o, i).mul_(0.02).bfloat16())
                 for name, o, i in (("qkv", (N_Q + 2 * N_KV) * D, HIDDEN), ("o", HIDDEN, N_Q * D), ("gate_up", 2 * FFN, HIDDEN), ("down", HIDDEN, FFN))}
            w |= {"attn_norm": gain(HIDDEN), "ffn_norm": gain(HIDDEN), "q_norm": gain(D), "k_norm": gain(D)}
            self.layers.append(w)
        self.kv = torch.zeros(n, n_blocks, 2, N_KV, q3.KV4_TILE, dtype=torch.uint8, device="cuda")
        self.tables = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)[:max_blocks].view(1, -1).contiguous()
        self.rope = q3.rope_table(32 * max_blocks, 1e6)
        self.final = gain(HIDDEN)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, x, pos, slot, prompt, seen=None):
        """x: f32 [T, HIDDEN], replaced by the layers' stream; returns (codes, scales) of the final norm."""
        q3, st = self.q3, self.status
        note = seen.append if seen is not None else lambda _: None
        delta = None
        for li, w in enumerate(self.layers):
            before = x.clone() if seen is not None else None
            c, s, _ = q3.op_i8_norm(x, w["attn_norm"], EPS, delta=delta, sum_out=x if delta is not None else None, status=st)
            note(("norm", before, delta, w["attn_norm"], x.clone(), c, s))
            qkv = q3.op_i8_matmul(c, s, *w["qkv"], status=st)
            note(("matmul", c, s, *w["qkv"], qkv))
            q = q3.op_kv4_append(qkv, w["q_norm"], w["k_norm"], self.rope, pos, slot, self.tables, self.kv[li], N_Q, EPS, status=st)
            if prompt is None:
                att = q3.op_kv4_decode_attention(q, pos, slot, self.tables, self.kv[li], status=st)
            else:
                att = q3.op_kv4_prefill_attention(q, *prompt, self.tables, self.kv[li], status=st)
            c, s = q3.op_i8_quantize(att.view(att.shape[0], -1), status=st)
            note(("quantize", att.view(att.shape[0], -1), c, s))
            delta = q3.op_i8_matmul(c, s, *w["o"], status=st)
            note(("matmul", c, s, *w["o"], delta))
            before = x.clone() if seen is not None else None
            c, s, _ = q3.op_i8_norm(x, w["ffn_norm"], EPS, delta=delta, sum_out=x, status=st)
            note(("norm", before, delta, w["ffn_norm"], x.clone(), c, s))
            gu = q3.op_i8_matmul(c, s, *w["gate_up"], status=st)
            note(("matmul", c, s, *w["gate_up"], gu))
            c, s = q3.op_i8_swiglu(gu, status=st)
            note(("swiglu", gu, c, s))
            delta = q3.op_i8_matmul(c, s, *w["down"], dtype=torch.bfloat16, status=st)
            note(("matmul", c, s, *w["down"], delta))
        return q3.op_i8_norm(x, self.final, EPS, delta=delta, sum_out=x, status=st)[:2]


def check(seen):
    for what, *t in seen:
        if what == "matmul":
            c, s, w, ws, out = t
            assert torch.equal(out, product(c, s, w, ws, out.dtype))
        elif what == "norm":
            x, delta, gain, total, c, s = t
            assert torch.equal(total, x if delta is None else (x + delta.float()))
            y = total.double()
            near_codes(c, s, y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * gain.double())
        elif what == "quantize":
            near_codes(t[1], t[2], t[0])
        else:
            g, u = t[0].double().chunk(2, 1)
            near_codes(t[1], t[2], g * torch.sigmoid(g) * u)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(first, n):
    return torch.arange(first, first + n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n", [9, 40, 300])
def test_prompt_then_single_tokens(q3, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n + 4, HIDDEN, generator=g, device="cuda")
    blocks = (n + 4 + 31) // 32
    whole, parts = (Layers(q3, 2, blocks + 3, blocks, 7) for _ in range(2))
    seen = []
    whole.step(x.clone(), *rows(0, n + 4), (ints(0, n + 4), ints(0)), seen)
    check(seen)
    seen = []
    parts.step(x[:n].clone(), *rows(0, n), (ints(0, n), ints(0)), seen)
    for i in range(n, n + 4):
        parts.step(x[i: i + 1].clone(), *rows(i, 1), None, seen)
    check(seen)
    q3.check_status(whole.status)
    q3.check_status(parts.status)
    assert torch.equal(whole.kv[0], parts.kv[0])


def test_a_captured_step_and_a_padded_batch(q3):
    """A decode step of 12 rows, three of them padding (negative positions, zero rows), replayed over new inputs."""
    m = Layers(q3, 2, 40, 8, 11)
    m.tables = torch.randperm(40, device="cuda").to(torch.int32)[:36].view(12, 3).contiguous()
    n = 12
    pos, slot = ints(*range(n)), ints(*range(n))
    pos[[2, 5, 11]] = -1
    x = torch.randn(n, HIDDEN, device="cuda")
    x[[2, 5, 11]] = 0
    first = x.clone()
    eager = m.step(x, pos, slot, None)
    kv = m.kv.clone()
    m.kv.zero_()
    x.copy_(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        m.step(x.clone(), pos, slot, None)                         # the kernels are loaded
    torch.cuda.current_stream().wait_stream(side)
    m.kv.zero_()
    buf = first.clone()
    with torch.cuda.graph(graph):
        x.copy_(buf)
        got = m.step(x, pos, slot, None)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, eager)) and torch.equal(m.kv, kv)
    assert not got[0][[2, 5, 11]].any() and not got[1][[2, 5, 11]].any()
    buf.copy_(torch.randn(n, HIDDEN, device="cuda"))
    buf[[2, 5, 11]] = 0
    m.kv.zero_()
    graph.replay()
    replayed = [t.clone() for t in got]
    m.kv.zero_()
    assert all(torch.equal(a, b) for a, b in zip(replayed, m.step(buf.clone(), pos, slot, None)))
    q3.check_status(m.status)
