"""The operators of a decoder layer in 8-bit integers: the sizes they are used
at, their inputs, their plain form in elementary torch operations and, where
`own` is set, the library's calls.

A row of values y is held as whole-number codes in [-127, 127] and one f32
scale: scale = max |y| / 127, code = round-half-even(y / scale); a row of zeros
has scale 0 and zero codes.  Activations have a scale for each token, weights
one for each output channel, and the product of two such matrices is a sum of
whole numbers times both scales.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
# (outputs, inputs) of a layer's projections: 0.6B, 4B, 8B and 14B shapes
PROJECTIONS = ((4096, 1024), (1024, 2048), (6144, 2560), (2560, 4096), (19456, 2560), (2560, 9728), (6144, 4096),
               (24576, 4096), (4096, 12288), (7168, 5120), (5120, 5120), (34816, 5120), (5120, 17408))
MOST = 2048 * 19456 * 2560             # products of the largest listed case


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one session's decode step (latency): the 4B gate and up projections
        {"name": "matmul_1_gateup4b", "op": "matmul", "rows": 1, "outs": 19456, "ins": 2560, "type": "f16"},
        # seven sessions' decode step: the 14B down projection
        {"name": "matmul_7_down14b", "op": "matmul", "rows": 7, "outs": 5120, "ins": 17408, "type": "bf16"},
        # a decode round of 32 sessions: the 4B output projection
        {"name": "matmul_32_o4b", "op": "matmul", "rows": 32, "outs": 2560, "ins": 4096, "type": "f16"},
        # a ragged round of 201 rows into a residual stream in f32, sizes that are no multiple of a tile
        {"name": "matmul_201_odd", "op": "matmul", "rows": 201, "outs": 5003, "ins": 4099, "type": "f32"},
        # a 2,048-token prompt: the 4B gate and up projections
        {"name": "matmul_2048_gateup4b", "op": "matmul", "rows": 2048, "outs": 19456, "ins": 2560, "type": "f16"},
        # one session's decode step (latency): the residual's addition and the norm before a projection
        {"name": "norm_1x2560", "op": "norm", "rows": 1, "ins": 2560, "type": "f32", "delta": "f16", "gap": 0},
        # a 2,048-token prompt, 14B width
        {"name": "norm_2048x5120", "op": "norm", "rows": 2048, "ins": 5120, "type": "bf16", "delta": "bf16", "gap": 0},
        # the first layer of a ragged round (nothing to add), an odd width, rows of a wider buffer
        {"name": "norm_701x2047", "op": "norm", "rows": 701, "ins": 2047, "type": "f16", "delta": "", "gap": 33},
        # a decode round of 32 sessions, 4B feed-forward width
        {"name": "swiglu_32x9728", "op": "swiglu", "rows": 32, "ins": 9728, "type": "f16", "gap": 0},
        # a 2,048-token prompt, 4B feed-forward width
        {"name": "swiglu_2048x9728", "op": "swiglu", "rows": 2048, "ins": 9728, "type": "f16", "gap": 0},
        # attention's outputs of 40 rows before the output projection, 8B heads
        {"name": "quantize_40x4096", "op": "quantize", "rows": 40, "ins": 4096, "type": "f16", "gap": 0},
        # a weight matrix by channel as it is loaded: the 14B gate and up projections
        {"name": "quantize_34816x5120", "op": "quantize", "rows": 34816, "ins": 5120, "type": "bf16", "gap": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("matmul", "matmul", "norm", "swiglu", "quantize"))
    if op == "matmul":
        outs, ins = rng.choice(PROJECTIONS)
        if rng.random() < 0.5:
            outs, ins = _log(rng, 64, 40000), _log(rng, 16, 20000)
        rows = _log(rng, 1, 2048)
        return {"op": op, "rows": max(1, min(rows, MOST // (outs * ins))), "outs": outs, "ins": ins,
                "type": rng.choice(("f32", "f16", "bf16"))}
    ins = rng.choice((1024, 2560, 4096, 5120, 9728, 17408, _log(rng, 16, 20000), _log(rng, 16, 20000)))
    if op == "quantize":
        rows = _log(rng, 1, min(34816, 34816 * 5120 // ins))
        return {"op": op, "rows": rows, "ins": ins, "type": rng.choice(("f32", "f16", "bf16")), "gap": rng.choice((0, 0, 64, 3))}
    rows = _log(rng, 1, 2048)
    if op == "swiglu":
        return {"op": op, "rows": rows, "ins": ins, "type": rng.choice(("f32", "f16", "bf16")), "gap": rng.choice((0, 0, 64, 3))}
    return {"op": op, "rows": rows, "ins": ins, "type": rng.choice(("f32", "f16", "bf16")),
            "delta": rng.choice(("f32", "f16", "bf16", "")), "gap": rng.choice((0, 0, 64, 3))}


def work(case):
    t, k, size = case["rows"], case["ins"], SIZE[case["type"]]
    if case["op"] == "matmul":
        m = case["outs"]
        return {"bytes": t * k + m * k + 4 * (t + m) + t * m * size, "flops": 2 * t * m * k}
    made = t * k * 3 + 4 * t                                     # codes, the values they stand for, scales
    if case["op"] == "norm":
        added = (SIZE[case["delta"]] + size) if case["delta"] else 0
        return {"bytes": t * k * (size + added) + 2 * k + made, "flops": 8 * t * k}
    if case["op"] == "swiglu":
        return {"bytes": 2 * t * k * size + made, "flops": 10 * t * k}
    return {"bytes": t * k * size + made, "flops": 4 * t * k}


# ---------------------------------------------------------------- inputs

def _codes(y):
    """f32 [T, K] -> whole-number codes f32 [T, K], scales f32 [T]."""
    scale = y.abs().amax(1) / 127.0
    s = scale.unsqueeze(1)
    return torch.round(y / torch.where(s > 0, s, 1.0)).clamp(-127, 127), scale


def _padded(codes):
    """int8 codes in rows that begin on 16-byte boundaries, as the quantisers lay them out."""
    t, k = codes.shape
    out = torch.empty(t, (k + 15) // 16 * 16, dtype=torch.int8, device=codes.device)[:, :k]
    out.copy_(codes)
    return out


def _rows(gen, t, k, kind, gap, spread=6.0):
    """Rows with a few channels several times the others' size, as a decoder's activations have them."""
    buf = torch.randn(t, k + gap, generator=gen, device="cuda")
    hot = torch.randint(0, k, (max(1, k // 512),), generator=gen, device="cuda")
    buf[:, hot] *= spread
    return buf.to(TYPES[kind])[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 11 + 5)
    op, t, k = case["op"], case["rows"], case["ins"]
    st = {"op": op, "type": TYPES[case["type"]]}
    if op == "matmul":
        x, xs = _codes(_rows(gen, t, k, "f32", 0))
        w, ws = _codes(torch.randn(case["outs"], k, generator=gen, device="cuda") * 0.02)
        return {**st, "x": _padded(x), "xs": xs, "w": _padded(w), "ws": ws}
    if op == "swiglu":
        st["x"] = _rows(gen, t, 2 * k, case["type"], case["gap"], 1.0)
        return st
    st["x"] = _rows(gen, t, k, case["type"], case["gap"])
    if op == "norm":
        st["gain"] = (1 + 0.1 * torch.randn(k, generator=gen, device="cuda")).bfloat16()
        st["delta"] = _rows(gen, t, k, case["delta"], 0, 2.0) if case["delta"] else None
    return st


# ---------------------------------------------------------------- the plain forms

def _held(y):
    """The values that y's rows are held as, and the rows' scales."""
    codes, scale = _codes(y)
    return (codes * scale.unsqueeze(1)).half(), scale


def _matmul(st):
    y = torch.matmul(st["x"].float(), st["w"].float().t())
    return (y * st["xs"].unsqueeze(1) * st["ws"]).to(st["type"])


def _norm(st):
    x = st["x"]
    if st["delta"] is not None:
        x = (x.float() + st["delta"].float()).to(x.dtype)
    s = x.float()
    values, scale = _held(s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * st["gain"].float())
    return {"values": values, "scale": scale, **({"sum": x} if st["delta"] is not None else {})}


def _swiglu(st):
    g, u = st["x"].float().chunk(2, 1)
    values, scale = _held(g / (1 + torch.exp(-g)) * u)
    return {"values": values, "scale": scale}


def _quantize(st):
    values, scale = _held(st["x"].float())
    return {"values": values, "scale": scale}


def run(state):
    op = state["op"]
    if own:
        import qwen3_dense_decoder_gb300 as q3
        if op == "matmul":
            return q3.op_i8_matmul(state["x"], state["xs"], state["w"], state["ws"], dtype=state["type"])
        x = state["x"]
        values = torch.empty(x.shape[0], x.shape[1] // (2 if op == "swiglu" else 1), dtype=torch.float16, device=x.device)
        if op == "norm":
            _, scale, total = q3.op_i8_norm(x, state["gain"], EPS, delta=state["delta"], values=values)
            return {"values": values, "scale": scale, **({"sum": total} if state["delta"] is not None else {})}
        _, scale = (q3.op_i8_swiglu if op == "swiglu" else q3.op_i8_quantize)(x, values=values)
        return {"values": values, "scale": scale}
    return {"matmul": _matmul, "norm": _norm, "swiglu": _swiglu, "quantize": _quantize}[op](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "matmul":
        t, m = st["x"].shape[0], st["w"].shape[0]
        out = torch.empty(t, m, dtype=torch.float64, device="cuda")
        x = st["x"].double()
        for at in range(0, m, 4096):
            w = st["w"][at: at + 4096].double()
            out[:, at: at + 4096] = (x @ w.T) * torch.outer(st["xs"].double(), st["ws"][at: at + 4096].double())
        return out
    values, scale, total = [], [], []
    for at in range(0, st["x"].shape[0], 2048):
        y = st["x"][at: at + 2048].double()
        if op == "norm":
            if st["delta"] is not None:
                y = (y + st["delta"][at: at + 2048].double()).to(st["type"]).double()
                total.append(y)
            y = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * st["gain"].double()
        elif op == "swiglu":
            half = y.shape[1] // 2
            y = y[:, half:] * y[:, :half] * torch.sigmoid(y[:, :half])
        step = y.abs().max(1, keepdim=True).values / 127
        values.append(torch.where(step > 0, (y / step).round() * step, 0.0).float())
        scale.append(step.squeeze(1))
    got = {"values": torch.cat(values), "scale": torch.cat(scale)}
    if total:
        got["sum"] = torch.cat(total)
    return got
