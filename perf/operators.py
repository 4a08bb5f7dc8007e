"""The operators of the 4-bit K/V cache and of token scoring: the sizes they
are used at, their inputs, their plain form in elementary torch operations
and, where `own` is set, the library's calls.

A cache tile (32 positions of K or V of one KV head) is 2,560 bytes: 4-bit
codes, then fp16 scales and biases per 32 dimensions; a stored value is
fp16(scale * code + bias).  K codes lie as [position][64 bytes], dimension
2 i in the low nibble of byte i, its parameters as [position][group](scale,
bias).  V codes lie as [position pair][g][group][even, odd position][four
dimensions 32 group + 4 g ..], its parameters as [pair][group](scale even,
scale odd, bias even, bias odd).
"""
import math

import torch

own = False

D = 128
TILE = 2560
BLOCK = 32
SCALE = 1.0 / math.sqrt(128.0)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode round of 32 sessions, 4B heads: the new token of each
        {"name": "append_decode32", "op": "append", "rows": 32, "n_q": 32, "n_kv": 8, "type": "f32", "seqs": 32, "ctx": 1184},
        # a 2,048-row prefill round of one session, 4B heads
        {"name": "append_prefill2048", "op": "append", "rows": 2048, "n_q": 32, "n_kv": 8, "type": "f32", "seqs": 1, "ctx": 2048},
        # chunks of three sessions, 14B heads, bf16 projections, an odd row count
        {"name": "append_mixed701", "op": "append", "rows": 701, "n_q": 40, "n_kv": 8, "type": "bf16", "seqs": 3, "ctx": 1500},
        # one session's decode step (latency)
        {"name": "decode_1x2176", "op": "decode", "rows": 1, "n_q": 32, "n_kv": 8, "type": "f16", "lo": 2176, "hi": 2176, "empty": 0},
        # 32 sessions of unequal contexts, mean near 1,184
        {"name": "decode_32x1184", "op": "decode", "rows": 32, "n_q": 32, "n_kv": 8, "type": "f32", "lo": 129, "hi": 2239, "empty": 0},
        # eight long sessions, 14B heads
        {"name": "decode_8x16384", "op": "decode", "rows": 8, "n_q": 40, "n_kv": 8, "type": "f16", "lo": 16384, "hi": 16384, "empty": 0},
        # a padded batch of short contexts, 0.6B heads, some rows without a session
        {"name": "decode_61_padded", "op": "decode", "rows": 61, "n_q": 16, "n_kv": 8, "type": "f16", "lo": 1, "hi": 611, "empty": 5},
        # a 2,048-token prompt, 4B heads
        {"name": "prefill_2048", "op": "prefill", "seqs": 1, "lo": 2048, "hi": 2048, "before": 0, "n_q": 32, "n_kv": 8},
        # five ragged chunks, each with context before it, 0.6B heads
        {"name": "prefill_ragged5", "op": "prefill", "seqs": 5, "lo": 3, "hi": 701, "before": 333, "n_q": 16, "n_kv": 8},
        # a late chunk of a long prompt, 14B heads
        {"name": "prefill_late512", "op": "prefill", "seqs": 1, "lo": 512, "hi": 512, "before": 10240, "n_q": 40, "n_kv": 8},
        # one decode step's logits with 20 alternatives (latency)
        {"name": "logprobs_1", "op": "logprobs", "rows": 1, "vocab": 151936, "type": "f32", "top": 20},
        # every row of a 2,048-token prompt scored
        {"name": "logprobs_2048", "op": "logprobs", "rows": 2048, "vocab": 151936, "type": "f32", "top": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill", "logprobs"))
    n_q, n_kv = rng.choice(((16, 8), (32, 8), (40, 8), (8, 8), (24, 8), (64, 8), (14, 2)))
    if op == "append":
        seqs = rng.randint(1, 8)
        rows = max(seqs, _log(rng, 1, 2048 if n_q <= 40 else 1024))
        return {"op": op, "rows": rows, "n_q": n_q, "n_kv": n_kv, "type": rng.choice(("f32", "f16", "bf16")), "seqs": seqs,
                "ctx": rows + rng.randint(0, 3000)}
    if op == "decode":
        rows = _log(rng, 1, 64)
        hi = _log(rng, 2, 131072 // rows // max(1, n_q // 32))
        return {"op": op, "rows": rows, "n_q": n_q, "n_kv": n_kv, "type": rng.choice(("f32", "f16")), "lo": rng.randint(1, hi),
                "hi": hi, "empty": rng.choice((0, 0, 1, rows // 4))}
    if op == "prefill":
        seqs = rng.randint(1, 6)
        hi = _log(rng, 2, 1500 // seqs)
        return {"op": op, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "before": _log(rng, 1, 4000) - 1, "n_q": n_q,
                "n_kv": n_kv}
    rows, vocab = _log(rng, 1, 1024), rng.choice((151936, 4096, 50257, 32003, 1000, _log(rng, 40, 200000)))
    return {"op": op, "rows": rows, "vocab": vocab, "type": rng.choice(("f32", "f32", "f16", "bf16")),
            "top": min(rng.choice((0, 1, 5, 20, 32)), vocab)}


def _spread(n, lo, hi):
    """n lengths of [lo, hi], spread evenly and out of order."""
    return [lo + int((hi - lo) * ((0.5 + 0.6180339887498949 * i) % 1.0) + 0.5) for i in range(n)]


def _decode_lens(case):
    """The context of each row; `empty` of them belong to no session."""
    n, empty = case["rows"], case["empty"]
    lens = _spread(n, case["lo"], case["hi"])
    if n > 2 and empty:
        for i in range(empty):
            lens[i * (n // empty) + n // empty // 2] = 0
    return lens


def _prefill_seqs(case):
    """(rows, position of the first row) of each sequence."""
    n = _spread(case["seqs"], case["lo"], case["hi"])
    before = case["before"]
    return [(r, before if case["seqs"] == 1 else (before * (i % 3)) // 2) for i, r in enumerate(n)]


def _append_rows(case):
    """(sequence, position) of each row: the rows split over the sequences, each ending at `ctx` or a little before."""
    rows, seqs, ctx = case["rows"], case["seqs"], case["ctx"]
    n = [rows // seqs + (i < rows % seqs) for i in range(seqs)]
    first = [max(0, ctx - n[i] - 7 * i) for i in range(seqs)]
    return [(i, first[i] + j) for i in range(seqs) for j in range(n[i])]


def _append_len(case):
    return max(p for _, p in _append_rows(case)) + 1


def work(case):
    if case["op"] == "append":
        size = 4 if case["type"] == "f32" else 2
        t, n_q, n_kv = case["rows"], case["n_q"], case["n_kv"]
        return {"bytes": t * ((n_q + 2 * n_kv) * D * size + n_q * 256 + n_kv * (160 + 512) + 512 + 12),
                "flops": t * (n_q + 2 * n_kv) * D * 10}
    if case["op"] == "decode":
        size = 4 if case["type"] == "f32" else 2
        total = sum(_decode_lens(case))
        return {"bytes": total * case["n_kv"] * 160 + case["rows"] * case["n_q"] * D * (size + 2),
                "flops": 4 * D * case["n_q"] * total}
    if case["op"] == "prefill":
        s = _prefill_seqs(case)
        return {"bytes": sum(n + p for n, p in s) * case["n_kv"] * 160 + sum(n for n, _ in s) * case["n_q"] * 512,
                "flops": 4 * D * case["n_q"] * sum(n * p + n * (n + 1) // 2 for n, p in s)}
    size = 4 if case["type"] == "f32" else 2
    return {"bytes": case["rows"] * (case["vocab"] * size + 12 + 8 * case["top"]), "flops": 5 * case["rows"] * case["vocab"]}


# ---------------------------------------------------------------- the cache format

def _quantise(x):
    """f32 [..., 128] -> codes uint8 [..., 128], scale and bias fp16 [..., 4]."""
    g = x.unflatten(-1, (4, 32))
    lo, hi = g.amin(-1), g.amax(-1)
    scale, bias = ((hi - lo) / 15.0).half(), lo.half()
    s, b = scale.float().unsqueeze(-1), bias.float().unsqueeze(-1)
    code = torch.where(s > 0, torch.round((g - b) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0.0)
    return code.to(torch.uint8).flatten(-2), scale, bias


def _stored(code, scale, bias):
    """The fp16 values that codes [..., 128] with parameters [..., 4] stand for."""
    c = code.unflatten(-1, (4, 32)).float()
    return (scale.float().unsqueeze(-1) * c + bias.float().unsqueeze(-1)).half().flatten(-2)


def _tiles(k, v):
    """f32 K and V [blocks, n_kv, 32, 128] -> cache uint8 [blocks, 2, n_kv, 2560]."""
    nb, n_kv = k.shape[:2]
    kv = torch.empty(nb, 2, n_kv, TILE, dtype=torch.uint8, device=k.device)
    c, s, b = _quantise(k)
    kv[:, 0, :, :2048] = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(2)
    kv[:, 0, :, 2048:] = torch.stack((s, b), -1).flatten(2).view(torch.uint8)
    c, s, b = _quantise(v)
    c = c.view(nb, n_kv, 16, 2, 4, 8, 4).permute(0, 1, 2, 5, 4, 3, 6).contiguous()
    kv[:, 1, :, :2048] = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(2)
    sb = torch.stack((s.view(nb, n_kv, 16, 2, 4), b.view(nb, n_kv, 16, 2, 4)), 3)      # pair, s/b, parity, group
    kv[:, 1, :, 2048:] = sb.permute(0, 1, 2, 5, 3, 4).contiguous().flatten(2).view(torch.uint8)
    return kv


def _untile(kv):
    """cache [..., 2, n_kv, 2560] -> the stored K and V, fp16 [..., n_kv, 32, 128]."""
    k, v = kv.select(-3, 0), kv.select(-3, 1)
    lead = k.shape[:-1]
    by = k[..., :2048].unflatten(-1, (32, 64))
    code = torch.stack((by & 15, by >> 4), -1).flatten(-2)
    sb = k[..., 2048:].contiguous().view(torch.float16).unflatten(-1, (32, 4, 2))
    kk = _stored(code, sb[..., 0], sb[..., 1])
    by = v[..., :2048].unflatten(-1, (16, 8, 4, 2, 2))
    code = torch.stack((by & 15, by >> 4), -1).flatten(-2)                              # pair, g, group, parity, dim
    n = len(lead)
    code = code.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).reshape(*lead, 32, 128)
    sb = v[..., 2048:].contiguous().view(torch.float16).unflatten(-1, (16, 4, 2, 2))    # pair, group, s/b, parity
    sb = sb.permute(*range(n), n, n + 3, n + 1, n + 2).reshape(*lead, 32, 4, 2)
    return kk, _stored(code, sb[..., 0], sb[..., 1])


# ---------------------------------------------------------------- inputs

def _cache(gen, lens, n_kv):
    """A pool whose blocks hold random rows, and a permuted table for sequences of these lengths."""
    per = max(1, max((n + BLOCK - 1) // BLOCK for n in lens))
    blocks = len(lens) * per + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    tables = perm[: len(lens) * per].view(len(lens), per).contiguous()
    kv = torch.empty(blocks, 2, n_kv, TILE, dtype=torch.uint8, device="cuda")
    step = 4096
    for at in range(0, blocks, step):
        n = min(step, blocks - at)
        kv[at: at + n] = _tiles(torch.randn(n, n_kv, BLOCK, D, generator=gen, device="cuda"),
                                torch.randn(n, n_kv, BLOCK, D, generator=gen, device="cuda"))
    return kv, tables


def _rope(n, theta=1e6):
    inv = torch.pow(torch.tensor(theta, dtype=torch.float64, device="cuda"),
                    -torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = torch.arange(n, dtype=torch.float64, device="cuda").unsqueeze(1) * inv
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()                     # [n][64][2]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7 + 1)
    st = {"op": case["op"]}
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        x = torch.randn(n, v, generator=gen, device="cuda") * 2.0
        hot = torch.randint(0, v, (n,), generator=gen, device="cuda")
        x.scatter_add_(1, hot.unsqueeze(1), torch.rand(n, 1, generator=gen, device="cuda") * 16)
        x[:, torch.randint(0, v, (max(1, v // 500),), generator=gen, device="cuda")] = -math.inf   # tokens never offered
        other = torch.randint(0, v, (n,), generator=gen, device="cuda")
        pick = torch.rand(n, generator=gen, device="cuda") < 0.5
        # a target that is never offered has log probability -inf; a scored text has none
        t = torch.where(pick, hot, other)
        t = torch.where(torch.isinf(x.gather(1, t.unsqueeze(1)).squeeze(1)), x.argmax(1), t)
        return {**st, "logits": x.to(TYPES[case["type"]]), "targets": t.to(torch.int32), "top": case["top"]}
    n_q, n_kv = case["n_q"], case["n_kv"]
    st["n_q"] = n_q
    if case["op"] == "append":
        rows = _append_rows(case)
        per = (_append_len(case) + BLOCK - 1) // BLOCK
        blocks = case["seqs"] * per + 3
        st["kv"] = torch.zeros(blocks, 2, n_kv, TILE, dtype=torch.uint8, device="cuda")
        perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        st["tables"] = perm[: case["seqs"] * per].view(case["seqs"], per).contiguous()
        st["row_slot"], st["row_pos"] = _ints([s for s, _ in rows]), _ints([p for _, p in rows])
        st["rope"] = _rope(_append_len(case))
        st["qkv"] = torch.randn(len(rows), (n_q + 2 * n_kv) * D, generator=gen, device="cuda").clamp_(-2.6, 2.6).to(TYPES[case["type"]])
        st["q_gain"], st["k_gain"] = ((1 + 0.02 * torch.randn(D, generator=gen, device="cuda")).bfloat16() for _ in range(2))
        return st
    if case["op"] == "decode":
        lens = _decode_lens(case)
        st["kv"], st["tables"] = _cache(gen, lens, n_kv)
        st["row_pos"] = _ints([n - 1 for n in lens])
        st["row_slot"] = torch.arange(len(lens), dtype=torch.int32, device="cuda")
        st["q"] = torch.randn(len(lens), n_q, D, generator=gen, device="cuda").to(TYPES[case["type"]])
        return st
    seqs = _prefill_seqs(case)
    st["kv"], st["tables"] = _cache(gen, [n + p for n, p in seqs], n_kv)
    at = [0]
    for n, _ in seqs:
        at.append(at[-1] + n)
    st["seq_rows"], st["seq_pos"] = _ints(at), _ints([p for _, p in seqs])
    st["most"] = max(n for n, _ in seqs)
    st["q"] = torch.randn(at[-1], n_q, D, generator=gen, device="cuda").half()
    return st


# ---------------------------------------------------------------- the plain forms

def _append(st):
    qkv, n_q = st["qkv"].float(), st["n_q"]
    t = qkv.shape[0]
    x = qkv.view(t, -1, D)
    n_kv = (x.shape[1] - n_q) // 2
    cs = st["rope"][st["row_pos"].long()].unsqueeze(1)                                  # [T][1][64][2]

    def turned(h, gain):
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gain.float()
        a, b = y[..., :64], y[..., 64:]
        return torch.cat((a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]), -1)

    q, k, v = turned(x[:, :n_q], st["q_gain"]), turned(x[:, n_q: n_q + n_kv], st["k_gain"]), x[:, n_q + n_kv:]
    kc, ks, kb = _quantise(k)
    vc, vs, vb = _quantise(v)
    pos, kv = st["row_pos"].long(), st["kv"]
    blk = st["tables"][st["row_slot"].long(), pos // BLOCK].long()
    r = pos % BLOCK
    flat = kv.view(kv.shape[0], 2, n_kv, TILE)
    byte = torch.arange(64, device=kv.device)
    head = torch.arange(n_kv, device=kv.device).view(1, -1, 1)
    flat[blk.view(-1, 1, 1), 0, head, r.view(-1, 1, 1) * 64 + byte] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    par = torch.stack((ks, kb), -1).flatten(2).view(torch.uint8)                        # [T][n_kv][16]
    flat[blk.view(-1, 1, 1), 0, head, 2048 + r.view(-1, 1, 1) * 16 + byte[:16]] = par
    # V: byte j of a row's 64 is dimensions 2 j, 2 j + 1: group j / 16, g (j % 16) / 2
    place = (byte % 16 // 2) * 16 + (byte // 16) * 4 + byte % 2
    flat[blk.view(-1, 1, 1), 1, head, (r // 2 * 128 + r % 2 * 2).view(-1, 1, 1) + place] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    par = torch.stack((vs, vb), -1).flatten(2).view(torch.uint8)                        # group, s/b, byte
    j = byte[:16]
    place = 2048 + (j // 4) * 8 + (j % 4 // 2) * 4 + j % 2
    flat[blk.view(-1, 1, 1), 1, head, (r // 2 * 32 + r % 2 * 2).view(-1, 1, 1) + place] = par
    return {"q": q.half(), "kv": torch.stack((_stored(kc, ks, kb), _stored(vc, vs, vb)), 1)}


def _decode(st):
    q = st["q"].float()
    t, n_q = q.shape[:2]
    k, v = _untile(st["kv"][st["tables"][st["row_slot"].long()].long()])               # [T][blocks][n_kv][32][128]
    n_kv = k.shape[2]
    k, v = (x.transpose(1, 2).flatten(2, 3).float() for x in (k, v))                    # [T][n_kv][ctx][128]
    s = torch.matmul(q.view(t, n_kv, n_q // n_kv, D), k.transpose(-1, -2)) * SCALE
    seen = (torch.arange(k.shape[2], device=q.device) <= st["row_pos"].view(-1, 1)).view(t, 1, 1, -1)
    s = torch.where(seen, s, -math.inf)
    e = torch.where(seen, torch.exp(s - torch.nan_to_num(s.amax(-1, keepdim=True), neginf=0.0)), 0.0)
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.reshape(t, n_q, D).half()


def _prefill(st):
    q, rows, pos0, most = st["q"].float(), st["seq_rows"].long(), st["seq_pos"].long(), st["most"]
    n_q, ns = q.shape[1], pos0.numel()
    k, v = _untile(st["kv"][st["tables"].long()])
    n_kv = k.shape[2]
    k, v = (x.transpose(1, 2).flatten(2, 3).float() for x in (k, v))                    # [seqs][n_kv][ctx][128]
    at = rows[:-1].view(-1, 1) + torch.arange(most, device=q.device)                    # [seqs][most]
    used = at < rows[1:].view(-1, 1)
    qq = q[torch.where(used, at, 0)].view(ns, most, n_kv, n_q // n_kv, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qq, k.unsqueeze(2).transpose(-1, -2)) * SCALE                      # [seqs][n_kv][G][most][ctx]
    pos = pos0.view(-1, 1) + torch.arange(most, device=q.device)
    seen = (torch.arange(k.shape[2], device=q.device) <= pos.unsqueeze(-1)).view(ns, 1, 1, most, -1)
    s.masked_fill_(~seen, -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s, v.unsqueeze(2)) / s.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(ns, most, n_q, D)[used].half()


def _logprobs(st):
    x, top = st["logits"].float(), st["top"]
    v = x.shape[1]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    logprob = (x.gather(1, st["targets"].long().unsqueeze(1)) - lse).squeeze(1)
    entropy = torch.log(total).squeeze(1) - (torch.where(e > 0, x - m, 0.0) * e).sum(1) / total.squeeze(1)
    # by value, the lowest index first among equals: the value's bits as a whole number that sorts like it, then the index
    bits = x.view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (v - 1 - torch.arange(v, device=x.device))
    ids = v - 1 - (torch.topk(key, top, dim=1).values & 0xFFFFFFFF) if top else torch.empty(x.shape[0], 0, dtype=torch.int64, device=x.device)
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.to(torch.int32), "top_logprobs": x.gather(1, ids) - lse}


def run(state):
    op = state["op"]
    if own:
        import qwen3_dense_decoder_gb300 as q3
        if op == "append":
            t, n_kv = state["qkv"].shape[0], state["kv"].shape[2]
            stored = torch.empty(t, 2, n_kv, D, dtype=torch.float16, device=state["qkv"].device)
            q = q3.op_kv4_append(state["qkv"], state["q_gain"], state["k_gain"], state["rope"], state["row_pos"], state["row_slot"],
                                 state["tables"], state["kv"], state["n_q"], kv_out=stored)
            return {"q": q, "kv": stored}
        if op == "decode":
            return q3.op_kv4_decode_attention(state["q"], state["row_pos"], state["row_slot"], state["tables"], state["kv"])
        if op == "prefill":
            return q3.op_kv4_prefill_attention(state["q"], state["seq_rows"], state["seq_pos"], state["tables"], state["kv"])
        logprob, entropy, ids, values = q3.op_token_logprobs(state["logits"], state["targets"], state["top"])
        return {"logprob": logprob, "entropy": entropy, "top_ids": ids, "top_logprobs": values}
    return {"append": _append, "decode": _decode, "prefill": _prefill, "logprobs": _logprobs}[op](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _row64(tile_k, tile_v, r):
    """K and V of place r of one head's two tiles, each value from its nibble, fp16(scale * code + bias), in 64 bits."""
    d = torch.arange(D, device=tile_k.device)
    g = d // 32
    half = lambda t, at: t[..., at: at + 2]  # noqa: E731
    word = lambda t, at: (t[..., at].long() | (t[..., at + 1].long() << 8)).to(torch.int16).view(torch.float16).double()  # noqa: E731
    code = (tile_k[..., r * 64 + d // 2].long() >> (4 * (d % 2))) & 15
    k = word(tile_k, 2048 + r * 16 + g * 4) * code + word(tile_k, 2048 + r * 16 + g * 4 + 2)
    i = d % 4
    at = (r // 2) * 128 + (d % 32 // 4) * 16 + g * 4 + (r % 2) * 2 + i // 2
    code = (tile_v[..., at].long() >> (4 * (i % 2))) & 15
    at = 2048 + (r // 2) * 32 + g * 8 + (r % 2) * 2
    v = word(tile_v, at) * code + word(tile_v, at + 4)
    return k.half().double(), v.half().double()


def _seq64(kv, table, n):
    """The first n positions of a sequence: K and V, f64 [n_kv][n][128]."""
    nb = (n + BLOCK - 1) // BLOCK
    t = kv[table[:nb].long()]
    n_kv = kv.shape[2]
    k = torch.empty(n_kv, nb, BLOCK, D, dtype=torch.float64, device=kv.device)
    v = torch.empty_like(k)
    for r in range(BLOCK):
        a, b = _row64(t[:, 0], t[:, 1], r)
        k[:, :, r], v[:, :, r] = a.transpose(0, 1), b.transpose(0, 1)
    return k.flatten(1, 2)[:, :n], v.flatten(1, 2)[:, :n]


def _attend64(q, k, v, pos):
    """q f64 [rows][n_q][128] at positions pos, over one sequence."""
    n_q, n_kv = q.shape[1], k.shape[0]
    out = torch.empty_like(q)
    hidden = torch.arange(k.shape[1], device=q.device) > pos.unsqueeze(1)
    for h in range(n_q):
        s = (q[:, h] @ k[h * n_kv // n_q].T) / math.sqrt(128.0)
        s[hidden] = -math.inf
        out[:, h] = torch.softmax(s, -1) @ v[h * n_kv // n_q]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "logprobs":
        n, v = st["logits"].shape
        top = st["top"]
        logprob, entropy, ids, values = [], [], [], []
        for at in range(0, n, 64):
            lp = torch.log_softmax(st["logits"][at: at + 64].double(), 1)
            logprob.append(lp.gather(1, st["targets"][at: at + 64].long().unsqueeze(1)).squeeze(1))
            entropy.append(-(lp.exp() * lp.clamp_min(-1e300)).sum(1))
            order = torch.sort(lp, dim=1, descending=True, stable=True)
            ids.append(order.indices[:, :top].to(torch.int32))
            values.append(order.values[:, :top])
        return {"logprob": torch.cat(logprob), "entropy": torch.cat(entropy), "top_ids": torch.cat(ids), "top_logprobs": torch.cat(values)}
    if op == "append":
        n_q, n_kv = case["n_q"], case["n_kv"]
        x = st["qkv"].double().view(-1, n_q + 2 * n_kv, D)
        c = st["rope"].double()[st["row_pos"].long()]
        z = torch.complex(c[..., 0], c[..., 1]).unsqueeze(1)

        def turned(h, gain):
            y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * gain.double()
            w = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * z
            return torch.cat((w.real, w.imag), -1)

        rows = torch.stack((turned(x[:, n_q: n_q + n_kv], st["k_gain"]), x[:, n_q + n_kv:]), 1)
        for g in range(4):
            part = rows[..., 32 * g: 32 * g + 32]
            lo = part.amin(-1, keepdim=True)
            s, b = ((part.amax(-1, keepdim=True) - lo) / 15).half().double(), lo.half().double()
            part.copy_(s * ((part - b) / s).round().clamp(0, 15) + b)
        return {"q": turned(x[:, :n_q], st["q_gain"]), "kv": rows}
    q = st["q"].double()
    out = torch.zeros_like(q)
    if op == "decode":
        for i, n in enumerate(_decode_lens(case)):
            if n:
                k, v = _seq64(st["kv"], st["tables"][i], n)
                out[i: i + 1] = _attend64(q[i: i + 1], k, v, st["row_pos"][i: i + 1].long())
        return out
    at = 0
    for i, (n, p) in enumerate(_prefill_seqs(case)):
        k, v = _seq64(st["kv"], st["tables"][i], n + p)
        out[at: at + n] = _attend64(q[at: at + n], k, v, p + torch.arange(n, device=q.device))
        at += n
    return out
