"""A plain reading of the 4-bit cache's tile format as include/q3.h states it,
and attention over it in 64 bits, for the operator tests."""
import numpy as np

TILE, D, BLOCK = 2560, 128, 32


def f16(lo, hi):
    return (lo.astype(np.uint16) | (hi.astype(np.uint16) << 8)).view(np.float16).astype(np.float64)


def read_tiles(kv):
    """kv: uint8 [n_blocks, 2, n_kv, 2560] -> dict of K and V parts:
    codes [n_blocks, n_kv, 32, 128], scale and bias [n_blocks, n_kv, 32, 4]."""
    nb, _, n_kv, _ = kv.shape
    out = {}
    for which, name in ((0, "k"), (1, "v")):
        t = kv[:, which]
        codes = np.zeros((nb, n_kv, BLOCK, D), np.int64)
        scale = np.zeros((nb, n_kv, BLOCK, 4))
        bias = np.zeros((nb, n_kv, BLOCK, 4))
        for r in range(BLOCK):
            for grp in range(4):
                for i in range(32):
                    if which == 0:
                        byte = t[:, :, r * 64 + grp * 16 + i // 2]
                        shift = 4 * (i % 2)
                    else:
                        g, e = i // 4, i % 4
                        byte = t[:, :, (r // 2) * 128 + g * 16 + grp * 4 + (r % 2) * 2 + e // 2]
                        shift = 4 * (e % 2)
                    codes[:, :, r, grp * 32 + i] = (byte >> shift) & 15
                if which == 0:
                    s = 2048 + r * 16 + grp * 4
                    b = s + 2
                else:
                    s = 2048 + (r // 2) * 32 + grp * 8 + (r % 2) * 2
                    b = s + 4
                scale[:, :, r, grp] = f16(t[:, :, s], t[:, :, s + 1])
                bias[:, :, r, grp] = f16(t[:, :, b], t[:, :, b + 1])
        out[name] = (codes, scale, bias)
    return out


def values(part):
    """The values a part stands for: fp16(scale * code + bias), as f64 [..., 128]."""
    codes, scale, bias = part
    v = np.repeat(scale, 32, -1) * codes + np.repeat(bias, 32, -1)
    return v.astype(np.float16).astype(np.float64)


def stored(kv):
    """K and V values [n_blocks, n_kv, 32, 128] of a pool."""
    p = read_tiles(kv)
    return values(p["k"]), values(p["v"])


def attend(q, K, V, table, pos, n_kv):
    """Rows q f64 [T, n_q, 128] at positions pos over one table: f64 [T, n_q, 128] (zeros where pos < 0)."""
    T, n_q, _ = q.shape
    G = n_q // n_kv
    out = np.zeros_like(q)
    n = max(int(np.max(pos)) + 1, 0)
    if n == 0:
        return out
    nb = (n + BLOCK - 1) // BLOCK
    kk = K[table[:nb]].transpose(1, 0, 2, 3).reshape(n_kv, nb * BLOCK, D)
    vv = V[table[:nb]].transpose(1, 0, 2, 3).reshape(n_kv, nb * BLOCK, D)
    for t in range(T):
        m = int(pos[t]) + 1
        if m <= 0:
            continue
        for h in range(n_kv):
            s = q[t, h * G:(h + 1) * G] @ kk[h, :m].T / np.sqrt(128.0)
            e = np.exp(s - s.max(-1, keepdims=True))
            out[t, h * G:(h + 1) * G] = (e / e.sum(-1, keepdims=True)) @ vv[h, :m]
    return out


def random_pool(n_blocks, n_kv, seed):
    """A pool of random codes with ordinary scales and biases (uint8 numpy)."""
    r = np.random.default_rng(seed)
    kv = r.integers(0, 256, (n_blocks, 2, n_kv, TILE), dtype=np.uint8)
    s = r.uniform(0.1, 0.4, (n_blocks, 2, n_kv, 128))
    b = -7.5 * s + r.normal(0, 0.3, s.shape)
    s, b = s.astype(np.float16), b.astype(np.float16)
    k = np.stack([s[:, 0], b[:, 0]], -1).reshape(n_blocks, n_kv, 256)                   # [position][group](s, b)
    v = np.stack([s[:, 1].reshape(n_blocks, n_kv, 16, 4, 2), b[:, 1].reshape(n_blocks, n_kv, 16, 4, 2)], -2)
    kv[:, 0, :, 2048:] = np.ascontiguousarray(k).view(np.uint8)
    kv[:, 1, :, 2048:] = np.ascontiguousarray(v.reshape(n_blocks, n_kv, 256)).view(np.uint8)
    return kv
