"""fp64 definitions of the gated expert activation with dropout and of the
few-token MoE layer, with element-wise error bounds (test infrastructure)."""
import math

import numpy as np

U_BF16 = 2.0 ** -8    # half a step of bf16, relative to the value
U_F32 = 2.0 ** -24
TINY = 2.0 ** -126    # below this a rounding error is absolute

_M32 = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key):
    """Philox4x32-10: counter four and key two broadcastable uint32 arrays."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k0, k1 = (np.asarray(v, np.uint64) for v in key)
    for _ in range(10):
        p0 = np.uint64(0xD2511F53) * c[0]
        p1 = np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ k0, p1 & _M32, (p0 >> np.uint64(32)) ^ c[3] ^ k1, p0 & _M32]
        k0 = (k0 + np.uint64(0x9E3779B9)) & _M32
        k1 = (k1 + np.uint64(0xBB67AE85)) & _M32
    return c


def kept_mask(entries, I, p, seed, offset):
    """[len(entries), I] kept elements and the scale of a kept one."""
    drop = int(np.rint(p * 65536))
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    vec = np.arange(-(-I // 8))[None, :]
    ent = np.asarray(entries)[:, None]
    w = philox4x32((vec + 0 * ent, ent + 0 * vec, offset & 0xFFFFFFFF, offset >> 32),
                   (seed & 0xFFFFFFFF, seed >> 32))
    out = np.empty((ent.shape[0], vec.shape[1], 8), bool)
    for j in range(8):
        out[:, :, j] = (np.broadcast_to(w[j // 2], out.shape[:2]) >> np.uint64(16 * (j % 2))
                        & np.uint64(0xFFFF)) >= drop
    return out.reshape(ent.shape[0], -1)[:, :I], 65536.0 / (65536 - drop)


def gate(act, g):
    """a(g) and a'(g) in fp64."""
    if act == "silu":
        c, dc = g, np.ones_like(g)
    else:
        r = 2.0 * math.sqrt(2.0 / math.pi)
        c, dc = r * (g + 0.044715 * g ** 3), r * (1.0 + 3 * 0.044715 * g * g)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-c))
    return g * s, s, g * s * (1.0 - s) * dc


def act_rows(gu, w, act, mask, scale):
    I = gu.shape[1] // 2
    a, _, _ = gate(act, gu[:, :I].astype(np.float64))
    v = w.astype(np.float64)[:, None] * scale * a * gu[:, I:].astype(np.float64)
    return np.where(mask, v, 0.0)


def act_rows_bwd(ghs, gu, w, act, mask, scale):
    """(ggu, gw, sum |terms| of ggate, sum |terms| of gw)."""
    I = gu.shape[1] // 2
    g, u = gu[:, :I].astype(np.float64), gu[:, I:].astype(np.float64)
    a, s, t = gate(act, g)
    d = np.where(mask, ghs.astype(np.float64) * scale, 0.0)
    dw = d * w.astype(np.float64)[:, None]
    ggu = np.concatenate([dw * u * (s + t), dw * a], 1)
    return ggu, (d * a * u).sum(1), np.abs(dw * u) * (s + np.abs(t)), np.abs(d * a * u).sum(1)


def layer(x, idx, w, w13, w2, num_shared, E, act):
    """(out, bound) of the few-token layer in fp64: x [T, H], idx [T, K] (outside
    [0, E): no expert; a repeated expert counts once), w [T, K], w13
    [E + S, 2I, H], w2 [E + S, H, I] as values.

    bound: gate and up are fp32 sums of H products (error H u32 sum|w x|), the
    activation moves by at most 1.13 per gate error and by its own 1e-5
    relative, a is rounded to bf16, the second sum has I fp32 terms and the
    weighted sum K + S; then out is rounded to bf16."""
    T, H = x.shape
    I = w2.shape[2]
    x = x.astype(np.float64)
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        pairs = []
        for k, e in enumerate(idx[t]):
            if 0 <= e < E and e not in [p[0] for p in pairs]:
                pairs.append((int(e), float(w[t, k])))
        pairs += [(E + j, 1.0) for j in range(num_shared)]
        for e, wt in pairs:
            m13, m2 = w13[e].astype(np.float64), w2[e].astype(np.float64)
            z = m13 @ x[t]
            dz = (H + 2) * U_F32 * (np.abs(m13) @ np.abs(x[t]))
            a, _, _ = gate(act, z[:I])
            h = a * z[I:]
            dh = 1.13 * dz[:I] * (np.abs(z[I:]) + dz[I:]) + np.abs(a) * dz[I:] + 1e-5 * np.abs(h)
            dh = dh + U_BF16 * (np.abs(h) + dh)
            y = m2 @ h
            dy = np.abs(m2) @ (dh + (I + len(pairs) + 4) * U_F32 * (np.abs(h) + dh))
            out[t] += wt * y
            bound[t] += abs(wt) * (dy + 2 * len(pairs) * U_F32 * np.abs(y))
    return out, bound + U_BF16 * (np.abs(out) + bound) + TINY
