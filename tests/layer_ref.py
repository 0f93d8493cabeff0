"""The few-token MoE layer at the precision its interface states (test
infrastructure): an element-wise bound, layers whose result is exact, and a
model on the host that can plant a mistake.

Stated: fp32 sums; with bf16 weights the activation between the products as the
sum of two bf16 numbers (what is left is half a bf16 step of half a bf16 step,
2^-16); with e4m3 weights x and the activation in fp16 times a power of two per
token and per entry, which brings the largest to [2^14, 2^15): half a step of
2^-11, and below 2^-14 half a step of 2^-24, 2^-39 of the largest; out in bf16."""
import numpy as np
import torch

from tests import expert_ref as ref

FAULTS = ("low parts lost", "low parts of the next column", "low parts of another token",
          "last 8 columns of the activation lost", "last 8 columns of x lost")
FAULTS_E4M3 = ("activation in 8 bits", "last 8 columns of the activation lost",
               "last 8 columns of x lost", "scales of the next row of blocks")


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float64)).to(torch.bfloat16).double().numpy()


def pairs_of(idx_t, w_t, E, shared):
    out = []
    for k, e in enumerate(idx_t):
        if 0 <= e < E and e not in [p[0] for p in out]:
            out.append((int(e), float(w_t[k])))
    return out + [(E + j, 1.0) for j in range(shared)]


def layer(x, idx, w, w13, w2, shared, E, act, e4m3):
    """(out, bound) in fp64, arguments as in expert_ref.layer.

    An fp32 sum of n terms is off by at most n 2^-24 of the terms' magnitudes in
    any order; a gate's error moves the activation by at most 1.13 of itself,
    and the activation's own arithmetic is good to 1e-5."""
    T, H = x.shape
    I = w2.shape[2]
    x = x.astype(np.float64)
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        pairs = pairs_of(idx[t], w[t], E, shared)
        dx = np.abs(x[t]).max() * 2.0 ** -39 if e4m3 else 0.0
        for e, wt in pairs:
            m13, m2 = w13[e].astype(np.float64), w2[e].astype(np.float64)
            z = m13 @ x[t]
            dz = np.abs(m13) @ ((H + 2) * ref.U_F32 * np.abs(x[t]) + dx)
            a, _, _ = ref.gate(act, z[:I])
            h = a * z[I:]
            dh = 1.13 * dz[:I] * (np.abs(z[I:]) + dz[I:]) + np.abs(a) * dz[I:] + 1e-5 * np.abs(h)
            kept = 2.0 ** -11 if e4m3 else 2.0 ** -16
            dh = dh + kept * (np.abs(h) + dh) + (np.abs(h).max() * 2.0 ** -39 if e4m3 else ref.TINY)
            y = m2 @ h
            dy = np.abs(m2) @ (dh + (I + len(pairs) + 4) * ref.U_F32 * (np.abs(h) + dh))
            out[t] += wt * y
            bound[t] += abs(wt) * (dy + 2 * len(pairs) * ref.U_F32 * np.abs(y))
    return out, bound + ref.U_BF16 * (np.abs(out) + bound) + ref.TINY


def model(x, idx, w, w13, w2, shared, E, act, e4m3, fault=None):
    """The layer with its stated roundings and nothing else (fp64 sums), out not
    yet rounded; `fault` plants a mistake."""
    T, H = x.shape
    I = w2.shape[2]
    x = x.astype(np.float64).copy()
    if fault == "last 8 columns of x lost":
        x[:, -8:] = 0.0
    out = np.zeros((T, H))
    acts = {}
    for t in range(T):
        for e, wt in pairs_of(idx[t], w[t], E, shared):
            z = w13[e].astype(np.float64) @ x[t]
            a, _, _ = ref.gate(act, z[:I])
            acts[t, e] = a * z[I:]
    entries = list(acts)
    for i, (t, e) in enumerate(entries):
        h = acts[t, e]
        if e4m3:
            f = 2.0 ** (14 - np.floor(np.log2(np.abs(h).max()))) if np.abs(h).max() > 0 else 1.0
            v = bf16(h) if fault == "activation in 8 bits" else (h * f).astype(np.float16).astype(np.float64) / f
        else:
            hi = bf16(h)
            lo = bf16(h - hi)
            if fault == "low parts lost":
                lo = 0.0 * lo
            elif fault == "low parts of the next column":
                lo = np.roll(lo, 1)
            elif fault == "low parts of another token":
                o = acts[entries[(i + 1) % len(entries)]]
                lo = bf16(o - bf16(o))
            v = hi + lo
        if fault == "last 8 columns of the activation lost":
            v = np.concatenate([v[:-8], np.zeros(8)])
        wt = dict(pairs_of(idx[t], w[t], E, shared))[e]
        out[t] += wt * (w2[e].astype(np.float64) @ v)
    return out


class Exact:
    """A layer whose every intermediate value is exact, so that out is the exact
    sum rounded once.

    Column 0 of x is 64 and feeds the gates: silu(64) and gelu(64) are 64 to
    more digits than fp32 has.  Column 1 is 4; the up rows take it and, with a
    sign, one of the other columns, r / (64 D) for an integer r: an activation is
    256 + r / D.  With bf16 weights D = 64 and |r| < 64, 16 bits, so that the
    second bf16 number holds r; with e4m3 weights D = 4 and |r| <= 120, 11 bits.
    Every W2 row subtracts columns from as many others, so that the 256 cancel
    and out holds what the last bits hold.  Every column of the activation is in
    some W2 row, and every column of x in some up row if the reached experts
    have that many.  The block scales are powers of two and the weights their
    inverses."""

    def __init__(self, T, E, K, H, I, shared=0, e4m3=False, seed=0):
        g = np.random.default_rng(seed)
        n = E + shared
        D, top = (4, 120) if e4m3 else (64, 63)
        self.T, self.E, self.K, self.H, self.I, self.S, self.e4m3 = T, E, K, H, I, shared, e4m3
        self.r = g.integers(-top, top + 1, (T, H))
        self.x = self.r / (64.0 * D)
        self.x[:, 0], self.x[:, 1] = 64.0, 4.0
        self.idx = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
        self.w = 2.0 ** g.integers(-2, 2, (T, K)).astype(np.float64)
        self.w13, self.w2 = np.zeros((n, 2 * I, H)), np.zeros((n, H, I))
        i, row = np.arange(I), np.arange(H)
        for e in range(n):
            sign = g.choice([-1.0, 1.0], I)
            self.w13[e, i, 0] = 1.0
            self.w13[e, I + i, 1] = 1.0
            self.w13[e, I + i, 2 + (i + e * I + g.integers(H)) % (H - 2)] = sign
            # pairs of columns j and j + I / 2, dealt out to the rows
            half = I // 2
            for k in range(max(1, -(-half // H))):
                j = row + k * H
                ok = (j < half) | (k == 0)
                j = j % half
                s = np.where(row // half % 2 == 0, 1.0, -1.0)
                self.w2[e, row[ok], j[ok]] += s[ok]
                self.w2[e, row[ok], j[ok] + half] -= s[ok]
        self.s13 = self.s2 = None
        if e4m3:
            self.s13, self.q13 = self.scaled(self.w13)
            self.s2, self.q2 = self.scaled(self.w2)

    @staticmethod
    def scaled(w):
        shape = (w.shape[0], -(-w.shape[1] // 128), -(-w.shape[2] // 128))
        e, a, b = np.indices(shape)
        s = 2.0 ** ((a + 2 * b + e) % 4 - 1)
        big = np.repeat(np.repeat(s, 128, 1), 128, 2)[:, :w.shape[1], :w.shape[2]]
        return s.astype(np.float32), w / big

    def values(self, fault=None):
        """The weights' values (with mistaken scales)."""
        if fault != "scales of the next row of blocks":
            return self.w13, self.w2
        out = []
        for s, q in ((self.s13, self.q13), (self.s2, self.q2)):
            s = np.roll(s, 1, 1)
            out.append(q * np.repeat(np.repeat(s, 128, 1), 128, 2)[:, :q.shape[1], :q.shape[2]])
        return out

    def out(self, fault=None):
        """Out in bf16, act silu or gelu."""
        w13, w2 = self.values(fault)
        return bf16(model(self.x, self.idx, self.w, w13, w2, self.S, self.E, "silu", self.e4m3, fault))

    def want(self):
        """The same from the integers r."""
        out = np.zeros((self.T, self.H))
        D = 4.0 if self.e4m3 else 64.0
        for t in range(self.T):
            for e, wt in pairs_of(self.idx[t], self.w[t], self.E, self.S):
                up = self.w13[e, self.I:].copy()
                up[:, :2] = 0.0
                out[t] += wt * (self.w2[e] @ (up @ self.r[t])) / D
        return bf16(out)
