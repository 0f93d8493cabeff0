"""fp64 definitions of the router's balance loss and of the norms around a block,
their gradients, and element-wise bounds of an fp32 implementation's error (test
infrastructure).

U32 is half a step of fp32 relative to a value.  A row's sum of squares is held
in a tree of at most 16 additions in a thread and 10 across threads, a sum of
positive terms over tokens in chains of at most CHAIN additions in all."""
import numpy as np

U_BF16 = 2.0 ** -8
U32 = 2.0 ** -24
TINY = 2.0 ** -126
TREE = 26
CHAIN = 200


# ---------------------------------------------------------------------------
# balance loss

def probabilities(logits, score):
    """(p, q, skipped): probabilities, the gradient's own factor, and rows whose
    NaN or +inf logit makes them count for nothing."""
    l = np.asarray(logits, np.float64)
    bad = (np.isnan(l) | (l == np.inf)).any(1)
    l = np.where(bad[:, None], -np.inf, l)
    m = l.max(1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(over="ignore"):
        if score == "softmax":
            v, q = np.exp(l - m), None
        else:
            # sigmoid / e^min(m, 0): the common factor leaves p and q as they are
            c = np.minimum(m, 0.0)
            v = np.exp(np.minimum(l, 0.0) - c) / (1.0 + np.exp(-np.abs(l)))
            q = v / (1.0 + np.exp(l))
    z = v.sum(1, keepdims=True)
    inv = np.where(z > 0, 1.0 / np.where(z > 0, z, 1.0), 0.0)
    return v * inv, (v if q is None else q) * inv, bad


def counts(idx, off, E):
    """Valid entries per sequence and expert: -1, others outside [0, E) and a
    token's repeats are not counted."""
    cnt = np.zeros((len(off) - 1, E), np.int64)
    for s in range(len(off) - 1):
        for row in idx[off[s]:off[s + 1]]:
            for e in {int(e) for e in row if 0 <= e < E}:
                cnt[s, e] += 1
    return cnt


def balance(logits, idx, off, E, score, coef):
    """(loss, counts, mean probabilities)."""
    p, _, _ = probabilities(logits, score)
    K, cnt = idx.shape[1], counts(idx, off, E)
    n = np.diff(off)
    loss, prob = 0.0, np.zeros(cnt.shape)
    for s in np.nonzero(n)[0]:
        P = p[off[s]:off[s + 1]].sum(0)
        prob[s] = P / n[s]
        loss += E / (K * float(n[s]) ** 2) * (cnt[s] * P).sum()
    return coef * loss / max(1, (n > 0).sum()), cnt, prob


def balance_bwd(logits, cnt, off, K, score, coef, gloss=1.0):
    """(glogits, bound): 0 outside the sequences; the bound without the rounding
    of a sum with a base."""
    T, E = logits.shape
    p, q, _ = probabilities(logits, score)
    n = np.diff(off)
    g, bound = np.zeros((T, E)), np.zeros((T, E))
    rel = probability_error(logits, score)
    for s in np.nonzero(n)[0]:
        r = slice(off[s], off[s + 1])
        B = gloss * coef / (n > 0).sum() * E / (K * float(n[s]) ** 2)
        d = cnt[s] - float(int(K * int(n[s]) // E))
        pd = p[r] * d
        dot = np.where(p[r].sum(1, keepdims=True) > 0, pd.sum(1, keepdims=True), 0.0)
        g[r] = B * q[r] * (d - dot)
        away = np.abs(d) + np.abs(pd).sum(1, keepdims=True)
        bound[r] = np.abs(B) * q[r] * away * (2 * rel[r] + (16 + TREE) * U32)
    return g, bound


def probability_error(logits, score):
    """Relative error of p (and q) per token, [T, 1]: the fast exponential's 2 +
    1.16 |x| ulp (an ulp is 2^-23) on the argument range of the row, the argument's
    own rounding, the division's 2 ulp, the sum over the experts."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isfinite(l), l, 0.0)
    x = l.max(1) - l.min(1) if score == "softmax" else np.maximum(np.abs(l).max(1), l.max(1) - l.min(1))
    e = (2 + 1.16 * x) * 2.0 ** -23 + x * U32
    return (2 * (e + 2.0 ** -22) + (16 + TREE) * U32)[:, None]


# ---------------------------------------------------------------------------
# norms around a block

def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def _norm_of(err, v):
    """Relative error of a row's norm from element errors."""
    n = np.sqrt((v * v).sum(1, keepdims=True))
    return np.sqrt((err * err).sum(1, keepdims=True)) / np.where(n > 0, n, 1.0)


def block_norm(res, y=None, gate=None, w_post=None, w_pre=None, scale=1.0, eps=1e-6, u_row=U32,
               y_error=None):
    """Outputs and bounds, two dicts of res_out, x, c, rstd_post and rstd_pre.
    y [T, H]: the block's output with what is added to it, y_error its error; gate
    [T, H]; weights with their offset; u_row: half a step of the rows' type."""
    out, bound = {}, {}
    if y is not None:
        ec = np.zeros_like(y) if y_error is None else y_error
        out["c"], bound["c"] = y, ec + u_row * np.abs(y)
        u, eu = y, ec
        if w_post is not None:
            r = _rstd(y, eps)
            rel = TREE * U32 + _norm_of(ec, y)
            out["rstd_post"], bound["rstd_post"] = r[:, 0], (r * rel)[:, 0]
            u = y * r * w_post
            eu = ec * np.abs(r * w_post) + np.abs(u) * (rel + 4 * U32)
        if gate is not None:
            u, eu = u * gate, eu * np.abs(gate) + np.abs(u * gate) * U32
        base = scale * res
        res = base + u
        er = eu + 2 * U32 * (np.abs(base) + np.abs(u))
        out["res_out"], bound["res_out"] = res, er + u_row * np.abs(res) + TINY
    else:
        er = np.zeros_like(res)
    if w_pre is not None:
        r = _rstd(res, eps)
        rel = TREE * U32 + _norm_of(er, res)
        out["rstd_pre"], bound["rstd_pre"] = r[:, 0], (r * rel)[:, 0]
        x = res * r * w_pre
        out["x"] = x
        bound["x"] = er * np.abs(r * w_pre) + np.abs(x) * (rel + 4 * U32 + u_row) + TINY
    return out, bound


def _through(v, ev, row, rstd, w):
    """Gradient v (error ev) of n w, n = row * rstd, to the row and to w's terms:
    (gradient, its error, weight terms, their error)."""
    n = row * rstd
    vw, evw = v * w, ev * np.abs(w) + 3 * U32 * np.abs(v * w)
    m = (vw * n).mean(1, keepdims=True)
    em = (evw * np.abs(n)).mean(1, keepdims=True) + (TREE + 2) * U32 * np.abs(vw * n).mean(1, keepdims=True)
    g = rstd * (vw - n * m)
    eg = rstd * (evw + np.abs(n) * em + 4 * U32 * (np.abs(vw) + np.abs(n * m)))
    return g, eg, v * n, ev * np.abs(n) + 2 * U32 * np.abs(v * n)


def block_norm_bwd(gres_out=None, gx=None, res_out=None, c=None, gate=None, group=None,
                   groups=0, w_post=None, w_pre=None, rstd_post=None, rstd_pre=None, scale=1.0,
                   u_row=U32):
    """Gradients and bounds, two dicts of gres, gy, ggate, gw_post and gw_pre.
    gate [groups, H], group [T]; rstd [T] as the forward gave them."""
    out, bound = {}, {}
    D = np.zeros_like(gx if gres_out is None else gres_out) if gres_out is None else gres_out
    eD = np.zeros_like(D)
    # additions in a row of a column sum: 1024 tokens, the sets of them that a team
    # takes, a 32nd of the teams' sums, 32 of those
    tokens = min(D.shape[0], 1024) + 112

    def total(terms, err):
        return terms.sum(0), err.sum(0) + tokens * U32 * np.abs(terms).sum(0)

    if gx is not None:
        g, eg, w, ew = _through(gx, eD, res_out, rstd_pre[:, None], w_pre)
        out["gw_pre"], bound["gw_pre"] = total(w, ew)
        eD = eg + 2 * U32 * (np.abs(D) + np.abs(g))
        D = D + g
    out["gres"] = scale * D
    bound["gres"] = np.abs(scale) * eD + (u_row + U32) * np.abs(scale * D) + TINY
    G, eG = D, eD
    if gate is not None:
        u = c if w_post is None else c * rstd_post[:, None] * w_post
        terms = D * u
        err = eD * np.abs(u) + 5 * U32 * np.abs(terms)
        out["ggate"], eg, ab = (np.zeros(gate.shape) for _ in range(3))
        np.add.at(out["ggate"], group, terms)
        np.add.at(eg, group, err)
        np.add.at(ab, group, np.abs(terms))
        bound["ggate"] = eg + tokens * U32 * ab + u_row * np.abs(out["ggate"]) + TINY
        G = D * gate[group]
        eG = eD * np.abs(gate[group]) + U32 * np.abs(G)
    if w_post is not None:
        G, eG, w, ew = _through(G, eG, c, rstd_post[:, None], w_post)
        out["gw_post"], bound["gw_post"] = total(w, ew)
    out["gy"], bound["gy"] = G, eG + u_row * np.abs(G) + TINY
    return out, bound
