"""Cases, plain forms and exact forms of the gated expert activation with
dropout (forward and backward) and of the whole MoE layer for a few tokens.

A case of kind "act" or "act_bwd" is one expert activation over the receive
rows of a dispatch layout; a case of kind "layer" is one MoE layer (routing,
experts, weighted sum) over a decode batch.  Where ``own`` is true, ``run``
calls the library; otherwise it computes the same results from elementary
torch operations in fp32, rounded once at the end.
"""
import functools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases

def _act(kind, T, E, K, I, dtype="bf16", act="silu", p=0.0, absorb=True, pad=1):
    return dict(kind=kind, T=T, E=E, K=K, I=I, dtype=dtype, act=act, p=p, absorb=absorb, pad=pad)


def _layer(T, E, K, H, I, live=None, score="softmax", groups=1, top_groups=1, group_top=1,
           scale=1.0, shared=0, weights="bf16", act="silu"):
    return dict(kind="layer", T=T, live=T if live is None else live, E=E, K=K, H=H, I=I,
                score=score, groups=groups, top_groups=top_groups, group_top=group_top,
                scale=scale, shared=shared, weights=weights, act=act)


def listed():
    return [
        # the tiny fp32 workload: a unit-test-sized layer, bound by the launch
        dict(_act("act", 256, 8, 2, 256, "f32", p=0.1), name="act tiny f32"),
        # inference or dropout-free training of the Qwen3-30B-A3B-shaped layer
        dict(_act("act", 8192, 128, 8, 768), name="act qwen3-30b"),
        # a training step's largest activation, scores absorbed, expert dropout
        dict(_act("act", 16384, 256, 8, 2048, p=0.1), name="act deepseek-v3 dropout"),
        # backward of a small fp32 layer with GELU experts
        dict(_act("act_bwd", 256, 8, 2, 256, "f32", act="gelu", p=0.1), name="act_bwd tiny f32"),
        # backward over segments padded to a GEMM tile, scores applied at the
        # combine, a width that fills no power of two
        dict(_act("act_bwd", 1500, 64, 4, 1000, act="gelu", p=0.25, absorb=False, pad=128),
             name="act_bwd padded ragged"),
        # backward of the largest training activation
        dict(_act("act_bwd", 16384, 256, 8, 2048, p=0.1), name="act_bwd deepseek-v3 dropout"),
        # one user's next token: weights of 8 experts, latency counts
        dict(_layer(1, 128, 8, 2048, 768), name="layer 1 token qwen3-30b"),
        # a small decode batch: most experts get a token or none
        dict(_layer(16, 128, 8, 2048, 768), name="layer 16 tokens qwen3-30b"),
        # odd sizes: fits no tile, GELU experts, one expert count off a power of two
        dict(_layer(7, 60, 6, 1000, 360, act="gelu"), name="layer ragged"),
        # speculative decoding of one user on the DeepSeek-V3-shaped layer
        dict(_layer(4, 256, 8, 7168, 2048, score="sigmoid", groups=8, top_groups=4, group_top=2,
                    scale=2.5, shared=1), name="layer 4 tokens deepseek-v3"),
        # a captured decode batch of 64 places with 37 live requests, 8-bit
        # weights with 128 x 128 block scales, a shared expert
        dict(_layer(64, 256, 8, 7168, 2048, live=37, score="sigmoid", groups=8, top_groups=4,
                    group_top=2, scale=2.5, shared=1, weights="e4m3"),
             name="layer 37 of 64 e4m3 deepseek-v3"),
        # few wide experts and the largest batch: every expert gets many tokens
        dict(_layer(128, 8, 2, 4096, 2048), name="layer 128 tokens 8 experts"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["act", "act_bwd", "layer", "layer"])
    if kind != "layer":
        E = _log_int(rng, 4, 256)
        K = _log_int(rng, 1, min(E, 8))
        I = _log_int(rng, 64, 2048, 8)
        T = _log_int(rng, 1, min(16384, 16384 * 8 * 2048 // (K * I)))
        return _act(kind, T, E, K, I, rng.choice(["bf16", "bf16", "f32"]) if T * K * I < 1 << 27
                    else "bf16", rng.choice(["silu", "gelu"]), rng.choice([0.0, 0.1, 0.25, 0.5]),
                    rng.random() < 0.6, rng.choice([1, 1, 16, 128]))
    weights = rng.choice(["bf16", "bf16", "e4m3"])
    step = 16 if weights == "e4m3" else 8
    T = _log_int(rng, 1, 128)
    H = _log_int(rng, 256, 7168, step)
    I = _log_int(rng, 64, 2048, step)
    sigmoid = rng.random() < 0.5
    most = (6 << 30) // (3 * H * I)
    E = _log_int(rng, 4, max(4, min(256, most)))
    groups, top_groups, group_top = 1, 1, 1
    if sigmoid and E >= 16:
        E = E // 8 * 8
        groups, top_groups, group_top = rng.choice([(1, 1, 1), (4, 2, 2), (8, 4, 2)])
    K = _log_int(rng, 1, min(8, E // groups * top_groups))
    live = T if rng.random() < 0.6 else rng.randint(1, T)
    return _layer(T, E, K, H, I, live, "sigmoid" if sigmoid else "softmax", groups, top_groups,
                  group_top, rng.choice([1.0, 2.5]), rng.choice([0, 0, 1, 2]), weights,
                  rng.choice(["silu", "silu", "gelu"]))


def work(case):
    if case["kind"] == "layer":
        T, E, K, H, I = case["live"], case["E"], case["K"], case["H"], case["I"]
        # experts that a token reaches, in the mean, under even routing
        active = E * (1.0 - (1.0 - K / E) ** T) + (case["shared"] if T else 0)
        wb = 1 if case["weights"] == "e4m3" else 2
        scales = active * 3 * -(-H // 128) * -(-I // 128) * 4 if wb == 1 else 0
        return {"bytes": active * 3 * H * I * wb + scales + T * (4 * E + 4 * H + 8 * K) + 8,
                "flops": 6.0 * T * (K + case["shared"]) * H * I + 1}
    rows, I = case["T"] * case["K"], case["I"]
    eb = 2 if case["dtype"] == "bf16" else 4
    per_row = 3 * I * eb if case["kind"] == "act" else 5 * I * eb
    score = (4 if case["kind"] == "act" else 8) if case["absorb"] else 0
    return {"bytes": rows * (per_row + score), "flops": rows * I * (12.0 if case["kind"] == "act" else 24.0)}


# ---------------------------------------------------------------------------
# inputs

def _routing(gen, T, E, K):
    """[T, K] distinct experts per token, int32."""
    r = torch.rand(T, E, generator=gen, device="cuda")
    return torch.topk(r, K, dim=1).indices.to(torch.int32)


def _rows_of(idx, E, pad):
    """Entry t*K + k of every receive row (-1: pad row or beyond the last
    segment), and whether the row lies in a segment; rows are grouped by
    expert, stable by entry, segments rounded up to `pad` rows."""
    n = idx.numel()
    order = torch.argsort(idx.reshape(-1), stable=True)
    cnt = torch.bincount(idx.reshape(-1), minlength=E)
    seg = (cnt + pad - 1) // pad * pad
    first = torch.cumsum(cnt, 0) - cnt
    start = torch.cumsum(seg, 0) - seg
    e = idx.reshape(-1)[order].long()
    row = start[e] + torch.arange(n, device="cuda") - first[e]
    entry = torch.full((n + E * (pad - 1),), -1, dtype=torch.int64, device="cuda")
    entry[row] = order
    inside = torch.arange(entry.numel(), device="cuda") < seg.sum()
    return entry, inside


def _prepare_act(case, seed):
    T, E, K, I, dt = case["T"], case["E"], case["K"], case["I"], DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    idx = _routing(gen, T, E, K)
    entry, inside = _rows_of(idx, E, case["pad"])
    rows = entry.numel()
    s = dict(case=case, idx=idx, entry=entry, inside=inside,
             gu=torch.empty(rows, 2 * I, dtype=dt, device="cuda").normal_(generator=gen),
             # [seed, offset] of the dropout generator, one pair per step
             rng=torch.tensor([seed * 1000003 + 17, 5 * seed + 1], dtype=torch.int64, device="cuda"),
             recv_w=None)
    if case["absorb"]:
        s["recv_w"] = torch.rand(rows, generator=gen, device="cuda") * 0.5
    out = torch.full((rows, I if case["kind"] == "act" else 2 * I), 0.5, dtype=dt, device="cuda")
    if case["kind"] == "act":
        s["hs"] = out
    else:
        s["ggu"] = out
        s["ghs"] = torch.empty(rows, I, dtype=dt, device="cuda").normal_(generator=gen)
        s["gw"] = torch.zeros(T, K, device="cuda") if case["absorb"] else None
    if own:
        import combine_moe_route_05_gb300 as moe
        s["router"] = moe.MoeRouter(E, K, 1, T, pad_align=case["pad"])
        s["router"].layout(idx)
    return s


def _weights(gen, shape, fan_in, kind):
    """Weights of standard deviation fan_in^-1/2, and their block scales."""
    if kind == "bf16":
        w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return w.normal_(0.0, fan_in ** -0.5, generator=gen), None
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(shape[0]):
        v = torch.empty(shape[1:], dtype=torch.bfloat16, device="cuda").normal_(0.0, 100.0, generator=gen)
        q[e] = v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    blocks = (shape[0], -(-shape[1] // 128), -(-shape[2] // 128))
    s = (torch.rand(blocks, generator=gen, device="cuda") + 0.5) * (0.01 * fan_in ** -0.5)
    return q, s


def _prepare_layer(case, seed):
    T, E, K, H, I = case["T"], case["E"], case["K"], case["H"], case["I"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case, bias=None, live=None,
             x=torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen),
             logits=torch.randn(T, E, generator=gen, device="cuda"))
    if case["score"] == "sigmoid":
        s["bias"] = 0.01 * torch.randn(E, generator=gen, device="cuda")
    n = E + case["shared"]
    s["w13"], s["s13"] = _weights(gen, (n, 2 * I, H), H, case["weights"])
    s["w2"], s["s2"] = _weights(gen, (n, H, I), I, case["weights"])
    # a decode loop's own buffers; places behind the live requests keep theirs
    s["out"] = torch.full((T, H), 0.25, dtype=torch.bfloat16, device="cuda")
    s["idx"] = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    s["w"] = torch.zeros(T, K, device="cuda")
    if case["live"] < T:
        s["live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
        s["logits"][case["live"]:] = float("nan")
    if own:
        import combine_moe_route_05_gb300 as moe
        s["router"] = moe.MoeRouter(E, K, 1, T, score_fn=case["score"], num_groups=case["groups"],
                                    topk_groups=case["top_groups"],
                                    group_score_topk=case["group_top"], route_scale=case["scale"])
        s["workspace"] = moe.layer_workspace(s["router"].h, H, I, case["shared"])
    return s


def prepare(case, seed):
    return _prepare_layer(case, seed) if case["kind"] == "layer" else _prepare_act(case, seed)


# ---------------------------------------------------------------------------
# one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_layer(state) if kind == "layer" else _own_act(state)
    if kind == "layer":
        return _plain_layer(state)
    return _plain_act(state) if kind == "act" else _plain_act_bwd(state)


def _own_act(s):
    import combine_moe_route_05_gb300 as moe
    c, h = s["case"], s["router"].h
    if c["kind"] == "act":
        moe.moe_act_rows(h, s["gu"], s["recv_w"], s["hs"], act=c["act"], p=c["p"], rng=s["rng"])
        return s["hs"]
    moe.moe_act_rows_bwd(h, s["ghs"], s["gu"], s["recv_w"], s["ggu"], s["gw"], act=c["act"],
                         p=c["p"], rng=s["rng"])
    return {"ggu": s["ggu"], "gw": s["gw"]} if c["absorb"] else {"ggu": s["ggu"]}


def _own_layer(s):
    import combine_moe_route_05_gb300 as moe
    c = s["case"]
    moe.moe_layer(s["router"].h, s["x"], s["logits"], s["w13"], s["w2"], s["out"], s["idx"], s["w"],
                  s["workspace"], bias=s["bias"], s13=s["s13"], s2=s["s2"], live=s["live"],
                  act=c["act"], num_shared=c["shared"])
    return {"out": s["out"], "idx": s["idx"], "w": s["w"]}


# Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
# as 1, 2, 3", 2011) on 32-bit values held in int64.
_LOW = 0xFFFFFFFF


def _philox_round(state, r):
    c0, c1, c2, c3, k0, k1 = state
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return ((p1 >> 32) & _LOW ^ c1 ^ k0, p1 & _LOW, (p0 >> 32) & _LOW ^ c3 ^ k1, p0 & _LOW,
            (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW)


def _kept(entry, I, p, rng):
    """[rows, I] mask of kept elements: element i of entry (t*K + k) compares 16
    bits of the Philox block (i div 8, entry, offset) under key seed."""
    drop = round(p * 65536)
    vec = torch.arange(-(-I // 8), device=entry.device)
    zero = torch.zeros(entry.numel(), vec.numel(), dtype=torch.int64, device=entry.device)
    start = (zero + vec, zero + entry.clamp(min=0)[:, None], zero + (rng[1] & _LOW),
             zero + ((rng[1] >> 32) & _LOW), rng[0] & _LOW, (rng[0] >> 32) & _LOW)
    words = torch.stack(functools.reduce(_philox_round, range(10), start)[:4], -1)
    halves = torch.stack((words & 0xFFFF, words >> 16), -1)
    return halves.reshape(entry.numel(), -1)[:, :I] >= drop, 65536.0 / (65536 - drop)


def _slope(act, g):
    """sigmoid argument c(g) of g * sigmoid(c(g)), and its derivative."""
    if act == "silu":
        return g, torch.ones_like(g)
    r = 2.0 * math.sqrt(2.0 / math.pi)
    return r * (g + 0.044715 * g * g * g), r * (1.0 + 3 * 0.044715 * g * g)


def _masked(v, case, s):
    """v with dropout: dropped elements are 0, kept ones scaled."""
    if case["p"] == 0.0:
        return v
    kept, scale = _kept(s["entry"], case["I"], case["p"], s["rng"])
    return torch.where(kept, v * scale, torch.zeros_like(v))


def _into(s, buffer, v):
    """Rows of entries get v, pad rows of the segments 0; rows behind the last
    segment keep what they hold."""
    v = torch.where((s["entry"] >= 0)[:, None], v, torch.zeros_like(v)).to(buffer.dtype)
    return torch.where(s["inside"][:, None], v, buffer)


def _plain_act(s):
    c = s["case"]
    g, u = s["gu"].float().split(c["I"], 1)
    v = _masked(g / (1.0 + torch.exp(-_slope(c["act"], g)[0])) * u, c, s)
    if c["absorb"]:
        v = v * s["recv_w"][:, None]
    return _into(s, s["hs"], v)


def _plain_act_bwd(s):
    c = s["case"]
    g, u = s["gu"].float().split(c["I"], 1)
    arg, darg = _slope(c["act"], g)
    sig = 1.0 / (1.0 + torch.exp(-arg))
    d = _masked(s["ghs"].float(), c, s)
    dw = d * s["recv_w"][:, None] if c["absorb"] else d
    ggu = torch.cat((dw * u * (sig + g * sig * (1.0 - sig) * darg), dw * g * sig), 1)
    out = {"ggu": _into(s, s["ggu"], ggu)}
    if c["absorb"]:
        gw = torch.zeros_like(s["gw"]).reshape(-1)
        rows = (d * g * sig * u).sum(1)
        live = s["entry"] >= 0
        gw.index_put_((s["entry"].clamp(min=0),), torch.where(live, rows, 0.0), accumulate=True)
        out["gw"] = gw.reshape(s["gw"].shape)
    return out


def _select(case, logits, bias):
    """Experts in descending key order (ties to the lower index) and their
    weights, on fp64 keys."""
    l = logits.double()
    if case["score"] == "softmax":
        vals, idx = torch.sort(l, dim=1, descending=True, stable=True)
        e = torch.exp(vals[:, :case["K"]] - vals[:, :1])
        return idx[:, :case["K"]], e / e.sum(1, keepdim=True) * case["scale"]
    sig = 1.0 / (1.0 + torch.exp(-l))
    key = sig + bias.double()
    if case["groups"] > 1:
        per = key.reshape(key.shape[0], case["groups"], -1)
        score = torch.sort(per, dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        rank = torch.argsort(torch.argsort(score, dim=1, descending=True, stable=True), dim=1)
        key = torch.where((rank < case["top_groups"])[:, :, None], per, -math.inf).reshape(key.shape)
    idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["K"]]
    v = torch.gather(sig, 1, idx)
    return idx, v / v.sum(1, keepdim=True) * case["scale"]


def _values(w, scale, at=None):
    """fp32 values of the weights of experts `at` (all: None)."""
    v = (w if at is None else w.view(torch.uint8)[at].view(w.dtype) if scale is not None else w[at]).float()
    if scale is None:
        return v
    sc = scale if at is None else scale[at]
    sc = sc.repeat_interleave(128, 1)[:, :v.shape[1]].repeat_interleave(128, 2)[:, :, :v.shape[2]]
    return v.mul_(sc)


def _experts(case, x, s, at=None):
    """x [n, m, H] through n experts: [n, m, H] fp32."""
    g, u = torch.bmm(x, _values(s["w13"], s["s13"], at).transpose(1, 2)).split(case["I"], 2)
    a = g / (1.0 + torch.exp(-_slope(case["act"], g)[0])) * u
    return torch.bmm(a, _values(s["w2"], s["s2"], at).transpose(1, 2))


def _plain_layer(s):
    c = s["case"]
    live, E, n = c["live"], c["E"], c["E"] + c["shared"]
    idx, w = _select(c, s["logits"][:live], s["bias"])
    x = s["x"][:live].float()
    full_idx = torch.cat((idx, torch.arange(E, n, device="cuda").expand(live, -1)), 1)
    full_w = torch.cat((w, torch.ones(live, c["shared"], dtype=w.dtype, device="cuda")), 1).float()
    if full_idx.numel() < n:  # the weights of each entry's expert
        y = _experts(c, x.repeat_interleave(full_idx.shape[1], 0)[:, None, :], s, full_idx.reshape(-1))
        y = (y.reshape(live, -1, c["H"]) * full_w[:, :, None]).sum(1)
    else:                     # every expert on every token, weighted
        dense = torch.zeros(live, n, device="cuda").scatter_(1, full_idx, full_w)
        y = torch.einsum("eth,te->th", _experts(c, x.expand(n, -1, -1), s), dense)
    return {"out": torch.cat((y.to(torch.bfloat16), s["out"][live:])),
            "idx": torch.cat((idx.to(torch.int32), s["idx"][live:])),
            "w": torch.cat((w.float(), s["w"][live:]))}


# ---------------------------------------------------------------------------
# exact forms: the definitions in fp64

def _mul32(a, m):
    """High and low 32 bits of a * m by 16-bit limbs (a: int64 tensor below 2^32)."""
    ah, al, mh, ml = a >> 16, a & 0xFFFF, m >> 16, m & 0xFFFF
    mid = al * mh + (al * ml >> 16)
    t = ah * ml + (mid & 0xFFFF)
    return ah * mh + (mid >> 16) + (t >> 16), ((t & 0xFFFF) << 16) | (al * ml & 0xFFFF)


def _exact_kept(rows_entry, I, drop, seed, offset):
    """Kept elements of the given entries, one Philox word at a time."""
    n, m = rows_entry.numel(), (I + 7) // 8
    c = [torch.arange(m, device="cuda").repeat(n, 1), rows_entry[:, None].repeat(1, m),
         torch.full((n, m), offset % 2 ** 32, device="cuda"),
         torch.full((n, m), offset // 2 ** 32 % 2 ** 32, device="cuda")]
    k = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for _ in range(10):
        h0, l0 = _mul32(c[0], 0xD2511F53)
        h1, l1 = _mul32(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    kept = torch.empty(n, m, 8, dtype=torch.bool, device="cuda")
    for j in range(8):
        kept[:, :, j] = (c[j // 2] // (65536 if j % 2 else 1)) % 65536 >= drop
    return kept.reshape(n, -1)[:, :I]


def _exact_act(case, seed):
    s = _prepare_act(case, seed)
    I = case["I"]
    drop = int(math.floor(case["p"] * 65536 + 0.5))
    seed64, off64 = (int(v) for v in s["rng"].tolist())
    out = s["hs" if case["kind"] == "act" else "ggu"].double()
    out[s["inside"]] = 0.0
    gw = torch.zeros(case["T"] * case["K"], dtype=torch.float64, device="cuda")
    rows = torch.nonzero(s["entry"] >= 0).reshape(-1)
    for r in rows.split(max(1, (1 << 25) // I)):
        e = s["entry"][r]
        g, u = s["gu"][r, :I].double(), s["gu"][r, I:].double()
        m = _exact_kept(e, I, drop, seed64, off64).double() * (65536.0 / (65536 - drop))
        w = s["recv_w"][r].double()[:, None] if case["absorb"] else 1.0
        if case["act"] == "silu":
            sg = torch.sigmoid(g)
            a, da = g * sg, sg * (1.0 + g * (1.0 - sg))
        else:
            z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
            th = torch.tanh(z)
            a = 0.5 * g * (1.0 + th)
            da = 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * g * g)
        if case["kind"] == "act":
            out[r] = w * m * a * u
        else:
            d = s["ghs"][r].double() * m
            out[r, :I] = d * w * u * da
            out[r, I:] = d * w * a
            gw[e] = (d * a * u).sum(1)
    if case["kind"] == "act":
        return out
    return {"ggu": out, "gw": gw.reshape(case["T"], case["K"])} if case["absorb"] else {"ggu": out}


def _exact_layer(case, seed):
    s = _prepare_layer(case, seed)
    live, E, K, I = case["live"], case["E"], case["K"], case["I"]
    out, w_out = s["out"].double(), s["w"].double()
    out[:live] = 0.0
    l = s["logits"][:live].double()
    sig = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = (sig + s["bias"].double() if case["score"] == "sigmoid" else l).cpu()
    per = E // case["groups"]
    chosen = []
    for t in range(live):
        row = key[t].tolist()
        best = [sorted(row[g * per:(g + 1) * per], reverse=True) for g in range(case["groups"])]
        score = [sum(b[:case["group_top"]]) for b in best]
        ok = sorted(range(case["groups"]), key=lambda g: (-score[g], g))[:case["top_groups"]]
        pick = sorted((e for e in range(E) if e // per in ok), key=lambda e: (-row[e], e))[:K]
        chosen.append(pick)
    if live:
        at = torch.tensor(chosen, device="cuda")
        v = torch.gather(sig, 1, at)
        w_out[:live] = v / v.sum(1, keepdim=True) * case["scale"]
    tokens = {}
    for t, pick in enumerate(chosen):
        for k, e in enumerate(pick):
            tokens.setdefault(e, []).append((t, k))
    for j in range(case["shared"] if live else 0):
        tokens[E + j] = [(t, -1) for t in range(live)]
    x = s["x"].double()
    for e, pairs in tokens.items():
        t = torch.tensor([p[0] for p in pairs], device="cuda")
        k = torch.tensor([p[1] for p in pairs], device="cuda")
        w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        if s["s13"] is not None:
            w13 *= torch.kron(s["s13"][e].double(), torch.ones(128, 128, device="cuda"))[:w13.shape[0], :w13.shape[1]]
            w2 *= torch.kron(s["s2"][e].double(), torch.ones(128, 128, device="cuda"))[:w2.shape[0], :w2.shape[1]]
        z = x[t] @ w13.T
        g, u = z[:, :I], z[:, I:]
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
        weight = torch.where(k >= 0, w_out[t, k.clamp(min=0)], 1.0)
        out.index_add_(0, t, ((a * u) @ w2.T) * weight[:, None])
    return {"out": out, "idx": None, "w": w_out}


def exact(case, seed):
    return _exact_layer(case, seed) if case["kind"] == "layer" else _exact_act(case, seed)
