"""Cases, plain forms and exact forms of the router's balance loss (forward and
backward) and of the norms around the MoE block (forward and backward).

A case of kind "balance" or "balance_bwd" is one balance loss over a batch of
packed sequences, or its gradient to the router logits.  A case of kind "norm"
or "norm_bwd" is one block boundary: the block's output rows (or the weighted
sum of their receive rows), normed, gated and added to the residual stream, and
the next block's norm; or its backward.  Where ``own`` is true, ``run`` calls
the library; otherwise it computes the same results from elementary torch
operations in fp32, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases

def _balance(kind, T, E, K, score="softmax", seqs=1, live=None, drop=0.0, base=False):
    """seqs: packed sequences over the first `live` tokens (1 and live None: one
    sequence, no offsets); drop: share of entries without an expert; base: the
    gradient is added to the routing's own."""
    return dict(kind=kind, T=T, E=E, K=K, score=score, seqs=seqs, live=T if live is None else live,
                drop=drop, base=base)


def _norm(kind, T, H, dtype="bf16", weights="bf16", K=0, E=8, add=False, post=True, pre=True,
          gate=0, save=False, scale=1.0, offset=0.0):
    """K: entries of a token whose receive rows are summed (0: token rows); gate:
    tokens to a row of the gate (0: none); save: what the backward needs is kept
    (the sums of rows, where there are any, and the norms' factors)."""
    return dict(kind=kind, T=T, H=H, dtype=dtype, weights=weights, K=K, E=E, add=add, post=post,
                pre=pre, gate=gate, save=save, scale=scale, offset=offset)


def listed():
    return [
        # the tiny workload's router: bound by the launches
        dict(_balance("balance", 256, 8, 2), name="balance tiny"),
        # a DeepSeek-V3-shaped training batch: sequence-wise loss over packed
        # sequences of different lengths, some places left empty behind them
        dict(_balance("balance", 16384, 256, 8, "sigmoid", seqs=9, live=15000),
             name="balance packed deepseek-v3"),
        # the largest router: a batch of 131072 tokens, 512 experts, and a few
        # entries that a capacity limit dropped
        dict(_balance("balance", 131072, 512, 8, drop=0.02), name="balance 131072 tokens 512 experts"),
        # its gradient on the Qwen3-30B-A3B-shaped router, the batch as one sequence
        dict(_balance("balance_bwd", 8192, 128, 8), name="balance_bwd qwen3-30b"),
        # packed sequences, added to the gradient that the routing weights left
        dict(_balance("balance_bwd", 16384, 256, 8, "sigmoid", seqs=9, live=15000, base=True),
             name="balance_bwd packed deepseek-v3"),
        # one user's next token between two layers: latency counts
        dict(_norm("norm", 1, 2048), name="norm 1 token"),
        # inference over a prompt in a model without post-norms: residual sum and
        # the next norm
        dict(_norm("norm", 8192, 2048, post=False), name="norm qwen3-30b"),
        # fp32 rows of a width that fills no power of two, weights stored as
        # their distance from 1, an own gate row per token
        dict(_norm("norm", 1500, 1000, "f32", "f32", gate=1, save=True, scale=0.5, offset=1.0),
             name="norm ragged f32"),
        # a training step's combine with shared experts, post-norm and next
        # pre-norm, what the backward needs kept
        dict(_norm("norm", 16384, 7168, K=8, E=256, add=True, save=True),
             name="norm combined deepseek-v3"),
        # backward of a small fp32 layer, one gate vector for all tokens
        dict(_norm("norm_bwd", 256, 256, "f32", "f32", gate=256), name="norm_bwd tiny f32"),
        # backward on the Qwen3-30B-A3B shape, a gate row for each of 7 images'
        # tokens (conditioned blocks), the last one shorter
        dict(_norm("norm_bwd", 8192, 2048, gate=1300, scale=0.7), name="norm_bwd gated qwen3-30b"),
        # backward of the largest training batch
        dict(_norm("norm_bwd", 16384, 7168), name="norm_bwd deepseek-v3"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["balance", "balance_bwd", "norm", "norm", "norm_bwd"])
    if kind.startswith("balance"):
        E = _log_int(rng, 4, 512)
        K = _log_int(rng, 1, min(E, 16))
        T = _log_int(rng, 1, min(131072, (1 << 25) // E))
        live = T if rng.random() < 0.5 else rng.randint(1, T)
        return _balance(kind, T, E, K, rng.choice(["softmax", "sigmoid"]),
                        1 if live == T and rng.random() < 0.5 else _log_int(rng, 1, max(1, min(64, T))),
                        live, rng.choice([0.0, 0.02, 0.3]), kind == "balance_bwd" and rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H = _log_int(rng, 64, 8192, 8)
    K = rng.choice([0, 0, _log_int(rng, 1, 8)]) if kind == "norm" else 0
    T = _log_int(rng, 1, min(16384, (1 << 25) // (H * max(1, K))))
    post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
    gate = rng.choice([0, 0, 1, T, _log_int(rng, 1, T)])
    return _norm(kind, T, H, dtype, rng.choice(["bf16", "f32"]), K, _log_int(rng, max(4, K), 256),
                 kind == "norm" and rng.random() < 0.4, post, pre, gate, rng.random() < 0.5,
                 rng.choice([1.0, 1.0, 0.5]), rng.choice([0.0, 1.0]))


def work(case):
    T, K = case["T"], case["K"]
    if case["kind"].startswith("balance"):
        live, E, S = case["live"], case["E"], case["seqs"]
        if case["kind"] == "balance":
            return {"bytes": live * (4 * E + 4 * K) + S * 4 * (2 * E + 1) + 4, "flops": live * E * 6.0 + 1}
        return {"bytes": live * 4 * E * (3 if case["base"] else 2) + S * 4 * (E + 1) + 4,
                "flops": live * E * 9.0 + 1}
    H, eb = case["H"], 2 if case["dtype"] == "bf16" else 4
    wb = 2 if case["weights"] == "bf16" else 4
    G = 0 if case["gate"] == 0 else -(-T // case["gate"])
    if case["kind"] == "norm":
        rows = T * (max(1, K) + case["add"] + 2 + case["pre"] +
                    (case["save"] and (K > 0 or case["add"]))) + G
        small = (case["post"] + case["pre"]) * H * wb + T * K * 8 + (8 * T if case["save"] else 0)
        return {"bytes": rows * H * eb + small, "flops": T * H * (2.0 * K + 12)}
    # gradients of the residual stream and the norm, their rows, two gradients back
    rows = T * (1 + 2 * case["pre"] + (case["post"] or G > 0) + 2) + 2 * G
    return {"bytes": rows * H * eb + (case["post"] + case["pre"]) * H * (wb + 4) + 8 * T,
            "flops": T * H * 24.0}


# ---------------------------------------------------------------------------
# inputs

def _routing(gen, T, E, K):
    """[T, K] distinct experts per token, int32."""
    r = torch.rand(T, E, generator=gen, device="cuda")
    return torch.topk(r, K, dim=1).indices.to(torch.int32)


def _offsets(case, seed):
    """Sequence offsets over the live tokens, some sequences perhaps empty."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, case["live"] + 1, (case["seqs"] - 1,), generator=g)
    ends = torch.tensor([0, case["live"]])
    return torch.sort(torch.cat((cuts, ends))).values.to(torch.int32)


def _prepare_balance(case, seed):
    T, E, K = case["T"], case["E"], case["K"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case, coef=0.01, off=None, base=None,
             logits=torch.randn(T, E, generator=gen, device="cuda"))
    # some experts are more popular than others
    s["logits"] += torch.randn(E, generator=gen, device="cuda")
    s["idx"] = torch.topk(s["logits"] + 0.5 * torch.randn(T, E, generator=gen, device="cuda"), K,
                          dim=1).indices.to(torch.int32)
    if case["drop"]:
        s["idx"].masked_fill_(torch.rand(T, K, generator=gen, device="cuda") < case["drop"], -1)
    if case["seqs"] > 1 or case["live"] < T:
        s["off"] = _offsets(case, seed).cuda()
        s["logits"][case["live"]:] = float("nan")  # places that hold nothing
    if case["kind"] == "balance":
        s["loss"] = torch.zeros(1, device="cuda")
        s["cnt"] = torch.zeros(case["seqs"], E, dtype=torch.int32, device="cuda")
        s["prob"] = torch.zeros(case["seqs"], E, device="cuda")
    else:
        s["cnt"] = _counts(s)
        # the gradient of a scaled loss, and the gradient buffer of a training
        # loop; empty places keep what it holds
        s["gloss"] = 65536.0 * (torch.rand(1, generator=gen, device="cuda") + 0.5)
        s["glogits"] = torch.full((T, E), 1e-4, device="cuda")
        if case["base"]:
            s["base"] = 1e-4 * torch.randn(T, E, generator=gen, device="cuda")
    if own:
        import combine_moe_route_05_gb300 as moe
        s["router"] = moe.MoeRouter(E, K, 1, T, score_fn=case["score"])
        s["workspace"] = moe.balance_workspace(s["router"].h, case["seqs"])
    return s


def _positions(idx, E):
    """Receive row of every entry: rows grouped by expert, stable by entry."""
    order = torch.argsort(idx.reshape(-1), stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return pos.reshape(idx.shape)


def _prepare_norm(case, seed):
    T, H, K, dt, wt = case["T"], case["H"], case["K"], DTYPES[case["dtype"]], DTYPES[case["weights"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rows(n, std=1.0):
        return torch.empty(n, H, dtype=dt, device="cuda").normal_(0.0, std, generator=gen)

    def weight():
        return (torch.rand(H, generator=gen, device="cuda") + (0.5 - case["offset"])).to(wt)

    s = dict(case=case, eps=1e-6, add=None, gate=None, cw=None, w_post=None, w_pre=None)
    if case["post"]:
        s["w_post"] = weight()
    if case["pre"]:
        s["w_pre"] = weight()
    if case["gate"]:
        s["gate"] = rows(-(-T // case["gate"]), 0.5)
    E, router = max(case["E"], K), None
    if own:
        import combine_moe_route_05_gb300 as moe
        router = moe.MoeRouter(E, max(1, K), 1, T)
        s["router"] = router
    if case["kind"] == "norm":
        s["res"] = rows(T, 2.0)
        if K:
            idx = _routing(gen, T, E, K)
            s["pos"] = _positions(idx, E)
            s["cw"] = torch.rand(T, K, generator=gen, device="cuda") * (2.0 / K)
            if own:
                router.layout(idx)
        s["y"] = rows(T * max(1, K))
        if case["add"]:
            s["add"] = rows(T)
        # buffers that the call fills
        s["res_out"] = torch.empty_like(s["res"])
        s["x"] = torch.empty_like(s["res"]) if case["pre"] else None
        s["c"] = torch.empty_like(s["res"]) if case["save"] and (K or case["add"]) else None
        for k, on in (("rstd_post", case["post"]), ("rstd_pre", case["pre"])):
            s[k] = torch.empty(T, device="cuda") if case["save"] and on else None
        return s
    s["gres_out"] = rows(T)
    s["gx"] = rows(T) if case["pre"] else None
    s["res_out"] = rows(T, 2.0) if case["pre"] else None
    s["c"] = rows(T) if case["post"] or case["gate"] else None
    for k, v in (("rstd_post", s["c"] if case["post"] else None), ("rstd_pre", s["res_out"])):
        s[k] = None if v is None else 1.0 / torch.sqrt((v.float() ** 2).mean(1) + s["eps"])
    s["gres"] = torch.empty_like(s["gres_out"])
    s["gy"] = torch.empty_like(s["gres_out"])
    s["ggate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    s["gw_post"] = torch.empty(H, device="cuda") if case["post"] else None
    s["gw_pre"] = torch.empty(H, device="cuda") if case["pre"] else None
    if own:
        s["workspace"] = moe.block_norm_workspace(router.h, T, H, max(1, case["gate"]))
    return s


def prepare(case, seed):
    return (_prepare_balance if case["kind"].startswith("balance") else _prepare_norm)(case, seed)


# ---------------------------------------------------------------------------
# one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"balance": _own_balance, "balance_bwd": _own_balance_bwd, "norm": _own_norm,
                "norm_bwd": _own_norm_bwd}[kind](state)
    return {"balance": _plain_balance, "balance_bwd": _plain_balance_bwd, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd}[kind](state)


def _given(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _own_balance(s):
    import combine_moe_route_05_gb300 as moe
    moe.moe_balance(s["router"].h, s["logits"], s["idx"], s["loss"], s["cnt"], s["workspace"],
                    prob=s["prob"], seq_off=s["off"], coef=s["coef"])
    return {"loss": s["loss"], "cnt": s["cnt"], "prob": s["prob"]}


def _own_balance_bwd(s):
    import combine_moe_route_05_gb300 as moe
    moe.moe_balance_bwd(s["router"].h, s["logits"], s["cnt"], s["glogits"], seq_off=s["off"],
                        coef=s["coef"], gloss=s["gloss"], base=s["base"])
    return s["glogits"]


def _own_norm(s):
    import combine_moe_route_05_gb300 as moe
    c = s["case"]
    moe.moe_block_norm(s["router"].h, s["res"], s["res_out"], s["x"], y=s["y"], gather=c["K"] > 0,
                       cw=s["cw"], add=s["add"], gate=s["gate"], gate_tokens=max(1, c["gate"]),
                       w_post=s["w_post"], w_pre=s["w_pre"], c=s["c"], rstd_post=s["rstd_post"],
                       rstd_pre=s["rstd_pre"], res_scale=c["scale"], eps=s["eps"],
                       weight_offset=c["offset"])
    return _given(res_out=s["res_out"], x=s["x"], c=s["c"], rstd_post=s["rstd_post"],
                  rstd_pre=s["rstd_pre"])


def _own_norm_bwd(s):
    import combine_moe_route_05_gb300 as moe
    c = s["case"]
    moe.moe_block_norm_bwd(s["router"].h, s["workspace"], gres_out=s["gres_out"], gx=s["gx"],
                           res_out=s["res_out"], c=s["c"], gate=s["gate"],
                           gate_tokens=max(1, c["gate"]), w_post=s["w_post"], w_pre=s["w_pre"],
                           rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], gres=s["gres"],
                           gy=s["gy"], ggate=s["ggate"], gw_post=s["gw_post"], gw_pre=s["gw_pre"],
                           res_scale=c["scale"], weight_offset=c["offset"])
    return _given(gres=s["gres"], gy=s["gy"], ggate=s["ggate"], gw_post=s["gw_post"],
                  gw_pre=s["gw_pre"])


def _sequence_of(s):
    """Sequence of each live token, and the sequences' lengths."""
    live, dev = s["case"]["live"], s["logits"].device
    if s["off"] is None:
        return torch.zeros(live, dtype=torch.int64, device=dev), torch.full((1,), live, device=dev)
    off = s["off"].long()
    n = off[1:] - off[:-1]
    t = torch.arange(live, device=dev)
    return (t[:, None] >= off[None, 1:]).sum(1), n


def _counts(s):
    c, (seq, _) = s["case"], _sequence_of(s)
    idx = s["idx"][:c["live"]].long()
    cnt = torch.zeros(c["seqs"] * c["E"], dtype=torch.int32, device=idx.device)
    cell = (seq[:, None] * c["E"] + idx)[idx >= 0]
    return cnt.index_add_(0, cell, torch.ones_like(cell, dtype=torch.int32)).reshape(c["seqs"], -1)


def _scores(case, l):
    """Scores before normalisation: e^(l - max), or the sigmoid."""
    if case["score"] == "softmax":
        return torch.exp(l - l.max(1, keepdim=True).values)
    return 1.0 / (1.0 + torch.exp(-l))


def _per_sequence(s, n):
    """Factor of each sequence's sum over its experts of counts times sums of p."""
    c = s["case"]
    f = torch.where(n > 0, c["E"] / (c["K"] * n.clamp(min=1).float() ** 2), 0.0)
    return f * (s["coef"] / (n > 0).sum().clamp(min=1))


def _plain_balance(s):
    c = s["case"]
    seq, n = _sequence_of(s)
    v = _scores(c, s["logits"][:c["live"]])
    p = v / v.sum(1, keepdim=True)
    if c["seqs"] == 1:
        P = p.sum(0, keepdim=True)
    else:
        P = torch.zeros(c["seqs"], c["E"], device=p.device).index_add_(0, seq, p)
    cnt = _counts(s)
    return {"loss": (_per_sequence(s, n) * (cnt.float() * P).sum(1)).sum().reshape(1), "cnt": cnt,
            "prob": P / n.clamp(min=1)[:, None]}


def _plain_balance_bwd(s):
    c = s["case"]
    seq, n = _sequence_of(s)
    v = _scores(c, s["logits"][:c["live"]])
    p = v / v.sum(1, keepdim=True)
    cnt = s["cnt"].float()[seq]
    slope = p if c["score"] == "softmax" else p * (1.0 - v)
    g = slope * (cnt - (cnt * p).sum(1, keepdim=True)) * (_per_sequence(s, n) * s["gloss"])[seq][:, None]
    if c["base"]:
        g = g + s["base"][:c["live"]]
    return torch.cat((g, s["glogits"][c["live"]:]))


def _gate_rows(s):
    """The gate's row of each token, fp32."""
    c = s["case"]
    return s["gate"].float()[torch.arange(c["T"], device=s["gate"].device) // c["gate"]]


def _weight(s, name):
    return s[name].float() + s["case"]["offset"]


def _rstd(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1) + eps)


def _plain_norm(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if case["K"]:
        c = torch.zeros(case["T"], case["H"], device=s["y"].device)
        for k in range(case["K"]):
            c += s["cw"][:, k, None] * s["y"][s["pos"][:, k]].float()
    else:
        c = s["y"].float()
    if case["add"]:
        c = c + s["add"].float()
    u, out = c, {}
    if case["post"]:
        out["rstd_post"] = _rstd(c, s["eps"])
        u = c * out["rstd_post"][:, None] * _weight(s, "w_post")
    if case["gate"]:
        u = u * _gate_rows(s)
    res = case["scale"] * s["res"].float() + u
    x = None
    if case["pre"]:
        out["rstd_pre"] = _rstd(res, s["eps"])
        x = (res * out["rstd_pre"][:, None] * _weight(s, "w_pre")).to(dt)
    if not case["save"]:
        return _given(res_out=res.to(dt), x=x)
    return _given(res_out=res.to(dt), x=x, c=None if s["c"] is None else c.to(dt), **out)


def _plain_norm_bwd(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    D, out = s["gres_out"].float(), {}
    if case["pre"]:
        r = s["rstd_pre"][:, None]
        hat, gx = s["res_out"].float() * r, s["gx"].float()
        v = gx * _weight(s, "w_pre")
        D = D + r * (v - hat * (v * hat).mean(1, keepdim=True))
        out["gw_pre"] = (gx * hat).sum(0)
    out["gres"] = (case["scale"] * D).to(dt)
    hat = None if s["c"] is None else s["c"].float()
    if case["post"]:
        hat = hat * s["rstd_post"][:, None]
    U = D
    if case["gate"]:
        U = D * _gate_rows(s)
        v = D * hat * _weight(s, "w_post") if case["post"] else D * hat
        group = torch.arange(case["T"], device=v.device) // case["gate"]
        sums = torch.zeros(s["gate"].shape, device=v.device)
        out["ggate"] = (v if case["gate"] == 1 else sums.index_add_(0, group, v)).to(dt)
    if case["post"]:
        out["gw_post"] = (U * hat).sum(0)
        v = U * _weight(s, "w_post")
        U = s["rstd_post"][:, None] * (v - hat * (v * hat).mean(1, keepdim=True))
    out["gy"] = U.to(dt)
    return {k: out[k] for k in ("gres", "gy", "ggate", "gw_post", "gw_pre") if k in out}


# ---------------------------------------------------------------------------
# exact forms: the definitions in fp64

def _exact_probabilities(case, l):
    """p and dp_j / dl_j's own factor, a chunk of tokens' logits in fp64."""
    if case["score"] == "softmax":
        p = torch.softmax(l, 1)
        return p, p
    v = torch.sigmoid(l)
    z = v.sum(1, keepdim=True)
    return v / z, v * torch.sigmoid(-l) / z


def _exact_balance(case, seed):
    s = _prepare_balance(case, seed)
    off = [0, case["live"]] if s["off"] is None else s["off"].tolist()
    E, K = case["E"], case["K"]
    full = [b - a for a, b in zip(off, off[1:]) if b > a]
    loss, prob = 0.0, torch.zeros(case["seqs"], E, dtype=torch.float64, device="cuda")
    glogits = None
    if case["kind"] == "balance_bwd":
        glogits = s["glogits"].double()
    for q, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        chosen = s["idx"][a:b].reshape(-1)
        cnt = torch.bincount(chosen[chosen >= 0].long(), minlength=E).double()
        factor = s["coef"] / len(full) * E / (K * float(b - a) ** 2)
        for t in range(a, b, 16384):
            rows = slice(t, min(t + 16384, b))
            p, own_factor = _exact_probabilities(case, s["logits"][rows].double())
            if glogits is None:
                loss += factor * float((p @ cnt).sum())
                prob[q] += p.sum(0) / (b - a)
            else:
                # sum_e cnt_e dp_e / dl_j
                g = own_factor * (cnt[None, :] - (p @ cnt)[:, None])
                g *= factor * float(s["gloss"])
                glogits[rows] = g + s["base"][rows].double() if case["base"] else g
    if glogits is not None:
        return glogits
    return {"loss": torch.tensor([loss], dtype=torch.float64), "cnt": None, "prob": prob}


def _exact_norm(case, seed):
    s = _prepare_norm(case, seed)
    T, H, K = case["T"], case["H"], case["K"]
    parts = []
    wp, wn = ((None if s[k] is None else s[k].double() + case["offset"]) for k in ("w_post", "w_pre"))
    for t in range(0, T, 1024):
        r = slice(t, min(t + 1024, T))
        n = r.stop - r.start
        if K:
            y = s["y"][s["pos"][r].reshape(-1)].reshape(n, K, H).double()
            c = torch.einsum("tk,tkh->th", s["cw"][r].double(), y)
        else:
            c = s["y"][r].double()
        if case["add"]:
            c = c + s["add"][r].double()
        part = {"c": c}
        u = c
        if case["post"]:
            part["rstd_post"] = (c.square().sum(1) / H + s["eps"]).rsqrt()
            u = torch.einsum("th,t,h->th", c, part["rstd_post"], wp)
        if case["gate"]:
            u = u * torch.stack([s["gate"][i // case["gate"]] for i in range(r.start, r.stop)]).double()
        res = s["res"][r].double() * case["scale"] + u
        part["res_out"] = res
        if case["pre"]:
            part["rstd_pre"] = (res.square().sum(1) / H + s["eps"]).rsqrt()
            part["x"] = torch.einsum("th,t,h->th", res, part["rstd_pre"], wn)
        parts.append(part)
    names = ["res_out", "x"] + (["rstd_post", "rstd_pre"] if case["save"] else [])
    names += ["c"] if s["c"] is not None else []
    return {k: torch.cat([p[k] for p in parts]) for k in names if k in parts[0]}


def _exact_norm_bwd(case, seed):
    s = _prepare_norm(case, seed)
    T, H = case["T"], case["H"]
    wp, wn = ((None if s[k] is None else s[k].double() + case["offset"]) for k in ("w_post", "w_pre"))
    gw_post, gw_pre = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    ggate = None if s["gate"] is None else torch.zeros(s["gate"].shape, dtype=torch.float64, device="cuda")
    gres, gy = [], []

    def through(v, row, rstd, w, grad_w):
        """Gradient v of w * row * rstd(row) to the row; adds the weight's."""
        grad_w += torch.einsum("th,th,t->h", v, row, rstd)
        along = torch.einsum("th,th,h->t", v, row, w) / H
        return v * w * rstd[:, None] - row * (along * rstd ** 3)[:, None]

    for t in range(0, T, 1024):
        r = slice(t, min(t + 1024, T))
        D = s["gres_out"][r].double()
        if case["pre"]:
            D = D + through(s["gx"][r].double(), s["res_out"][r].double(), s["rstd_pre"][r].double(),
                            wn, gw_pre)
        gres.append(D * case["scale"])
        c = None if s["c"] is None else s["c"][r].double()
        g = D
        if case["gate"]:
            at = torch.tensor([i // case["gate"] for i in range(r.start, r.stop)], device="cuda")
            u = c if wp is None else torch.einsum("th,t,h->th", c, s["rstd_post"][r].double(), wp)
            ggate.index_add_(0, at, D * u)
            g = D * s["gate"].double()[at]
        gy.append(g if wp is None else through(g, c, s["rstd_post"][r].double(), wp, gw_post))
    return _given(gres=torch.cat(gres), gy=torch.cat(gy), ggate=ggate,
                  gw_post=gw_post if case["post"] else None, gw_pre=gw_pre if case["pre"] else None)


def exact(case, seed):
    if case["kind"].startswith("balance"):
        return _exact_balance(case, seed)
    return (_exact_norm if case["kind"] == "norm" else _exact_norm_bwd)(case, seed)
