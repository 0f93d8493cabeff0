"""The few-token MoE layer on the GPU against its fp64 definition, within the
element-wise bound that tests/expert_ref.py derives; its routing against the
oracle; and the calls around it (padded batches, given routes, graphs, streams,
in place, the separate calls of the same layer)."""
import ctypes
import threading
import time

import numpy as np
import pytest
import torch

import combine_moe_route_05_gb300 as moe
import oracle
from tests import expert_ref as ref
from tests.gpu_util import dev, to_dev, to_host

pytestmark = pytest.mark.gpu


def weights(g, n, I, H, e4m3):
    """(w13, w2, s13, s2) on the device, and their fp64 values."""
    out, scales, vals = [], [], []
    for shape, fan in (((n, 2 * I, H), H), ((n, H, I), I)):
        if not e4m3:
            t = torch.from_numpy(g.standard_normal(shape).astype(np.float32) * fan ** -0.5).to(dev(), torch.bfloat16)
            out.append(t)
            scales.append(None)
            vals.append(t.double().cpu().numpy())
            continue
        q = torch.from_numpy((g.standard_normal(shape) * 100).clip(-448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
        s = ((g.random((n, -(-shape[1] // 128), -(-shape[2] // 128))) + 0.5) * 0.01 * fan ** -0.5).astype(np.float32)
        big = np.repeat(np.repeat(s, 128, 1), 128, 2)[:, :shape[1], :shape[2]]
        out.append(q.to(dev()))
        scales.append(torch.from_numpy(s).to(dev()))
        vals.append(q.double().numpy() * big)
    return out + scales, vals


class Problem:
    def __init__(self, T, E, K, H, I, shared=0, e4m3=False, act="silu", score="softmax", groups=1,
                 top_groups=1, group_top=1, scale=1.0, renorm=True, seed=0, max_tokens=None):
        g = np.random.default_rng(seed)
        self.T, self.E, self.K, self.H, self.I, self.S, self.act = T, E, K, H, I, shared, act
        self.r = moe.MoeRouter(E, K, 1, max_tokens or T, score_fn=score, num_groups=groups,
                               topk_groups=top_groups, group_score_topk=group_top, renorm=renorm,
                               route_scale=scale)
        (self.w13, self.w2, self.s13, self.s2), (self.v13, self.v2) = weights(g, E + shared, I, H, e4m3)
        self.x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(dev(), torch.bfloat16)
        self.logits = g.standard_normal((T, E)).astype(np.float32)
        self.bias = (g.standard_normal(E) * 0.01).astype(np.float32) if score == "sigmoid" else None
        if score == "sigmoid":
            self.route = oracle.route_sigmoid_grouped(self.logits, self.bias, K, groups, top_groups,
                                                      group_top, renorm, scale) if T else None
        else:
            self.route = oracle.route_softmax(self.logits, K, renorm, scale) if T else None
        self.ws = moe.layer_workspace(self.r.h, H, I, shared)
        # sentinels in the outputs, and in the workspace what an earlier call may leave
        self.ws.fill_(0xff)
        self.out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=dev())
        self.idx = torch.full((T, K), -9, dtype=torch.int32, device=dev())
        self.w = torch.full((T, K), -9.0, device=dev())

    def call(self, logits=True, x=None, out=None, live=None, ws=None, stream=None):
        moe.moe_layer(self.r.h, self.x if x is None else x,
                      to_dev(self.logits) if logits is True else logits, self.w13, self.w2,
                      self.out if out is None else out, self.idx, self.w,
                      self.ws if ws is None else ws, bias=to_dev(self.bias) if logits is not None else None,
                      s13=self.s13, s2=self.s2, live=live, act=self.act, num_shared=self.S,
                      stream=stream)

    def want(self, idx, w, tokens=None):
        n = self.T if tokens is None else tokens
        x = self.x[:n].double().cpu().numpy()
        return ref.layer(x, idx[:n], w[:n], self.v13, self.v2, self.S, self.E, self.act)

    def check(self, tokens=None, out=None, flags=0):
        n = self.T if tokens is None else tokens
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(self.r.h) == flags
        idx, w = to_host(self.idx), to_host(self.w)
        want, bound = self.want(idx, w, n)
        got = (self.out if out is None else out).double().cpu().numpy()
        bad = ~(np.abs(got[:n] - want) <= bound)
        assert not bad.any(), "%d of %d out of bound: worst %.3g, bound %.3g" % (
            bad.sum(), bad.size, np.abs(got[:n] - want)[bad].max(), bound[bad].max())
        return idx, w, got

    def check_route(self, n=None):
        n = self.T if n is None else n
        oi, ow = self.route
        assert np.array_equal(to_host(self.idx)[:n], oi[:n])
        assert np.abs(to_host(self.w)[:n].view(np.int32) - ow[:n].view(np.int32)).max() <= 1


CASES = [
    dict(T=1, E=4, K=1, H=8, I=8),
    dict(T=1, E=8, K=2, H=256, I=64),
    dict(T=2, E=13, K=3, H=264, I=72, act="gelu"),
    dict(T=3, E=16, K=16, H=136, I=200),
    dict(T=7, E=60, K=6, H=1000, I=360, act="gelu", shared=2),
    dict(T=9, E=512, K=8, H=64, I=40),
    dict(T=16, E=32, K=4, H=2048, I=96, shared=1),
    dict(T=33, E=8, K=2, H=120, I=136, renorm=False),
    dict(T=64, E=4, K=4, H=72, I=64, shared=4),
    dict(T=128, E=8, K=2, H=200, I=48),
    dict(T=127, E=3, K=1, H=48, I=1024),
    dict(T=5, E=32, K=4, H=512, I=256, score="sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5),
    dict(T=1, E=8, K=2, H=16, I=16, e4m3=True),
    dict(T=4, E=16, K=3, H=400, I=176, e4m3=True, shared=1),     # blocks cut at 2I, H and I
    dict(T=20, E=6, K=2, H=128, I=336, e4m3=True, act="gelu"),
    dict(T=70, E=4, K=2, H=272, I=128, e4m3=True, score="sigmoid", scale=0.5),
    # between 2 and 6 tokens an expert in the mean, shared experts with more
    dict(T=24, E=16, K=3, H=328, I=152, shared=1),
    dict(T=24, E=16, K=3, H=336, I=160, shared=1, e4m3=True),
    dict(T=31, E=32, K=5, H=128, I=104, act="gelu"),
    # more than 6, rows cut inside the last tile of 4 x 16
    dict(T=60, E=6, K=2, H=392, I=264, shared=1),
    dict(T=100, E=12, K=5, H=464, I=304, e4m3=True, act="gelu"),
    # 32 entries and one more (the grouping of one warp, of the block)
    dict(T=8, E=9, K=4, H=64, I=64),
    dict(T=11, E=9, K=2, H=64, I=64, shared=1),
    # thousands of jobs on teams of 8 and 4: all but the first two or so of a
    # team come from the counter
    dict(T=8, E=16, K=4, H=4096, I=1152),
    dict(T=8, E=16, K=4, H=4096, I=1152, e4m3=True),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_layer(kw):
    p = Problem(**kw)
    p.call()
    p.check()
    p.check_route()
    first = p.out.clone()
    p.call()   # the same workspace again: the same bits
    assert torch.equal(p.out, first)


@pytest.mark.parametrize("live", [0, 1, 5, 12, 13, -4, 1000])
@pytest.mark.parametrize("shared", [0, 1])
def test_live_tokens(live, shared):
    """Places behind the live tokens: x and logits hold NaN, outputs keep theirs."""
    p = Problem(T=13, E=12, K=3, H=96, I=64, shared=shared, max_tokens=40)
    n = min(max(live, 0), 13)
    p.logits[n:] = np.nan
    p.x[n:] = float("nan")
    p.call(live=torch.tensor([live], dtype=torch.int32, device=dev()))
    idx, w, got = p.check(n)
    if n:
        p.check_route(n)
    assert (idx[n:] == -9).all() and (w[n:] == -9.0).all() and (got[n:] == 7.0).all()


def test_given_routes_with_empty_tokens():
    """Routes of the caller's own: no expert (-1), out of range, repeated."""
    p = Problem(T=11, E=6, K=3, H=88, I=48)
    idx = np.argsort(np.random.default_rng(1).random((11, 6)), axis=1)[:, :3].astype(np.int32)
    idx[2] = -1
    idx[5, 1] = -1
    p.idx.copy_(to_dev(idx))
    p.w.copy_(torch.rand(11, 3, device=dev()))
    p.call(logits=None)
    i2, _, got = p.check()
    assert np.array_equal(i2, idx) and (got[2] == 0).all()
    idx[7] = [4, 9, -2]
    idx[8] = [1, 1, 1]
    p.idx.copy_(to_dev(idx))
    p.call(logits=None)
    p.check(flags=moe.MOE_DEVERR_BAD_EXPERT | moe.MOE_DEVERR_DUP_EXPERT)


@pytest.mark.parametrize("shared", [0, 2])
def test_no_token_has_an_expert(shared):
    p = Problem(T=6, E=4, K=2, H=40, I=32, shared=shared)
    p.idx.fill_(-1)
    p.w.fill_(1.0)
    p.call(logits=None)
    _, _, got = p.check()
    assert shared or (got == 0).all()


@pytest.mark.parametrize("T", [8, 9, 31, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_all_tokens_on_the_same_experts(T, e4m3):
    p = Problem(T=T, E=16, K=2, H=144, I=48, e4m3=e4m3)
    p.logits[:, [3, 15]] += 50.0
    p.call()
    idx, _, _ = p.check()
    assert set(idx.reshape(-1)) == {3, 15}


def test_a_bad_token_stays_its_own():
    """NaN and infinity in one token's row, and a non-finite logit of another."""
    p = Problem(T=10, E=8, K=2, H=64, I=32)
    p.call()
    want = p.out.clone()
    p.x[4, 7] = float("nan")
    p.x[6, 0] = float("inf")
    p.logits[8, 3] = np.nan
    p.call()
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(p.r.h) == moe.MOE_DEVERR_NONFINITE
    keep = [t for t in range(10) if t not in (4, 6, 8)]
    assert torch.equal(p.out[keep], want[keep])
    assert p.out[4].isnan().any() and not p.out[6].isfinite().all()


@pytest.mark.parametrize("T,e4m3", [(10, True), (100, False), (100, True)])
def test_a_bad_token_stays_its_own_in_every_kernel(T, e4m3):
    p = Problem(T=T, E=8, K=2, H=144, I=48, e4m3=e4m3, shared=1)
    p.call()
    want = p.out.clone()
    p.x[4, 7] = float("nan")
    p.x[6, 0] = float("inf")
    p.call()
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (4, 6)]
    assert torch.equal(p.out[keep], want[keep])
    assert p.out[4].isnan().any() and not p.out[6].isfinite().all()


@pytest.mark.parametrize("T,live,e4m3", [(13, 5, True), (100, 7, False), (100, 61, True), (128, 0, True)])
def test_live_tokens_in_every_kernel(T, live, e4m3):
    p = Problem(T=T, E=6, K=2, H=160, I=48, shared=1, e4m3=e4m3)
    p.logits[live:] = np.nan
    p.x[live:] = float("nan")
    p.call(live=torch.tensor([live], dtype=torch.int32, device=dev()))
    idx, w, got = p.check(live)
    assert (idx[live:] == -9).all() and (w[live:] == -9.0).all() and (got[live:] == 7.0).all()


@pytest.mark.parametrize("T,H,I,e4m3", [(3, 264, 72, False), (100, 264, 72, False),
                                        (3, 272, 80, True), (100, 272, 80, True)])
def test_unreached_experts_are_not_read_into_the_sums(T, H, I, e4m3):
    """Experts that no token takes hold NaN; the reached ones lie between them,
    their last rows and columns cut inside a tile."""
    p = Problem(T=T, E=7, K=2, H=H, I=I, e4m3=e4m3)
    p.logits[:, [1, 4]] += 60.0
    for e in (0, 2, 3, 5, 6):
        for t in (p.w13, p.w2):
            (t.view(torch.uint8) if e4m3 else t)[e] = 0x7f if e4m3 else float("nan")
    p.call()
    idx, _, _ = p.check()
    assert set(idx.reshape(-1)) == {1, 4}


@pytest.mark.parametrize("kw", [
    dict(T=8, E=1, K=1, H=8, I=8),                  # 32 entries and less, smallest sizes
    dict(T=40, E=2, K=2, H=8, I=16, shared=1),
    dict(T=9, E=1, K=1, H=16, I=16, e4m3=True),
    dict(T=128, E=2, K=1, H=16, I=32, e4m3=True),
    dict(T=128, E=3, K=3, H=136, I=136, shared=4),  # 128 tokens an expert, a 128-column block and 8
    dict(T=128, E=3, K=2, H=144, I=144, shared=2, e4m3=True, act="gelu"),
    dict(T=64, E=4, K=2, H=1032, I=520, act="gelu"),
    dict(T=37, E=2, K=1, H=4096, I=2048),           # jobs for some blocks only
    dict(T=17, E=4, K=1, H=272, I=80, e4m3=True),   # 16 and 32 columns and one more
    dict(T=33, E=1, K=1, H=128, I=64, e4m3=True),
    dict(T=65, E=1, K=1, H=256, I=64, e4m3=True),
], ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_layer_with_many_tokens_an_expert(kw):
    p = Problem(**kw)
    p.call()
    p.check()
    p.check_route()
    first = p.out.clone()
    p.call()
    assert torch.equal(p.out, first)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tokens_given_routes_some_without_an_expert(e4m3):
    p = Problem(T=90, E=5, K=3, H=176, I=96, e4m3=e4m3)
    g = np.random.default_rng(3)
    idx = np.argsort(g.random((90, 5)), axis=1)[:, :3].astype(np.int32)
    idx[g.random((90, 3)) < 0.3] = -1
    idx[7] = -1
    idx[idx == 2] = -1                 # an expert that nobody takes
    p.idx.copy_(to_dev(idx))
    p.w.copy_(torch.rand(90, 3, device=dev()))
    p.call(logits=None)
    _, _, got = p.check()
    assert (got[7] == 0).all()
    idx[11] = [0, 0, 99]
    p.idx.copy_(to_dev(idx))
    p.call(logits=None)
    p.check(flags=moe.MOE_DEVERR_BAD_EXPERT | moe.MOE_DEVERR_DUP_EXPERT)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tokens_in_a_captured_graph_in_place(e4m3):
    p = Problem(T=80, E=6, K=2, H=160, I=96, shared=1, e4m3=e4m3)
    logits = to_dev(p.logits)
    live = torch.tensor([80], dtype=torch.int32, device=dev())
    x = p.x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.call(logits=logits, live=live, x=x, out=x)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        x.copy_(p.x)
        p.call(logits=logits, live=live, x=x, out=x)
        p.call(logits=logits, live=live)
    for n in (80, 33, 1):
        live.fill_(n)
        graph.replay()
        p.check(n)
        assert torch.equal(x[:n], p.out[:n]) and torch.equal(x[n:], p.x[n:])


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tokens_a_wait_that_gives_up(e4m3):
    p = Problem(T=60, E=4, K=2, H=512, I=256, e4m3=e4m3)
    moe.moe_set_wait_limit(p.r.h, 1)
    p.call()
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(p.r.h) == moe.MOE_DEVERR_TIMEOUT
    moe.moe_set_wait_limit(p.r.h, 0)
    moe.moe_clear_device_status(p.r.h)
    p.call()
    p.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tokens_weights_past_32_bit_offsets(e4m3):
    """Experts 39 and 40 of 41 begin past 2^31 elements of w13."""
    E, H, I, T = 41, 7168, 4096, 128
    r = moe.MoeRouter(E, 2, 1, T)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.uint8 if e4m3 else dt, device=dev())
    w2 = torch.zeros(E, H, I, dtype=torch.uint8 if e4m3 else dt, device=dev())
    one = torch.tensor([1.0]).to(dt).view(torch.uint8).item() if e4m3 else 1.0
    for e, col in ((39, 6), (40, 4000)):
        w13[e, col, 11] = one
        w13[e, I + col, 12] = one
        w2[e, 7000 + e, col] = one
    if e4m3:
        w13, w2 = w13.view(dt), w2.view(dt)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=dev())
    x[:, 11], x[:, 12] = 64.0, 0.5
    logits = torch.zeros(T, E, device=dev())
    logits[:, 39:] = 8.0
    scales = dict(s13=torch.ones(E, 64, 56, device=dev()), s2=torch.ones(E, 56, 32, device=dev())) if e4m3 else {}
    out, idx, w = r.layer(x, logits, w13, w2, **scales)
    assert (idx.sort(1).values == torch.tensor([39, 40], device=dev())).all()
    assert (out[:, 7039] == 16.0).all() and (out[:, 7040] == 16.0).all()
    assert (out != 0).sum().item() == 2 * T


def test_routes_without_an_expert_hide_their_scores():
    p = Problem(T=5, E=6, K=3, H=88, I=48)
    p.idx.copy_(torch.tensor([[0, -1, 2]] * 5, dtype=torch.int32))
    p.w.copy_(torch.tensor([[0.5, float("nan"), 0.25]] * 5))
    p.call(logits=None)
    torch.cuda.synchronize()
    got = p.out.clone()
    assert got.isfinite().all()
    p.w[:, 1] = 0.0
    p.call(logits=None)
    p.check()
    assert torch.equal(p.out, got)


def test_most_entries_and_experts():
    """128 tokens of 16 + 4 experts, 512 + 4 experts: the largest tables."""
    p = Problem(T=128, E=512, K=16, H=32, I=16, shared=4)
    p.call()
    p.check()
    p.check_route()


def test_e4m3_codes_read_as_their_values():
    """Every finite e4m3 code, subnormals among them, as a W2 weight: with one
    expert, I = 16 and a one-hot activation, out is scale * code * a, one
    rounding each for a (exact here) and out."""
    H, I = 256, 16
    r = moe.MoeRouter(1, 1, 1, 1)
    codes = torch.arange(256, dtype=torch.uint8)
    codes[0x7f] = codes[0xff] = 0
    w2 = codes.view(torch.float8_e4m3fn).reshape(1, H, 1).repeat(1, 1, I).contiguous().to(dev())
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device=dev())
    one = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    w13[0, 3, 0] = one          # gate 3 = x0
    w13[0, I + 3, 1] = one      # up 3 = x1
    w13 = w13.view(torch.float8_e4m3fn)
    s13 = torch.ones(1, 1, 2, device=dev())
    s2 = torch.full((1, 2, 1), 0.25, device=dev())
    x = torch.zeros(1, H, dtype=torch.bfloat16, device=dev())
    x[0, 0], x[0, 1] = 64.0, 0.03125   # silu(64) = 64 to 28 digits: a = 2
    out, _, _ = r.layer(x, torch.zeros(1, 1, device=dev()), w13, w2, s13=s13, s2=s2)
    want = codes.view(torch.float8_e4m3fn).float() * 0.5
    assert torch.equal(out.float().cpu()[0], want)


def test_same_layer_as_the_separate_calls():
    """Routing, layout, dispatch, gate/up products, activation with the score
    absorbed, the W2 GEMM and the plain combine, against the layer; the handle
    keeps its layout across the layer call."""
    T, E, K, H, I = 48, 16, 4, 512, 192
    p = Problem(T=T, E=E, K=K, H=H, I=I)
    r = p.r
    logits = to_dev(p.logits)
    idx, w = r.route(logits)
    lay = {k: v.clone() for k, v in r.layout(idx).items()}
    p.call()
    for k, v in moe.layout_tensors(r.h).items():
        assert torch.equal(v, lay[k]), k
    recv, recv_w, _ = r.dispatch(p.x, w)
    off = lay["off_e"].tolist()
    gu = torch.cat([recv[a:b].float() @ p.w13[e].float().T for e, (a, b) in enumerate(zip(off, off[1:]))]).to(torch.bfloat16)
    y = r.w2_absorbed(r.act_rows(gu), recv_w, p.w2)
    sep = r.combine(y).double().cpu().numpy()
    _, _, got = p.check()
    # the separate calls round gate/up (2), the activation (1), its product with
    # the score (1) and the expert rows (1) to bf16: five roundings more, each
    # half a step of a term; the terms add up to at most sum |w| |w2| |a|
    want, bound = p.want(to_host(idx), to_host(w))
    assert (np.abs(sep - want) <= 7 * bound).all()
    assert (np.abs(got - want) <= bound).all()


def test_in_place_output():
    p = Problem(T=12, E=8, K=2, H=160, I=64, shared=1)
    p.call()
    want = p.out.clone()
    x = p.x.clone()
    p.call(x=x, out=x)
    assert torch.equal(x, want)


def test_captured_graph_replays_with_new_inputs():
    p = Problem(T=24, E=12, K=2, H=128, I=96, shared=1)
    logits = to_dev(p.logits)
    live = torch.tensor([24], dtype=torch.int32, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.call(logits=logits, live=live)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.call(logits=logits, live=live)
        p.call(logits=logits, live=live)   # back to back on one workspace
    for step, n in ((0, 24), (1, 9), (2, 17)):
        g = torch.Generator().manual_seed(step)
        p.logits[:] = torch.randn(24, 12, generator=g).numpy()
        p.x.copy_(torch.randn(24, 128, generator=g).to(torch.bfloat16))
        logits.copy_(to_dev(p.logits))
        live.fill_(n)
        p.out.fill_(7.0)
        graph.replay()
        _, _, got = p.check(n)
        assert (got[n:] == 7.0).all()


def test_a_wait_that_gives_up_is_reported_and_the_next_call_works():
    """With a wait limit of 1 ns the blocks that reach a grid barrier first give
    up: the call returns, the status word says so, and with the usual limit
    the same workspace works again."""
    for e4m3 in (False, True):
        p = Problem(T=6, E=8, K=2, H=512, I=256, e4m3=e4m3)
        moe.moe_set_wait_limit(p.r.h, 1)
        p.call()
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(p.r.h) == moe.MOE_DEVERR_TIMEOUT
        moe.moe_set_wait_limit(p.r.h, 0)
        moe.moe_clear_device_status(p.r.h)
        p.call()
        p.check()


def test_two_streams_with_a_workspace_each():
    ps = [Problem(T=32, E=8, K=2, H=256, I=128, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in ps]
    logits = [to_dev(p.logits) for p in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s, l in zip(ps, streams, logits):
            p.call(logits=l, stream=s)
    for p in ps:
        p.check()


def test_calls_on_streams_of_three_priorities():
    """Many calls in flight at once, one a part of the GPU and two all of it,
    beside a plain product: none waits for blocks that cannot start."""
    kws = (dict(T=1, E=8, K=2, H=512, I=256), dict(T=100, E=8, K=2, H=1024, I=512),
           dict(T=24, E=8, K=2, H=1024, I=512, e4m3=True))
    ps = [Problem(seed=s, **kw) for s, kw in enumerate(kws)]
    low, high = torch.cuda.Stream.priority_range() if hasattr(torch.cuda.Stream, "priority_range") else (0, -1)
    streams = [torch.cuda.Stream(priority=q) for q in (low, high, low)]
    side = torch.cuda.Stream(priority=high)
    logits = [to_dev(p.logits) for p in ps]
    bias = [to_dev(p.bias) for p in ps]
    a = torch.randn(4096, 4096, device=dev(), dtype=torch.bfloat16)
    torch.cuda.synchronize()
    for i in range(200):
        for p, s, l in zip(ps, streams, logits):
            p.call(logits=l, stream=s)
        if i % 8 == 0:
            with torch.cuda.stream(side):
                a @ a
    for p in ps:
        p.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_beside_the_w2_product_on_another_stream(e4m3):
    """Both kernels want whole SMs and their tensor memory: they take turns."""
    p = Problem(T=100, E=8, K=2, H=1024, I=512, e4m3=e4m3)
    T, H, I = 2048, 1024, 512
    r = moe.MoeRouter(8, 2, 1, T)
    g = torch.Generator().manual_seed(5)
    idx, w = r.route(torch.randn(T, 8, generator=g).to(dev()))
    r.layout(idx)
    h = torch.randn(r.h.recv_rows, I, generator=g).to(dev(), torch.bfloat16)
    rw = torch.rand(r.h.recv_rows, generator=g).to(dev())
    w2 = (torch.randn(8, H, I, generator=g) * I ** -0.5).to(dev(), torch.bfloat16)
    want = r.w2_absorbed(h, rw, w2)
    logits = to_dev(p.logits)
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for _ in range(60):
        moe.moe_w2_absorbed(r.h, h, rw, w2, y, stream=a)
        p.call(logits=logits, stream=b)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(r.h) == 0 and torch.equal(y, want)
    p.check()


def test_method_on_another_stream_keeps_its_workspace(monkeypatch):
    """The workspace freed when the method returns is not given to the current
    stream while the other one may still use it."""
    p = Problem(T=9, E=8, K=2, H=64, I=32)
    p.call()
    torch.cuda.synchronize()
    real, seen = moe.layer_workspace, []

    def recorded(*a):
        ws = real(*a)
        seen.append((ws.data_ptr(), ws.numel()))
        return ws
    monkeypatch.setattr(moe, "layer_workspace", recorded)
    s = torch.cuda.Stream()
    logits = to_dev(p.logits)
    torch.cuda.synchronize()
    out, idx, w = p.r.layer(p.x, logits, p.w13, p.w2, stream=s)
    mine = [torch.empty(seen[0][1], dtype=torch.uint8, device=dev()) for _ in range(3)]
    assert seen[0][0] not in [t.data_ptr() for t in mine]
    s.synchronize()
    assert torch.equal(out, p.out) and torch.equal(idx, p.idx) and torch.equal(w, p.w)


def test_method_without_logits_is_refused():
    p = Problem(T=4, E=8, K=2, H=64, I=32)
    with pytest.raises(ValueError):
        p.r.layer(p.x, None, p.w13, p.w2)


def test_binding_method_with_and_without_live():
    p = Problem(T=9, E=8, K=2, H=64, I=32)
    out, idx, w = p.r.layer(p.x, to_dev(p.logits), p.w13, p.w2)
    p.call()
    assert torch.equal(out, p.out) and torch.equal(idx, p.idx) and torch.equal(w, p.w)
    out, idx, w = p.r.layer(p.x, to_dev(p.logits), p.w13, p.w2,
                            live=torch.tensor([4], dtype=torch.int32, device=dev()))
    assert torch.equal(out[:4], p.out[:4]) and (out[4:] == 0).all() and (idx[4:] == -1).all()


@pytest.mark.parametrize("kw,status", [
    (dict(H=60), moe.MOE_ERR_INVALID),
    (dict(I=36), moe.MOE_ERR_INVALID),
    (dict(num_shared=5), moe.MOE_ERR_INVALID),
    (dict(act=7), moe.MOE_ERR_INVALID),
    (dict(weight_dtype=1), moe.MOE_ERR_INVALID),
    (dict(weight_dtype=2), moe.MOE_ERR_INVALID),          # e4m3 without scales
    (dict(d_s13=0x1000, d_s2=0x1000), moe.MOE_ERR_INVALID),  # bf16 with scales
    (dict(d_x=None), moe.MOE_ERR_INVALID),
    (dict(d_x=0x1008), moe.MOE_ERR_INVALID),
    (dict(d_w13=None), moe.MOE_ERR_INVALID),
    (dict(d_idx=None), moe.MOE_ERR_INVALID),
    (dict(d_w=0x1002), moe.MOE_ERR_INVALID),
    (dict(d_bias=0x1000), moe.MOE_ERR_INVALID),           # bias with softmax scores
    (dict(T=17), moe.MOE_ERR_CAPACITY),
    (dict(T=-1), moe.MOE_ERR_INVALID),
    (dict(ws=0x1010), moe.MOE_ERR_INVALID),
    (dict(ws=None), moe.MOE_ERR_INVALID),
    (dict(ws_bytes=1000), moe.MOE_ERR_INVALID),
    (dict(T=0), moe.MOE_OK),
])
def test_refusals(kw, status):
    """Host checks of the C entry point (addresses that no kernel gets)."""
    h = moe.Handle(moe.make_config(8, 2, 1, 16))
    f = dict(d_x=0x1000, d_logits=0x1000, d_w13=0x1000, d_w2=0x1000, d_out=0x1000, d_idx=0x1000,
             d_w=0x1000, H=64, I=32)
    c = dict(T=16, ws=0x1000, ws_bytes=1 << 24)
    for k, v in kw.items():
        (c if k in c else f)[k] = v
    a = moe.MoeLayerArgs(**f)
    assert moe.lib().moe_layer(h.ptr, ctypes.byref(a), c["T"], c["ws"], c["ws_bytes"], None) == status


def test_more_than_the_layer_takes():
    r = moe.MoeRouter(8, 2, 1, 4096)
    assert moe.moe_layer_workspace_bytes(r.h.cfg, 64, 32) == \
        moe.moe_layer_workspace_bytes(moe.make_config(8, 2, 1, 128), 64, 32)
    x = torch.zeros(129, 64, dtype=torch.bfloat16, device=dev())
    with pytest.raises(moe.MoeError) as e:
        r.layer(x, torch.zeros(129, 8, device=dev()),
                torch.zeros(8, 64, 64, dtype=torch.bfloat16, device=dev()),
                torch.zeros(8, 64, 32, dtype=torch.bfloat16, device=dev()))
    assert e.value.status == moe.MOE_ERR_CAPACITY


def test_weights_past_32_bit_offsets():
    """Expert 40 of 41 begins past 2^31 elements of w13 (4.7 GB)."""
    E, H, I = 41, 7168, 4096
    r = moe.MoeRouter(E, 1, 1, 1)
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device=dev())
    w2 = torch.zeros(E, H, I, dtype=torch.bfloat16, device=dev())
    w13[40, 5, 11] = 1.0
    w13[40, I + 5, 12] = 1.0
    w2[40, 7000, 5] = 1.0
    x = torch.zeros(1, H, dtype=torch.bfloat16, device=dev())
    x[0, 11], x[0, 12] = 64.0, 0.5
    logits = torch.zeros(1, E, device=dev())
    logits[0, 40] = 5.0
    out, idx, _ = r.layer(x, logits, w13, w2)
    assert idx.item() == 40 and out[0, 7000].item() == 32.0 and out.abs().sum().item() == 32.0


@pytest.mark.parametrize("large,small", [
    (dict(T=128, E=512, K=8, H=16, I=16), dict(T=1, E=4, K=1, H=16, I=16)),
    (dict(T=128, E=160, K=5, H=16, I=16), dict(T=4, E=1, K=1, H=16, I=16)),
    (dict(T=6, E=512, K=8, H=16, I=16, e4m3=True), dict(T=1, E=4, K=1, H=16, I=16, e4m3=True)),
    (dict(T=128, E=40, K=16, H=16, I=16, shared=4), dict(T=8, E=1, K=1, H=16, I=16)),
    (dict(T=128, E=40, K=16, H=16, I=16, shared=4, e4m3=True), dict(T=8, E=1, K=1, H=16, I=16, e4m3=True)),
], ids=["packed", "unpacked", "e4m3", "many", "many-e4m3"])
def test_two_host_threads_with_tables_of_other_sizes(large, small):
    """The same kernel called from two threads, each with its own handle, stream
    and workspace, once with the largest tables and once with the smallest."""
    ps = [Problem(**kw) for kw in (large, small)]
    streams = [torch.cuda.Stream() for _ in ps]
    logits = [to_dev(p.logits) for p in ps]
    torch.cuda.synchronize()
    start, refused = threading.Barrier(2), [0, 0]

    def work(i):
        p, L = ps[i], moe.lib()
        a = moe.MoeLayerArgs(p.x.data_ptr(), logits[i].data_ptr(), None, None, p.w13.data_ptr(), p.w2.data_ptr(),
                             p.s13.data_ptr() if p.s13 is not None else None,
                             p.s2.data_ptr() if p.s2 is not None else None, p.out.data_ptr(), p.idx.data_ptr(),
                             p.w.data_ptr(), p.H, p.I, p.S, moe.MOE_BF16 if p.s13 is None else moe.MOE_E4M3, 0)
        with torch.cuda.device(dev()):
            start.wait()
            for _ in range(1500):
                refused[i] += L.moe_layer(p.r.h.ptr, ctypes.byref(a), p.T, p.ws.data_ptr(), p.ws.numel(),
                                          streams[i].cuda_stream) != moe.MOE_OK
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for p in ps:
        p.check()


@pytest.mark.parametrize("kw", [dict(T=60, E=4, K=2, H=512, I=256), dict(T=60, E=4, K=2, H=512, I=256, e4m3=True),
                                dict(T=6, E=8, K=2, H=512, I=256), dict(T=4, E=8, K=2, H=512, I=256, e4m3=True)],
                         ids=["many", "many-e4m3", "few", "few-e4m3"])
def test_a_wait_that_gives_up_ends_the_call_soon(kw):
    """The kernel ends within the handle's limit and the time of the copies under
    way, not after the default limit of a second."""
    p = Problem(**kw)
    logits = to_dev(p.logits)
    p.call(logits=logits)
    moe.moe_set_wait_limit(p.r.h, 1)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    p.call(logits=logits)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 0.5
    assert moe.moe_read_device_status(p.r.h) == moe.MOE_DEVERR_TIMEOUT
    moe.moe_set_wait_limit(p.r.h, 0)
    moe.moe_clear_device_status(p.r.h)
    p.call()
    p.check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_waits_that_give_up_anywhere_in_the_kernel(e4m3):
    """Limits from nothing to about the kernel's time: the waits of every part run
    out in some block.  Each call ends soon, and the next one is right."""
    p = Problem(T=128, E=8, K=2, H=2048, I=1024, shared=1, e4m3=e4m3)
    logits = to_dev(p.logits)
    p.call(logits=logits)
    want = p.check()[2]
    for limit in (1, 1000, 2000, 4000, 8000, 16000, 32000, 64000):
        moe.moe_set_wait_limit(p.r.h, limit)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        for _ in range(3):
            p.call(logits=logits)
        torch.cuda.synchronize()
        assert time.monotonic() - t0 < 0.5
        assert moe.moe_read_device_status(p.r.h) in (0, moe.MOE_DEVERR_TIMEOUT)
        moe.moe_set_wait_limit(p.r.h, 0)
        moe.moe_clear_device_status(p.r.h)
        p.call(logits=logits)
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(p.r.h) == 0
        assert np.array_equal(p.out.double().cpu().numpy(), want)


class KernelNodeParams(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p)]


def kernels_of(call):
    """Names of the kernels in a captured graph of `call`, in order."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call()
    rt, raw, n = ctypes.CDLL("libcudart.so.13"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert rt.cudaGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert rt.cudaGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes:
        p, name = KernelNodeParams(), ctypes.c_char_p()
        assert rt.cudaGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        assert rt.cudaFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)) == 0
        names.append(name.value.decode())
    return names


@pytest.mark.parametrize("kw,many", [
    (dict(T=128, E=64, K=1, H=64, I=64, shared=2), True),    # 128 tokens' passes over the shared experts
    (dict(T=128, E=64, K=1, H=64, I=64), False),             # 2 tokens an expert
    (dict(T=16, E=64, K=1, H=64, I=64, shared=1), False),
    (dict(T=48, E=64, K=1, H=64, I=64, shared=2, e4m3=True), True),
    (dict(T=48, E=64, K=1, H=64, I=64, e4m3=True), False),
    (dict(T=5, E=64, K=1, H=64, I=64, shared=2, e4m3=True), False),
])
def test_the_kernel_is_chosen_with_the_shared_experts_in_mind(kw, many):
    p = Problem(**kw)
    logits = to_dev(p.logits)
    p.call(logits=logits)
    p.check()
    names = kernels_of(lambda: p.call(logits=logits))
    assert len(names) == 2 and "route" in names[0]
    assert ("layer_many_kernel" in names[1]) == many and "layer" in names[1]
