"""The norms around a block and their backward on the GPU against their fp64
definitions, within the element-wise bounds of tests/block_ref.py: one rounding
of each output, and the roundings of the fp32 products and sums in front of it."""
import numpy as np
import pytest
import torch

import combine_moe_route_05_gb300 as moe
from tests import block_ref as ref
from tests.gpu_util import dev, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, ref.U_BF16), "f32": (torch.float32, ref.U32)}
EPS = 1e-5


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, bound, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d out of bound, worst ratio %.3g" % (
        what, bad.sum(), bad.size, (np.abs(got - want) / np.maximum(bound, 1e-300)).max())


class Problem:
    """Tensors of one block boundary; K: receive rows of K entries a token."""

    def __init__(self, T, H, dtype="bf16", weights="bf16", K=0, E=8, pad=1, weighted=True, drop=0.0,
                 block=True, add=False, post=True, pre=True, gate=0, scale=1.0, offset=0.0, seed=0,
                 max_tokens=None):
        g = np.random.default_rng(seed)
        self.T, self.H, self.K, self.scale, self.offset = T, H, K, scale, offset
        self.dt, self.u = TYPES[dtype]
        self.wt = TYPES[weights][0]
        self.r = moe.MoeRouter(max(E, K), max(1, K), 1, max_tokens or max(T, 1), pad_align=pad)
        self.gate_tokens = max(1, gate)

        def rows(n, std=1.0):
            return torch.from_numpy((std * g.standard_normal((n, H))).astype(np.float32)).to(dev(), self.dt)

        def weight():
            return torch.from_numpy((g.random(H) + 0.5 - offset).astype(np.float32)).to(dev(), self.wt)

        self.res = rows(T, 2.0)
        self.y = self.cw = self.pos = None
        if block and K:
            idx = np.argsort(g.random((T, max(E, K))), axis=1)[:, :K].astype(np.int32)
            idx[g.random((T, K)) < drop] = -1
            self.pos = self.r.layout(to_dev(idx))["pos"].cpu().numpy()
            moe.moe_clear_device_status(self.r.h)
            self.y = rows(self.r.h.recv_rows)
            if weighted:
                self.cw = torch.from_numpy(g.random((T, K)).astype(np.float32)).to(dev())
        elif block:
            self.y = rows(T)
        self.add = rows(T) if add else None
        groups = -(-T // self.gate_tokens)
        self.gate = rows(groups) if gate else None
        self.group = np.arange(T) // self.gate_tokens
        self.w_post, self.w_pre = weight() if post else None, weight() if pre else None
        self.gres_out, self.gx = rows(T), rows(T) if pre else None

    def shared(self):
        return dict(gate=self.gate, gate_tokens=self.gate_tokens, w_post=self.w_post, w_pre=self.w_pre,
                    res_scale=self.scale, weight_offset=self.offset)

    def forward(self, stream=None, res_out=None):
        empty = lambda: torch.full_like(self.res, 77.0)  # noqa: E731
        o = dict(res_out=res_out if res_out is not None else empty() if self.y is not None else None,
                 x=empty() if self.w_pre is not None else None,
                 c=empty() if self.y is not None else None)
        for k, w in (("rstd_post", self.w_post), ("rstd_pre", self.w_pre)):
            o[k] = None if w is None else torch.full((self.T,), 77.0, device=dev())
        moe.moe_block_norm(self.r.h, self.res, y=self.y, gather=self.K > 0, cw=self.cw, add=self.add,
                           eps=EPS, stream=stream, **o, **self.shared())
        return o

    def weights64(self):
        return [None if w is None else f64(w) + self.offset for w in (self.w_post, self.w_pre)]

    def check_forward(self):
        got = self.forward()
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(self.r.h) == 0
        y = err = None
        if self.y is not None:
            if self.K:
                y, mag = np.zeros((self.T, self.H)), np.zeros((self.T, self.H))
                rows = f64(self.y)
                for k in range(self.K):
                    w = np.ones(self.T) if self.cw is None else f64(self.cw)[:, k]
                    term = np.where(self.pos[:, k] >= 0, w, 0.0)[:, None] * rows[self.pos[:, k].clip(0)]
                    y, mag = y + term, mag + np.abs(term)
            else:
                y = f64(self.y)
                mag = np.abs(y)
            if self.add is not None:
                y, mag = y + f64(self.add), mag + np.abs(f64(self.add))
            terms = max(1, self.K) + (self.add is not None)
            err = (terms - 1 + (self.cw is not None)) * ref.U32 * mag
        w_post, w_pre = self.weights64()
        gate = None if self.gate is None else f64(self.gate)[self.group]
        want, bound = ref.block_norm(f64(self.res), y, gate, w_post, w_pre, self.scale, EPS, self.u, err)
        for k, v in got.items():
            if v is not None:
                within(v, want[k], bound[k], k)
        return got

    def backward(self, saved, outs=None, stream=None):
        has_c = self.gate is not None or self.w_post is not None
        o = outs or dict(
            gres=torch.full_like(self.res, 77.0), gy=torch.full_like(self.res, 77.0),
            ggate=None if self.gate is None else torch.full_like(self.gate, 77.0),
            gw_post=None if self.w_post is None else torch.full((self.H,), 77.0, device=dev()),
            gw_pre=None if self.w_pre is None else torch.full((self.H,), 77.0, device=dev()))
        ws = moe.block_norm_workspace(self.r.h, self.T, self.H, self.gate_tokens)
        moe.moe_block_norm_bwd(self.r.h, ws, self.gres_out, self.gx,
                               saved["res_out"] if self.w_pre is not None else None,
                               saved["c"] if has_c else None, rstd_post=saved["rstd_post"],
                               rstd_pre=saved["rstd_pre"], stream=stream, **o, **self.shared())
        return o

    def saved(self):
        s = self.forward()
        if s["res_out"] is None:
            s["res_out"] = self.res
        return s

    def check_backward(self, saved=None):
        s = saved or self.saved()
        gres_out = f64(self.gres_out)
        got = self.backward(s)
        torch.cuda.synchronize()
        assert moe.moe_read_device_status(self.r.h) == 0
        w_post, w_pre = self.weights64()
        want, bound = ref.block_norm_bwd(
            gres_out, f64(self.gx), f64(s["res_out"]), f64(s["c"]), f64(self.gate), self.group,
            -(-self.T // self.gate_tokens), w_post, w_pre, f64(s["rstd_post"]), f64(s["rstd_pre"]),
            self.scale, self.u)
        for k, v in got.items():
            if v is not None:
                within(v, want[k], bound[k], k)
        return got


WIDTHS = [  # T, H, dtype: one warp and several, ragged teams, the widest
    (1, 8, "bf16"), (1, 4, "f32"), (3, 64, "bf16"), (37, 256, "f32"), (130, 512, "bf16"),
    (130, 516, "f32"), (5, 520, "bf16"), (64, 1000, "f32"), (64, 1000, "bf16"), (33, 2048, "bf16"),
    (9, 4096, "f32"), (20, 7168, "bf16"), (6, 8192, "bf16"), (5, 8200, "bf16"), (3, 16384, "bf16"),
    (3, 16384, "f32"), (2, 12292, "f32"),
]


@pytest.mark.parametrize("T,H,dtype", WIDTHS)
@pytest.mark.parametrize("weights", ["bf16", "f32"])
def test_widths(T, H, dtype, weights):
    p = Problem(T, H, dtype, weights, seed=H)
    p.check_forward()
    p.check_backward()


FORMS = [dict(post=False), dict(pre=False), dict(post=False, pre=False), dict(block=False, post=False),
         dict(add=True), dict(gate=1), dict(gate=7), dict(gate=10 ** 9), dict(gate=5, post=False),
         dict(gate=3, pre=False, add=True), dict(scale=0.25, offset=1.0), dict(scale=-1.0, gate=1),
         dict(scale=0.0)]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join("%s_%s" % i for i in f.items()))
@pytest.mark.parametrize("T,H,dtype", [(50, 96, "bf16"), (41, 1032, "bf16"), (41, 1036, "f32")])
def test_forms(T, H, dtype, form):
    p = Problem(T, H, dtype, **form)
    p.check_forward()
    p.check_backward()


@pytest.mark.parametrize("K,E,pad,weighted,drop,add", [
    (1, 4, 1, True, 0.0, False), (8, 16, 1, True, 0.1, True), (8, 16, 16, False, 0.0, False),
    (3, 5, 7, True, 0.5, True), (9, 20, 1, True, 0.0, True), (16, 16, 1, False, 0.2, False),
    (2, 8, 1, True, 1.0, False)])
@pytest.mark.parametrize("H,dtype", [(72, "bf16"), (2056, "bf16"), (516, "f32"), (9000, "bf16")])
def test_receive_rows(K, E, pad, weighted, drop, add, H, dtype):
    Problem(45, H, dtype, K=K, E=E, pad=pad, weighted=weighted, drop=drop, add=add, gate=4).check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
def test_the_sum_of_receive_rows_is_the_combines(dtype, weighted):
    p = Problem(70, 1024, dtype, K=6, E=9, weighted=weighted)
    got = p.forward()
    assert torch.equal(got["c"], p.r.combine(p.y, p.cw))


@pytest.mark.parametrize("gate", [1, 2, 5, 64, 999, 4999, 5000])
@pytest.mark.parametrize("T,H,dtype", [(5000, 64, "bf16"), (5000, 60, "f32"), (3001, 1032, "bf16")])
def test_column_sums_over_units_and_groups(T, H, dtype, gate):
    """More tokens than units, groups inside a unit, across two and across many."""
    Problem(T, H, dtype, gate=gate, seed=gate).check_backward()


@pytest.mark.parametrize("H,dtype", [(7168, "bf16"), (7168, "f32"), (4096, "f32"), (9000, "bf16"),
                                     (16384, "bf16"), (104, "bf16"), (256, "f32")])
@pytest.mark.parametrize("gate", [0, 1, 5, 300])
def test_many_tokens_a_team(H, dtype, gate):
    """Several tokens a team, so that places in shared memory are taken again."""
    p = Problem(700 if H > 1000 else 20000, H, dtype, gate=gate, seed=H + gate)
    p.check_forward()
    p.check_backward()


@pytest.mark.parametrize("T,H,dtype,K,add", [
    (700, 2056, "bf16", 8, False), (500, 7168, "bf16", 8, True), (900, 1500, "f32", 5, True),
    (500, 7168, "f32", 3, False), (400, 9000, "bf16", 2, True), (900, 2048, "bf16", 16, False),
    (30000, 96, "bf16", 4, True)])
def test_many_tokens_of_receive_rows_a_team(T, H, dtype, K, add):
    Problem(T, H, dtype, K=K, E=24, add=add, drop=0.05, gate=0, seed=T).check_forward()


def test_column_sums_of_very_many_tokens():
    """Units of more tokens than are added up in registers, with groups that
    end inside one."""
    T = 2600000  # 1070 tokens a unit on 152 SMs
    for gate in (1064, T):
        Problem(T, 8, "f32", gate=gate, seed=gate).check_backward()


@pytest.mark.parametrize("H", [96, 2048])
def test_gradients_of_one_side_alone(H):
    p = Problem(60, H, "f32")
    s = p.saved()
    gres_out, gx, w_pre = p.gres_out, p.gx, p.w_pre
    both = {k: f64(v) for k, v in p.check_backward(s).items() if v is not None}
    # no gradient of the residual sum: the same as one of zeros, bit for bit
    p.gres_out = torch.zeros_like(gres_out)
    zeros = p.backward(s)
    ws = moe.block_norm_workspace(p.r.h, 60, H)
    outs = {k: torch.empty_like(v) for k, v in zeros.items() if v is not None}
    moe.moe_block_norm_bwd(p.r.h, ws, None, gx, s["res_out"], s["c"], rstd_post=s["rstd_post"],
                           rstd_pre=s["rstd_pre"], **outs, **p.shared())
    for k, v in outs.items():
        assert torch.equal(v, zeros[k]), k
    # gradients are linear: the residual's part alone adds up with the norm's
    p.gres_out, p.gx, p.w_pre = gres_out, None, None
    alone = p.check_backward(s)
    for k in ("gres", "gy"):
        assert np.allclose(f64(alone[k]) + f64(outs[k]), both[k], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("H,dtype", [(256, "f32"), (1024, "bf16")])
def test_in_place(H, dtype):
    p = Problem(100, H, dtype, gate=9)
    want = p.forward()
    res = p.res.clone()
    p.res = res
    got = p.forward(res_out=res)
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = p.backward(want)
    outs = {k: torch.empty_like(v) for k, v in g.items()}
    outs["gres"] = p.gres_out
    again = p.backward(want, outs)
    assert all(torch.equal(again[k], g[k]) for k in g)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_row_that_is_not_finite_stays_alone(value):
    p = Problem(40, 1024, "bf16")
    want = p.forward()
    p.y[17, 3] = value
    got = p.forward()
    keep = [i for i in range(40) if i != 17]
    assert all(torch.equal(got[k][keep], want[k][keep]) for k in got)
    assert not torch.isfinite(got["x"][17]).any() or torch.isnan(got["x"][17]).any()


def test_rows_of_zeros():
    p = Problem(10, 640, "f32")
    p.res.zero_()
    p.y.zero_()
    s = p.check_forward()
    assert not s["x"].any() and not s["res_out"].any()
    p.check_backward()


@pytest.mark.parametrize("T,H,gate", [(700, 256, 50), (333, 2048, 100)])
def test_repeated_calls_give_the_same_bits(T, H, gate):
    p = Problem(T, H, "bf16", gate=gate)
    s = p.saved()
    g = p.backward(s)
    for _ in range(5):
        again, h = p.forward(), p.backward(s)
        assert all(torch.equal(again[k], s[k]) for k in s if s[k] is not None)
        assert all(torch.equal(h[k], g[k]) for k in g)


def test_another_stream_and_a_captured_graph():
    p, q = Problem(300, 2048, gate=90, seed=1), Problem(300, 2048, gate=90, seed=2)
    ws, qs = p.saved(), q.saved()
    wg, qg = p.backward(ws), q.backward(qs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = p.forward(stream=side)
    side.wait_stream(torch.cuda.current_stream())
    g = p.backward(s, stream=side)
    side.synchronize()
    assert all(torch.equal(g[k], wg[k]) for k in g) and torch.equal(s["x"], ws["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = p.forward()
        g = p.backward(s)
    for name in ("res", "y", "gate", "w_post", "w_pre", "gres_out", "gx"):
        getattr(p, name).copy_(getattr(q, name))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s[k], qs[k]) for k in s)
    assert all(torch.equal(g[k], qg[k]) for k in g)


def test_two_backward_calls_at_once():
    ps = [Problem(2000, 1024, gate=300, seed=i) for i in range(2)]
    saved = [p.saved() for p in ps]
    want = [p.backward(s) for p, s in zip(ps, saved)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in ps], []
    for _ in range(8):
        for p, s, st in zip(ps, saved, streams):
            with torch.cuda.stream(st):
                outs.append(p.backward(s))
    torch.cuda.synchronize()
    for n, o in enumerate(outs):
        assert all(torch.equal(o[k], want[n % 2][k]) for k in o)


def test_two_graphs_replayed_at_once():
    """Each with its own workspace, on one handle."""
    ps = [Problem(900, 1024, gate=200, seed=i) for i in range(2)]
    ps[1].r = ps[0].r
    saved = [p.saved() for p in ps]
    want = [p.backward(s) for p, s in zip(ps, saved)]
    graphs, outs = [], []
    for p, s in zip(ps, saved):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.backward(s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[k], w[k]) for k in w)


def test_methods_give_the_same():
    p = Problem(64, 512, "bf16", K=4, E=8, add=True, gate=8)
    want = p.forward()
    res_out, x, saved = p.r.block_norm(p.res, p.y, gather=True, cw=p.cw, add=p.add, eps=EPS, save=True,
                                       **p.shared())
    assert torch.equal(res_out, want["res_out"]) and torch.equal(x, want["x"])
    assert all(torch.equal(saved[k], want[k]) for k in ("res_out", "c", "rstd_post", "rstd_pre"))
    wg = p.backward(want)
    got = p.r.block_norm_bwd(p.gres_out, p.gx, saved, **p.shared())
    for v, k in zip(got, ("gres", "gy", "ggate", "gw_post", "gw_pre")):
        assert torch.equal(v, wg[k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = p.r.block_norm_bwd(p.gres_out, p.gx, saved, stream=side, **p.shared())
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[1], wg["gy"])
    # the norm alone, and without what the backward needs
    none, x, saved = p.r.block_norm(p.res, w_pre=p.w_pre, eps=EPS)
    assert none is None and saved is None
    q = Problem(64, 512, "bf16", block=False, post=False)
    q.res, q.w_pre = p.res, p.w_pre
    assert torch.equal(x, q.forward()["x"])
    _, _, saved = p.r.block_norm(p.res, w_pre=p.w_pre, eps=EPS, save=True)
    gres, gy, ggate, gw_post, gw_pre = p.r.block_norm_bwd(None, p.gx, saved, w_pre=p.w_pre)
    assert gy is None and ggate is None and gw_post is None and gw_pre is not None


def test_no_tokens():
    p = Problem(0, 64, "f32", gate=5, max_tokens=10)
    p.forward()
    g = p.backward(p.forward())
    torch.cuda.synchronize()
    assert not g["gw_post"].any() and not g["gw_pre"].any()  # sums of nothing


def test_a_workspace_of_the_largest_batch_serves_every_smaller_one():
    h = moe.Handle(moe.make_config(8, 2, 1, 4096))
    for H in (64, 1024, 16384):
        for gate in (1, 3):
            n = [moe.moe_block_norm_workspace_bytes(h, T, H, gate) for T in range(0, 4097)]
            assert n == sorted(n) and n[0] > 0
    for bad in ((-1, 64, 1), (4097, 64, 1), (8, 0, 1), (8, 16385, 1), (8, 64, 0)):
        assert moe.moe_block_norm_workspace_bytes(h, *bad) == 0


def test_refusals():
    import ctypes
    p = Problem(32, 64, "bf16", K=2, gate=4, add=True, max_tokens=40)
    h, L = p.r.h, moe.lib()
    o = p.saved()
    ws = moe.block_norm_workspace(h, 32, 64, 4)
    a = dict(d_res=p.res, d_y=p.y, d_cw=p.cw, d_add=p.add, d_gate=p.gate, d_w_post=p.w_post,
             d_w_pre=p.w_pre, d_res_out=o["res_out"], d_x=o["x"], d_c=o["c"],
             d_rstd_post=o["rstd_post"], d_rstd_pre=o["rstd_pre"], res_scale=1.0, eps=1e-6,
             weight_offset=0.0, H=64, dtype=0, weight_dtype=0, gate_tokens=4, gather=1)
    b = {k: a[k] for k in ("d_gate", "d_w_post", "d_w_pre", "d_rstd_post", "d_rstd_pre", "d_c", "d_res_out",
                           "res_scale", "weight_offset", "H", "dtype", "weight_dtype", "gate_tokens")}
    g = p.backward(o)
    b.update(d_gres_out=p.gres_out, d_gx=p.gx, **{"d_" + k: v for k, v in g.items()})

    def struct(cls, base, kw):
        s = cls()
        for k, v in {**base, **kw}.items():
            setattr(s, k, v.data_ptr() if torch.is_tensor(v) else v)
        return ctypes.byref(s)

    def fwd(T=32, **kw):
        return L.moe_block_norm(h.ptr, struct(moe.MoeBlockNormArgs, a, kw), T, None)

    def bwd(T=32, space=ws.data_ptr(), n=ws.numel(), **kw):
        return L.moe_block_norm_bwd(h.ptr, struct(moe.MoeBlockNormBwdArgs, b, kw), T, space, n, None)

    assert fwd() == moe.MOE_OK and bwd() == moe.MOE_OK
    assert fwd(T=41) == moe.MOE_ERR_CAPACITY and bwd(T=41) == moe.MOE_ERR_CAPACITY
    assert L.moe_block_norm(h.ptr, None, 32, None) == moe.MOE_ERR_INVALID
    off = lambda t, n: t.data_ptr() + n  # noqa: E731
    both = [dict(H=0), dict(H=63), dict(H=16392), dict(dtype=2), dict(weight_dtype=2), dict(weight_dtype=-1),
            dict(gate_tokens=0), dict(res_scale=float("nan")), dict(weight_offset=float("inf")),
            dict(res_scale=1e60), dict(d_gate=off(p.gate, 8)), dict(d_w_post=off(p.w_post, 2)),
            dict(d_w_pre=None), dict(T=-1)]
    for bad in both + [dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60), dict(eps=float("inf")),
                       dict(gather=2), dict(T=31), dict(d_res=None), dict(d_res=off(p.res, 2)),
                       dict(d_res_out=None), dict(d_x=None), dict(d_x=off(o["x"], 8)), dict(gather=0),
                       dict(d_y=None), dict(d_w_post=None), dict(d_cw=off(p.cw, 2)),
                       dict(d_c=off(o["c"], 4)), dict(d_rstd_pre=off(o["rstd_pre"], 1))]:
        assert fwd(**bad) == moe.MOE_ERR_INVALID, bad
    for bad in both + [dict(d_gres_out=None, d_gx=None), dict(d_gx=None), dict(d_res_out=None),
                       dict(d_rstd_pre=None), dict(d_rstd_post=None), dict(d_c=None), dict(d_gate=None),
                       dict(d_w_post=None), dict(d_gy=off(g["gy"], 2)), dict(d_gw_pre=off(g["gw_pre"], 2)),
                       dict(space=None), dict(space=ws.data_ptr() + 128), dict(n=ws.numel() - 1)]:
        assert bwd(**bad) == moe.MOE_ERR_INVALID, bad
    fresh = moe.Handle(moe.make_config(8, 2, 1, 40))
    assert L.moe_block_norm(fresh.ptr, struct(moe.MoeBlockNormArgs, a, {}), 32, None) == moe.MOE_ERR_STATE
    with pytest.raises(ValueError):
        moe.moe_block_norm(h, p.res, o["res_out"], o["x"], y=p.y[:32], w_pre=p.w_pre[:32])
    with pytest.raises(ValueError):
        moe.moe_block_norm_bwd(h, ws)
    with pytest.raises(ValueError):
        moe.moe_block_norm(h, p.res, o["res_out"], y=p.res, gate=p.gate, gate_tokens=3)
    with pytest.raises(TypeError):
        moe.moe_block_norm(h, p.res.half(), o["res_out"])
    with pytest.raises(TypeError):
        moe.moe_block_norm(h, p.res, o["res_out"], o["x"], y=p.res, w_post=p.w_post, w_pre=p.w_pre.float())
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(h) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pad", [1, 16])
def test_a_training_step_of_a_block(score, pad):
    """Pre-norm, routing, balance loss, dispatch, experts (here y = v * row), combine
    with post-norm, gate and residual sum, the next pre-norm; and all of it backward,
    against fp64 autograd with the routing's choice held fixed.  fp32 rows.  A chain
    of some twenty fp32 operations whose sums have at most H = 512 terms or K = 4:
    relative to each gradient's norm 1e-5 covers them (512 * 2^-24 = 3e-5 at worst for
    one sum, typically its root); what the chain could lose, a term, is of order 1."""
    T, H, E, K, coef, groups = 200, 512, 16, 4, 0.1, 3
    g = np.random.default_rng(11)
    f = lambda *s: g.standard_normal(s)  # noqa: E731
    res0, wr, v = f(T, H), f(E, H) / np.sqrt(H), 1 + 0.3 * f(E, H)
    w0, wpost, w1, gate = 1 + 0.1 * f(H), 1 + 0.1 * f(H), 1 + 0.1 * f(H), f(groups, H)
    gres, gx = f(T, H), f(T, H)
    off = np.array([0, 70, 70, 200], np.int32)
    gate_tokens = -(-T // groups)
    d32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev())  # noqa: E731
    r = moe.MoeRouter(E, K, 4, T, score_fn=score, pad_align=pad)
    # forward
    _, x0, s0 = r.block_norm(d32(res0), w_pre=d32(w0), eps=EPS, save=True)
    logits = x0 @ d32(wr).T
    idx, w = r.route(logits)
    lay = r.layout(idx)
    loss, cnt, _ = r.balance(logits, idx, seq_off=torch.from_numpy(off).to(dev()), coef=coef)
    recv, _, _ = r.dispatch(x0, w)
    expert = torch.zeros(r.h.recv_rows, dtype=torch.long, device=dev())
    ends = lay["off_e"].long()
    expert = torch.searchsorted(ends[1:].contiguous(), torch.arange(r.h.recv_rows, device=dev()), right=True).clamp(max=E - 1)
    vd = d32(v)
    y = recv * vd[expert]
    kw = dict(gate=d32(gate), gate_tokens=gate_tokens, w_post=d32(wpost), res_scale=0.8)
    res1, x1, s1 = r.block_norm(d32(res0), y, gather=True, cw=w, w_pre=d32(w1), eps=EPS, save=True, **kw)
    # backward
    gres1, gc, ggate, gwpost, gw1 = r.block_norm_bwd(d32(gres), d32(gx), s1, w_pre=d32(w1), **kw)
    gy, gw = r.combine_bwd(gc, y, w)
    gxd, glogits = r.dispatch_bwd_route(gy * vd[expert], logits, idx, gw)
    glogits = r.balance_bwd(logits, cnt, seq_off=torch.from_numpy(off).to(dev()), coef=coef, base=glogits)
    gx0 = gxd + glogits @ d32(wr)
    gres0, _, _, _, gw0 = r.block_norm_bwd(gres1, gx0, s0, w_pre=d32(w0))
    gwr = glogits.T @ x0
    assert moe.moe_read_device_status(r.h) == 0
    # the same in fp64
    t = lambda a: torch.tensor(np.float32(a).astype(np.float64), requires_grad=True)  # noqa: E731
    P = dict(res=t(res0), wr=t(wr), w0=t(w0), wpost=t(wpost), w1=t(w1), gate=t(gate))
    norm = lambda a, b: a / torch.sqrt((a * a).mean(1, keepdim=True) + EPS) * b  # noqa: E731
    a0 = norm(P["res"], P["w0"])
    l = a0 @ P["wr"].T
    ix = idx.long().cpu()
    if score == "softmax":
        p, sel = torch.softmax(l, 1), torch.softmax(torch.gather(l, 1, ix), 1)
    else:
        sg = torch.sigmoid(l)
        p, sel = sg / sg.sum(1, keepdim=True), torch.gather(sg, 1, ix)
        sel = sel / sel.sum(1, keepdim=True)
    c = torch.zeros(T, H, dtype=torch.float64)
    v64 = torch.from_numpy(np.float32(v).astype(np.float64))
    for k in range(K):
        c = c + sel[:, k, None] * a0 * v64[ix[:, k]]
    r1 = 0.8 * P["res"] + P["gate"][torch.arange(T) // gate_tokens] * norm(c, P["wpost"])
    b1 = norm(r1, P["w1"])
    L = torch.zeros((), dtype=torch.float64)
    for q in range(3):
        a, b = int(off[q]), int(off[q + 1])
        if b > a:
            n = torch.bincount(ix[a:b].reshape(-1), minlength=E).double()
            L = L + coef / 2 * E / (K * (b - a) ** 2) * (n * p[a:b].sum(0)).sum()
    (L + (r1 * torch.from_numpy(np.float32(gres).astype(float))).sum()
     + (b1 * torch.from_numpy(np.float32(gx).astype(float))).sum()).backward()

    def close(got, want, what):
        want = want.detach().numpy()
        err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert err <= 1e-5, "%s: %.3g" % (what, err)

    close(loss, L.reshape(1), "loss")
    close(res1, r1, "res1")
    close(x1, b1, "x1")
    for got, name in ((gres0, "res"), (gwr, "wr"), (gw0, "w0"), (gwpost, "wpost"), (gw1, "w1"),
                      (ggate, "gate")):
        close(got, P[name].grad, name)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [2, 5, 10 ** 6])
@pytest.mark.parametrize("T,H", [(3, 14340), (330, 14336), (330, 14340), (330, 16384)])
def test_widest_fp32_rows_with_a_gate_of_groups(T, H, gate, post):
    """Weights, the gate's row and its product with them do not all fit into a
    block's shared memory from 14340 on."""
    p = Problem(T, H, "f32", "f32", gate=gate, post=post, seed=H + gate)
    p.check_forward()
    p.check_backward()


@pytest.mark.parametrize("T,H,dtype", [(70, 96, "f32"), (700, 2056, "bf16"), (40, 9000, "bf16")])
def test_the_kept_sum_in_place_of_what_is_added_or_of_the_block(T, H, dtype):
    for K, add in ((3, True), (0, True), (0, False)):
        p = Problem(T, H, dtype, K=K, add=add, gate=9)
        want = p.forward()
        for name in ("add",) * add + ("y",) * (K == 0):
            kept = getattr(p, name)
            setattr(p, name, kept.clone())
            o = {k: torch.empty_like(v) for k, v in want.items()}
            o["c"] = getattr(p, name)
            moe.moe_block_norm(p.r.h, p.res, y=p.y, gather=K > 0, cw=p.cw, add=p.add, eps=EPS, **o,
                               **p.shared())
            assert all(torch.equal(o[k], want[k]) for k in o), name
            setattr(p, name, kept)


@pytest.mark.parametrize("gate", [0, 1, 7, 300])
@pytest.mark.parametrize("T,H,dtype", [(300, 96, "bf16"), (300, 1036, "f32"), (300, 16384, "f32")])
def test_each_output_alone(T, H, dtype, gate):
    p = Problem(T, H, dtype, gate=gate)
    want = p.saved()
    o = dict.fromkeys(want)
    o["res_out"] = torch.empty_like(p.res)
    for alone in ("res_out", "x", "c", "rstd_post", "rstd_pre"):
        q = dict(o, **{alone: torch.empty_like(want[alone])})
        if alone == "rstd_pre":
            q["x"] = torch.empty_like(want["x"])
        kw = p.shared()
        if q["x"] is None:
            kw["w_pre"] = None
        moe.moe_block_norm(p.r.h, p.res, y=p.y, eps=EPS, **q, **kw)
        assert all(torch.equal(v, want[k]) for k, v in q.items() if v is not None), alone
    grads = p.backward(want)
    for alone in grads:
        if grads[alone] is not None:
            got = p.backward(want, dict(dict.fromkeys(grads), **{alone: torch.empty_like(grads[alone])}))
            assert torch.equal(got[alone], grads[alone]), alone
