"""The router's balance loss, its counts and its gradient on the GPU against their
fp64 definitions.

Tolerances (tests/block_ref.py): a probability carries the fast exponential's
documented error on its row's range of logits, twice (once in the row's sum), and
the sum's additions; a mean or the loss, whose terms are positive, at most CHAIN
additions more.  Counts are exact."""
import numpy as np
import pytest
import torch

import combine_moe_route_05_gb300 as moe
from tests import block_ref as ref
from tests.gpu_util import dev, to_dev, to_host

pytestmark = pytest.mark.gpu

SENTINEL = 7.25


def routed(g, T, E, K, drop=0.0):
    idx = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
    idx[g.random((T, K)) < drop] = -1
    return idx


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def outside(T, off):
    """Tokens of no sequence."""
    t = np.arange(T)
    return (t < off[0]) | (t >= off[-1])


class Problem:
    def __init__(self, T, E, K, score, off=None, drop=0.0, seed=0, scale=1.0, shift=0.0, shifted=0):
        g = np.random.default_rng(seed)
        self.T, self.E, self.K, self.score = T, E, K, score
        self.table = off is not None
        self.off = np.array([0, T], np.int32) if off is None else off
        self.logits = (g.standard_normal((T, E)) * scale + shift).astype(np.float32)
        self.idx = routed(g, T, E, K, drop)
        self.base = (1e-3 * g.standard_normal((T, E))).astype(np.float32)
        self.logits[outside(T, self.off)] = np.nan
        self.r = moe.MoeRouter(E, K, 1, max(T, 1), score_fn=score)
        self.S = len(self.off) - 1
        self.shifted = shifted  # elements from a 16-byte boundary

    def dev(self, a):
        if not self.shifted:
            return to_dev(a)
        flat = torch.empty(a.size + self.shifted, dtype=torch.from_numpy(a).dtype, device=dev())
        view = flat[self.shifted:].view(a.shape)
        view.copy_(torch.from_numpy(a))
        assert view.is_contiguous()
        return view

    def forward(self, coef=0.02, prob=True, stream=None):
        off = to_dev(self.off) if self.table else None
        loss = torch.full((1,), SENTINEL, device=dev())
        cnt = torch.full((self.S, self.E), -9, dtype=torch.int32, device=dev())
        p = torch.full((self.S, self.E), SENTINEL, device=dev()) if prob else None
        moe.moe_balance(self.r.h, self.dev(self.logits), self.dev(self.idx), loss, cnt,
                        moe.balance_workspace(self.r.h, self.S), prob=p, seq_off=off, coef=coef,
                        stream=stream)
        torch.cuda.synchronize()
        return loss, cnt, p

    def backward(self, cnt, coef=0.02, gloss=None, base=None, in_place=False):
        off = to_dev(self.off) if self.table else None
        gl = None if gloss is None else torch.tensor([gloss], device=dev())
        b = None if base is None else self.dev(base)
        out = b if in_place else self.dev(np.full((self.T, self.E), SENTINEL, np.float32))
        moe.moe_balance_bwd(self.r.h, self.dev(self.logits), cnt, out, seq_off=off, coef=coef,
                            gloss=gl, base=b)
        torch.cuda.synchronize()
        return out

    def check(self, status=0, with_base=True):
        loss, cnt, prob = self.forward()
        assert moe.moe_read_device_status(self.r.h) == status
        wl, wc, wp = ref.balance(self.logits, self.idx, self.off, self.E, self.score, 0.02)
        assert np.array_equal(to_host(cnt), wc)
        live = ~outside(self.T, self.off)
        rel = ref.probability_error(self.logits[live], self.score).max() if live.any() else 0.0
        rel += ref.CHAIN * ref.U32
        assert (np.abs(to_host(prob) - wp) <= rel * wp + ref.TINY).all()
        assert abs(float(loss) - wl) <= (rel + 40 * ref.U32) * wl, (float(loss), wl)
        for gloss, base, in_place in ((None, None, False), (3.0, self.base, False),
                                      (0.5, self.base, True)):
            if base is not None and not with_base:
                continue
            got = to_host(self.backward(cnt, gloss=gloss, base=base, in_place=in_place)).astype(np.float64)
            want, bound = ref.balance_bwd(self.logits, wc, self.off, self.K, self.score, 0.02,
                                          1.0 if gloss is None else gloss)
            if base is not None:
                want = np.where(live[:, None], want + base, want)
                bound = bound + ref.U32 * np.abs(want)
            # rows outside the sequences are left as they were
            kept = base if in_place else np.full_like(self.base, SENTINEL)
            assert np.array_equal(got[~live], kept[~live].astype(np.float64))
            bad = ~(np.abs(got - want)[live] <= bound[live] + ref.TINY)
            assert not bad.any(), "%d of %d out of bound, worst ratio %.3g" % (
                bad.sum(), bad.size, (np.abs(got - want)[live] / (bound[live] + ref.TINY)).max())
        assert moe.moe_read_device_status(self.r.h) == status
        return loss, cnt, prob


SIZES = [
    # T, E, K: every team width, experts off a multiple of four, one tile and many
    (1, 1, 1), (1, 8, 2), (3, 5, 5), (37, 13, 3), (256, 8, 2), (300, 16, 4), (511, 31, 8),
    (700, 64, 16), (1000, 100, 6), (2049, 128, 8), (777, 129, 1), (1500, 256, 8), (650, 300, 16),
    (400, 384, 8), (333, 511, 3), (900, 512, 8),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_one_sequence(T, E, K, score):
    Problem(T, E, K, score, drop=0.1, seed=T).check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("name,T,E,K,lens,first", [
    ("ends", 100, 8, 2, [0, 100, 0], 0),
    ("gaps", 1000, 16, 2, [300, 0, 1, 400, 0, 0, 200], 50),
    ("ones", 200, 32, 4, [1] * 200, 0),
    ("long", 3000, 128, 8, [1, 2998, 1], 0),
    ("packed", 5000, 64, 4, [700, 1, 1300, 0, 64, 63, 65, 2000, 400], 7),
    ("many", 9000, 20, 3, [9] * 990, 3),
    ("most", 4000, 12, 2, [0, 3, 1, 0, 5] * 440, 0),
])
def test_packed_sequences(name, T, E, K, lens, first, score):
    Problem(T, E, K, score, offsets(lens, first), drop=0.05, seed=len(lens)).check()


def test_no_sequence_holds_a_token():
    p = Problem(40, 8, 2, "softmax", offsets([0, 0, 0], 11))
    loss, cnt, prob = p.check()
    assert float(loss) == 0.0 and not cnt.any() and not prob.any()


def test_no_tokens():
    p = Problem(0, 8, 2, "softmax")
    loss, cnt, prob = p.forward()
    assert float(loss) == 0.0 and not cnt.any() and not prob.any()
    p.backward(cnt)
    assert moe.moe_read_device_status(p.r.h) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 50, 256])
def test_rows_off_a_16_byte_boundary(E, score):
    Problem(333, E, 4, score, offsets([100, 200]), shifted=1).check()


@pytest.mark.parametrize("scale,shift", [(8.0, 0.0), (1.0, -60.0), (1.0, 60.0), (0.0, 0.0), (3.0, -29.0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ranges_of_logits(scale, shift, score):
    Problem(500, 64, 4, score, scale=scale, shift=shift, seed=1).check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 72, 512])
def test_masked_experts_and_rows(E, score):
    p = Problem(300, E, 2, score, seed=2)
    p.logits[:, 3] = -np.inf
    p.logits[10:20, : E - 1] = -np.inf
    p.logits[30:40] = -np.inf
    p.check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_of_the_lowest_value(score):
    p = Problem(300, 40, 2, score, seed=3)
    low = np.finfo(np.float32).min
    p.logits[:, 7] = low
    p.logits[5:9, : 39] = low
    loss, cnt, prob = p.forward()
    wl, wc, wp = ref.balance(p.logits, p.idx, p.off, 40, score, 0.02)
    assert np.array_equal(to_host(cnt), wc)
    # 2 (2 + 1.16 x) ulp for unmasked logits, which are within x = 10 of each other
    rel = 2 * (2 + 1.16 * 10) * 2.0 ** -23 + ref.CHAIN * ref.U32
    assert (np.abs(to_host(prob) - wp) <= rel * wp + ref.TINY).all() and (to_host(prob)[0, 7] == 0)
    assert abs(float(loss) - wl) <= (rel + 40 * ref.U32) * wl
    g = to_host(p.backward(cnt))
    assert np.isfinite(g).all() and (g[:, 7] == 0).all()
    assert moe.moe_read_device_status(p.r.h) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_inf_logits_are_flagged_and_count_for_nothing(score):
    for value in (np.nan, np.inf):
        p = Problem(300, 24, 2, score, seed=4)
        p.logits[7, 5] = value
        p.logits[299, 23] = value
        loss, _, _ = p.check(status=moe.MOE_DEVERR_NONFINITE)
        assert np.isfinite(float(loss))


def test_entries_that_do_not_count_are_flagged():
    for value, flag in ((24, moe.MOE_DEVERR_BAD_EXPERT), (-2, moe.MOE_DEVERR_BAD_EXPERT),
                        (2 ** 31 - 1, moe.MOE_DEVERR_BAD_EXPERT), (None, moe.MOE_DEVERR_DUP_EXPERT)):
        p = Problem(300, 24, 4, "softmax", seed=4)
        p.idx[200, 3] = p.idx[200, 1] if value is None else value
        p.check(status=flag)


@pytest.mark.parametrize("off", [[0, 200, 100, 300], [-5, 100, 200, 300], [0, 100, 200, 301],
                                 [300, 0, 0, 0], [2 ** 31 - 1, 5, -2 ** 31, 7]])
def test_offsets_that_are_no_table_are_flagged(off):
    p = Problem(300, 24, 4, "softmax")
    p.table, p.S, p.off = True, 3, np.array(off, np.int32)
    _, cnt, _ = p.forward()
    assert moe.moe_read_device_status(p.r.h) & moe.MOE_DEVERR_BAD_LAYOUT
    p.backward(cnt.clamp(0, 300))  # comes back


@pytest.mark.parametrize("T,E,S", [(400000, 128, 1), (400000, 128, 3), (140000, 8, 1000)])
def test_long_batches(T, E, S):
    """Tiles of more than one set of register sums; fp64 torch on the GPU."""
    K = 4
    g = torch.Generator(device="cuda").manual_seed(T + S)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices.to(torch.int32)
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")
    off = torch.cat([cuts, torch.tensor([0, T], device="cuda")]).sort().values.to(torch.int32)
    r = moe.MoeRouter(E, K, 1, T)
    loss, cnt, prob = r.balance(logits, idx, seq_off=off, coef=1.0)
    o = off.long()
    seq = torch.searchsorted(o[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
    n = (o[1:] - o[:-1]).double()
    want_cnt = torch.bincount((seq[:, None] * E + idx).reshape(-1), minlength=S * E).reshape(S, E)
    assert torch.equal(cnt.long(), want_cnt)
    P = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seq, torch.softmax(logits.double(), 1))
    want = (E / (K * n.clamp(min=1) ** 2) * (want_cnt * P).sum(1)).sum() / (n > 0).sum()
    rel = 3e-6 + ref.CHAIN * ref.U32  # logits within 11 of each other: 2 (15 + 6) ulp
    assert ((prob.double() * n[:, None] - P).abs() <= rel * P).all()
    assert abs(float(loss) - float(want)) <= rel * float(want)
    assert moe.moe_read_device_status(r.h) == 0


def test_repeated_calls_give_the_same_bits():
    p = Problem(9000, 64, 4, "sigmoid", offsets([2000, 1, 6000, 900]), seed=9)
    first = p.forward()
    g = p.backward(first[1])
    for _ in range(5):
        again = p.forward()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert torch.equal(g, p.backward(again[1]))


def test_prob_is_optional_and_coef_scales():
    p = Problem(500, 32, 4, "softmax")
    a, _, none = p.forward(coef=1.0, prob=False)
    b, _, _ = p.forward(coef=-4.0)
    assert none is None and float(b) == -4.0 * float(a)
    assert float(p.forward(coef=0.0)[0]) == 0.0


def test_another_stream_and_a_captured_graph():
    """Forward and backward captured once, replayed on new logits, routes and
    offsets; and called on a stream of their own."""
    T, E, K = 3000, 64, 4
    probs = [Problem(T, E, K, "softmax", offsets(l), seed=s) for s, l in enumerate(([1000, 2000], [2500, 400]))]
    r = probs[0].r
    logits, idx, off = (to_dev(a).clone() for a in (probs[0].logits, probs[0].idx, probs[0].off))
    side = torch.cuda.Stream()
    ws = moe.balance_workspace(r.h, 2)
    loss, gl = torch.empty(1, device=dev()), torch.zeros(T, E, device=dev())
    cnt = torch.empty(2, E, dtype=torch.int32, device=dev())

    def both():
        moe.moe_balance(r.h, logits, idx, loss, cnt, ws, seq_off=off, coef=0.02)
        moe.moe_balance_bwd(r.h, logits, cnt, gl, seq_off=off, coef=0.02)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    want = probs[0].forward()
    assert torch.equal(loss, want[0]) and torch.equal(cnt, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for p in probs[::-1]:
        for to, a in ((logits, p.logits), (idx, p.idx), (off, p.off)):
            to.copy_(to_dev(a))
        gl.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        want = p.forward()
        assert torch.equal(loss, want[0]) and torch.equal(cnt, want[1])
        assert torch.equal(gl, p.backward(want[1]))


def test_two_calls_at_once():
    """Two handles on two streams, each with its own workspace."""
    ps = [Problem(20000, 128, 8, s, offsets([7000, 13000]), seed=i)
          for i, s in enumerate(("softmax", "sigmoid"))]
    want = [p.forward() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    data = [(to_dev(p.logits), to_dev(p.idx), to_dev(p.off), moe.balance_workspace(p.r.h, 2)) for p in ps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for p, st, (l, i, o, ws) in zip(ps, streams, data):
            with torch.cuda.stream(st):
                out = (torch.empty(1, device=dev()), torch.empty(2, 128, dtype=torch.int32, device=dev()))
                moe.moe_balance(p.r.h, l, i, out[0], out[1], ws, seq_off=o, coef=0.02)
                outs.append(out)
    torch.cuda.synchronize()
    for n, out in enumerate(outs):
        assert torch.equal(out[0], want[n % 2][0]) and torch.equal(out[1], want[n % 2][1])


def test_two_graphs_replayed_at_once():
    """Each with its own workspace, on one handle."""
    ps = [Problem(5000, 64, 4, "softmax", offsets([1500 + i, 3000]), seed=i) for i in range(2)]
    h = ps[0].r.h
    graphs, outs = [], []
    want = [p.forward() for p in ps]
    for p in ps:
        l, i, o, ws = to_dev(p.logits), to_dev(p.idx), to_dev(p.off), moe.balance_workspace(h, 2)
        out = (torch.empty(1, device=dev()), torch.empty(2, 64, dtype=torch.int32, device=dev()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_balance(h, l, i, out[0], out[1], ws, seq_off=o, coef=0.02)
        graphs.append((g, l, i, o, ws))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_methods_allocate_what_they_return():
    p = Problem(900, 32, 4, "sigmoid", offsets([100, 500]))
    l, i, o = to_dev(p.logits), to_dev(p.idx), to_dev(p.off)
    loss, cnt, prob = p.r.balance(l, i, seq_off=o, coef=0.02)
    want = p.forward()
    assert torch.equal(loss, want[0]) and torch.equal(cnt, want[1]) and torch.equal(prob, want[2])
    g = p.r.balance_bwd(l, cnt, seq_off=o, coef=0.02)
    wg = p.backward(cnt)
    assert torch.equal(g[:600], wg[:600]) and not g[600:].any()  # places of no sequence: 0
    base = to_dev(p.base)
    g = p.r.balance_bwd(l, cnt, seq_off=o, coef=0.02, base=base)
    assert torch.equal(g[:600], p.backward(cnt, base=p.base)[:600]) and torch.equal(g[600:], base[600:])


def test_refusals():
    p = Problem(64, 8, 2, "softmax")
    h, L = p.r.h, moe.lib()
    l, i, o = to_dev(p.logits), to_dev(p.idx), to_dev(p.off)
    loss, gl = torch.zeros(1, device=dev()), torch.zeros(64, 8, device=dev())
    cnt = torch.zeros(1, 8, dtype=torch.int32, device=dev())
    ws = moe.balance_workspace(h, 1)

    def fwd(**kw):
        a = dict(l=l.data_ptr(), i=i.data_ptr(), T=64, o=None, S=1, c=1.0, loss=loss.data_ptr(),
                 cnt=cnt.data_ptr(), p=None, ws=ws.data_ptr(), n=ws.numel())
        a.update(kw)
        return L.moe_balance(h.ptr, a["l"], a["i"], a["T"], a["o"], a["S"], a["c"], a["loss"],
                             a["cnt"], a["p"], a["ws"], a["n"], None)

    def bwd(**kw):
        a = dict(l=l.data_ptr(), cnt=cnt.data_ptr(), T=64, o=None, S=1, c=1.0, g=None, b=None,
                 out=gl.data_ptr())
        a.update(kw)
        return L.moe_balance_bwd(h.ptr, a["l"], a["cnt"], a["T"], a["o"], a["S"], a["c"], a["g"],
                                 a["b"], a["out"], None)

    assert fwd() == moe.MOE_OK and bwd() == moe.MOE_OK
    assert fwd(T=65) == moe.MOE_ERR_CAPACITY and bwd(T=65) == moe.MOE_ERR_CAPACITY
    for bad in (dict(T=-1), dict(l=None), dict(i=None), dict(loss=None), dict(cnt=None), dict(S=0),
                dict(S=2), dict(o=o.data_ptr() + 2), dict(l=l.data_ptr() + 1), dict(p=loss.data_ptr() + 2),
                dict(c=float("nan")), dict(c=1e300), dict(ws=None), dict(ws=ws.data_ptr() + 16),
                dict(n=ws.numel() - 1)):
        assert fwd(**bad) == moe.MOE_ERR_INVALID, bad
    for bad in (dict(T=-1), dict(l=None), dict(cnt=None), dict(out=None), dict(S=0), dict(S=2),
                dict(c=float("inf")), dict(g=loss.data_ptr() + 1), dict(b=gl.data_ptr() + 3)):
        assert bwd(**bad) == moe.MOE_ERR_INVALID, bad
    for call in (lambda: moe.moe_balance(h, l, i, loss, cnt, ws, seq_off=o[:1]),
                 lambda: moe.moe_balance(h, l, i, loss, cnt, ws, seq_off=to_dev(np.array([0, 3, 64], np.int32))),
                 lambda: moe.moe_balance(h, l, i[:, :1], loss, cnt, ws),
                 lambda: moe.moe_balance(h, l[:, ::2], i, loss, cnt, ws),
                 lambda: moe.moe_balance_bwd(h, l, cnt, gl[:32])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_balance(h, l.double(), i, loss, cnt, ws),
                 lambda: moe.moe_balance(h, l, i.long(), loss, cnt, ws),
                 lambda: moe.moe_balance(h, l, i, loss, cnt, ws, seq_off=o.long()),
                 lambda: moe.moe_balance_bwd(h, l, cnt.float(), gl)):
        with pytest.raises(TypeError):
            call()
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(h) == 0


def test_too_many_sequences_are_refused():
    p = Problem(64, 8, 2, "softmax")
    h, L = p.r.h, moe.lib()
    l, i, o = to_dev(p.logits), to_dev(p.idx), to_dev(p.off)
    loss, gl = torch.zeros(1, device=dev()), torch.zeros(64, 8, device=dev())
    cnt = torch.zeros(1, 8, dtype=torch.int32, device=dev())
    ws = moe.balance_workspace(h, 1)
    for S in ((1 << 30) + 1, 2 ** 31 - 1):
        assert L.moe_balance(h.ptr, l.data_ptr(), i.data_ptr(), 64, o.data_ptr(), S, 1.0,
                             loss.data_ptr(), cnt.data_ptr(), None, ws.data_ptr(), ws.numel(),
                             None) == moe.MOE_ERR_INVALID
        assert L.moe_balance_bwd(h.ptr, l.data_ptr(), cnt.data_ptr(), 64, o.data_ptr(), S, 1.0,
                                 None, None, gl.data_ptr(), None) == moe.MOE_ERR_INVALID


def gradient_of_one_sequence(logits, cnt, T, K, score, coef):
    """(gradient, bound) of some tokens of one sequence of T, whatever its counts.
    A constant m may be taken off the counts, as p sums to 1: with d = c - m the
    gradient is B q (d - sum p d).  A relative error r of p and q makes one of at
    most r B q (|d| + sum p |d|) of it, and so do the additions: the bound of
    block_ref.balance_bwd, whose m is K T / E.  The counts' own mean, as here, is
    that if no entry was dropped; where some were, or where the counts are any
    numbers, another m would leave a part of |m| in d and in the error."""
    E = logits.shape[1]
    p, q, _ = ref.probabilities(logits, score)
    c = cnt.astype(np.float64)
    d = c - np.rint(c.mean())
    B = coef * E / (K * float(T) ** 2)
    want = B * q * (d - (p * d).sum(1, keepdims=True))
    away = np.abs(d) + (p * np.abs(d)).sum(1, keepdims=True)
    rel = 2 * ref.probability_error(logits, score) + (16 + ref.TREE) * ref.U32
    return want, abs(B) * q * away * rel


@pytest.mark.parametrize("E", [8, 24, 256])
@pytest.mark.parametrize("top", [0.0, -15.0, 30.0])
def test_slopes_of_sigmoids_far_below_the_rows_largest(top, E):
    """One expert at `top`, the others at -69 to -87: their slope is their sigmoid
    itself, within the bound of every other logit.  coef keeps the gradient above
    fp32's smallest normal value."""
    p = Problem(6, E, 2, "sigmoid", seed=E)
    g = np.random.default_rng(E)
    p.logits[:] = g.uniform(-87.0, -69.0, p.logits.shape)
    p.logits[np.arange(6), g.integers(0, E, 6)] = top
    cnt = to_dev(g.integers(0, 7, (1, E)).astype(np.int32))
    got = to_host(p.backward(cnt, coef=1e6)).astype(np.float64)
    want, bound = gradient_of_one_sequence(p.logits, to_host(cnt)[0], 6, 2, "sigmoid", 1e6)
    assert (np.abs(want) > 1e3 * ref.TINY).mean() > 0.5
    bad = ~(np.abs(got - want) <= bound + ref.TINY)
    assert not bad.any(), "%d of %d out of bound, worst ratio %.3g" % (
        bad.sum(), bad.size, (np.abs(got - want) / (bound + ref.TINY)).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(400000, 8, 2), (400000, 100, 16), (100000, 384, 16)])
def test_gradient_of_even_counts_with_dropped_entries(T, E, K, score):
    """A long sequence whose counts differ by some tens, 30% of its entries dropped:
    the gradient, which is made of those differences, keeps their digits."""
    r = moe.MoeRouter(E, K, 1, T, score_fn=score)
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    even = K * T * 7 // (E * 10)
    cnt = (even + torch.randint(-20, 21, (1, E), generator=g, device="cuda")).to(torch.int32)
    glogits = torch.empty_like(logits)
    moe.moe_balance_bwd(r.h, logits, cnt, glogits, coef=1.0)
    for rows in (slice(0, 1000), slice(T - 1000, T)):
        l, got = to_host(logits[rows]), to_host(glogits[rows]).astype(np.float64)
        want, bound = gradient_of_one_sequence(l, to_host(cnt)[0], T, K, score, 1.0)
        bad = ~(np.abs(got - want) <= bound + ref.TINY)
        assert not bad.any(), "%d of %d out of bound, worst ratio %.3g" % (
            bad.sum(), bad.size, (np.abs(got - want) / (bound + ref.TINY)).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gloss", [np.inf, -np.inf, np.nan])
def test_tokens_without_probabilities_get_the_base_whatever_the_gradient(gloss, score):
    """A scaled loss whose gradient overflowed spoils the tokens that have a part in
    the loss, no others."""
    p = Problem(300, 24, 2, score, seed=5)
    p.logits[30:40] = -np.inf
    p.logits[7, 5] = np.nan
    p.logits[299, 23] = np.inf
    none = np.zeros(300, bool)
    none[[7, 299]] = none[30:40] = True
    _, cnt, _ = p.forward()
    for in_place in (False, True):
        got = to_host(p.backward(cnt, gloss=gloss, base=p.base, in_place=in_place))
        assert np.array_equal(got[none], p.base[none])
        assert not np.isfinite(got[~none]).any()
