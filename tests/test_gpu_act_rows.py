"""The gated expert activation with dropout and its backward on the GPU against
their fp64 definitions.

Tolerances: an output is one rounding of an fp32 product.  The fp32 factors
carry the exponential's documented error (fast: 2 + floor(1.16 |c|) ulp; the
tests keep |c| below 24, so 30 ulp, 3.6e-6; accurate: 2 ulp), the fast
division's 2 ulp and at most six product roundings: REL = 5e-6 for bf16 rows,
1e-6 for fp32 rows.  A sum of terms is held to REL of its terms' magnitudes
plus I fp32 additions.  Masked elements and pad rows are exactly 0."""
import numpy as np
import pytest
import torch

import combine_moe_route_05_gb300 as moe
import synth
from tests import expert_ref as ref
from tests.gpu_util import dev, to_dev, to_host

pytestmark = pytest.mark.gpu

REL = {"bf16": 5e-6, "f32": 1e-6}
U = {"bf16": ref.U_BF16, "f32": ref.U_F32}
SENTINEL = 0.5


def f64(bits):
    a = to_host(bits)
    return (synth.bf16_bits_to_f32(a) if a.dtype == np.uint16 else a).astype(np.float64)


def problem(T, E, K, I, dtype, pad=1, seed=0, idx=None, scale=1.0):
    g = np.random.default_rng(seed)
    if idx is None:
        idx = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
    r = moe.MoeRouter(E, K, 1, max(T, 1), pad_align=pad)
    lay = {k: v.cpu().numpy() for k, v in r.layout(to_dev(idx)).items()}
    rows = r.h.recv_rows
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    gu = torch.from_numpy(g.standard_normal((rows, 2 * I)) * scale).to(dev(), td)
    ghs = torch.from_numpy(g.standard_normal((rows, I))).to(dev(), td)
    rw = torch.from_numpy(g.random(rows).astype(np.float32)).to(dev())
    ent = np.where(lay["recv_token"] >= 0, lay["recv_token"].astype(np.int64) * K + lay["recv_k"], -1)
    return r, ent, int(lay["off_e"][-1]), gu, ghs, rw


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=dev())


def ok(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d out of bound, worst %.3g over %.3g" % (
        what, bad.sum(), bad.size, np.abs(got - want)[bad].max(), bound[bad].max())


def check_fwd(r, ent, end, gu, rw, act, p, seed, offset, dtype):
    I = gu.shape[1] // 2
    hs = torch.full((gu.shape[0], I), SENTINEL, dtype=gu.dtype, device=dev())
    moe.moe_act_rows(r.h, gu, rw, hs, act=act, p=p, rng=rng_of(seed, offset) if p else None)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(r.h) == 0
    got = f64(hs)
    assert (got[end:] == SENTINEL).all()
    w = to_host(rw) if rw is not None else np.ones(gu.shape[0])
    mask, scale = ref.kept_mask(np.maximum(ent, 0), I, p, seed, offset)
    mask &= (ent >= 0)[:, None]
    want = ref.act_rows(f64(gu), w, act, mask, scale)[:end]
    assert (got[:end][~mask[:end]] == 0.0).all()
    ok(got[:end], want, np.abs(want) * (U[dtype] + REL[dtype]) + ref.TINY, "hs")


def check_bwd(r, ent, end, gu, ghs, rw, act, p, seed, offset, dtype, in_place=False):
    I, T, K = ghs.shape[1], r.h.T, r.h.K
    gu64 = f64(gu)
    ggu = gu if in_place else torch.full_like(gu, SENTINEL)
    gw = torch.full((T, K), -3.0, device=dev()) if rw is not None else None
    moe.moe_act_rows_bwd(r.h, ghs, gu, rw, ggu, gw, act=act, p=p,
                         rng=rng_of(seed, offset) if p else None)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(r.h) == 0
    got = f64(ggu)
    if not in_place:
        assert (got[end:] == SENTINEL).all()
    w = to_host(rw) if rw is not None else np.ones(gu.shape[0])
    mask, scale = ref.kept_mask(np.maximum(ent, 0), I, p, seed, offset)
    mask &= (ent >= 0)[:, None]
    want, wgw, tg, tw = ref.act_rows_bwd(f64(ghs), gu64, w, act, mask, scale)
    both = np.concatenate([mask, mask], 1)[:end]
    assert (got[:end][~both] == 0.0).all()
    bound = np.abs(want) * U[dtype] + ref.TINY
    bound[:, :I] += REL[dtype] * 2 * tg
    bound[:, I:] += REL[dtype] * np.abs(want[:, I:])
    ok(got[:end], want[:end], bound[:end], "ggu")
    if gw is not None:
        full, fb = np.zeros(T * K), np.zeros(T * K)
        real = ent >= 0
        full[ent[real]] = wgw[real]
        fb[ent[real]] = (tw * (I * ref.U_F32 + 2 * REL[dtype]))[real]
        ok(to_host(gw).reshape(-1).astype(np.float64), full, fb, "gw")


CASES = [
    # T, E, K, I, dtype, act, p, absorb, pad
    (1, 4, 1, 8, "bf16", "silu", 0.0, True, 1),
    (1, 4, 2, 4, "f32", "gelu", 0.5, True, 1),
    (3, 8, 2, 12, "f32", "silu", 0.1, False, 1),       # half a generator block at the row's end
    (37, 13, 3, 264, "bf16", "gelu", 0.1, True, 1),
    (64, 16, 16, 40, "bf16", "silu", 0.9, True, 7),
    (100, 5, 2, 1000, "bf16", "silu", 0.25, False, 128),
    (100, 5, 2, 1000, "f32", "gelu", 0.25, True, 128),
    (257, 512, 8, 72, "bf16", "gelu", 0.0, False, 3),
    (700, 64, 4, 2048, "bf16", "silu", 0.1, True, 1),
    (5, 8, 2, 20000, "bf16", "silu", 0.3, True, 1),
]


@pytest.mark.parametrize("T,E,K,I,dtype,act,p,absorb,pad", CASES)
def test_forward(T, E, K, I, dtype, act, p, absorb, pad):
    r, ent, end, gu, _, rw = problem(T, E, K, I, dtype, pad)
    check_fwd(r, ent, end, gu, rw if absorb else None, act, p, 99, 5, dtype)


@pytest.mark.parametrize("T,E,K,I,dtype,act,p,absorb,pad", CASES)
def test_backward(T, E, K, I, dtype, act, p, absorb, pad):
    r, ent, end, gu, ghs, rw = problem(T, E, K, I, dtype, pad)
    check_bwd(r, ent, end, gu, ghs, rw if absorb else None, act, p, 99, 5, dtype)


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward_in_place(p):
    r, ent, end, gu, ghs, rw = problem(50, 8, 2, 136, "bf16", 16)
    check_bwd(r, ent, end, gu, ghs, rw, "silu", p, 3, 4, "bf16", in_place=True)


@pytest.mark.parametrize("seed,offset", [(0, 0), (-1, -1), (2 ** 63 - 1, 2 ** 32), (1 << 33, 1 << 40)])
def test_seed_and_offset_are_64_bits(seed, offset):
    r, ent, end, gu, ghs, rw = problem(20, 8, 2, 64, "f32")
    check_fwd(r, ent, end, gu, rw, "silu", 0.4, seed, offset, "f32")
    check_bwd(r, ent, end, gu, ghs, rw, "silu", 0.4, seed, offset, "f32")


@pytest.mark.parametrize("p", [1e-9, 2.0 ** -16, 0.99998])
def test_extreme_probabilities(p):
    """D = 0 (nothing dropped, no generator needed), 1 and 65535."""
    r, ent, end, gu, ghs, rw = problem(40, 8, 2, 512, "bf16")
    check_fwd(r, ent, end, gu, rw, "silu", p, 8, 9, "bf16")
    if p == 1e-9:
        hs = torch.empty(gu.shape[0], 512, dtype=gu.dtype, device=dev())
        moe.moe_act_rows(r.h, gu, rw, hs, p=p)


def test_large_gates_and_values():
    """Gates of +-100 and +-1e4: the sigmoid saturates; no NaN, 0 or identity."""
    for act in ("silu", "gelu"):
        r, ent, end, gu, ghs, rw = problem(8, 4, 2, 64, "f32")
        I = 64
        gu[:, :I] = torch.tensor([100.0, -100.0, 1e4, -1e4], device=dev()).repeat(I // 4)
        hs, ggu = torch.empty_like(ghs), torch.empty_like(gu)
        moe.moe_act_rows(r.h, gu, None, hs, act=act)
        moe.moe_act_rows_bwd(r.h, ghs, gu, None, ggu, act=act)
        g, u, d = gu[:, :I], gu[:, I:], ghs
        pos = g > 0
        assert torch.equal(hs[pos], (g * u)[pos]) and (hs[~pos].abs() < 1e-30).all()
        assert torch.equal(ggu[:, :I][pos], (d * u)[pos]) and (ggu[:, :I][~pos].abs() < 1e-30).all()
        assert torch.equal(ggu[:, I:][pos], (d * g)[pos]) and (ggu[:, I:][~pos].abs() < 1e-30).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_whose_square_is_infinite(dtype, act):
    """Gates of +-2^70 and +-2^127: a is the identity or 0 and its derivative 1
    or 0, as for any saturated gate."""
    r, ent, end, gu, ghs, rw = problem(8, 4, 2, 64, dtype)
    I = 64
    gu[:, :I] = torch.tensor([2.0 ** 70, -2.0 ** 70, 2.0 ** 127, -2.0 ** 127], device=dev()).repeat(I // 4)
    gu[:, I:].clamp_(-1, 1)
    ghs.clamp_(-1, 1)
    hs, ggu = torch.empty_like(ghs), torch.empty_like(gu)
    moe.moe_act_rows(r.h, gu, None, hs, act=act)
    moe.moe_act_rows_bwd(r.h, ghs, gu, None, ggu, act=act)
    g, u, d = gu[:, :I], gu[:, I:], ghs
    one = (g > 0).to(g.dtype)
    assert torch.equal(hs, one * g * u)
    assert torch.equal(ggu[:, :I], one * d * u) and torch.equal(ggu[:, I:], one * d * g)


def test_masked_places_hide_nan_and_infinity():
    """NaN and infinity in dropped elements and pad rows reach no output."""
    p, seed, off = 0.5, 11, 12
    r, ent, end, gu, ghs, rw = problem(30, 6, 2, 128, "bf16", 8)
    mask, _ = ref.kept_mask(np.maximum(ent, 0), 128, p, seed, off)
    hidden = torch.from_numpy(~(mask & (ent >= 0)[:, None])).to(dev())
    clean = [gu.clone(), ghs.clone(), rw.clone()]
    gu[:, :128][hidden] = float("nan")
    gu[:, 128:][hidden] = float("inf")
    ghs[hidden] = float("-inf")
    rw[torch.from_numpy(ent < 0).to(dev())] = float("nan")

    def both(gu, ghs, rw):
        hs, ggu = torch.zeros_like(ghs), torch.zeros_like(gu)
        gw = torch.empty(30, 2, device=dev())
        moe.moe_act_rows(r.h, gu, rw, hs, p=p, rng=rng_of(seed, off))
        moe.moe_act_rows_bwd(r.h, ghs, gu, rw, ggu, gw, p=p, rng=rng_of(seed, off))
        return hs, ggu, gw
    for a, b in zip(both(gu, ghs, rw), both(*clean)):
        assert torch.equal(a, b)


def test_dropped_entries_get_no_row_and_a_zero_gradient():
    g = np.random.default_rng(2)
    idx = np.argsort(g.random((40, 9)), axis=1)[:, :3].astype(np.int32)
    idx[4, 1] = 77
    idx[9, 2] = idx[9, 0]
    idx[20] = -1
    r, ent, end, gu, ghs, rw = problem(40, 9, 3, 64, "bf16", idx=idx)
    moe.moe_clear_device_status(r.h)
    assert end == 40 * 3 - 5
    check_fwd(r, ent, end, gu, rw, "silu", 0.2, 1, 1, "bf16")
    check_bwd(r, ent, end, gu, ghs, rw, "silu", 0.2, 1, 1, "bf16")


def test_mask_does_not_depend_on_the_layout():
    """The same routing packed and padded: each entry's row is the same."""
    idx = np.argsort(np.random.default_rng(5).random((60, 10)), axis=1)[:, :4].astype(np.int32)
    out = []
    for pad in (1, 32):
        r, ent, end, _, _, _ = problem(60, 10, 4, 96, "f32", pad, idx=idx)
        gu = torch.ones(r.h.recv_rows, 192, device=dev())
        hs = r.act_rows(gu, p=0.5, rng=rng_of(6, 7))
        rows = np.empty(240, np.int64)
        rows[ent[ent >= 0]] = np.nonzero(ent >= 0)[0]
        out.append(to_host(hs)[rows])
    assert np.array_equal(out[0], out[1])


def test_captured_graph_draws_a_new_mask_per_replay():
    r, ent, end, gu, ghs, rw = problem(64, 8, 2, 256, "bf16")
    state = rng_of(21, 0)
    hs, ggu, gw = torch.empty_like(ghs), torch.empty_like(gu), torch.empty(64, 2, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            state[1] += 1
            moe.moe_act_rows(r.h, gu, rw, hs, p=0.5, rng=state)
            moe.moe_act_rows_bwd(r.h, ghs, gu, rw, ggu, gw, p=0.5, rng=state)
    torch.cuda.current_stream().wait_stream(s)
    seen = []
    for step in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert state.tolist() == [21, step]
        eager = r.act_rows(gu, rw, p=0.5, rng=rng_of(21, step))
        e_ggu, e_gw = r.act_rows_bwd(ghs, gu, rw, p=0.5, rng=rng_of(21, step))
        assert torch.equal(hs, eager) and torch.equal(ggu, e_ggu) and torch.equal(gw, e_gw)
        seen.append(hs.clone())
    assert not torch.equal(seen[0], seen[1])


def test_gradients_against_differences():
    """fp32 rows, the dropped mask held fixed: central differences of the
    kernel's own forward.  h = 2^-7: truncation h^2/6 |a'''| |u| < 5e-5, fp32
    rounding of an output below 8 over 2h: 8 * 2^-23 / 2^-6 = 6e-5."""
    r, ent, end, gu, ghs, rw = problem(6, 4, 2, 32, "f32")
    I, h, kw = 32, 2.0 ** -7, dict(act="gelu", p=0.25, rng=rng_of(5, 6))
    gu = gu.clamp(-3, 3)
    ggu, gw = r.act_rows_bwd(torch.ones_like(ghs), gu, rw, **kw)
    for half in (0, 1):
        step = torch.zeros_like(gu)
        step[:, half * I:(half + 1) * I] = h
        diff = (r.act_rows(gu + step, rw, **kw) - r.act_rows(gu - step, rw, **kw)) / (2 * h)
        assert (diff - ggu[:, half * I:(half + 1) * I]).abs().max() < 1.5e-3
    gain = (r.act_rows(gu, rw + h, **kw) - r.act_rows(gu, rw - h, **kw)).sum(1) / (2 * h)
    real = torch.from_numpy(ent).to(dev())
    assert (gain - gw.reshape(-1)[real]).abs().max() < 32 * 6e-5


@pytest.mark.parametrize("bad", ["p1", "pneg", "pnan", "no_rng", "gw_without_w", "width", "act", "state"])
def test_refusals(bad):
    r, ent, end, gu, ghs, rw = problem(8, 4, 2, 64, "bf16")
    hs, ggu, gw = torch.empty_like(ghs), torch.empty_like(gu), torch.empty(8, 2, device=dev())
    kw = dict(p1=dict(p=1.0), pneg=dict(p=-0.1), pnan=dict(p=float("nan")), no_rng=dict(p=0.5),
              act=dict(act=2)).get(bad, {})
    status = moe.MOE_ERR_INVALID
    if bad == "p1":
        kw["rng"] = rng_of(1, 1)
    if bad == "state":
        r, status = moe.MoeRouter(4, 2, 1, 8), moe.MOE_ERR_STATE
    if bad == "width":  # rows of 8 bytes
        gu, hs, ggu, ghs = (t[:, :w].contiguous() for t, w in ((gu, 8), (hs, 4), (ggu, 8), (ghs, 4)))
    if bad != "gw_without_w":
        with pytest.raises(moe.MoeError) as e:
            moe.moe_act_rows(r.h, gu, rw, hs, **kw)
        assert e.value.status == status
    with pytest.raises(moe.MoeError) as e:
        moe.moe_act_rows_bwd(r.h, ghs, gu, None if bad == "gw_without_w" else rw, ggu, gw, **kw)
    assert e.value.status == status


def test_empty_batch_and_other_stream():
    r, ent, end, gu, ghs, rw = problem(0, 4, 2, 64, "bf16")
    assert r.act_rows(gu, rw).shape == (0, 64)
    r, ent, end, gu, ghs, rw = problem(500, 4, 2, 64, "bf16")
    want = r.act_rows(gu, rw, p=0.1, rng=rng_of(1, 2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r.act_rows(gu, rw, p=0.1, rng=rng_of(1, 2), stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def outputs_of(method, stream):
    """Their (address, bytes), freed, after the current stream has been made to wait
    for `stream` and given some 50 ms of work."""
    out = method(stream)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda._sleep(100000000)
    return [(t.data_ptr(), t.numel() * t.element_size()) for t in out]


@pytest.mark.parametrize("name", ["act_rows", "act_rows_bwd", "layer"])
def test_methods_on_another_stream_keep_their_outputs(name):
    """What a method returns, once freed, is given neither to the current stream
    while the other one may still write it nor to the other one while the current
    one may still read it."""
    r, ent, end, gu, ghs, rw = problem(100, 4, 2, 64, "bf16")
    x = torch.randn(8, 64, device=dev()).to(torch.bfloat16)
    w13, w2 = torch.zeros(4, 64, 64, device=dev()).to(torch.bfloat16), torch.zeros(4, 64, 32, device=dev()).to(torch.bfloat16)
    logits = torch.randn(8, 4, device=dev())
    method = {"act_rows": lambda s: (r.act_rows(gu, rw, stream=s),),
              "act_rows_bwd": lambda s: r.act_rows_bwd(ghs, gu, rw, stream=s),
              "layer": lambda s: r.layer(x, logits, w13, w2, stream=s)}[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = outputs_of(method, s)
    here = [torch.empty(n, dtype=torch.uint8, device=dev()) for _, n in seen for _ in range(2)]
    with torch.cuda.stream(s):
        there = [torch.empty(n, dtype=torch.uint8, device=dev()) for _, n in seen for _ in range(2)]
    assert not torch.cuda.current_stream().query()  # the current stream is not done with them
    assert not {p for p, _ in seen} & {t.data_ptr() for t in here + there}
    torch.cuda.synchronize()


def test_methods_on_a_forked_stream_of_a_captured_graph():
    """Both activations and the layer on a second stream inside a capture, an output
    freed before the capture ends."""
    r, ent, end, gu, ghs, rw = problem(60, 4, 2, 64, "bf16")
    g = torch.Generator().manual_seed(3)
    x = torch.randn(8, 64, generator=g).to(dev(), torch.bfloat16)
    w13 = (torch.randn(4, 64, 64, generator=g) / 8).to(dev(), torch.bfloat16)
    w2 = (torch.randn(4, 64, 32, generator=g) / 6).to(dev(), torch.bfloat16)
    logits = torch.randn(8, 4, generator=g).to(dev())
    side = torch.cuda.Stream()

    def both(stream):
        hs = r.act_rows(gu, rw, stream=stream)
        ggu, gw = r.act_rows_bwd(ghs, gu, rw, stream=stream)
        out = r.layer(x, logits, w13, w2, stream=stream)[0]
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        doubled = hs * 2
        del hs
        return doubled, ggu * 1, gw * 1, out * 1
    want = both(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = both(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
