"""The few-token layer at the precision its interface states: layers whose result
is exact, bit for bit, and random ones within a bound that leaves no room for a
lost low part (tests/layer_ref.py; that it does not is tested without a GPU)."""
import numpy as np
import pytest
import torch

import combine_moe_route_05_gb300 as moe
from tests import layer_ref as ref
from tests.gpu_util import dev, to_host

# sizes on both sides of the kernels' rule: a token an expert and less, several,
# tens; columns that end inside a stage, a tile, a block of scales
EXACT = [
    dict(T=1, E=4, K=1, H=16, I=16),
    dict(T=3, E=8, K=2, H=64, I=48),
    dict(T=7, E=16, K=4, H=520, I=136, shared=1),
    dict(T=9, E=12, K=2, H=72, I=1032),
    dict(T=6, E=32, K=2, H=200, I=400, shared=1),
    dict(T=13, E=16, K=2, H=24, I=200, shared=1),
    dict(T=20, E=16, K=2, H=264, I=72),
    dict(T=24, E=16, K=3, H=136, I=104),
    dict(T=4, E=4, K=3, H=264, I=136, shared=1),
    dict(T=24, E=16, K=3, H=136, I=104, shared=2),
    dict(T=40, E=4, K=2, H=264, I=72),
    dict(T=60, E=6, K=2, H=392, I=264, shared=1),
    dict(T=128, E=3, K=3, H=136, I=136, shared=4),
    dict(T=128, E=2, K=1, H=1032, I=520),
    dict(T=1, E=8, K=2, H=16, I=16, e4m3=True),
    dict(T=4, E=8, K=2, H=160, I=288, e4m3=True, shared=1),
    dict(T=6, E=16, K=2, H=1040, I=144, e4m3=True),
    dict(T=14, E=32, K=2, H=144, I=272, e4m3=True),
    dict(T=20, E=6, K=2, H=128, I=336, e4m3=True),
    dict(T=40, E=4, K=2, H=272, I=144, e4m3=True, shared=2),
    dict(T=100, E=2, K=2, H=400, I=176, e4m3=True),
    dict(T=128, E=5, K=1, H=144, I=528, e4m3=True, shared=1),
]

RANDOM = [
    dict(T=5, E=8, K=2, H=64, I=64),
    dict(T=8, E=16, K=2, H=72, I=48, shared=1),
    dict(T=16, E=8, K=2, H=64, I=56),
    dict(T=33, E=4, K=2, H=120, I=136, act="gelu"),
    dict(T=64, E=3, K=2, H=64, I=72, shared=1),
    dict(T=4, E=8, K=2, H=64, I=48, e4m3=True),
    dict(T=8, E=16, K=2, H=96, I=32, e4m3=True, act="gelu"),
    dict(T=40, E=4, K=2, H=64, I=48, e4m3=True),
    dict(T=70, E=3, K=1, H=80, I=32, e4m3=True, shared=1),
]


class RandomProblem:
    """Weights of standard deviation fan-in^-1/2, tokens of 1; with e4m3 weights the
    block scales are powers of two."""

    def __init__(self, T, E, K, H, I, shared=0, e4m3=False, act="silu", seed=0):
        g = np.random.default_rng(seed)
        self.T, self.E, self.K, self.H, self.I, self.S, self.e4m3 = T, E, K, H, I, shared, e4m3
        n = E + shared
        x = ref.bf16(g.standard_normal((T, H)))
        self.idx = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
        self.w = g.random((T, K)).astype(np.float32).astype(np.float64)
        self.s13 = self.s2 = None
        if not e4m3:
            w13, w2 = (ref.bf16(g.standard_normal(s) * s[2] ** -0.5) for s in ((n, 2 * I, H), (n, H, I)))
        else:
            v = []
            for s in ((n, 2 * I, H), (n, H, I)):
                q = torch.from_numpy((g.standard_normal(s) * 64).clip(-448, 448).astype(np.float32))
                q = q.to(torch.float8_e4m3fn).double().numpy()
                c = 2.0 ** (g.integers(-1, 2, (n, -(-s[1] // 128), -(-s[2] // 128))) - 6 -
                            np.round(np.log2(s[2]) / 2))
                v += [q, c.astype(np.float32),
                      q * np.repeat(np.repeat(c, 128, 1), 128, 2)[:, :s[1], :s[2]]]
            self.q13, self.s13, w13, self.q2, self.s2, w2 = v
        self.x, self.w13, self.w2 = x, w13, w2
        self.args = (x, self.idx, self.w, w13, w2, shared, E, act, e4m3)


def run(p, act="silu"):
    """Out of the routes p.idx, p.w on the GPU."""
    def t(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dev(), dtype)
    wt = torch.float8_e4m3fn if p.e4m3 else torch.bfloat16
    h = moe.Handle(moe.make_config(p.E, p.K, 1, p.T))
    out = torch.full((p.T, p.H), float("nan"), dtype=torch.bfloat16, device=dev())
    ws = moe.layer_workspace(h, p.H, p.I, p.S).fill_(0xff)
    moe.moe_layer(h, t(p.x, torch.bfloat16), None, t(p.q13 if p.e4m3 else p.w13, wt),
                  t(p.q2 if p.e4m3 else p.w2, wt), out, torch.from_numpy(p.idx).to(dev()),
                  t(p.w, torch.float32), ws, s13=t(p.s13, torch.float32) if p.e4m3 else None,
                  s2=t(p.s2, torch.float32) if p.e4m3 else None, act=act, num_shared=p.S)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(h) == 0
    return to_host(out.double())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kw", EXACT, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_exact_layers(kw, act):
    p = ref.Exact(**kw)
    got, want = run(p, act), p.want()
    bad = got != want
    assert not bad.any(), "%d of %d differ, the first at %s: %r for %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


@pytest.mark.gpu
@pytest.mark.parametrize("kw", RANDOM, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_stated_precision(kw):
    p = RandomProblem(**kw)
    want, bound = ref.layer(*p.args)
    err = np.abs(run(p, kw.get("act", "silu")) - want)
    assert (err <= bound).all(), "worst %.3g of its bound" % (err / bound).max()
