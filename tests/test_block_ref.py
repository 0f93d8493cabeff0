"""The fp64 definitions of the balance loss and the norms around a block: closed
forms, invariants, and their gradients against central differences (CPU)."""
import ctypes

import numpy as np
import pytest

from tests import block_ref as ref


def routed(rng, T, E, K):
    return np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_even_routing_costs_the_coefficient(score):
    """Equal logits and an even count: E / (K n^2) * E * (K n / E) * (n / E) = 1."""
    E, K, n = 8, 2, 16
    idx = np.stack([(np.arange(K) + K * t) % E for t in range(n)]).astype(np.int32)
    loss, cnt, prob = ref.balance(np.full((n, E), -0.7), idx, np.array([0, n]), E, score, 0.25)
    assert (cnt == K * n // E).all() and np.allclose(prob, 1.0 / E)
    assert loss == pytest.approx(0.25, rel=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_expert_for_all_costs_most(score):
    E, n = 8, 16
    logits = np.full((n, E), -60.0)
    logits[:, 3] = 60.0
    loss, _, _ = ref.balance(logits, np.full((n, 1), 3, np.int32), np.array([0, n]), E, score, 1.0)
    assert loss == pytest.approx(E, rel=1e-12)


def test_entries_that_do_not_count():
    idx = np.array([[0, 0], [-1, 2], [5, 1], [-7, 3]], np.int32)
    assert ref.counts(idx, np.array([0, 4]), 4).tolist() == [[1, 1, 1, 1]]


def test_rows_that_count_for_nothing():
    l = np.zeros((4, 3))
    l[0] = -np.inf
    l[1, 0] = np.nan
    l[2, 1] = np.inf
    l[3, 2] = -np.inf
    for score in ("softmax", "sigmoid"):
        p, q, bad = ref.probabilities(l, score)
        assert (p[:3] == 0).all() and (q[:3] == 0).all() and bad.tolist() == [False, True, True, False]
        assert np.allclose(p[3], [0.5, 0.5, 0.0])


def test_far_negative_sigmoids_normalise_like_the_softmax():
    l = np.random.default_rng(0).standard_normal((5, 7)) - 800.0
    assert np.allclose(ref.probabilities(l, "sigmoid")[0], ref.probabilities(l, "softmax")[0], rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [0.0, -50.0])
def test_balance_gradient_equals_differences(score, shift):
    rng = np.random.default_rng(3)
    T, E, K = 11, 6, 2
    off = np.array([0, 4, 4, 9])
    logits, idx = rng.standard_normal((T, E)) + shift, routed(rng, T, E, K)
    _, cnt, _ = ref.balance(logits, idx, off, E, score, 0.3)
    g, _ = ref.balance_bwd(logits, cnt, off, K, score, 0.3, 1.7)
    step = 1e-5
    for t in range(T):
        for e in range(E):
            d = []
            for sgn in (1, -1):
                moved = logits.copy()
                moved[t, e] += sgn * step
                d.append(ref.balance(moved, idx, off, E, score, 0.3)[0])
            # differences: third derivative times step^2, and 1e-16 / step
            assert g[t, e] == pytest.approx(1.7 * (d[0] - d[1]) / (2 * step), rel=1e-6, abs=1e-9)
    assert (g[9:] == 0).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_norm_gradients_equal_differences(post, gated, pre):
    rng = np.random.default_rng(5)
    T, H, groups = 5, 6, 2
    group = np.arange(T) // 3
    a = dict(res=rng.standard_normal((T, H)), y=rng.standard_normal((T, H)))
    if gated:
        a["gate"] = rng.standard_normal((groups, H))
    if post:
        a["w_post"] = rng.standard_normal(H)
    if pre:
        a["w_pre"] = rng.standard_normal(H)
    gr, gx = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def forward(a):
        b = dict(a)
        if gated:
            b["gate"] = a["gate"][group]
        return ref.block_norm(**b, scale=0.7, eps=1e-3)[0]

    def loss(a):
        o = forward(a)
        return (o["res_out"] * gr).sum() + ((o["x"] * gx).sum() if pre else 0.0)

    o = forward(a)
    got, _ = ref.block_norm_bwd(gr, gx if pre else None, o["res_out"], o["c"], a.get("gate"), group,
                                groups, a.get("w_post"), a.get("w_pre"), o.get("rstd_post"),
                                o.get("rstd_pre"), 0.7)
    for name, out in (("res", "gres"), ("y", "gy"), ("gate", "ggate"), ("w_post", "gw_post"),
                      ("w_pre", "gw_pre")):
        if name not in a:
            assert out not in got
            continue
        want = np.zeros_like(a[name])
        for at in np.ndindex(want.shape):
            d = []
            for sgn in (1, -1):
                moved = {k: v.copy() for k, v in a.items()}
                moved[name][at] += sgn * 1e-5
                d.append(loss(moved))
            want[at] = (d[0] - d[1]) / 2e-5
        assert np.allclose(got[out], want, rtol=1e-6, atol=1e-8), name


def test_bounds_hold_for_a_plain_fp32_form():
    """A straightforward fp32 evaluation lies within the bounds, one with its
    weight off by a bf16 step does not."""
    rng = np.random.default_rng(7)
    f = np.float32
    res, y = (rng.standard_normal((64, 128)).astype(f) for _ in range(2))
    w = rng.random(128).astype(f) + f(0.5)

    def plain(w):
        r = f(1) / np.sqrt((y * y).mean(1, keepdims=True, dtype=f) + f(1e-6))
        return res * f(0.5) + y * r * w

    want, bound = ref.block_norm(res.astype(float), y.astype(float), w_post=w.astype(float), scale=0.5)
    assert (np.abs(plain(w) - want["res_out"]) <= bound["res_out"]).all()
    assert (np.abs(plain(w * f(1 + 2.0 ** -8)) - want["res_out"]) > bound["res_out"]).mean() > 0.9


def test_sizes_and_null_handles_are_refused_without_a_gpu():
    import combine_moe_route_05_gb300 as moe
    from combine_moe_route_05_gb300 import build
    build.build()
    L = moe.lib()
    cfg = moe.make_config(64, 4, 1, 128)
    small, large = (moe.moe_balance_workspace_bytes(cfg, S) for S in (1, 1000))
    assert 0 < small <= large
    assert moe.moe_balance_workspace_bytes(cfg, 0) == 0
    assert moe.moe_balance_workspace_bytes(moe.make_config(600, 4, 1, 128), 1) == 0
    assert L.moe_block_norm_workspace_bytes(None, 4, 64, 1) == 0
    A = 0x10000
    assert L.moe_balance(None, A, A, 4, None, 1, 1.0, A, A, None, A, 1 << 30, None) == moe.MOE_ERR_INVALID
    assert L.moe_balance_bwd(None, A, A, 4, None, 1, 1.0, None, None, A, None) == moe.MOE_ERR_INVALID
    a, b = moe.MoeBlockNormArgs(), moe.MoeBlockNormBwdArgs()
    assert L.moe_block_norm(None, ctypes.byref(a), 4, None) == moe.MOE_ERR_INVALID
    assert L.moe_block_norm_bwd(None, ctypes.byref(b), 4, A, 1 << 30, None) == moe.MOE_ERR_INVALID


def test_sequences_of_a_balance_loss_are_limited():
    """The kernels count sequences in steps of a grid, in 32 bits."""
    import combine_moe_route_05_gb300 as moe
    cfg = moe.make_config(64, 4, 1, 128)
    most = 1 << 30
    assert moe.moe_balance_workspace_bytes(cfg, most) > 0
    for S in (most + 1, 2 ** 31 - 1, -1):
        assert moe.moe_balance_workspace_bytes(cfg, S) == 0


def test_structs_match_the_header():
    """Field order and types of the binding's structs are the header's."""
    import os
    import re
    import combine_moe_route_05_gb300 as moe
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_route.h")).read(), flags=re.S)
    kinds = {"double": ctypes.c_double, "int32_t": ctypes.c_int32}
    for name, cls in (("moe_block_norm_args", moe.MoeBlockNormArgs),
                      ("moe_block_norm_bwd_args", moe.MoeBlockNormBwdArgs)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        want = [(m[2], ctypes.c_void_p if m[1] else kinds[m[0]])
                for m in re.findall(r"(?:const )?(\w+)(\*?) (\w+);", body)]
        assert list(cls._fields_) == want
    import struct
    for form, cls in (("12P3d5i4x", moe.MoeBlockNormArgs), ("14P2d4i", moe.MoeBlockNormBwdArgs)):
        assert struct.calcsize(form) == ctypes.sizeof(cls)
        kinds = {ctypes.c_void_p: "P", ctypes.c_double: "d", ctypes.c_int32: "i"}
        each = "".join(n * c for n, c in ((int(n or 1), c) for n, c in re.findall(r"(\d*)([Pdi])", form)))
        assert each == "".join(kinds[t] for _, t in cls._fields_)
