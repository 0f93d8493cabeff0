"""The fp64 references of the expert activation and the few-token layer
(published generator vectors, differences), and the host-side refusals of
moe_act_rows, moe_act_rows_bwd and moe_layer that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import expert_ref as ref


@pytest.fixture(scope="module")
def lib():
    from combine_moe_route_05_gb300 import build
    build.build()
    import combine_moe_route_05_gb300 as m
    return m


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(int(v) for v in ref.philox4x32(counter, key)) == want


def test_mask_rate_and_independence_of_the_row_order():
    ent = np.arange(400)
    m, scale = ref.kept_mask(ent, 1000, 0.25, 12345, 7)
    # 400000 Bernoulli(0.75) draws: standard deviation 6.8e-4 of the rate
    assert abs(m.mean() - 0.75) < 5 * 6.9e-4 and scale == 4.0 / 3.0
    perm = np.random.default_rng(0).permutation(400)
    assert np.array_equal(ref.kept_mask(ent[perm], 1000, 0.25, 12345, 7)[0], m[perm])
    assert not np.array_equal(ref.kept_mask(ent, 1000, 0.25, 12345, 8)[0], m)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_gradient_against_differences(act):
    rng = np.random.default_rng(3)
    gu, ghs, w = rng.standard_normal((5, 48)), rng.standard_normal((5, 24)), rng.random(5)
    mask, scale = ref.kept_mask(np.arange(5), 24, 0.3, 1, 2)
    loss = lambda gu, w: float((ref.act_rows(gu, w, act, mask, scale) * ghs).sum())  # noqa: E731
    ggu, gw, _, _ = ref.act_rows_bwd(ghs, gu, w, act, mask, scale)
    h = 1e-5  # central differences: error about h^2 = 1e-10 and 1e-16 / h = 1e-11
    for r, c in [(0, 0), (1, 7), (2, 23), (3, 24), (4, 47)]:
        d = np.zeros_like(gu)
        d[r, c] = h
        assert abs((loss(gu + d, w) - loss(gu - d, w)) / (2 * h) - ggu[r, c]) < 1e-7
    for r in range(5):
        d = np.zeros_like(w)
        d[r] = h
        assert abs((loss(gu, w + d) - loss(gu, w - d)) / (2 * h) - gw[r]) < 1e-7


@pytest.mark.parametrize("H,I,S,ok", [
    (64, 32, 0, True), (7168, 2048, 1, True), (65536, 65536, 4, True), (8, 8, 0, True),
    (60, 32, 0, False), (64, 36, 0, False), (0, 32, 0, False), (64, -8, 0, False),
    (65544, 32, 0, False), (64, 32, 5, False), (64, 32, -1, False),
])
def test_layer_workspace_validates_sizes(lib, H, I, S, ok):
    cfg = lib.make_config(8, 2, 1, 1000)
    n = lib.moe_layer_workspace_bytes(cfg, H, I, S)
    assert (n > 0) == ok
    if ok:  # 128 tokens' bf16 activations and fp32 output rows
        assert n >= 128 * (2 + S) * (2 * I + 4 * H)
    small = lib.moe_layer_workspace_bytes(lib.make_config(8, 2, 1, 4), H, I, S)
    assert (small > 0) == ok and small <= n


def test_null_handles_are_refused(lib):
    L = lib.lib()
    P = 0x1000
    assert L.moe_act_rows(None, P, 64, 0, 0, None, 0.0, None, P, None) == lib.MOE_ERR_INVALID
    assert L.moe_act_rows_bwd(None, P, P, 64, 0, 0, None, 0.0, None, P, None, None) == lib.MOE_ERR_INVALID
    a = lib.MoeLayerArgs()
    assert L.moe_layer(None, ctypes.byref(a), 1, P, 1 << 20, None) == lib.MOE_ERR_INVALID
    assert L.moe_layer_workspace_bytes(None, 64, 64, 0) == 0


def test_layer_args_match_the_header(lib):
    """11 pointers, then 5 int32, padded to 8 bytes."""
    assert ctypes.sizeof(lib.MoeLayerArgs) == 11 * 8 + 5 * 4 + 4
    assert lib.MoeLayerArgs.H.offset == 88 and lib.MoeLayerArgs.act.offset == 104


class _Fake:
    """Stands in for a CUDA tensor (no GPU needed)."""
    is_cuda = True

    def __init__(self, shape, dtype, contiguous=True, device="cuda:0"):
        self.shape, self.dtype, self.c, self.device = shape, dtype, contiguous, torch.device(device)

    def is_contiguous(self):
        return self.c

    def numel(self):
        return int(np.prod(self.shape))

    def data_ptr(self):
        return 0x1000


class _FakeHandle:
    device = torch.device("cuda", 0)
    E, K, T, recv_rows = 8, 2, 4, 8
    ptr = None


def layer_call(lib, **kw):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    a = dict(x=_Fake((4, 64), bf), logits=_Fake((4, 8), f32), w13=_Fake((8, 64, 64), bf),
             w2=_Fake((8, 64, 32), bf), out=_Fake((4, 64), bf), idx=_Fake((4, 2), i32),
             w=_Fake((4, 2), f32), workspace=_Fake((1 << 20,), torch.uint8))
    a.update(kw)
    lib.moe_layer(_FakeHandle(), **a)


@pytest.mark.parametrize("kw,err", [
    (dict(x=_Fake((4, 64), torch.float32)), TypeError),
    (dict(w13=_Fake((8, 64, 64), torch.float16)), TypeError),
    (dict(w2=_Fake((8, 64, 32), torch.float8_e4m3fn)), TypeError),     # w13 and w2 differ
    (dict(w13=_Fake((8, 66, 64), torch.bfloat16)), ValueError),
    (dict(num_shared=1), ValueError),                                  # no shared expert in w13
    (dict(w13=_Fake((8, 64, 64), torch.bfloat16, False)), ValueError),  # strided
    (dict(live=_Fake((1,), torch.int64)), TypeError),
    (dict(live=_Fake((4,), torch.int32)), ValueError),
    (dict(out=_Fake((4, 64), torch.bfloat16, device="cuda:1")), ValueError),
    (dict(idx=_Fake((4, 3), torch.int32)), ValueError),
    (dict(bias=_Fake((7,), torch.float32)), ValueError),
    (dict(s13=_Fake((8, 1, 2), torch.float32)), ValueError),
])
def test_layer_binding_refuses(lib, kw, err):
    with pytest.raises(err):
        layer_call(lib, **kw)


@pytest.mark.parametrize("kw,err", [
    (dict(gu=_Fake((8, 60), torch.bfloat16)), ValueError),
    (dict(gu=_Fake((8, 64), torch.float32)), TypeError),
    (dict(recv_w=_Fake((7,), torch.float32)), ValueError),
    (dict(rng=_Fake((2,), torch.int32)), TypeError),
    (dict(rng=_Fake((1,), torch.int64)), ValueError),
    (dict(hs=_Fake((8, 32), torch.bfloat16, False)), ValueError),
    (dict(gu=_Fake((8, 64), torch.float16), hs=_Fake((8, 32), torch.float16)), TypeError),
    (dict(act="relu"), KeyError),
])
def test_act_binding_refuses(lib, kw, err):
    a = dict(gu=_Fake((8, 64), torch.bfloat16), recv_w=_Fake((8,), torch.float32),
             hs=_Fake((8, 32), torch.bfloat16))
    a.update(kw)
    with pytest.raises(err):
        lib.moe_act_rows(_FakeHandle(), stream=type("S", (), dict(device=_FakeHandle.device, cuda_stream=0))(), **a)
