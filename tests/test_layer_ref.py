"""The references of the few-token layer at its stated precision: the exact layers
are what their integers say, and a mistake planted in the host model falls outside
what the GPU tests allow."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.test_gpu_layer_precision import EXACT, RANDOM, RandomProblem


@pytest.mark.parametrize("kw", EXACT, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_exact_layers_and_planted_mistakes(kw):
    p = ref.Exact(**kw)
    want = p.want()
    assert np.array_equal(p.out(), want)
    assert np.array_equal(ref.bf16(p.x), p.x) and np.array_equal(ref.bf16(p.w13), p.w13)
    assert np.array_equal(ref.bf16(p.w2), p.w2)
    if p.e4m3:
        for q in (p.q13, p.q2):
            assert np.array_equal(torch.from_numpy(q).to(torch.float8_e4m3fn).double().numpy(), q)
    for fault in ref.FAULTS_E4M3 if p.e4m3 else ref.FAULTS:
        if fault == "scales of the next row of blocks" and p.s13.shape[1] == 1 and p.s2.shape[1] == 1:
            continue  # there is no other row
        if fault == "low parts of another token" and p.T * (p.K + p.S) == 1:
            continue  # nor another entry
        assert not np.array_equal(p.out(fault), want), fault


@pytest.mark.parametrize("kw", RANDOM, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_planted_mistakes_leave_the_stated_bound(kw):
    p = RandomProblem(**kw)
    want, bound = ref.layer(*p.args)
    assert (np.abs(ref.bf16(ref.model(*p.args)) - want) <= bound).all()
    faults = ref.FAULTS_E4M3[:3] if p.e4m3 else ref.FAULTS
    for fault in faults:
        assert (np.abs(ref.bf16(ref.model(*p.args, fault=fault)) - want) > bound).any(), fault
