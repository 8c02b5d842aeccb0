"""Sigmoid router weights far below 0, where binary32 sigmoids lose bits and
vanish: the renormalised weights and the gradients stay those of the formula
down to the smallest binary32 sigmoid (logits of -103.9).  Bounds as in the
router's other tests."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from test_gpu_gate import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(16, 4), (130, 8), (129, 32)])
def test_logits_far_below_zero(E, K, dtype, normalize):
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(12, E, generator=g)
    logits[1] = logits[1] - 75.0
    logits[2] = logits[2] - 84.0
    logits[3] = logits[3] - 88.7            # expf(-l) overflows for some of them
    logits[4] = logits[4] - 95.0
    logits[5] = logits[5] * 0.3 - 102.0
    logits[6] = logits[6] * 0.1 - 103.0
    logits[7] = -95.0                       # 1 / K each
    logits[8, :3], logits[8, 3:] = -85.0, -110.0
    logits[9, :2], logits[9, 2:] = 1.5, -98.0
    logits[10] = -95.0
    logits[10, 1::2] = -float("inf")
    logits[11] = torch.linspace(-60.0, -100.0, E)
    _check(logits.to(dtype).cuda(), K, None, True, normalize, scale=1.5)


def test_all_below_the_smallest_sigmoid():
    """The 64-bit form takes such a sigmoid for 0, and their sum then gives weight 0."""
    logits = torch.randn(3, 16, generator=torch.Generator().manual_seed(1)).cuda() - 130.0
    flags = moedc.GATE_SIGMOID | moedc.GATE_NORMALIZE
    idx, w = moedc.gate(logits, 4, flags=flags)
    assert (w == 0).all() and (idx >= 0).all()
    assert (moedc.gate_grad(logits, idx, torch.ones_like(w), flags=flags) == 0).all()


def test_equal_logits_share_the_weight():
    for l in (-70.0, -90.0, -95.0, -103.0):
        logits = torch.full((3, 8), l).cuda()
        idx, w = moedc.gate(logits, 4, flags=moedc.GATE_SIGMOID | moedc.GATE_NORMALIZE)
        assert torch.equal(w, torch.full((3, 4), 0.25).cuda())
        dw = torch.tensor([[1.0, 0.0, 0.0, 0.0]] * 3).cuda()
        dl = moedc.gate_grad(logits, idx, dw, flags=moedc.GATE_SIGMOID | moedc.GATE_NORMALIZE)
        want = torch.tensor([0.1875, -0.0625, -0.0625, -0.0625, 0, 0, 0, 0]).cuda()
        assert torch.equal(dl, want.expand(3, 8))
