"""The example's training layer as automatic differentiation meets it: frozen parameters,
second derivatives, padding rows that hooks and anomaly detection see."""
import pytest
import torch

from test_gpu_moe_layer import _example

pytestmark = pytest.mark.gpu


def _layer(ex, dtype=torch.bfloat16, T=70, H=136, I=72, E=5, K=2, align=16):
    torch.manual_seed(2)
    layer = ex.MoeLayer(H, I, E, K, align=align, dtype=dtype)
    x = torch.randn(T, H, device="cuda", dtype=dtype)
    return layer, x, torch.randn(T, H, device="cuda", dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_second_derivatives_are_refused(dtype):
    ex = _example()
    layer, x, c = _layer(ex, dtype)
    x.requires_grad_(True)
    first, = torch.autograd.grad((layer(x) * c).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        first.float().square().sum().backward()


def test_second_derivatives_of_the_router_are_refused():
    ex = _example()
    logits = torch.randn(6, 4, device="cuda", requires_grad=True)
    _, w = ex.Gate.apply(logits, 2)
    first, = torch.autograd.grad(w.square().sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        first.sum().backward()
