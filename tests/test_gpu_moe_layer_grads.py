"""The example's training layer under losses whose gradients reach it expanded or
transposed."""
import pytest
import torch

from test_gpu_moe_layer import _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loss", [
    lambda y: y.sum(),                                        # an expanded scalar
    lambda y: (y.sum(1) * torch.arange(21.0, device="cuda")).sum(),   # one value a token
    lambda y: (y.T.contiguous() * 2.0).sum(),                 # columns first
    lambda y: y[3, 5]], ids=["sum", "rows", "transposed", "one"])
def test_expanded_and_transposed_gradients(loss):
    ex = _example()
    torch.manual_seed(1)
    T, H, I, E, K = 21, 40, 24, 5, 2
    layer = ex.MoeLayer(H, I, E, K, align=4, dtype=torch.float32)
    x = torch.randn(T, H, device="cuda", requires_grad=True)
    y = layer(x).detach().requires_grad_(True)
    dense = torch.autograd.grad(loss(y), y)[0].contiguous()
    loss(layer(x)).backward()
    got = [x.grad.clone()] + [p.grad.clone() for p in layer.parameters()]
    x.grad = None
    layer.zero_grad()
    layer(x).backward(dense)
    for a, b in zip(got, [x.grad] + [p.grad for p in layer.parameters()]):
        assert torch.equal(a, b)
