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


def _spoil(shapes, dtype):
    """NaN in the memory that the next tensors of these shapes get."""
    held = [torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in shapes for _ in range(4)]
    del held


def test_padding_rows_hold_no_old_memory():
    ex = _example()
    layer, x, c = _layer(ex)
    idx, _ = ex.Gate.apply((x @ layer.router.T).float(), layer.K)
    rows, _, src, offsets, counts = ex.Sort.apply(x.requires_grad_(True), idx, layer.E, layer.align)
    R, (H, I) = rows.shape[0], layer.down.shape[1:]
    pad = src < 0
    assert pad.any() and (rows[pad] == 0).all()
    _spoil([(R, I), (R, 2 * I), (R, H)], x.dtype)
    h = ex.Block.apply(rows, layer.gate_up, offsets, counts, layer.status)
    out = ex.Product.apply(h, layer.down, offsets, counts, layer.status)
    assert (h[pad] == 0).all() and (out[pad] == 0).all()
    seen = []
    h.register_hook(lambda g: seen.append(g.clone()))
    rows.register_hook(lambda g: seen.append(g.clone()))
    dout = torch.randn_like(out)
    _spoil([(R, I), (R, 2 * I), (R, H)], x.dtype)
    out.backward(dout)
    assert len(seen) == 2 and all((g[pad] == 0).all() and torch.isfinite(g).all() for g in seen)


def test_anomaly_detection_finds_nothing():
    ex = _example()
    layer, x, c = _layer(ex)
    R, (H, I) = 70 * 2 + 5 * 15, layer.down.shape[1:]
    with torch.autograd.detect_anomaly():
        for _ in range(3):
            _spoil([(R, I), (R, 2 * I), (R, H)], x.dtype)
            (layer(x) * c).sum().backward()
    assert all(torch.isfinite(p.grad).all() for p in layer.parameters())


@pytest.mark.parametrize("frozen", [("gate_up", "down"), ("gate_up",), ("down", "router"), ("router",)])
@pytest.mark.parametrize("with_x", [False, True])
def test_frozen_parameters(frozen, with_x, monkeypatch):
    """The gradients that are asked for are those of the whole layer; the others are not computed."""
    ex = _example()
    layer, x, c = _layer(ex)
    x.requires_grad_(with_x)
    (layer(x) * c).sum().backward()
    whole = {n: p.grad for n, p in layer.named_parameters()} | {"x": x.grad}
    layer.zero_grad(set_to_none=True)
    x.grad = None
    asked = []
    grad = ex.moedc.matmul_grad

    def counted(dout, rows, w, **kw):
        asked.append((w is not None, rows is not None))
        return grad(dout, rows, w, **kw)

    monkeypatch.setattr(ex.moedc, "matmul_grad", counted)
    for n in frozen:
        getattr(layer, n).requires_grad_(False)
    (layer(x) * c).sum().backward()
    for n, p in layer.named_parameters():
        assert p.grad is None if n in frozen else torch.equal(p.grad, whole[n])
    assert x.grad is None if not with_x else torch.equal(x.grad, whole["x"])
    # the down product's, then the block's: (dx, dw)
    block = with_x, "gate_up" not in frozen
    down = any(block), "down" not in frozen
    assert asked == [pair for pair in (down, block) if any(pair)]


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
