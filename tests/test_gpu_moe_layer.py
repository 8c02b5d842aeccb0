"""The operators together: the example's decode step against a 64-bit layer and
its training layer's gradients against 64-bit automatic differentiation."""
import importlib.util
import os

import pytest
import torch

from lm_util import int4_weights

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _topk(logits, K):
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    return order.indices[:, :K], torch.softmax(order.values[:, :K].double(), 1)


def test_decode_step_against_a_64_bit_layer():
    """Intermediate rows and outputs are rounded to bf16: half an ulp (2^-8) of
    each, the intermediate's carried on through the down product's weights."""
    ex = _example()
    g = torch.Generator().manual_seed(0)
    T, H, I, E, K = 9, 512, 256, 12, 3
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g)
    logits[3] = -float("inf")                              # a token that goes nowhere
    up = torch.randn(E, 2 * I, H, generator=g) * H ** -0.5
    down = torch.randn(E, H, I, generator=g) * I ** -0.5
    qu, su = ex.quantize_int4(up, 64)
    qd, sd = ex.quantize_int4(down, 128)
    experts = ex.Int4Experts(qu.cuda(), su.cuda(), qd.cuda(), sd.cuda())
    status = torch.zeros(1, dtype=torch.int32).cuda()
    y = ex.decode_step(x.cuda(), logits.cuda(), experts, K, status).cpu().double()
    assert int(status) == 0
    wu, wd = int4_weights(qu, su, None, 64), int4_weights(qd, sd, None, 128)
    idx, w = _topk(logits, K)
    for t in range(T):
        ref, bound = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        if t != 3:
            for k in range(K):
                e = int(idx[t, k])
                a, b = (wu[e] @ x[t].double()).chunk(2)
                h = a * torch.sigmoid(a) * b
                o = wd[e] @ h
                ref += w[t, k] * o
                # roundings of h and o, and binary32 sums well below them
                bound += w[t, k] * (2.0 ** -8 * (wd[e].abs() @ h.abs() + o.abs()) + 1e-4)
        assert ((y[t] - ref).abs() <= bound + 2.0 ** -8 * ref.abs()).all()
    assert (y[3] == 0).all()


def test_training_layer_gradients():
    """binary32 layer: every product and sum carries some H * 2^-24 relative, far
    below the 1e-4 of the largest gradient that is asked for."""
    ex = _example()
    torch.manual_seed(1)
    T, H, I, E, K = 21, 40, 24, 5, 2
    layer = ex.MoeLayer(H, I, E, K, align=4, dtype=torch.float32)
    x = torch.randn(T, H, device="cuda", requires_grad=True)
    c = torch.randn(T, H, device="cuda")
    allow = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        y = layer(x)
        (y * c).sum().backward()
        logits = (x @ layer.router.T).detach()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allow
    p = {n: v.detach().cpu().double().requires_grad_(True) for n, v in layer.named_parameters()}
    xr = x.detach().cpu().double().requires_grad_(True)
    lr = xr @ p["router"].T
    idx, _ = _topk(logits.cpu(), K)
    w = torch.softmax(lr.gather(1, idx), 1)
    rows = []
    for t in range(T):
        acc = 0
        for k in range(K):
            e = int(idx[t, k])
            a, b = (p["gate_up"][e] @ xr[t]).chunk(2)
            acc = acc + w[t, k] * (p["down"][e] @ (a * torch.sigmoid(a) * b))
        rows.append(acc)
    ref = torch.stack(rows)
    (ref * c.cpu().double()).sum().backward()
    assert (y.detach().cpu().double() - ref.detach()).abs().max() <= 1e-4 * ref.abs().max()
    got = {n: v.grad for n, v in layer.named_parameters()}
    for name in p:
        r = p[name].grad
        assert (got[name].cpu().double() - r).abs().max() <= 1e-4 * r.abs().max(), name
    assert (x.grad.cpu().double() - xr.grad).abs().max() <= 1e-4 * xr.grad.abs().max()


def test_decode_step_replays_as_a_graph_with_new_routing():
    ex = _example()
    g = torch.Generator().manual_seed(2)
    T, H, I, E, K = 16, 512, 256, 32, 4
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    qu, su = ex.quantize_int4(torch.randn(E, 2 * I, H, generator=g) * H ** -0.5, 128)
    qd, sd = ex.quantize_int4(torch.randn(E, H, I, generator=g) * I ** -0.5, 128)
    experts = ex.Int4Experts(qu.cuda(), su.cuda(), qd.cuda(), sd.cuda())
    status = torch.zeros(1, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ex.decode_step(x, logits, experts, K, status)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ex.decode_step(x, logits, experts, K, status)
    for seed in (3, 4):
        h = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=h).to(torch.bfloat16))
        logits.copy_(torch.randn(T, E, generator=h))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want = ex.decode_step(x, logits, experts, K, status)
        assert torch.equal(got, want)
    assert int(status) == 0
