"""The experts' dense layers as the example uses them: the training layer in 16 bits, the
decode step and the receive buffer's step with e4m3 experts."""
import pytest
import torch

from matmul_util import randn
from test_gpu_matmul_e4m3 import wide_w, wide_x
from test_gpu_moe_layer import _example, _topk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,I,E,K,align", [(1, 64, 32, 4, 2, 1), (70, 136, 72, 5, 2, 4), (300, 256, 128, 3, 1, 16)])
def test_training_layer_in_16_bits(T, H, I, E, K, align, dtype):
    """Against 64-bit automatic differentiation of the same layer.  On the way from a weight to
    the loss and back some eight tensors are rounded, each by 2^-8 (bf16; 2^-11) of its norm at
    most; weights and inputs of random signs carry a relative error on without making it larger."""
    ex = _example()
    torch.manual_seed(1)
    layer = ex.MoeLayer(H, I, E, K, align=align, dtype=dtype)
    x = torch.randn(T, H, device="cuda", dtype=dtype, requires_grad=True)
    c = torch.randn(T, H, device="cuda", dtype=dtype)
    y = layer(x)
    (y * c).sum().backward()
    logits = (x @ layer.router.T).float().detach()
    p = {n: v.detach().cpu().double().requires_grad_(True) for n, v in layer.named_parameters()}
    xr = x.detach().cpu().double().requires_grad_(True)
    idx, _ = _topk(logits.cpu(), K)
    w = torch.softmax((xr @ p["router"].T).gather(1, idx), 1)
    ref = []
    for t in range(T):
        acc = 0
        for k in range(K):
            e = int(idx[t, k])
            a, b = (p["gate_up"][e] @ xr[t]).chunk(2)
            acc = acc + w[t, k] * (p["down"][e] @ (a * torch.sigmoid(a) * b))
        ref.append(acc)
    ref = torch.stack(ref)
    (ref * c.cpu().double()).sum().backward()
    most = 8 * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11)

    def near(a, b):
        return (a.detach().cpu().double() - b).norm() <= most * b.norm()

    assert int(layer.status) == 0
    assert near(y, ref.detach())
    assert near(layer.gate_up.grad, p["gate_up"].grad) and near(layer.down.grad, p["down"].grad)
    assert near(x.grad, xr.grad)


def _experts(ex, g, E, H, I):
    return ex.E4m3Experts.of(randn(g, torch.bfloat16, E, 2 * I, H, scale=H ** -0.5),
                             randn(g, torch.bfloat16, E, H, I, scale=I ** -0.5))


def _expert_out(experts, e, q, qs):
    """(64-bit output row of expert e for an e4m3 token, its bound) with the rows between the
    products rounded to e4m3."""
    up = wide_w(experts.gate_up[e], experts.gate_up_scales[e], True)
    down = wide_w(experts.down[e], experts.down_scales[e], False)
    a, b = (up @ wide_x(q, qs)).chunk(2)
    h = a * torch.sigmoid(a) * b
    # half a step of e4m3: 2^-4 relative, or half the subnormal spacing of the group's scale
    step = h.abs().reshape(-1, 128).amax(1).clamp(min=1e-4) / 448.0
    off = h.abs() * 2.0 ** -4 + step.repeat_interleave(128) * 2.0 ** -10
    out = down @ h
    return out, down.abs() @ off + 2.0 ** -8 * out.abs() + 1e-4


def test_decode_step_with_e4m3_experts():
    ex = _example()
    g = torch.Generator().manual_seed(0)
    T, H, I, E, K = 9, 512, 256, 12, 3
    x = randn(g, torch.bfloat16, T, H)
    logits = torch.randn(T, E, generator=g)
    logits[3] = -float("inf")                              # a token that goes nowhere
    experts = _experts(ex, g, E, H, I)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    y = ex.decode_step(x, logits.cuda(), experts, K, status)
    assert int(status) == 0
    idx, w = _topk(logits, K)
    q, qs = ex.moedc.quant_e4m3(x)
    for t in range(T):
        ref, bound = torch.zeros(H, dtype=torch.float64, device="cuda"), 0.0
        for k in range(K if t != 3 else 0):
            out, off = _expert_out(experts, int(idx[t, k]), q[t], qs[t])
            ref, bound = ref + float(w[t, k]) * out, bound + float(w[t, k]) * off
        assert ((y[t].double() - ref).abs() <= bound + 2.0 ** -8 * ref.abs()).all()
    assert (y[3] == 0).all()


def test_slots_step_is_the_decode_step_of_the_same_routing():
    """The receive buffer holds the rows that quant_e4m3 gives; combine and unsort round the
    same sums once, one of them fused: an ulp apart."""
    ex = _example()
    g = torch.Generator().manual_seed(1)
    T, H, I, E, K = 40, 512, 256, 8, 2
    x = randn(g, torch.bfloat16, T, H)
    logits = torch.randn(T, E, generator=g).cuda()
    experts = _experts(ex, g, E, H, I)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    idx, w = ex.moedc.gate(logits, K, flags=ex.FLAGS)
    a = ex.decode_step(x, logits, experts, K, status).double()
    b = ex.slots_step(x, idx, w, E, 2, T, experts).double()
    assert int(status) == 0 and ((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-6).all()


def test_e4m3_decode_step_replays_as_a_graph():
    ex = _example()
    g = torch.Generator().manual_seed(2)
    T, H, I, E, K = 16, 512, 256, 32, 4
    x, logits = randn(g, torch.bfloat16, T, H), torch.randn(T, E, generator=g).cuda()
    experts = _experts(ex, g, E, H, I)
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
        assert torch.equal(y, ex.decode_step(x, logits, experts, K, status))
    assert int(status) == 0


def test_training_step_replays_as_a_graph():
    """Forward and backward of the 16-bit layer read nothing on the host: captured once, replayed
    with other tokens and weights."""
    ex = _example()
    torch.manual_seed(3)
    T, H, I, E, K = 120, 128, 64, 6, 2
    layer = ex.MoeLayer(H, I, E, K, align=8, dtype=torch.bfloat16)
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    c = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)

    def step():
        y = layer(x)
        (y * c).sum().backward()
        return y.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            layer.zero_grad(set_to_none=True)
            step()
    torch.cuda.current_stream().wait_stream(side)
    layer.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    grads = [p.grad for p in layer.parameters()]
    for seed in (4, 5):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g))
        with torch.no_grad():
            for p in layer.parameters():
                p.mul_(1.01)
        for v in grads:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone()] + [v.clone() for v in grads]
        other = ex.MoeLayer(H, I, E, K, align=8, dtype=torch.bfloat16)
        other.load_state_dict(layer.state_dict())
        z = other(x)
        (z * c).sum().backward()
        for a, b in zip(got, [z.detach()] + [p.grad for p in other.parameters()]):
            assert torch.equal(a, b)
    assert int(layer.status) == 0
