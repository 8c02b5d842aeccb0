"""Top-k router and its gradient against 64-bit forms.

Bounds: expf is good to 2 ulp and its argument l - max carries half an ulp of
its size; sums over at most 1024 experts in trees and short chains and one
division stay below 64 roundings: (64 + 4 max|l|) * 2^-24 relative."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, U32, assert_within, gate_grad_ref, gate_ref, rounding

pytestmark = pytest.mark.gpu

FORMS = [(False, True), (False, False), (True, True), (True, False)]


def _flags(sigmoid, normalize):
    return ((moedc.GATE_SIGMOID if sigmoid else moedc.GATE_SOFTMAX) |
            (moedc.GATE_NORMALIZE if normalize else 0))


def _logits(seed, T, E, dtype, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype).cuda()


def _check(logits, K, bias, sigmoid, normalize, scale=1.0, dw=None):
    flags = _flags(sigmoid, normalize)
    idx, w = moedc.gate(logits, K, bias=bias, flags=flags, scale=scale)
    ref_idx, ref_w = gate_ref(logits, K, bias, sigmoid, normalize, scale)
    assert torch.equal(idx.cpu(), ref_idx)
    finite = logits.float()[torch.isfinite(logits.float())]
    big = float(finite.abs().max()) if finite.numel() else 0.0
    rel = (64 + 4 * min(big, 200.0)) * U32
    assert_within(w, ref_w, rel * ref_w.abs() + 1e-37)
    if dw is None:
        dw = torch.randn(w.shape, generator=torch.Generator().manual_seed(3)).cuda()
    dl = moedc.gate_grad(logits, idx, dw, bias=bias, flags=flags, scale=scale)
    ref = gate_grad_ref(logits, ref_idx, dw, bias, sigmoid, normalize, scale)
    live = dw.cpu()[ref_idx >= 0]
    most = float(live.abs().max()) if live.numel() else 0.0
    # p (d - sum p d): two magnitudes of at most max|d| each, factors at most 1
    assert_within(dl, ref, 2 * rel * scale * most + rounding(ref, logits.dtype))
    return idx, w, dl


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (5, 60, 6), (33, 129, 8), (7, 288, 8), (2, 1024, 32),
                                   (3, 1, 1), (4, 7, 7), (6, 513, 3)])
def test_gate_and_gradient(T, E, K, dtype, sigmoid, normalize):
    _check(_logits(T * E, T, E, DTYPES[dtype]), K, None, sigmoid, normalize, scale=2.5)


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_bias_moves_the_choice_alone(sigmoid, normalize):
    logits = _logits(5, 17, 64, torch.float32)
    bias = (torch.randn(64, generator=torch.Generator().manual_seed(6)) * 2).cuda()
    idx, _, _ = _check(logits, 4, bias, sigmoid, normalize)
    plain, _ = moedc.gate(logits, 4, flags=_flags(sigmoid, normalize))
    assert not torch.equal(idx, plain)


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_masked_experts_and_rows_with_nothing_left(sigmoid, normalize):
    inf = float("inf")
    logits = _logits(7, 8, 40, torch.float32)
    logits[0] = -inf                              # nothing left
    logits[1] = -inf
    logits[1, 17] = 0.25                          # one left
    logits[2, 5] = float("nan")
    logits[2, 6] = -inf
    logits[3, ::2] = -inf
    logits[4] = float("nan")
    bias = torch.zeros(40).cuda()
    bias[11] = -inf                               # masked through the bias
    bias[12] = float("nan")
    dw = torch.randn(8, 8).cuda()
    dw[0], dw[1, 1:], dw[4] = float("nan"), inf, inf      # gradients of masked entries
    idx, w, dl = _check(logits, 8, bias, sigmoid, normalize, dw=dw)
    assert (idx[0] == -1).all() and (w[0] == 0).all() and (dl[0] == 0).all()
    assert (idx[4] == -1).all() and (dl[4] == 0).all()
    assert not ((idx == 11) | (idx == 12)).any()
    assert (dl[:, 11:13] == 0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_lowest_value_masks_and_infinity(dtype, sigmoid, normalize):
    dt = DTYPES[dtype]
    logits = _logits(8, 6, 33, dt)
    low = torch.finfo(dt).min
    logits[0, 3:] = low                           # more chosen than unmasked
    logits[1] = low                               # every expert at the lowest value
    logits[2, 4] = float("inf")
    logits[3, [4, 9]] = float("inf")
    idx, w = moedc.gate(logits, 5, flags=_flags(sigmoid, normalize))
    ref_idx, ref_w = gate_ref(logits, 5, None, sigmoid, normalize)
    assert torch.equal(idx.cpu(), ref_idx)
    assert_within(w, ref_w, 128 * U32 * ref_w + 1e-37)
    dl = moedc.gate_grad(logits, idx, torch.ones_like(w), flags=_flags(sigmoid, normalize))
    assert torch.isfinite(dl.float()).all()


def test_ties_go_to_the_lowest_expert():
    logits = torch.zeros(3, 100).cuda()
    logits[1, 50:] = 1.0
    logits[2, ::2] = -0.0                         # -0 ties with +0
    idx, _ = moedc.gate(logits, 6)
    assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]
    assert idx[1].tolist() == [50, 51, 52, 53, 54, 55]
    assert idx[2].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_gradient_against_differences(sigmoid, normalize):
    """Central differences of the 64-bit weights with step h: truncation
    h^2 |f'''| / 6 < 1e-7 here, so the kernel's binary32 error decides."""
    T, E, K, h = 4, 13, 3, 1e-4
    logits = _logits(9, T, E, torch.float32)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).cuda()
    flags = _flags(sigmoid, normalize)
    idx, _ = moedc.gate(logits, K, flags=flags)
    dl = moedc.gate_grad(logits, idx, dw, flags=flags).cpu().double()

    from lm_util import _weights

    def loss(l):
        return sum((_weights(l[t], idx[t].tolist(), list(range(E)), sigmoid, normalize) *
                    dw[t].cpu().double()).sum() for t in range(T))

    base = logits.cpu().double()
    for t in range(T):
        for e in range(E):
            up, down = base.clone(), base.clone()
            up[t, e] += h
            down[t, e] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - dl[t, e]) < 1e-5


def test_row_stride_empty_batch_and_reuse():
    wide = _logits(10, 9, 200, torch.bfloat16)
    part = wide[:, 3:67]
    idx, w = moedc.gate(part, 4)
    want = moedc.gate(part.contiguous(), 4)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    dw = torch.randn(9, 4).cuda()
    assert torch.equal(moedc.gate_grad(part, idx, dw),
                       moedc.gate_grad(part.contiguous(), idx, dw))
    again = moedc.gate(part, 4, out=(idx, w))
    assert again[0] is idx
    e = torch.empty(0, 16).cuda()
    idx, w = moedc.gate(e, 2)
    assert idx.shape == (0, 2)
    assert moedc.gate_grad(e, idx, w).shape == (0, 16)


def test_other_stream_and_many_tokens():
    logits = _logits(11, 20000, 256, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        idx, w = moedc.gate(logits, 8)
    side.synchronize()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(idx, order.indices[:, :8].to(torch.int32))
    assert_within(w, torch.softmax(order.values[:, :8].double(), 1).cpu(), 128 * U32)


def test_refusals():
    x = torch.zeros(4, 16).cuda()
    for bad in (lambda: moedc.gate(x, 17), lambda: moedc.gate(x, 0),
                lambda: moedc.gate(x, 2, flags=0x40)):
        with pytest.raises(moedc.MoedcError):
            bad()
    idx, w = moedc.gate(x, 2)
    for bad in (lambda: moedc.gate(x.double(), 2), lambda: moedc.gate(x.T, 2),
                lambda: moedc.gate(x.cpu(), 2), lambda: moedc.gate(x[:1].expand(4, 16), 2),
                lambda: moedc.gate(x, 2, bias=torch.zeros(15).cuda()),
                lambda: moedc.gate(x, 3, out=(idx, w)),
                lambda: moedc.gate_grad(x, idx.long(), w),
                lambda: moedc.gate_grad(x, idx, w[:, :1])):
        with pytest.raises(ValueError):
            bad()
