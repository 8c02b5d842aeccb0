"""The router's choice by score + bias against its definition in 64 bits.

A key is a score of at most 1, good to (64 + 4 max|l|) * 2^-24 as the weights
are, and one binary32 sum with a bias of at most 4 (half an ulp: 2^-22): two
keys closer than 1e-5 may come in either order, logits being below 16 here."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, U32, _weights, assert_within, gate_grad_ref, rounding

pytestmark = pytest.mark.gpu

FORMS = [(False, True), (False, False), (True, True), (True, False)]
NEAR = 1e-5
INF = float("inf")


def _flags(sigmoid, normalize):
    return ((moedc.GATE_SIGMOID if sigmoid else moedc.GATE_SOFTMAX) | moedc.GATE_BIAS_SCORE |
            (moedc.GATE_NORMALIZE if normalize else 0))


def _check(logits, K, bias, sigmoid, normalize, scale=1.0):
    flags = _flags(sigmoid, normalize)
    idx, w = moedc.gate(logits, K, bias=bias, flags=flags, scale=scale)
    got, l, b = idx.cpu(), logits.cpu().double(), bias.cpu().double()
    T, E = l.shape
    ref_w = torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        ok = [e for e in range(E) if l[t, e] > -INF and b[e] > -INF]
        k = min(K, len(ok))
        chosen = got[t].tolist()
        assert chosen[k:] == [-1] * (K - k) and len(set(chosen[:k])) == k
        assert set(chosen[:k]) <= set(ok)
        if not k:
            continue
        score = torch.full((E,), -INF, dtype=torch.float64)
        score[ok] = torch.sigmoid(l[t, ok]) if sigmoid else torch.softmax(l[t, ok], 0)
        key = score + b
        mine = key[chosen[:k]]
        assert (mine[:-1] >= mine[1:] - NEAR).all()
        rest = [float(key[e]) for e in ok if e not in chosen]
        assert not rest or float(mine.min()) >= max(rest) - NEAR
        ref_w[t, :k] = _weights(l[t], chosen[:k], ok, sigmoid, normalize) * scale
    rel = (64 + 4 * 16) * U32
    assert_within(w, ref_w, rel * ref_w.abs() + 1e-37)
    dw = torch.randn(w.shape, generator=torch.Generator().manual_seed(3)).cuda()
    dl = moedc.gate_grad(logits, idx, dw, bias=bias, flags=flags, scale=scale)
    ref = gate_grad_ref(logits, got, dw, bias, sigmoid, normalize, scale)
    assert_within(dl, ref, 2 * rel * scale * float(dw.abs().max()) + rounding(ref, logits.dtype))
    return idx, w, dl


def _inputs(seed, T, E, dtype, spread):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(T, E, generator=g) * 1.5).to(dtype).cuda(),
            (torch.randn(E, generator=g) * spread).cuda())


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (33, 129, 8), (7, 288, 8), (2, 1024, 32), (4, 7, 7),
                                   (6, 513, 3)])
def test_choice_weights_and_gradient(T, E, K, dtype, sigmoid, normalize):
    logits, bias = _inputs(T * E, T, E, DTYPES[dtype], 0.3)
    _check(logits, K, bias, sigmoid, normalize, scale=2.5)


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_the_score_and_not_the_logit_is_moved(sigmoid, normalize):
    logits = torch.tensor([[6.0, 0.0, -8.0]]).cuda()
    bias = torch.tensor([0.0, 1.2, 0.0]).cuda()      # scores 1, 0.5 or 0.002, 0
    idx, _, _ = _check(logits, 1, bias, sigmoid, normalize)
    assert idx.tolist() == [[1]]
    plain, _ = moedc.gate(logits, 1, bias=bias, flags=_flags(sigmoid, normalize) & ~moedc.GATE_BIAS_SCORE)
    assert plain.tolist() == [[0]]


@pytest.mark.parametrize("sigmoid,normalize", FORMS)
def test_masked_experts_and_rows_with_nothing_left(sigmoid, normalize):
    logits, bias = _inputs(2, 8, 40, torch.float32, 0.3)
    logits[0] = -INF
    logits[1] = -INF
    logits[1, 17] = 0.25
    logits[2, 5] = float("nan")
    logits[3, ::2] = -INF
    logits[4] = float("nan")
    bias[11], bias[12] = -INF, float("nan")
    idx, w, dl = _check(logits, 8, bias, sigmoid, normalize)
    assert (idx[0] == -1).all() and (w[0] == 0).all() and (dl[0] == 0).all()
    assert (idx[4] == -1).all() and (dl[4] == 0).all()
    assert not ((idx == 11) | (idx == 12)).any() and (dl[:, 11:13] == 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_equal_keys_go_to_the_lowest_expert_and_no_bias_to_the_logits(sigmoid):
    logits = torch.zeros(2, 100).cuda()
    bias = torch.zeros(100).cuda()
    bias[50:] = 0.5
    idx, _ = moedc.gate(logits, 6, bias=bias, flags=_flags(sigmoid, True))
    assert idx.tolist() == [[50, 51, 52, 53, 54, 55]] * 2
    logits, _ = _inputs(3, 9, 64, torch.float32, 0.0)
    a = moedc.gate(logits, 4, flags=_flags(sigmoid, True))
    b = moedc.gate(logits, 4, flags=_flags(sigmoid, True) & ~moedc.GATE_BIAS_SCORE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
