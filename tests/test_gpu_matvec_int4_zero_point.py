"""4-bit products where a large value of x meets weights at the zero point: the
product is exactly zero, so the other channels' sum keeps its bound (which
counts |q - z| |x|), in every form of the product.

x is N(0, 1) in bf16 beside values of about 2^22.  In the forms that bring x
into f16, a value below 2^-27 of the record's largest is rounded by at most
2^-35 of it: 2^-13 for the one value in 40 that lies below 2^-5, some 30 of
1280 channels, times at most 15 and of either sign.  That adds up to some
0.005 scales, a tenth of the 0.05 that the bound's (Kd / 8 + 64) roundings give
there."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import assert_within, int4_weights, matvec_ref, rounding
from test_gpu_matvec_int4 import _weights

pytestmark = pytest.mark.gpu

INF = float("inf")

# (T, E, K, N, Kd, group, swiglu): the one launch for few weights; prepared x with units of
# 8, 16 and 32 rows and one part of K or several; experts of many rows
SHAPES = [(5, 4, 2, 40, 512, 32, False), (5, 4, 2, 40, 512, 64, True), (9, 2, 1, 30, 1280, 128, False),
          (6, 1, 1, 110000, 512, 128, False), (6, 1, 1, 60000, 512, 64, True),
          (6, 1, 1, 110000, 512, 32, False), (6, 160, 2, 9000, 512, 128, False),
          (14, 1, 1, 60000, 512, 128, False), (14, 1, 1, 60000, 512, 64, False),
          (40, 2, 1, 9000, 1280, 32, False),
          (70, 1, 1, 6000, 1280, 64, False), (70, 1, 1, 6000, 1280, 128, True)]


def _inputs(T, E, K, N, Kd, group, swiglu, zeros, seed):
    g = torch.Generator().manual_seed(seed)
    n = 2 * N if swiglu else N
    wq, s, z = _weights(g, E, n, Kd, group, zeros, torch.bfloat16)
    x = torch.randn(T, Kd, generator=g).to(torch.bfloat16).cuda()
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    m = moedc.sort(None, idx.cuda(), E)
    return g, x, wq, s, z, m


def _run(x, wq, s, z, m, K, swiglu):
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = moedc.matvec_int4(x, wq, s, zeros=z, offsets=m.offsets, counts=m.counts, src=m.src,
                            top_k=K, swiglu=swiglu, status=status)
    assert int(status) == 0
    return out


def _experts(m):
    offsets, counts = m.offsets.tolist(), m.counts.tolist()
    for e, c in enumerate(counts):
        if c:
            yield e, slice(offsets[e], offsets[e] + c)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,E,K,N,Kd,group,swiglu", SHAPES)
def test_large_values_at_the_zero_point_add_nothing(T, E, K, N, Kd, group, swiglu, zeros):
    g, x, wq, s, z, m = _inputs(T, E, K, N, Kd, group, swiglu, zeros, T + group)
    for c in (3, 130, 301, Kd - 2):              # odd and even channels, several groups
        x[:, c] = (torch.rand(T, generator=g) + 3.0).to(torch.bfloat16).cuda() * 2.0 ** 20
        at = z[:, :, c // group] if zeros else torch.full_like(wq[:, :, 0], 8)
        b = wq[:, :, c // 2]
        wq[:, :, c // 2] = (b & 0x0f) | (at << 4) if c % 2 else (b & 0xf0) | at
    out = _run(x, wq, s, z, m, K, swiglu)
    for e, rows in _experts(m):
        w = int4_weights(wq[e], s[e], None if z is None else z[e], group)
        ref, err = matvec_ref(x[(m.src[rows] // K).long()], w, swiglu)
        assert_within(out[rows], ref.cuda(), err + rounding(ref, torch.bfloat16))


@pytest.mark.parametrize("T,E,K,N,Kd,group,swiglu", SHAPES)
def test_infinities_follow_the_formula_in_every_form(T, E, K, N, Kd, group, swiglu):
    """inf * 0 and inf - inf are NaN, everything else of an infinity is one, and
    only in its own token's rows."""
    _, x, wq, s, z, m = _inputs(T, E, K, N, Kd, group, swiglu, True, T + N)
    x[1, 7] = INF
    x[2, Kd - 1] = -INF
    x[3, 300] = float("nan")
    x[4, 0], x[4, 270] = INF, -INF
    out = _run(x, wq, s, z, m, K, swiglu)
    for e, rows in _experts(m):
        w = int4_weights(wq[e], s[e], z[e], group)
        ref, err = matvec_ref(x[(m.src[rows] // K).long()], w, swiglu)
        got = out[rows].double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        inf = torch.isinf(ref)
        assert torch.equal(got[inf], ref[inf])
        fine = torch.isfinite(ref)
        bound = err[fine] + rounding(ref[fine], torch.bfloat16)
        assert ((got[fine] - ref[fine]).abs() <= bound).all()
