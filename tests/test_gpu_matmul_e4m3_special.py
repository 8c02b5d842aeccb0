"""NaN and infinities in e4m3 products, in the form for few rows, in clusters and in the form for
many: which outputs and codes they reach."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def _inputs(rows, N, Kd, top):
    """Small whole numbers with scales of powers of two: every sum is exact.  Half of row 2's sums are
    beyond 2^top (values of one sign)."""
    g = torch.Generator().manual_seed(rows + Kd)
    x = torch.randint(-3, 4, (rows, Kd), generator=g).float()
    w = torch.randint(0, 4, (N, Kd), generator=g).float() * 2.0 ** torch.randint(-2, 2, (N, 1), generator=g)
    xs = 2.0 ** torch.randint(-1, 1, (rows, Kd // 128), generator=g).float()
    ws = 2.0 ** torch.randint(0, 2, (-(-N // 128), Kd // 128), generator=g).float()
    x[2:4], xs[2:4] = x[2].abs(), 1.0
    xs[2:4] = 2.0 ** (top - _sums(x[2:3], xs[2:3], w, ws).median().log2().round())
    x[3] *= -1.0
    x[0, 5] = NAN                       # its row, everywhere
    x[1, :128], x[4, :128] = 1.0, -1.0  # infinities, NaN where the group's sum is 0
    xs[1, 0] = xs[4, 0] = INF
    w[9, :128] = 0.0
    w[7, 3] = NAN                       # its column, everywhere
    return x, xs, w, ws


def _sums(x, xs, w, ws):
    """The binary32 values: exact in 64 bits, infinite from 2^128 on."""
    N, Kd = w.shape
    v = torch.zeros(x.shape[0], N, dtype=torch.float64)
    for k in range(Kd // 128):
        part = x[:, 128 * k:128 * k + 128].double() @ w[:, 128 * k:128 * k + 128].double().T
        v = v + part * (xs[:, k:k + 1].double() * ws[:, k].double().repeat_interleave(128)[:N])
    return v.float()


def _codes(v):
    """dispatch's rule: NaN is left out of the maximum; IEEE quotients."""
    a = torch.nan_to_num(v.abs(), nan=0.0, posinf=INF).reshape(v.shape[0], -1, 128)
    scale = a.amax(2).clamp(min=1e-4) / torch.tensor(448.0)
    return (v.reshape(a.shape) / scale[..., None]).reshape(v.shape), scale


# few rows, few rows in a cluster of blocks, many rows
@pytest.mark.parametrize("rows,Kd", [(5, 256), (5, 2048), (40, 2048), (300, 256)])
def test_infinities_and_nan(rows, Kd):
    N = 384
    x, xs, w, ws = _inputs(rows, N, Kd, 128)
    v = _sums(x, xs, w, ws)
    assert torch.isnan(v[0]).all() and torch.isnan(v[:, 7]).all() and torch.isnan(v[1, 9])
    assert torch.isinf(v[1]).sum() == N - 2 and 0 < torch.isinf(v[2]).sum() < N - 1 and (v[3] == -INF).any()
    args = x.cuda().to(E4M3), xs.cuda(), w.cuda().to(E4M3), ws.cuda()
    y = moedc.matmul_e4m3(*args).cpu()
    want = v.to(torch.bfloat16)
    assert torch.equal(torch.isnan(y), torch.isnan(v)) and torch.equal(y[~torch.isnan(v)], want[~torch.isnan(v)])
    codes, scales = (t.cpu() for t in moedc.matmul_e4m3(*args, out_dtype=moedc.FP8_E4M3))
    q, scale = _codes(v)
    assert torch.equal(scales, scale) and torch.isinf(scale[2]).any()
    nan = torch.isnan(q)
    assert torch.equal(torch.isnan(codes.float()), nan)
    assert torch.equal(codes.view(torch.uint8)[~nan], q.to(E4M3).view(torch.uint8)[~nan])


@pytest.mark.parametrize("rows,Kd", [(5, 256), (5, 2048), (300, 256)])
def test_infinities_and_nan_through_the_gate(rows, Kd):
    """silu(gate) * up as the formula has it: a gate of -inf gives NaN, of +inf an infinity of up's
    sign, 0 times an infinity NaN."""
    N = 256
    x, xs, gate, gs = _inputs(rows, N, Kd, 64)
    _, _, up, us = _inputs(rows + 1, N, Kd, 64)
    up[7, 3], up[30] = 1.0, 0.0
    a, b = _sums(x, xs, gate, gs), _sums(x, xs, up, us)
    ref = (a / (1.0 + torch.exp(-a.double()))).float() * b
    assert torch.isnan(ref[4]).all() and torch.isinf(ref[1]).any() and 50 < torch.isinf(ref[2]).sum() < N - 50
    args = (x.cuda().to(E4M3), xs.cuda(), torch.cat([gate, up]).cuda().to(E4M3), torch.cat([gs, us]).cuda())
    y = moedc.matmul_e4m3(*args, swiglu=True).cpu().float()
    assert torch.equal(torch.isnan(y), torch.isnan(ref)) and torch.equal(torch.isinf(y), torch.isinf(ref.to(torch.bfloat16)))
    fine = torch.isfinite(ref.to(torch.bfloat16))
    # one rounding, a few of binary32
    assert ((y - ref).abs()[fine] <= 2.0 ** -7 * ref.abs()[fine] + 1e-37).all()
    codes, scales = (t.cpu() for t in moedc.matmul_e4m3(*args, swiglu=True, out_dtype=moedc.FP8_E4M3))
    q, scale = _codes(ref)
    assert torch.equal(torch.isinf(scales), torch.isinf(scale))
    assert torch.equal(torch.isnan(codes.float()), torch.isnan(q))
    dead = torch.isinf(scale).repeat_interleave(128, 1) & ~torch.isnan(q)
    assert dead.sum() > 50 and (codes.float()[dead] == 0).all()
    live = torch.isfinite(scale).repeat_interleave(128, 1) & ~torch.isnan(q)
    # half a step of the codes and the roundings before them, of a value of magnitude 448 at most
    off = 2.0 ** -4 * q.abs() + 2.0 ** -10 + 448 * 2.0 ** -20
    assert ((codes.float() - q).abs()[live] <= off[live]).all()
