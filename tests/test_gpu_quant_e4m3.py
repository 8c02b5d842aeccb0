"""Rows and blocks to e4m3: bit for bit the rule in binary32, and what dispatch writes."""
import os
import subprocess

import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES

pytestmark = pytest.mark.gpu


def _nearest(q):
    """Nearest e4m3 value, ties to even, in 64 bits: three fraction bits, exponents from -6."""
    power = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -60))).clamp(min=-6.0)
    step = torch.exp2(power - 3.0)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _ref(x, block_rows):
    """(codes' values f64, scales f32) of one expert's [R, Kd]."""
    x = x.cpu().float()
    R, Kd = x.shape
    padded = torch.zeros(-(-R // block_rows) * block_rows, Kd)
    padded[:R] = x
    amax = padded.reshape(-1, block_rows, Kd // 128, 128).abs().amax((1, 3))
    scale = torch.maximum(amax, torch.tensor(1e-4)) / torch.tensor(448.0)
    wide = scale.repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)
    return _nearest((x / wide).double()), scale


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,R,Kd", [(None, 1, 128), (None, 37, 640), (None, 128, 256), (3, 129, 384), (2, 300, 1152),
                                    (None, 2000, 128)])
def test_against_the_rule(E, R, Kd, dtype, block_rows):
    g = torch.Generator().manual_seed(R)
    x = torch.randn(*([E] if E else []), R, Kd, generator=g)
    x[..., ::7, :] *= 100.0
    x[..., 0, :128] = 0.0                      # the smallest scale
    x[..., R // 2, -128:] *= 1e-6
    x = x.to(DTYPES[dtype])
    codes, scales = moedc.quant_e4m3(x.cuda(), block_rows=block_rows)
    for e in range(E or 1):
        want, scale = _ref(x[e] if E else x, block_rows)
        got, sc = (codes[e], scales[e]) if E else (codes, scales)
        assert torch.equal(sc.cpu(), scale)
        assert torch.equal(got.cpu().double(), want)


def test_every_e4m3_tie_and_step():
    """Every value, every midpoint between two and their neighbours go to their code: the scale is 1,
    but for the rows that hold 448 (1 + 2^-20), where the rule makes it the next binary32 numbers'."""
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    values = torch.unique(values[torch.isfinite(values)])
    ties = (values[1:] + values[:-1]) / 2
    x = torch.cat([values, ties, values * (1 + 2.0 ** -20), values * (1 - 2.0 ** -20)])
    x = torch.cat([x, torch.zeros(-x.numel() % 127)]).reshape(-1, 127)
    x = torch.cat([x, torch.full((x.shape[0], 1), 448.0)], 1)
    codes, scales = moedc.quant_e4m3(x.cuda())
    want, scale = _ref(x, 1)
    assert torch.equal(scales.cpu(), scale) and (scale == 1.0).sum() >= scale.numel() - 2
    assert torch.equal(codes.cpu().double(), want)


def test_nan_infinities_and_strides():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(9, 512, generator=g).cuda()
    x = wide[:, 128:384]
    x[2, 5], x[4, 200], x[6, 0] = float("nan"), float("inf"), -0.0
    for block_rows in (1, 128):
        codes, scales = moedc.quant_e4m3(x, block_rows=block_rows)
        again, same = moedc.quant_e4m3(x.contiguous(), block_rows=block_rows)
        assert torch.equal(codes.view(torch.uint8), again.view(torch.uint8)) and torch.equal(scales, same)
        v = codes.float()
        assert torch.isnan(v[2, 5]) and torch.isnan(v[4, 200])
        assert int(torch.isnan(v).sum()) == 2
        assert (v[4, 128:][torch.arange(128) != 72] == 0).all()      # others beside an infinity
        assert torch.isfinite(scales).sum() == scales.numel() - 1


def test_as_dispatch_does():
    g = torch.Generator().manual_seed(2)
    T, H = 50, 1024
    x = (torch.randn(T, H, generator=g) * torch.rand(T, 1, generator=g) * 50).to(torch.bfloat16).cuda()
    idx = torch.zeros(T, 1, dtype=torch.int32).cuda()
    lay = moedc.layout(idx, 1, 1, T)
    recv, scales, _ = moedc.dispatch(x, idx, lay, 1, T, moedc.FP8_E4M3)
    codes, mine = moedc.quant_e4m3(x)
    assert torch.equal(codes.view(torch.uint8), recv[0].view(torch.uint8)) and torch.equal(mine, scales[0])


def test_reused_buffers_empty_and_refused():
    x = torch.randn(4, 256).cuda()
    out = moedc.quant_e4m3(x)
    assert moedc.quant_e4m3(x, out=out) is out
    assert moedc.quant_e4m3(x[:0])[0].shape == (0, 256)
    for bad in (dict(x=x.cpu()), dict(x=x.long()), dict(block_rows=64), dict(block_rows=128, out=out),
                dict(x=x.T), dict(x=x[:3], out=out), dict(x=x.reshape(2, 2, 256).transpose(0, 1))):
        args = dict(x=x) | bad
        with pytest.raises(ValueError):
            moedc.quant_e4m3(args.pop("x"), **args)
    for bad in (x[:, :200], x.flatten()[1:1 + 768].view(3, 256), x[:, 1:129]):
        with pytest.raises(moedc.MoedcError):
            moedc.quant_e4m3(bad)


def test_quotients_are_the_divisions(tmp_path):
    """Every mantissa of a divisor with every one of a bf16 and an f16 dividend, and 2^33
    binary32 pairs; the program is built here, not into the library."""
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    exe = str(tmp_path / "quotient_sweep")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I" + os.path.join(root, "include"),
                    "-I" + os.path.join(root, "combine_moedc_layout_gb300", "csrc"),
                    os.path.join(here, "cuda", "quotient_sweep.cu"), "-o", exe], check=True, capture_output=True)
    done = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout + done.stderr


def test_zeros_keep_their_sign_as_in_dispatch():
    x = torch.tensor([0.0, -0.0, 1e-30, -1e-30] * 32).to(torch.bfloat16).reshape(1, 128).cuda()
    lay = moedc.layout(torch.zeros(1, 1, dtype=torch.int32).cuda(), 1, 1, 1)
    recv, _, _ = moedc.dispatch(x, torch.zeros(1, 1, dtype=torch.int32).cuda(), lay, 1, 1, moedc.FP8_E4M3)
    assert torch.equal(moedc.quant_e4m3(x)[0].view(torch.uint8), recv[0].view(torch.uint8))
    assert torch.equal(moedc.quant_e4m3(x, block_rows=128)[0].view(torch.uint8), recv[0].view(torch.uint8))
