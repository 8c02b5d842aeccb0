"""Rows and columns as many as the arguments can say, and more."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from matmul_util import randn
from test_gpu_dense_edges import _near, _need_bytes, _status

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


def _need(gib):
    torch.cuda.empty_cache()
    _need_bytes(gib << 30)


def test_as_many_rows_as_there_are_numbers():
    """One expert and two, whose rows end at the largest number: forward and dx."""
    _need(150)
    g = torch.Generator().manual_seed(0)
    x = torch.zeros(MOST, 8, dtype=torch.bfloat16, device="cuda")
    x[:300], x[-300:] = randn(g, torch.bfloat16, 300, 8), randn(g, torch.bfloat16, 300, 8)
    w = randn(g, torch.bfloat16, 2, 8, 8)
    status = _status()
    y = torch.empty_like(x)
    moedc.matmul(x, w[0], status=status, out=y)
    assert int(status) == 0
    _near(y[:300], x[:300], w[0])
    _near(y[-300:], x[-300:], w[0])
    assert not y[300:300 + (1 << 20)].any() and not y[-300 - (1 << 20):-300].any()
    o = torch.tensor([0, 300, MOST], dtype=torch.int32).cuda()
    c = torch.tensor([300, MOST - 300], dtype=torch.int32).cuda()
    y[300:-300] = 0
    dx = torch.empty_like(x)
    moedc.matmul_grad(y, None, w, offsets=o, counts=c, status=status, out=(dx, None))
    assert int(status) == 0
    for e, part in enumerate((slice(0, 300), slice(MOST - 300, MOST))):
        _near(dx[part], y[part], w[e].T.contiguous())


def test_as_many_columns_as_there_are_numbers():
    """dx and dW as wide as can be, a forward with as many outputs; the first and the last of them."""
    _need(160)
    g = torch.Generator().manual_seed(1)
    Kd = 2 ** 31 - 8
    status = _status()
    x, w = torch.zeros(2, Kd, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, Kd, dtype=torch.bfloat16, device="cuda")
    for part in (slice(0, 300), slice(Kd - 300, Kd)):
        x[:, part], w[:, part] = randn(g, torch.bfloat16, 2, 300), randn(g, torch.bfloat16, 8, 300)
    d = randn(g, torch.bfloat16, 2, 8)
    dx, dw = moedc.matmul_grad(d, x, w, status=status)
    assert int(status) == 0
    for part in (slice(0, 300), slice(Kd - 300, Kd)):
        _near(dx[:, part], d, w[:, part].T.contiguous())
        _near(dw[:, part], d.T.contiguous(), x[:, part].T.contiguous())
    del dx, dw, w
    Kd = 2 ** 30 + 8
    x = x.view(-1)[-2 * Kd:].view(2, Kd)
    x[0, :300] = 1.0
    _, dw = moedc.matmul_grad(d, x, None, dw_dtype=torch.float32, status=status)
    assert int(status) == 0
    for part in (slice(0, 300), slice(Kd - 300, Kd)):
        _near(dw[0][:, part], d.T.contiguous(), x[:, part].T.contiguous(), dtype=torch.float32)
    del x, dw
    N = 2 ** 30 - 8
    w = torch.zeros(2 * N, 8, dtype=torch.bfloat16, device="cuda")
    parts = (slice(0, 300), slice(N - 300, N), slice(2 * N - 300, 2 * N))
    for part in parts:
        w[part] = randn(g, torch.bfloat16, 300, 8)
    x = randn(g, torch.bfloat16, 3, 8)
    y = moedc.matmul(x, w[:N], status=status)
    h, kept = moedc.matmul(x, w, swiglu=True, keep=True, status=status)
    assert int(status) == 0
    for part in parts:
        _near(kept[:, part], x, w[part])
    for part in parts[:2]:
        _near(y[:, part], x, w[part])
    _near(h[:, -300:], x, torch.cat([w[parts[1]], w[parts[2]]]), True)


def test_more_rows_than_numbers_are_refused():
    """2^32 rows would arrive at the library as none."""
    _need(150)
    rows = 2 ** 32
    memory = torch.empty(16 * rows, dtype=torch.bfloat16, device="cuda")
    x, products = memory[:8 * rows].view(rows, 8), memory.view(rows, 16)
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: moedc.matmul(x, w), lambda: moedc.matmul_grad(x, x, w),
                 lambda: moedc.matmul_grad(x, None, w), lambda: moedc.swiglu_grad(x, products)):
        with pytest.raises(ValueError):
            call()
    e4m3, one = torch.float8_e4m3fn, torch.ones(1, 1, device="cuda")
    src = memory.view(torch.int32)[:rows]
    with pytest.raises(ValueError):
        moedc.matmul_e4m3(torch.zeros(1, 128, device="cuda").to(e4m3), one, torch.zeros(8, 128, device="cuda").to(e4m3), one,
                          src=src)
    wide = memory[:8 * (rows + 8)].view(8, rows + 8)
    with pytest.raises(ValueError):
        moedc.matmul(wide[:1], wide)
    with pytest.raises(ValueError):
        moedc.matmul_grad(w[:1], None, wide)
    with pytest.raises(ValueError):
        moedc.quant_e4m3(wide[None], block_rows=128)
