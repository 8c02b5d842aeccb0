"""The dense layers over contracted axes and calls that are long: sums that stay as exact as
short ones, waits that are bounded by a step of the work and not by the call."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import ROUND, U32
from test_gpu_dense_edges import _need_bytes, _status

pytestmark = pytest.mark.gpu


def _uniform(seed, dtype, *shape, lo=0.0, hi=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.rand(part.shape, generator=g, device="cuda") * (hi - lo) + lo)
    return out


def _dw64(d, x, step=1 << 22):
    return sum(d[a:a + step].double().T @ x[a:a + step].double() for a in range(0, len(x), step))


def test_weight_gradients_of_one_tile_over_many_tokens():
    """One pair of SMs for some 0.4 s.  Values of one sign: relative errors of the sum are at most
    an ulp (2 * 2^-24) for each of a piece's 48 products, half an ulp for each of the pieces."""
    _need_bytes(16 << 30)
    rows = 3 << 25
    x, d = _uniform(0, torch.bfloat16, rows, 8), _uniform(1, torch.bfloat16, rows, 8)
    status = _status()
    _, dw = moedc.matmul_grad(d, x, None, dw_dtype=torch.float32, status=status)
    assert int(status) == moedc.OK
    ref = _dw64(d, x)
    assert ((dw[0].double() - ref).abs() <= (96 + rows / 768) * U32 * ref).all()


def test_products_of_a_third_of_a_second():
    """Every pair of SMs is at work for the whole call."""
    _need_bytes(64 << 30)
    rows, N, Kd = 1 << 17, 1 << 16, 1 << 15
    x, w = _uniform(2, torch.bfloat16, rows, Kd), _uniform(3, torch.bfloat16, N, Kd)
    status = _status()
    y = moedc.matmul(x, w, status=status)
    assert int(status) == moedc.OK
    for r in (0, 70000, rows - 40):
        for n in (0, 40000, N - 200):
            ref = x[r:r + 40].double() @ w[n:n + 200].double().T
            got = y[r:r + 40, n:n + 200].double()
            # an ulp for each product of 16, one rounding
            assert ((got - ref).abs() <= (Kd / 8 * U32 + ROUND[torch.bfloat16]) * ref).all()


# A sum of 16-bit outputs: an ulp (2 * 2^-24) for each of at most 512 products of 16 in a piece, half an
# ulp for each piece and for the sums of up to four pairs, one rounding of the result.
def _bound(K, dtype):
    return (1024 + K / 8192 + 1 + 4) * U32 + ROUND[dtype]


@pytest.mark.parametrize("rows", [8200, 65536 + 24, 1 << 20])
def test_sixteen_bit_weight_gradients_of_many_tokens(rows):
    """Values of one sign, where what a sum loses adds up."""
    x, d = (_uniform(s, torch.float16, rows, n, lo=2.0 ** -4, hi=2.0 ** -3) for s, n in ((4, 72), (5, 264)))
    status = _status()
    _, dw = moedc.matmul_grad(d, x, None, status=status)
    ref = _dw64(d, x)
    assert int(status) == 0 and ((dw[0].double() - ref).abs() <= _bound(rows, torch.float16) * ref).all()
    # two experts, one of them short
    o = torch.tensor([0, 100, rows], dtype=torch.int32).cuda()
    c = torch.tensor([100, rows - 100], dtype=torch.int32).cuda()
    _, dw = moedc.matmul_grad(d, x, None, offsets=o, counts=c, status=status)
    for e, part in enumerate((slice(0, 100), slice(100, rows))):
        ref = _dw64(d[part], x[part])
        assert ((dw[e].double() - ref).abs() <= _bound(rows, torch.float16) * ref).all()


def test_sixteen_bit_gradients_of_one_tile_over_many_tokens():
    """One pair of SMs for some 0.4 s."""
    _need_bytes(16 << 30)
    rows = 3 << 25
    x, d = _uniform(10, torch.bfloat16, rows, 8), _uniform(11, torch.bfloat16, rows, 8)
    status = _status()
    _, dw = moedc.matmul_grad(d, x, None, status=status)
    assert int(status) == moedc.OK
    ref = _dw64(d, x)
    assert ((dw[0].double() - ref).abs() <= _bound(rows, torch.bfloat16) * ref).all()


# two and four pairs of SMs to a tile, one pair
@pytest.mark.parametrize("rows,n", [(40, 80), (200, 272), (300, 272), (700, 4112)])
@pytest.mark.parametrize("K", [8200, 131080, 1 << 20])
def test_rows_and_their_gradients_over_a_long_axis(rows, n, K):
    if rows * K + n * K > 1 << 30:
        K = 131080
    x = _uniform(6, torch.float16, rows, K, lo=2.0 ** -4, hi=2.0 ** -3)
    w = _uniform(7, torch.float16, n, K, lo=2.0 ** -4, hi=2.0 ** -3)
    ref = sum(x[:, k:k + 8192].double() @ w[:, k:k + 8192].double().T for k in range(0, K, 8192))
    status = _status()
    y = moedc.matmul(x, w, status=status)
    assert int(status) == 0 and ((y.double() - ref).abs() <= _bound(K, torch.float16) * ref).all()
    half = n // 2
    h, p = moedc.matmul(x[:, :K], w, swiglu=True, keep=True, status=status)
    assert torch.equal(p, y)
    # of x W: the weights' rows are contracted
    dx, _ = moedc.matmul_grad(x, None, w.T.contiguous(), status=status)
    assert int(status) == 0 and ((dx.double() - ref).abs() <= _bound(K, torch.float16) * ref).all()


def test_gated_block_over_a_long_axis():
    """SwiGLU of sums below 1, where it is not the rounding of one of them."""
    K = 131080
    x = _uniform(8, torch.float16, 50, K, lo=2.0 ** -9, hi=2.0 ** -8)
    w = _uniform(9, torch.float16, 144, K, lo=2.0 ** -9, hi=2.0 ** -8)
    status = _status()
    h = moedc.matmul(x, w, swiglu=True, status=status)
    v = x.double() @ w.double().T
    a, b = v[:, :72], v[:, 72:]
    ref = a * torch.sigmoid(a) * b
    # d log silu(a) / d log a = 1 + a (1 - s) <= 1 + a; 16 roundings of the epilogue
    off = (_bound(K, torch.float32) * (2 + a) + 16 * U32 + ROUND[torch.float16]) * ref
    assert int(status) == 0 and ((h.double() - ref).abs() <= off).all()


def test_one_tile_over_an_axis_of_many_elements():
    """Four pairs of SMs for some 0.3 s: each waits for a piece of its sum, not for all of it."""
    _need_bytes(32 << 30)
    N = 1 << 28
    d = _uniform(12, torch.bfloat16, 8, N)
    w = _uniform(13, torch.bfloat16, N, 8)
    status = _status()
    dx, _ = moedc.matmul_grad(d, None, w, status=status)
    assert int(status) == moedc.OK
    ref = sum(d[:, a:a + (1 << 22)].double() @ w[a:a + (1 << 22)].double() for a in range(0, N, 1 << 22))
    assert ((dx.double() - ref).abs() <= _bound(N, torch.bfloat16) * ref).all()
