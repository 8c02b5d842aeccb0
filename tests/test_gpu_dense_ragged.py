"""Weight gradients of experts that end anywhere in 16 rows, beside rows of NaN: both blocks of a
pair clear what the products must not see, over and over."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import assert_within, rounding
from matmul_util import groups, owned, product, randn
from test_gpu_dense_edges import _need_bytes, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dw_dtype", [None, torch.float32])
@pytest.mark.parametrize("counts", [[1, 15, 17, 31, 33, 47, 49, 63] * 8, [65, 769, 127, 770, 1, 783] * 2, [9] * 300])
def test_cleared_rows(counts, dw_dtype):
    g = torch.Generator().manual_seed(len(counts))
    offsets, cnt, rows = groups(counts, 16)
    x, d = randn(g, torch.bfloat16, rows, 520), randn(g, torch.bfloat16, rows, 264)
    mine = owned(offsets, cnt, rows)
    x[~mine], d[~mine] = float("nan"), float("inf")
    status = _status()
    args = dict(offsets=offsets, counts=cnt, dw_dtype=dw_dtype, status=status)
    _, first = moedc.matmul_grad(d, x, None, **args)
    for e in range(0, len(counts), 7):
        a, c = int(offsets[e]), counts[e]
        v, err = product(d[a:a + c].T.contiguous(), x[a:a + c].T.contiguous(), False)
        assert_within(first[e], v, err + rounding(v.abs() + err, first.dtype))
    again = torch.empty_like(first)
    for _ in range(40):
        moedc.matmul_grad(d, x, None, out=(None, again), **args)
        assert torch.equal(again, first)
    assert int(status) == 0


def test_rows_to_clear_behind_many_stages():
    """The warp that clears waits some 0.4 s for the one stage that it has to do with."""
    _need_bytes(16 << 30)
    rows = (3 << 25) + 5
    x = torch.ones(rows + 64, 8, dtype=torch.bfloat16, device="cuda")
    d = torch.ones(rows + 64, 8, dtype=torch.bfloat16, device="cuda")
    x[rows:], d[rows:] = float("nan"), float("nan")
    o = torch.tensor([0, rows], dtype=torch.int32).cuda()
    status = _status()
    for dw_dtype in (None, torch.float32):
        _, dw = moedc.matmul_grad(d, x, None, offsets=o, counts=o[1:], dw_dtype=dw_dtype, status=status)
        assert int(status) == moedc.OK
        # the pieces' sums are exact up to 2^24, then half an ulp of at most 2^27 each
        assert ((dw[0].double() - rows).abs() <= rows * (2.0 ** -8 if dw_dtype is None else rows / 768 * 2.0 ** -24)).all()
