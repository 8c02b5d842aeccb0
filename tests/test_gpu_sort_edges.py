"""Sorted rows at the edges: no tokens with a buffer of fixed size."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [64, 63, 4096])
@pytest.mark.parametrize("rows,align", [(1, 1), (64, 1), (1000, 16)])
def test_no_tokens_clear_every_row_of_the_buffer(rows, align, H, dtype):
    """A step without tokens on the buffers of the steps before it."""
    dt, E, K = DTYPES[dtype], 8, 2
    x = torch.randn(5, H).to(dt).cuda()
    idx = torch.randint(0, E, (5, K), dtype=torch.int32).cuda()
    none = idx[:0]
    m = moedc.sort(x[:0], none, E, align=align, rows=rows)
    m.rows.fill_(float("nan"))
    m.src.fill_(7)
    again = moedc.sort(x[:0], none, E, align=align, rows=rows, out=m)
    assert again is m and int(m.status) == 0
    assert (m.rows == 0).all() and (m.src == -1).all()
    assert (m.counts == 0).all() and (m.offsets == 0).all()
    # back, and the gradients
    w = torch.empty(0, K).cuda()
    assert moedc.unsort(m.rows, m.row, w).shape == (0, H)
    drows = torch.full((rows, H), float("nan"), dtype=dt).cuda()
    dw = torch.empty(0, K).cuda()
    moedc.unsort_grad(x[:0], m.rows, m.row, m.src, w, out=(drows, dw))
    assert (drows == 0).all()
    assert moedc.sort_grad(drows, m.row).shape == (0, H)
    # maps alone
    maps = moedc.sort(None, none, E, align=align, rows=rows)
    assert (maps.src == -1).all()


def test_a_buffer_without_rows_reads_and_writes_none():
    x = torch.randn(6, 40).cuda()
    idx = torch.zeros(6, 2, dtype=torch.int32).cuda()
    m = moedc.sort(x, idx, 4, rows=0)
    assert m.rows.shape == (0, 40) and (m.row == -1).all()
    assert int(m.status) == moedc.ERR_CAPACITY
