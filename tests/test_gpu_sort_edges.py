"""Sorted rows at the edges: no tokens with a buffer of fixed size, rows moved by
element, offsets past 32 bits."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, U32, sort_ref

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


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,K,E,H,align,mask", [(400, 4, 8, 63, 1, 0.0), (300, 8, 60, 1, 16, 0.1),
                                                (701, 2, 128, 517, 4, 0.2), (1500, 1, 5, 130, 8, 0.0)])
def test_many_entries_with_rows_moved_by_element(T, K, E, H, align, mask, dtype):
    """More entries than the single launch takes, with odd widths or rows that begin
    off a 16-byte boundary."""
    g = torch.Generator().manual_seed(T)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    idx[torch.rand(T, K, generator=g) < mask] = -1
    wide = torch.randn(T, H + 5, generator=g).to(DTYPES[dtype]).cuda()
    x = wide[:, 1:1 + H]
    m = moedc.sort(x, idx.cuda(), E, align=align)
    row, src, offsets, counts = sort_ref(idx, E, align, m.src.shape[0])
    assert torch.equal(m.row.cpu(), row) and torch.equal(m.src.cpu(), src)
    assert torch.equal(m.offsets.cpu(), offsets) and torch.equal(m.counts.cpu(), counts)
    want = torch.zeros(m.rows.shape, dtype=x.dtype)
    live = src >= 0
    want[live] = x.cpu()[(src[live] // K).long()]
    assert torch.equal(m.rows.cpu(), want) and int(m.status) == 0
    # back: K equal weights of 1 / K where nothing is masked, all of them powers of two
    if mask == 0.0:
        w = torch.full((T, K), 1.0 / K).cuda()
        assert torch.equal(moedc.unsort(m.rows, m.row, w), x)


def test_packed_rows_past_32_bit_offsets():
    """320000 rows of 7168: 2.3e9 elements.  Eight weights of 1/8 give x back exactly,
    and its gradient rows are x / 8 exactly; dweights is a sum of 7168 squares with
    chains of 7168 / 256 and some 16 partial sums."""
    T, K, E, H = 40000, 8, 64, 7168
    g = torch.Generator(device="cuda").manual_seed(0)
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    m = moedc.sort(x, idx, E)
    assert int(m.status) == 0 and m.rows.numel() > 2 ** 31
    for k in range(K):
        assert torch.equal(m.rows[m.row[:, k].long()], x)
    w = torch.full((T, K), 0.125).cuda()
    assert torch.equal(moedc.unsort(m.rows, m.row, w), x)
    drows, dw = moedc.unsort_grad(x, m.rows, m.row, m.src, w)
    for k in range(K):
        assert torch.equal(drows[m.row[:, k].long()], x * 0.125)
    ref = torch.cat([part.double().square().sum(1) for part in x.split(4000)])
    assert ((dw.double() - ref[:, None]).abs() <= (7168 / 256 + 32) * U32 * ref[:, None]).all()
    del drows
    assert torch.equal(moedc.sort_grad(m.rows, m.row), x * 8.0)
