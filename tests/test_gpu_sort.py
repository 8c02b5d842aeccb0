"""Rows sorted by expert and back, and the gradients, against 64-bit forms.

Bounds: sort copies bits.  unsort adds at most K products, each sum and
product rounded: (K + 2) * 2^-24 of the magnitudes, then one rounding to the
type.  drows is one product, rounded in binary32 and to the type.  dweights is
a sum over H whose longest chain is H / 32 elements and some 32 partial sums."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, U32, assert_within, rounding, sort_ref, unsort_ref

pytestmark = pytest.mark.gpu


def _routing(seed, T, K, E, mask=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    if K > E:
        idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    idx[torch.rand(T, K, generator=g) < mask] = -1
    return idx.contiguous().cuda(), torch.randn(T, K, generator=g).cuda()


def _rand(seed, *shape, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check(T, H, K, E, align, mask, dtype, seed=0, poison=False):
    idx, w = _routing(seed, T, K, E, mask)
    x = _rand(seed + 1, T, H, dtype=dtype)
    m = moedc.sort(x, idx, E, align=align)
    R = moedc.moedc_sort_rows(T, K, E, align)
    row, src, offsets, counts = sort_ref(idx, E, align, R)
    assert torch.equal(m.row.cpu(), row) and torch.equal(m.src.cpu(), src)
    assert torch.equal(m.offsets.cpu(), offsets) and torch.equal(m.counts.cpu(), counts)
    want = torch.zeros(R, H, dtype=dtype)
    live = src >= 0
    want[live] = x.cpu()[(src[live] // K).long()]
    assert torch.equal(m.rows.cpu(), want)
    assert int(m.status) == 0
    # the way back
    eo = _rand(seed + 2, R, H, dtype=dtype)
    if poison:                      # rows and weights that no entry reaches
        eo[m.src < 0] = float("nan")
        w[m.row < 0] = float("nan")
    y = moedc.unsort(eo, m.row, w)
    ref, mag = unsort_ref(eo, row, w)
    assert_within(y, ref, (K + 2) * U32 * mag + rounding(ref, dtype))
    # gradients
    dy = _rand(seed + 3, T, H, dtype=dtype)
    drows, dw = moedc.unsort_grad(dy, eo, m.row, m.src, w)
    ref_rows = torch.zeros(R, H, dtype=torch.float64)
    ref_dw, mag_dw = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(row[t, k])
            if r >= 0:
                d = dy[t].cpu().double()
                ref_rows[r] = float(w[t, k]) * d
                p = d * eo[r].cpu().double()
                ref_dw[t, k], mag_dw[t, k] = p.sum(), p.abs().sum()
    assert_within(drows, ref_rows, U32 * ref_rows.abs() * 2 + rounding(ref_rows, dtype))
    assert (drows[m.src < 0] == 0).all()
    assert_within(dw, ref_dw, (H / 32 + 32) * U32 * mag_dw)
    only, none = moedc.unsort_grad(dy, None, m.row, m.src, w)
    assert none is None and torch.equal(only, drows)
    dx = moedc.sort_grad(drows, m.row)
    ref, mag = unsort_ref(drows, row, None)
    assert_within(dx, ref, (K + 2) * U32 * mag + rounding(ref, dtype))
    return m, y, drows, dw, dx


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,H,K,E,align,mask", [
    (1, 8, 1, 1, 1, 0.0), (1, 1, 1, 4, 8, 0.0), (3, 7, 2, 5, 1, 0.3), (16, 128, 8, 128, 1, 0.0),
    (37, 264, 3, 6, 16, 0.1), (50, 129, 4, 9, 1, 0.5), (9, 2048, 6, 60, 8, 0.1),
    (130, 1000, 8, 288, 1, 0.05), (20, 40, 32, 32, 4, 0.0), (11, 4100, 12, 16, 1, 0.1)])
def test_sort_round_trip_and_gradients(T, H, K, E, align, mask, dtype):
    _check(T, H, K, E, align, mask, DTYPES[dtype], seed=T + H)


def test_wide_rows_and_poisoned_padding():
    _check(5, 16384, 4, 8, 4, 0.3, torch.bfloat16, seed=1, poison=True)
    _check(6, 9001, 4, 8, 4, 0.3, torch.float32, seed=2, poison=True)


def test_nothing_routed_and_no_tokens():
    m, y, drows, dw, dx = _check(6, 64, 2, 8, 4, 1.1, torch.bfloat16)
    assert (y == 0).all() and (dw == 0).all() and (dx == 0).all() and (m.rows == 0).all()
    idx = torch.empty((0, 2), dtype=torch.int32).cuda()
    x = torch.empty((0, 64), dtype=torch.bfloat16).cuda()
    m = moedc.sort(x, idx, 8)
    assert m.rows.shape == (0, 64) and (m.counts == 0).all() and (m.offsets == 0).all()
    assert moedc.unsort(m.rows, m.row, torch.empty(0, 2).cuda()).shape == (0, 64)
    moedc.unsort_grad(x, m.rows, m.row, m.src, torch.empty(0, 2).cuda())


@pytest.mark.parametrize("T,K,E", [(700, 8, 64), (513, 6, 60), (2200, 8, 256), (9000, 8, 128),
                                   (30000, 4, 16)])
def test_maps_on_every_layout_path(T, K, E):
    idx, _ = _routing(T, T, K, E, 0.05)
    m = moedc.sort(None, idx, E, align=8)
    R = moedc.moedc_sort_rows(T, K, E, 8)
    row, src, offsets, counts = sort_ref(idx, E, 8, R)
    assert m.rows is None
    assert torch.equal(m.row.cpu(), row) and torch.equal(m.src.cpu(), src)
    assert torch.equal(m.offsets.cpu(), offsets) and torch.equal(m.counts.cpu(), counts)


def test_one_expert_takes_everything_and_repeated_experts():
    T, K, E = 40, 4, 6
    idx = torch.full((T, K), 3, dtype=torch.int32).cuda()
    x = _rand(0, T, 96, dtype=torch.float16)
    m = moedc.sort(x, idx, E, align=32)
    row, src, offsets, counts = sort_ref(idx, E, 32, moedc.moedc_sort_rows(T, K, E, 32))
    assert torch.equal(m.row.cpu(), row) and torch.equal(m.offsets.cpu(), offsets)
    assert torch.equal(m.rows[:T * K].cpu(), x.cpu().repeat_interleave(K, 0))


@pytest.mark.parametrize("rows", [0, 1, 50, 77])
def test_a_buffer_that_is_too_small_drops_and_reports(rows):
    T, H, K, E, align = 20, 72, 4, 8, 4
    idx, w = _routing(4, T, K, E)
    x = _rand(5, T, H, dtype=torch.bfloat16)
    m = moedc.sort(x, idx, E, align=align, rows=rows)
    row, src, offsets, counts = sort_ref(idx, E, align, rows)
    assert torch.equal(m.row.cpu(), row) and torch.equal(m.src.cpu(), src)
    assert torch.equal(m.offsets.cpu(), offsets) and torch.equal(m.counts.cpu(), counts)
    assert int(m.status) == moedc.ERR_CAPACITY
    want = torch.zeros(rows, H, dtype=torch.bfloat16)
    live = src >= 0
    want[live] = x.cpu()[(src[live] // K).long()]
    assert torch.equal(m.rows.cpu(), want)


def test_index_out_of_range_is_masked_and_reported():
    idx, _ = _routing(6, 12, 3, 8)
    idx[2, 1], idx[5, 0] = 8, -7
    clean = idx.clone()
    clean[2, 1], clean[5, 0] = -1, -1
    x = _rand(7, 12, 48, dtype=torch.bfloat16)
    m, c = moedc.sort(x, idx, 8), moedc.sort(x, clean, 8)
    assert int(m.status) == moedc.ERR_EXPERT_RANGE and int(c.status) == 0
    for a, b in ((m.rows, c.rows), (m.row, c.row), (m.src, c.src), (m.offsets, c.offsets)):
        assert torch.equal(a, b)


def test_rows_outside_the_buffer_are_skipped():
    row = torch.tensor([[0, 5], [-3, 1], [2, 1 << 30]], dtype=torch.int32).cuda()
    s = _rand(8, 3, 40, dtype=torch.float32)
    y = moedc.unsort(s, row, torch.ones(3, 2).cuda())
    assert torch.equal(y, s[[0, 1, 2]])


@pytest.mark.parametrize("H,pad", [(64, 8), (64, 3), (63, 0)])
def test_strided_tokens(H, pad):
    idx, w = _routing(9, 14, 2, 5)
    wide = _rand(10, 14, H + pad + 8, dtype=torch.bfloat16)
    x = wide[:, pad:pad + H]
    a, b = moedc.sort(x, idx, 5), moedc.sort(x.contiguous(), idx, 5)
    assert torch.equal(a.rows, b.rows)
    ga = moedc.unsort_grad(x, a.rows, a.row, a.src, w)
    gb = moedc.unsort_grad(x.contiguous(), a.rows, a.row, a.src, w)
    assert torch.equal(ga[0], gb[0])
    assert_within(ga[1], gb[1].cpu().double(),
                  (H / 32 + 32) * U32 * 2 * (x.abs().float().sum().item()) * 8)


def test_gradients_against_differences():
    """The loss <y, g> is linear in the rows and in the weights: its
    differences are exact up to the 64-bit sums."""
    T, H, K, E = 5, 12, 2, 4
    idx, w = _routing(11, T, K, E, 0.2)
    m = moedc.sort(None, idx, E)
    R = m.src.shape[0]
    eo, g = _rand(12, R, H, dtype=torch.float32), _rand(13, T, H, dtype=torch.float32)
    drows, dw = moedc.unsort_grad(g, eo, m.row, m.src, w)
    row = m.row.cpu()

    def loss(rows, weights):
        return (unsort_ref(rows, row, weights)[0] * g.cpu().double()).sum()

    base = loss(eo, w)
    for t in range(T):
        for k in range(K):
            w2 = w.cpu().double()
            w2[t, k] += 1.0
            assert abs(loss(eo, w2) - base - dw[t, k].item()) < 1e-5
    for r in range(R):
        e2 = eo.cpu().double()
        e2[r, 3] += 1.0
        assert abs(loss(e2, w) - base - drows[r, 3].item()) < 1e-5
    # sort: <sorted, c> moves by c summed over a token's rows
    c = _rand(14, R, H, dtype=torch.float32)
    dx = moedc.sort_grad(c, m.row)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for r in range(R):
        i = int(m.src[r])
        if i >= 0:
            ref[i // K] += c[r].cpu().double()
    assert_within(dx, ref, 1e-5)


def test_equal_bits_on_every_call_stream_and_reused_buffers():
    idx, w = _routing(15, 300, 8, 64, 0.05)
    x = _rand(16, 300, 520, dtype=torch.bfloat16)
    m = moedc.sort(x, idx, 64, align=8)
    eo = _rand(17, m.src.shape[0], 520, dtype=torch.bfloat16)
    first = moedc.unsort_grad(x, eo, m.row, m.src, w)
    kept = [t.clone() for t in (m.rows, m.row, m.src, m.offsets, m.counts)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = moedc.sort(x, idx, 64, align=8, out=m)
        second = moedc.unsort_grad(x, eo, m.row, m.src, w)
    side.synchronize()
    assert again is m
    for a, b in zip(kept, (m.rows, m.row, m.src, m.offsets, m.counts)):
        assert torch.equal(a, b)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


def test_refusals():
    idx, w = _routing(18, 6, 2, 8)
    x = _rand(19, 6, 32, dtype=torch.bfloat16)
    for bad in (lambda: moedc.sort(x, idx, 0), lambda: moedc.sort(x, idx, 2000),
                lambda: moedc.sort(x, idx, 8, align=0), lambda: moedc.sort(x, idx, 8, align=4096)):
        with pytest.raises(moedc.MoedcError):
            bad()
    m = moedc.sort(x, idx, 8)
    for bad in (lambda: moedc.sort(x.double(), idx, 8), lambda: moedc.sort(x[:5], idx, 8),
                lambda: moedc.sort(x.T, idx, 8), lambda: moedc.sort(x, idx.long(), 8),
                lambda: moedc.sort(x, idx, 7, out=m), lambda: moedc.sort(None, idx, 8, out=m),
                lambda: moedc.sort(x, idx, 8, out=m, rows=3),
                lambda: moedc.unsort(m.rows, m.row, w[:, :1]),
                lambda: moedc.unsort(m.rows, m.row, w.double()),
                lambda: moedc.unsort_grad(x, m.rows[:3], m.row, m.src, w),
                lambda: moedc.unsort_grad(x.float(), m.rows, m.row, m.src, w)):
        with pytest.raises(ValueError):
            bad()
