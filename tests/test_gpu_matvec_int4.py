"""Products with 4-bit weights and group scales against 64-bit forms."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, assert_within, int4_weights, matvec_ref, rounding, sort_ref

pytestmark = pytest.mark.gpu


def _weights(g, E, n, Kd, group, zeros, sdtype):
    wq = torch.randint(0, 256, (E, n, Kd // 2), generator=g, dtype=torch.uint8)
    s = ((0.5 + torch.rand(E, n, Kd // group, generator=g)) * 0.2 / Kd ** 0.5).to(sdtype)
    z = torch.randint(0, 16, s.shape, generator=g, dtype=torch.uint8) if zeros else None
    return wq.cuda(), s.cuda(), z.cuda() if zeros else None


def _check(T, E, K, N, Kd, group, dtype, swiglu=False, zeros=False, align=1, mask=0.0,
           gather=True, sdtype=None, seed=0, idx=None, big=False):
    g = torch.Generator().manual_seed(seed + T + N)
    if big:       # enough outputs for the form with prepared x
        per = (min(E, T * K) + T * K // 8) * (2 if swiglu else 1) * Kd // 2
        N += (26 << 20) // per + 1
        rows = moedc.moedc_sort_rows(T, K, E, align)
        assert moedc.moedc_matvec_int4_workspace_bytes(T, Kd, E, N, int(swiglu), rows) > 0
    if idx is None:
        idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
        idx[torch.rand(T, K, generator=g) < mask] = -1
    x = torch.randn(T, Kd, generator=g).to(dtype).cuda()
    n = 2 * N if swiglu else N
    wq, s, z = _weights(g, E, n, Kd, group, zeros, sdtype or dtype)
    m = moedc.sort(x, idx.cuda(), E, align=align)
    R = m.src.shape[0]
    out = torch.full((R, N), 7.0, dtype=dtype).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    xin, src = (x, m.src) if gather else (m.rows, None)
    got = moedc.matvec_int4(xin, wq, s, zeros=z, offsets=m.offsets, counts=m.counts, src=src,
                            top_k=K, swiglu=swiglu, status=status, out=out)
    assert got is out and int(status) == 0
    _, src_ref, offsets, counts = sort_ref(idx, E, align, R)
    for e in range(E):
        rows = slice(int(offsets[e]), int(offsets[e]) + int(counts[e]))
        if counts[e] == 0:
            continue
        w = int4_weights(wq[e], s[e], None if z is None else z[e], group)
        ref, err = matvec_ref(x[(src_ref[rows] // K).long().cuda()], w, swiglu)
        assert_within(out[rows], ref, err + rounding(ref, dtype))
    assert (out[m.src < 0] == 7.0).all()           # rows of no expert stay as they were


# both forms of the product: one launch for few weights, prepared x for many
FORMS = pytest.mark.parametrize("big", [False, True], ids=["few", "many"])


@FORMS
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,K,N,mult", [
    (1, 1, 1, 1, 1), (1, 4, 2, 16, 3), (3, 8, 2, 17, 5), (16, 12, 4, 130, 4), (40, 6, 2, 33, 7),
    (9, 2, 1, 64, 16), (70, 3, 2, 48, 2), (150, 2, 2, 20, 3)])
def test_products(T, E, K, N, mult, group, dtype, big):
    _check(T, E, K, N, group * mult, group, DTYPES[dtype], big=big)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@FORMS
def test_swiglu_and_zero_points(group, zeros, dtype, big):
    _check(13, 6, 3, 37, group * 5, group, DTYPES[dtype], swiglu=True, zeros=zeros, big=big)
    _check(50, 3, 2, 24, group * 9, group, DTYPES[dtype], swiglu=False, zeros=zeros, seed=1,
           big=big)


# enough 128-row tiles of weights to give every SM one: experts of few and of many rows,
# odd output counts, channels that end inside a stage of 256
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,K,N,mult,swiglu,zeros", [
    (40, 160, 2, 40, 2, False, False), (64, 160, 4, 33, 3, True, True),
    (30, 20, 8, 1100, 5, False, True), (70, 12, 8, 900, 1, True, False),
    (100, 20, 12, 1030, 4, False, False), (260, 16, 4, 1300, 2, False, True)])
def test_many_tiles(T, E, K, N, mult, swiglu, zeros, group, dtype):
    _check(T, E, K, N, group * mult, group, DTYPES[dtype], swiglu=swiglu, zeros=zeros, align=4,
           mask=0.05)


@pytest.mark.parametrize("sdtype", list(DTYPES))
@pytest.mark.parametrize("group,mult", [(32, 11), (64, 7), (128, 5)])
def test_many_tiles_scale_types(group, mult, sdtype):
    _check(50, 160, 4, 60, group * mult, group, torch.bfloat16, zeros=True, sdtype=DTYPES[sdtype])


def test_many_tiles_at_one_expert():
    idx = torch.full((75, 1), 3, dtype=torch.int32)
    _check(75, 160, 1, 70, 512, 64, torch.float16, idx=idx)
    _check(21, 1, 1, 20000, 512, 128, torch.bfloat16, seed=2)


@pytest.mark.parametrize("Kd", [128, 512, 640, 1280])
def test_nothing_of_an_earlier_call_comes_through(Kd):
    """Channels that end inside the last stage, after a call that left NaN
    everywhere in the SMs' shared memory."""
    g = torch.Generator().manual_seed(6)
    wq, s, _ = _weights(g, 8, 4096, 2048, 64, False, torch.bfloat16)
    bad = torch.full((64, 2048), float("nan"), dtype=torch.bfloat16).cuda()
    idx = torch.arange(64, dtype=torch.int32).reshape(64, 1) % 8
    m = moedc.sort(None, idx.cuda(), 8)
    out = moedc.matvec_int4(bad, wq, s, offsets=m.offsets, counts=m.counts, src=m.src)
    assert torch.isnan(out).all()
    _check(5, 4, 2, 40, Kd, 64, torch.bfloat16, zeros=True, big=True)
    _check(5, 4, 2, 40, Kd, 64, torch.bfloat16, zeros=True)


@pytest.mark.parametrize("sdtype", list(DTYPES))
@FORMS
def test_scale_types(sdtype, big):
    _check(5, 4, 2, 40, 512, 64, torch.bfloat16, zeros=True, sdtype=DTYPES[sdtype], big=big)


@pytest.mark.parametrize("gather", [False, True])
@FORMS
def test_aligned_groups_masked_entries_and_gather(gather, big):
    _check(30, 9, 4, 50, 384, 128, torch.bfloat16, align=16, mask=0.4, gather=gather, big=big)
    _check(8, 9, 4, 50, 384, 128, torch.bfloat16, align=4, mask=1.1, gather=gather, big=big)


@FORMS
def test_long_rows_of_real_sizes(big):
    _check(4, 2, 2, 96, 7168, 128, torch.bfloat16, big=big)
    _check(33, 2, 1, 64, 14336, 128, torch.bfloat16, seed=3, big=big)
    _check(12, 3, 2, 64, 6144, 64, torch.bfloat16, swiglu=True, zeros=True, seed=4, big=big)


@FORMS
def test_every_row_at_one_expert(big):
    idx = torch.full((97, 1), 2, dtype=torch.int32)
    _check(97, 4, 1, 40, 256, 64, torch.float16, idx=idx, big=big)


def test_one_linear_layer_without_maps():
    g = torch.Generator().manual_seed(1)
    for rows in (1, 2, 8, 9, 31):
        x = torch.randn(rows, 256, generator=g).to(torch.bfloat16).cuda()
        wq, s, z = _weights(g, 1, 70, 256, 32, True, torch.float32)
        out = moedc.matvec_int4(x, wq[0], s[0], zeros=z[0])
        ref, err = matvec_ref(x, int4_weights(wq[0], s[0], z[0], 32), False)
        assert_within(out, ref, err + rounding(ref, torch.bfloat16))
    assert moedc.matvec_int4(x[:0], wq[0], s[0]).shape == (0, 70)


def test_strided_rows_other_stream_and_equal_bits():
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(6, 640, generator=g).to(torch.float16).cuda()
    wq, s, _ = _weights(g, 1, 48, 512, 128, False, torch.float16)
    want = moedc.matvec_int4(wide[:, 64:576].contiguous(), wq[0], s[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moedc.matvec_int4(wide[:, 64:576], wq[0], s[0])
    side.synchronize()
    assert torch.equal(got, want)


@FORMS
def test_infinite_inputs_stay_in_their_row(big):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 256, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, 1, 220000 if big else 40, 256, 64, False, torch.bfloat16)
    want = moedc.matvec_int4(x, wq[0], s[0])
    x[2, 100] = float("nan")
    x[3, 7] = float("inf")
    got = moedc.matvec_int4(x, wq[0], s[0])
    for r in (0, 1, 4):
        assert torch.equal(got[r], want[r])
    assert torch.isnan(got[2]).all()
    assert not torch.isfinite(got[3].float()).any()


@FORMS
def test_rows_past_the_end_and_bad_sources_are_reported(big):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(4, 128, generator=g).to(torch.bfloat16).cuda()
    n = 220000 if big else 20
    wq, s, _ = _weights(g, 2, n, 128, 64, False, torch.bfloat16)
    offsets = torch.tensor([0, 3, 6], dtype=torch.int32).cuda()
    counts = torch.tensor([3, 3], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = torch.zeros(4, n, dtype=torch.bfloat16).cuda()
    moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, status=status, out=out)
    assert int(status) == moedc.ERR_CAPACITY
    ref, err = matvec_ref(x[3:], int4_weights(wq[1], s[1], None, 64), False)
    assert_within(out[3:], ref, err + rounding(ref, torch.bfloat16))
    src = torch.tensor([0, 9, -1, 2], dtype=torch.int32).cuda()      # 9 and -1: no such token
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    counts = torch.tensor([2, 2], dtype=torch.int32).cuda()
    status.zero_()
    moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, src=src, status=status, out=out)
    assert int(status) == moedc.ERR_EXPERT_RANGE
    assert (out[1:3] == 0).all()


def test_refusals():
    x = torch.zeros(2, 256, dtype=torch.bfloat16).cuda()
    wq = torch.zeros(1, 16, 128, dtype=torch.uint8).cuda()
    s = torch.zeros(1, 16, 4, dtype=torch.bfloat16).cuda()
    moedc.matvec_int4(x, wq, s)
    i32 = torch.zeros(2, dtype=torch.int32).cuda()
    for bad in (lambda: moedc.matvec_int4(x.float(), wq, s),                      # f32 rows
                lambda: moedc.matvec_int4(x, wq, s[:, :, :1].contiguous()),       # groups of 256
                lambda: moedc.matvec_int4(x, wq, s, offsets=i32),                 # no counts
                lambda: moedc.matvec_int4(x, wq, s, src=i32, top_k=0),
                lambda: moedc.matvec_int4(x, wq.expand(2, 16, 128).contiguous(),
                                          s.expand(2, 16, 4).contiguous()),       # E = 2, no maps
                lambda: moedc.matvec_int4(torch.zeros(2, 260, dtype=torch.bfloat16).cuda()[:, 1:257],
                                          wq, s)):                                # rows not 16-byte aligned
        with pytest.raises(moedc.MoedcError):
            bad()
    for bad in (lambda: moedc.matvec_int4(x[:, :128], wq, s),
                lambda: moedc.matvec_int4(x, wq.int(), s),
                lambda: moedc.matvec_int4(x, wq, s[:, :8].contiguous()),
                lambda: moedc.matvec_int4(x, wq, s, zeros=torch.zeros(1, 16, 2, dtype=torch.uint8).cuda()),
                lambda: moedc.matvec_int4(x, wq[:, :15].contiguous(), s[:, :15].contiguous(), swiglu=True),
                lambda: moedc.matvec_int4(x, wq, s, out=torch.zeros(2, 15, dtype=torch.bfloat16).cuda())):
        with pytest.raises(ValueError):
            bad()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 512, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, 1, 110000, 512, 64, False, torch.bfloat16)
    want = moedc.matvec_int4(x, wq, s)
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    moedc.load().moedc_test_set_wait_extra(1)
    try:
        moedc.matvec_int4(x, wq, s, status=status)
        assert int(status) == moedc.ERR_TIMEOUT
    finally:
        moedc.load().moedc_test_set_wait_extra(0)
    status.zero_()
    assert torch.equal(moedc.matvec_int4(x, wq, s, status=status), want) and int(status) == 0
