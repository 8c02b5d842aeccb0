"""4-bit products of experts with many rows each, where tensor memory holds the
weights, against 64-bit forms."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, assert_within, int4_weights, matvec_ref, rounding
from test_gpu_matvec_int4 import _check, _weights

pytestmark = pytest.mark.gpu


# experts of one, two and three chunks of 64 rows, chunks of a few rows at the end, odd
# output counts, channels that end inside a stage of 256, one stage and many
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("T,E,K,N,mult,swiglu,zeros", [
    (70, 3, 2, 48, 2, False, False), (97, 2, 1, 130, 3, True, True), (66, 1, 1, 1, 1, False, True),
    (200, 5, 2, 65, 5, True, False), (130, 2, 2, 700, 4, False, True), (33, 1, 1, 257, 17, True, True)])
def test_many_rows(T, E, K, N, mult, swiglu, zeros, group, dtype):
    _check(T, E, K, N, group * mult, group, DTYPES[dtype], swiglu=swiglu, zeros=zeros, mask=0.05,
           big=True)


@pytest.mark.parametrize("gather", [False, True])
def test_aligned_groups_and_gather(gather):
    _check(100, 4, 2, 50, 384, 128, torch.bfloat16, align=16, mask=0.1, gather=gather, big=True)
    _check(100, 4, 2, 50, 384, 64, torch.float16, align=64, gather=gather, swiglu=True, big=True)


@pytest.mark.parametrize("sdtype", list(DTYPES))
@pytest.mark.parametrize("group,mult", [(64, 7), (128, 5), (64, 8), (128, 4)])
def test_scale_types(group, mult, sdtype):
    _check(80, 2, 1, 60, group * mult, group, torch.bfloat16, zeros=True, sdtype=DTYPES[sdtype],
           big=True)


def test_uneven_experts():
    idx = torch.full((150, 1), 3, dtype=torch.int32)
    idx[:2] = 1
    _check(150, 4, 1, 70, 512, 64, torch.float16, idx=idx, big=True)
    idx[:] = 0
    _check(150, 4, 1, 70, 512, 128, torch.bfloat16, idx=idx, big=True)
    idx[:] = -1
    _check(150, 4, 1, 70, 512, 128, torch.bfloat16, idx=idx, big=True)


def test_more_units_than_blocks_and_equal_bits():
    _check(300, 8, 2, 9000, 512, 128, torch.bfloat16, swiglu=True, zeros=True)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(90, 2048, generator=g).to(torch.bfloat16).cuda()
    wq, s, z = _weights(g, 1, 30000, 2048, 64, True, torch.bfloat16)
    want = moedc.matvec_int4(x, wq, s, zeros=z)
    for _ in range(4):
        assert torch.equal(moedc.matvec_int4(x, wq, s, zeros=z), want)


def test_infinite_inputs_stay_in_their_row():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(70, 256, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, 1, 220000, 256, 64, False, torch.bfloat16)
    want = moedc.matvec_int4(x, wq, s)
    x[2, 100] = float("nan")
    x[66, 7] = float("inf")
    got = moedc.matvec_int4(x, wq, s)
    keep = [r for r in range(70) if r not in (2, 66)]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[2]).all()
    assert not torch.isfinite(got[66].float()).any()


def test_rows_past_the_end_and_bad_sources_are_reported():
    g = torch.Generator().manual_seed(4)
    n = 220000
    x = torch.randn(60, 128, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, 2, n, 128, 64, False, torch.bfloat16)
    offsets = torch.tensor([0, 40, 80], dtype=torch.int32).cuda()
    counts = torch.tensor([40, 40], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = torch.zeros(60, n, dtype=torch.bfloat16).cuda()
    moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, status=status, out=out)
    assert int(status) == moedc.ERR_CAPACITY
    ref, err = matvec_ref(x[40:], int4_weights(wq[1], s[1], None, 64), False)
    assert_within(out[40:], ref, err + rounding(ref, torch.bfloat16))
    src = torch.arange(60, dtype=torch.int32)
    src[33], src[59] = 60, -1                                   # no such tokens
    counts = torch.tensor([40, 20], dtype=torch.int32).cuda()
    status.zero_()
    moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, src=src.cuda(), status=status, out=out)
    assert int(status) == moedc.ERR_EXPERT_RANGE
    assert (out[33] == 0).all() and (out[59] == 0).all()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 512, generator=g).to(torch.bfloat16).cuda()
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
