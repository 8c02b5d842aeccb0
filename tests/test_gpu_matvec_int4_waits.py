"""A bounded wait that runs out ends the 4-bit products with a status, in whatever
unit the copies stand when it does."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from test_gpu_matvec_int4 import _weights

pytestmark = pytest.mark.gpu


# one part of K and several; units of 8 and 32 rows; more units than blocks; rows that are
# gathered (a lane's copies are under conditions of its own)
@pytest.mark.parametrize("rows,E,N,Kd,group,swiglu", [
    (3, 1, 120000, 512, 64, False), (5, 16, 9000, 640, 32, True), (70, 2, 9000, 1280, 32, False),
    (9, 3, 1000, 14336, 128, False)])
def test_every_wait_that_runs_out_ends_the_call(rows, E, N, Kd, group, swiglu):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, Kd, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, E, 2 * N if swiglu else N, Kd, group, False, torch.bfloat16)
    idx = (torch.arange(rows, dtype=torch.int32) % E).reshape(rows, 1).cuda()
    m = moedc.sort(None, idx, E)
    status = torch.zeros(1, dtype=torch.int32).cuda()

    def run():
        status.zero_()
        y = moedc.matvec_int4(x, wq, s, offsets=m.offsets, counts=m.counts, src=m.src,
                              swiglu=swiglu, status=status)
        return y, int(status)

    assert moedc.moedc_matvec_int4_workspace_bytes(rows, Kd, E, N, int(swiglu), rows) > 0
    want, code = run()
    assert code == moedc.OK
    moedc.load().moedc_test_set_wait_extra(1)
    try:
        assert [run()[1] for _ in range(3)] == [moedc.ERR_TIMEOUT] * 3
    finally:
        moedc.load().moedc_test_set_wait_extra(0)
    got, code = run()
    assert code == moedc.OK and torch.equal(got, want)
