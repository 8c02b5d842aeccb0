"""Tensors that a kernel would write through are refused when they are not the
CUDA tensors of the type and shape that it takes."""
import dataclasses

import pytest
import torch

from combine_moedc_layout_gb300 import moedc

pytestmark = pytest.mark.gpu


def test_sort_refuses_status_and_buffers_of_other_kinds():
    idx = torch.zeros(6, 2, dtype=torch.int32).cuda()
    x = torch.zeros(6, 32, dtype=torch.bfloat16).cuda()
    for status in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64).cuda()):
        with pytest.raises(ValueError, match="status"):
            moedc.sort(x, idx, 8, status=status)
    m = moedc.sort(x, idx, 8)
    for name in ("row", "src", "offsets", "counts", "workspace", "status"):
        good = getattr(m, name)
        for bad in (good.cpu(), good.to(torch.int16)):
            with pytest.raises(ValueError, match=name):
                moedc.sort(x, idx, 8, out=dataclasses.replace(m, **{name: bad}))
    with pytest.raises(ValueError, match="offsets"):
        moedc.sort(x, idx, 8, out=dataclasses.replace(m, offsets=m.offsets[:8]))
    assert moedc.sort(x, idx, 8, out=m) is m


def test_matvec_refuses_status_and_workspace_of_other_kinds():
    x = torch.zeros(2, 256, dtype=torch.bfloat16).cuda()
    wq = torch.zeros(1, 16, 128, dtype=torch.uint8).cuda()
    s = torch.zeros(1, 16, 4, dtype=torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    for bad in (status.cpu(), status.long()):
        with pytest.raises(ValueError, match="status"):
            moedc.matvec_int4(x, wq, s, status=bad)
    for bad in (torch.empty(4096, dtype=torch.uint8), torch.empty(4096, dtype=torch.int32).cuda()):
        with pytest.raises(ValueError, match="workspace"):
            moedc.matvec_int4(x, wq, s, status=status, workspace=bad)
    moedc.matvec_int4(x, wq, s, status=status, workspace=torch.empty(4096, dtype=torch.uint8).cuda())
