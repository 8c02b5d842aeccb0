"""e4m3 products of rows that are gathered through src: the copy into packed order that a
workspace allows changes no bit of the outputs."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import assert_within
from matmul_util import codes_bound, groups, product
from test_gpu_matmul_e4m3 import E4M3, OUT, check, rows_of, weights, wide_w, wide_x

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32).cuda()


def _bits(out):
    return [t.view(torch.uint8) for t in (out if isinstance(out, tuple) else (out,))]


def _both(*args, **kw):
    """The call as it is, and with a workspace too small for the copy."""
    return (moedc.matmul_e4m3(*args, **kw),
            moedc.matmul_e4m3(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw))


# few tiles, whose channels clusters of blocks can share: more rows than the form for few of
# them takes, as many as it takes with few tiles, several experts
@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,Kd", [([100], 256, 4096), ([49], 128, 7168), ([130], 384, 1024), ([60, 2, 40], 256, 2048),
                                         ([40], 256, 4096), ([30, 3], 128, 4096)])
def test_equal_bits_with_and_without_a_workspace(counts, N, Kd, swiglu, out):
    g = torch.Generator().manual_seed(sum(counts) + N)
    w, ws = weights(g, len(counts), N, Kd, swiglu)
    x, xs = rows_of(g, 70, Kd)
    offsets, cnt, rows = groups(counts)
    src = torch.randint(0, 140, (rows,), generator=g).to(torch.int32).cuda()
    assert moedc.moedc_matmul_e4m3_workspace_bytes(Kd, len(counts), rows) > 16 or len(counts) > 1
    status = _status()
    a, b = _both(x, xs, w, ws, offsets=offsets, counts=cnt, src=src, top_k=2, swiglu=swiglu, out_dtype=OUT[out],
                 status=status)
    assert int(status) == 0
    assert all(torch.equal(p, q) for p, q in zip(_bits(a), _bits(b)))
    token = src.long() // 2
    for e, c in enumerate(counts):
        o = int(offsets[e])
        t = token[o:o + c]
        v, err = product(wide_x(x.view(torch.uint8)[t].view(E4M3), xs[t]), wide_w(w[e], ws[e], swiglu), swiglu)
        check((a[0][o:o + c], a[1][o:o + c]) if out == "e4m3" else a[o:o + c], v, err, out)
