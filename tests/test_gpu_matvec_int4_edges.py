"""4-bit products at the edges of their arguments."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from test_gpu_matvec_int4 import _weights

pytestmark = pytest.mark.gpu


# few weights; prepared x; the form for many rows an expert (by its rows)
@pytest.mark.parametrize("E,N,Kd,rows", [(8, 40, 256, 64), (8, 30000, 512, 64), (2, 30000, 512, 200)])
@pytest.mark.parametrize("gather", [False, True])
def test_no_tokens_on_buffers_of_fixed_size(E, N, Kd, rows, gather):
    g = torch.Generator().manual_seed(rows)
    wq, s, _ = _weights(g, E, N, Kd, 64, False, torch.bfloat16)
    x = torch.randn(4, Kd, generator=g).to(torch.bfloat16).cuda()[:0]
    idx = torch.empty(0, 2, dtype=torch.int32).cuda()
    m = moedc.sort(None if gather else x, idx, E, rows=rows)
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16).cuda()
    moedc.matvec_int4(x if gather else m.rows, wq, s, offsets=m.offsets, counts=m.counts,
                      src=m.src if gather else None, top_k=2, status=m.status, out=out)
    assert int(m.status) == 0
    assert (out == 7.0).all()
    assert moedc.unsort(out, m.row, torch.empty(0, 2).cuda()).shape == (0, N)


@pytest.mark.parametrize("n", [20, 220000])          # few weights; prepared x
def test_without_a_status_errors_are_raised(n):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(4, 128, generator=g).to(torch.bfloat16).cuda()
    wq, s, _ = _weights(g, 2, n, 128, 64, False, torch.bfloat16)
    counts = torch.tensor([2, 2], dtype=torch.int32).cuda()
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    want = moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts)
    src = torch.tensor([0, 9, 1, 2], dtype=torch.int32).cuda()
    with pytest.raises(moedc.MoedcError) as e:
        moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, src=src)
    assert e.value.code == moedc.ERR_EXPERT_RANGE
    with pytest.raises(moedc.MoedcError) as e:
        moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts + 1)
    assert e.value.code == moedc.ERR_CAPACITY
    # a status takes them instead, and nothing waits: such a call can be captured
    status = torch.zeros(1, dtype=torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts, status=status)
        with pytest.raises(ValueError, match="status"):
            moedc.matvec_int4(x, wq, s, offsets=offsets, counts=counts)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and int(status) == 0
