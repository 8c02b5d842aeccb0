"""4-bit products at the edges of their arguments."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import assert_within, int4_weights, matvec_ref, rounding
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


# few weights read, prepared x, and many rows an expert, out of the same 2.3e9 bytes
@pytest.mark.parametrize("T", [1, 40, 960])
def test_weights_past_32_bit_offsets(T):
    E, N, Kd, group = 320, 2048, 7168, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    wq = torch.randint(0, 256, (E, N, Kd // 2), dtype=torch.uint8, generator=g, device="cuda")
    assert wq.numel() > 2 ** 31
    s = ((0.5 + torch.rand(E, N, Kd // group, generator=g, device="cuda")) * 0.2 / Kd ** 0.5).to(torch.bfloat16)
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, generator=g, device="cuda")
    x = torch.randn(T, Kd, generator=g, device="cuda").to(torch.bfloat16)
    K = 2 if T == 1 else 8
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    idx[0, 0], idx[0, 1] = E - 1, E - 2
    m = moedc.sort(None, idx, E)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = moedc.matvec_int4(x, wq, s, zeros=z, offsets=m.offsets, counts=m.counts, src=m.src,
                            top_k=K, status=status)
    assert int(status) == 0
    for e in (E - 1, E - 2, E - 3, 0):
        a, n = int(m.offsets[e]), int(m.counts[e])
        if n:
            ref, err = matvec_ref(x[(m.src[a:a + n] // K).long()],
                                  int4_weights(wq[e], s[e], z[e], group), False)
            assert_within(out[a:a + n], ref.cuda(), err + rounding(ref, torch.bfloat16))


def test_outputs_past_32_bit_offsets():
    """300032 rows of 7424 outputs, 2.2e9 elements, by the form for many rows."""
    rows, N, Kd = 300032, 7424, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    wq = torch.randint(0, 256, (1, N, Kd // 2), dtype=torch.uint8, generator=g, device="cuda")
    s = ((0.5 + torch.rand(1, N, 1, generator=g, device="cuda")) * 0.02).to(torch.bfloat16)
    x = torch.randn(rows, Kd, generator=g, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = moedc.matvec_int4(x, wq, s, status=status)
    assert int(status) == 0 and out.numel() > 2 ** 31
    for a in (0, 150000, rows - 128):
        ref, err = matvec_ref(x[a:a + 128], int4_weights(wq[0], s[0], None, 128), False)
        assert_within(out[a:a + 128], ref.cuda(), err + rounding(ref, torch.bfloat16))
