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


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", ["packed", "slots"])
def test_lost_rows_are_zeros_beside_weights_of_nan(form, swiglu, out):
    """Rows that src leads outside have outputs of 0 whatever the weights hold, in the copied form and
    in the other one."""
    g = torch.Generator().manual_seed(5)
    E, cap, N, Kd = 2, 60, 256, 512
    w, ws = weights(g, E, N, Kd, swiglu)
    w.view(torch.uint8)[:, 3, 7] = 0x7f
    ws[:, 1, 2] = float("inf")
    x, xs = rows_of(g, 50, Kd)
    counts = [60, 47]
    src = torch.randint(0, 50, (E * cap,), generator=g).to(torch.int32)
    lost = [0, 17, 59, 60, 101, 106]
    src[lost] = torch.tensor([50, -1, 2 ** 31 - 1, 51, -(2 ** 31), 1000], dtype=torch.int32)
    maps = dict(counts=torch.tensor(counts, dtype=torch.int32).cuda(), src=src.cuda())
    if form == "packed":
        maps["offsets"] = torch.tensor([0, cap, cap + 47], dtype=torch.int32).cuda()
    else:
        maps["src"] = maps["src"].view(E, cap)
    assert moedc.moedc_matmul_e4m3_workspace_bytes(Kd, E, E * cap) > 0
    status = _status()
    a, b = _both(x, xs, w, ws, swiglu=swiglu, out_dtype=OUT[out], status=status, **maps)
    assert int(status) == moedc.ERR_EXPERT_RANGE
    mine = torch.zeros(E * cap, dtype=torch.bool)
    mine[:60], mine[60:107] = True, True
    for got in (a, b):
        parts = [t.reshape(E * cap, -1) for t in (got if out == "e4m3" else (got,))]
        assert (parts[0][lost].float() == 0).all()
        if out == "e4m3":
            assert (parts[1][lost] == torch.tensor(1e-4) / torch.tensor(448.0)).all()
    for p, q in zip(*[[t.reshape(E * cap, -1)[mine] for t in _bits(v)] for v in (a, b)]):
        assert torch.equal(p, q)
    first = a[0] if out == "e4m3" else a
    assert torch.isnan(first.reshape(E * cap, -1)[1, 3].float())      # the others have the weights' NaN


def test_scales_of_minus_zero_are_zeros():
    """No scale of the caller's is taken for a lost row's."""
    g = torch.Generator().manual_seed(6)
    w, ws = weights(g, 1, 256, 512, False)
    x, xs = rows_of(g, 20, 512)
    src = torch.arange(100, dtype=torch.int32).cuda() % 20
    for cols in (slice(3, 4), slice(0, 4)):
        s = xs.clone()
        s[::3, cols] = 0.0
        want = moedc.matmul_e4m3(x, s, w, ws, src=src)
        s[::3, cols] = -0.0
        assert all(torch.equal(y, want) for y in _both(x, s, w, ws, src=src))
        assert want[1].any() and want[0].any() == (cols.start == 3)


# copied for the form for many rows, and for clusters of the other one
@pytest.mark.parametrize("cap,Kd", [(60, 512), (40, 4096), (24, 1024)])
@pytest.mark.parametrize("layout", [0, moedc.SCALES_PER_TOKEN])
def test_lost_rows_in_every_form_and_scale_layout(cap, Kd, layout):
    g = torch.Generator().manual_seed(cap)
    E, N = 2, 256
    w, ws = weights(g, E, N, Kd, False)
    w.view(torch.uint8)[:, 3, 7] = 0x7f
    x, xs = rows_of(g, 31, Kd)
    if layout:
        xs = xs[:, 0].contiguous()
    src = torch.randint(0, 31, (E, cap), generator=g).to(torch.int32)
    src[0, 1], src[1, cap - 1] = 31, -7
    status = _status()
    maps = dict(counts=torch.full((E,), cap, dtype=torch.int32).cuda(), src=src.cuda(), scale_layout=layout, status=status)
    a, b = _both(x, xs, w, ws, **maps)
    assert int(status) == moedc.ERR_EXPERT_RANGE
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    lost = torch.zeros(E, cap, dtype=torch.bool)
    lost[0, 1] = lost[1, cap - 1] = True
    assert (a[lost] == 0).all() and torch.isnan(a[~lost][:, 3]).all() and not torch.isnan(a[~lost][:, 4:]).any()
    t = src.long().clamp(0, 30).cuda()
    for e in range(E):
        s = xs[t[e]][:, None].expand(cap, Kd // 128) if layout else xs[t[e]]
        keep = ~lost[e]
        v, err = product(wide_x(x.view(torch.uint8)[t[e]].view(E4M3), s)[keep], wide_w(w[e], ws[e], False)[4:], False)
        check(a[e][keep][:, 4:], v, err, "bf16")
