"""Products of packed expert rows in e4m3 with block scales, against 64-bit forms: packed,
gathered and receive-buffer rows, every output type, the edges of tiles and groups."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, assert_within, rounding
from matmul_util import codes_bound, groups, owned, product, randn

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
OUT = {"bf16": moedc.BF16, "f16": moedc.F16, "e4m3": moedc.FP8_E4M3}


def _status():
    return torch.zeros(1, dtype=torch.int32).cuda()


def weights(g, E, N, Kd, swiglu):
    parts = 2 if swiglu else 1
    w = randn(g, E4M3, E, parts * N, Kd)
    ws = (torch.rand(E, parts * -(-N // 128), Kd // 128, generator=g) + 0.5).cuda() * Kd ** -0.5
    return w, ws


def rows_of(g, R, Kd):
    return randn(g, E4M3, R, Kd), (torch.rand(R, Kd // 128, generator=g) + 0.25).cuda()


def wide_x(x, xs):
    return x.double() * xs.double().repeat_interleave(128, -1)


def wide_w(w, ws, swiglu):
    """f64 weights [.., n, Kd] of one expert."""
    parts = 2 if swiglu else 1
    N = w.shape[0] // parts
    s = ws.double().reshape(parts, -1, ws.shape[-1]).repeat_interleave(128, 1)[:, :N]
    return w.double() * s.reshape(parts * N, -1).repeat_interleave(128, 1)


def check(got, v, err, out):
    if out != "e4m3":
        assert_within(got, v, err + rounding(v.abs() + err, DTYPES[out]))
        return
    codes, scales = got
    bound, scale, off = codes_bound(v, err)
    assert_within(scales, scale, off)
    assert_within(codes.double() * scales.double().repeat_interleave(128, 1), v, bound)


# rows around the tile's 256 and 128, none, one; columns that end inside a tile and a block
CASES = [
    ([1], 128, 128, 1),
    ([3], 200, 384, 1),
    ([0, 1, 127, 128, 129, 0, 2], 256, 256, 1),
    ([255, 256, 257, 0], 384, 640, 8),
    ([513, 31], 130, 1152, 16),
    ([4] * 40, 520, 512, 1),
    ([7, 0, 12], 77, 256, 4),
]


@pytest.mark.parametrize("out", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("counts,N,Kd,align", CASES)
def test_packed_rows(counts, N, Kd, align, swiglu, out, many):
    """`many`: rows of nobody behind the groups, so that the call expects many rows to an expert;
    else experts without rows behind them, so that it expects few, and takes its other form."""
    if not many:
        counts = counts + [0] * (sum(counts) // 12)
    if out == "e4m3":
        N = -(-N // 128) * 128
    g = torch.Generator().manual_seed(len(counts) + N)
    offsets, cnt, rows = groups(counts, align, tail=300 * len(counts) if many else 5)
    w, ws = weights(g, len(counts), N, Kd, swiglu)
    x, xs = rows_of(g, rows, Kd)
    mine = owned(offsets, cnt, rows)
    x.view(torch.uint8)[~mine] = 0x7f                     # NaN in rows of nobody
    xs[~mine] = float("inf")
    status = _status()
    y = torch.full((rows, N), 7.0, device="cuda").to(E4M3 if out == "e4m3" else DTYPES[out])
    buf = (y, torch.full((rows, N // 128), 7.0, device="cuda")) if out == "e4m3" else y
    got = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=swiglu,
                            out_dtype=OUT[out], status=status, out=buf)
    assert got is buf and int(status) == 0
    assert (y[~mine].float() == 7.0).all()
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if not c:
            continue
        v, err = product(wide_x(x[a:a + c], xs[a:a + c]), wide_w(w[e], ws[e], swiglu), swiglu)
        check((buf[0][a:a + c], buf[1][a:a + c]) if out == "e4m3" else buf[a:a + c], v, err, out)
    fresh = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=swiglu,
                              out_dtype=OUT[out], status=status)
    for p, q in zip(fresh if out == "e4m3" else [fresh], buf if out == "e4m3" else [buf]):
        assert torch.equal(p[mine].float(), q[mine].float())


@pytest.mark.parametrize("T,E,K", [(1, 2, 1), (1, 8, 2), (9, 12, 3), (130, 4, 2), (600, 3, 1)])
def test_gathered_rows(T, E, K):
    g = torch.Generator().manual_seed(T)
    N, Kd = 256, 384
    w, ws = weights(g, E, N, Kd, True)
    x, xs = rows_of(g, T, Kd)
    idx = torch.rand(T, E, generator=g).topk(K, dim=1).indices.to(torch.int32).cuda()
    m = moedc.sort(None, idx, E, align=4)
    y = moedc.matmul_e4m3(x, xs, w, ws, offsets=m.offsets, counts=m.counts, src=m.src, top_k=K,
                          swiglu=True, status=m.status)
    token = (m.src.long() // K).clamp(min=0)
    flat = moedc.matmul_e4m3(x.view(torch.uint8)[token].view(E4M3), xs[token], w, ws, offsets=m.offsets,
                             counts=m.counts, swiglu=True, status=m.status)
    mine = m.src >= 0
    # gathered as the products need them, where the call would copy the rows first
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    z = moedc.matmul_e4m3(x, xs, w, ws, offsets=m.offsets, counts=m.counts, src=m.src, top_k=K,
                          swiglu=True, status=m.status, workspace=small)
    assert torch.equal(y[mine], z[mine])
    assert torch.equal(y[mine], flat[mine]) and int(m.status) == 0
    for e in range(E):
        a, c = int(m.offsets[e]), int(m.counts[e])
        if c:
            t = token[a:a + c]
            v, err = product(wide_x(x.view(torch.uint8)[t].view(E4M3), xs[t]), wide_w(w[e], ws[e], True), True)
            check(y[a:a + c], v, err, "bf16")


@pytest.mark.parametrize("layout", [0, moedc.SCALES_COL_MAJOR, moedc.SCALES_PER_TOKEN])
def test_behind_dispatch(layout):
    """dispatch's receive buffer, in its three scale layouts, through an expert layer to combine."""
    g = torch.Generator().manual_seed(3)
    T, H, E, K, N, cap = 70, 512, 6, 3, 256, 70
    x = randn(g, torch.bfloat16, T, H)
    idx = torch.rand(T, E, generator=g).topk(K, dim=1).indices.to(torch.int32)
    idx[5] = -1
    idx = idx.cuda()
    lay = moedc.layout(idx, E, 2, cap)
    recv, scales, src_idx = moedc.dispatch(x, idx, lay, E, cap, moedc.FP8_E4M3 | layout)
    w, ws = weights(g, E, N, H, False)
    y = moedc.matmul_e4m3(recv, scales, w, ws, counts=lay.num_tokens_per_expert, scale_layout=layout, status=lay.status)
    assert y.shape == (E, cap, N) and int(lay.status) == 0
    G = H // 128
    for e in range(E):
        c = int(lay.num_tokens_per_expert[e])
        s = scales[e].T[:c] if layout == moedc.SCALES_COL_MAJOR else scales[e][:c]
        if layout == moedc.SCALES_PER_TOKEN:
            s = s[:, None].expand(c, G)
        v, err = product(wide_x(recv[e][:c], s), wide_w(w[e], ws[e], False), False)
        check(y[e][:c], v, err, "bf16")
    moedc.combine(y, idx, lay.slot, torch.ones(T, K, device="cuda"))
    # the same rows from quantised tokens, through src_idx
    if layout == 0:
        q, qs = moedc.quant_e4m3(x)
        z = moedc.matmul_e4m3(q, qs, w, ws, counts=lay.num_tokens_per_expert, src=src_idx, status=lay.status)
        live = src_idx >= 0
        assert torch.equal(z[live], y[live]) and int(lay.status) == 0


def test_two_layers_in_8_bits_and_back():
    """router's choice -> gate/up to e4m3 rows -> down -> weighted way back, against 64 bits of
    the same e4m3 rows."""
    g = torch.Generator().manual_seed(4)
    T, H, I, E, K = 33, 512, 256, 10, 2
    logits = torch.randn(T, E, generator=g).cuda()
    x = randn(g, torch.bfloat16, T, H)
    up, us = weights(g, E, I, H, True)
    down, ds = weights(g, E, H, I, False)
    idx, wt = moedc.gate(logits, K)
    m = moedc.sort(None, idx, E)
    maps = dict(offsets=m.offsets, counts=m.counts, status=m.status)
    q, qs = moedc.quant_e4m3(x)
    h, hs = moedc.matmul_e4m3(q, qs, up, us, src=m.src, top_k=K, swiglu=True, out_dtype=moedc.FP8_E4M3, **maps)
    o = moedc.matmul_e4m3(h, hs, down, ds, **maps)
    y = moedc.unsort(o, m.row, wt)
    assert int(m.status) == 0 and torch.isfinite(y).all()
    for e in range(E):
        a, c = int(m.offsets[e]), int(m.counts[e])
        if c:
            v, err = product(wide_x(h[a:a + c], hs[a:a + c]), wide_w(down[e], ds[e], False), False)
            check(o[a:a + c], v, err, "bf16")


def test_rows_out_of_range_count_as_zeros():
    g = torch.Generator().manual_seed(5)
    w, ws = weights(g, 2, 128, 256, False)
    x, xs = rows_of(g, 4, 256)
    src = torch.tensor([0, 9, 3, -1, 1, 2, 8], dtype=torch.int32).cuda()
    offsets, cnt, _ = groups([4, 3])
    status = _status()
    y = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, src=src, top_k=2, status=status)
    assert int(status) == moedc.ERR_EXPERT_RANGE
    assert (y[[3, 6]] == 0).all() and (y[1] == 0).all()
    for r, t in ((0, 0), (2, 1), (4, 0), (5, 1)):
        v, err = product(wide_x(x[t:t + 1], xs[t:t + 1]), wide_w(w[int(r >= 4)], ws[int(r >= 4)], False), False)
        check(y[r:r + 1], v, err, "bf16")
    with pytest.raises(moedc.MoedcError) as err:
        moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, src=src, top_k=2)
    assert err.value.code == moedc.ERR_EXPERT_RANGE
    # where the rows are copied first
    src = (torch.arange(80, dtype=torch.int32) % 8).cuda()
    src[[7, 50]] = torch.tensor([8, -1], dtype=torch.int32).cuda()
    offsets, cnt, _ = groups([40, 40])
    assert moedc.moedc_matmul_e4m3_workspace_bytes(256, 2, 80) > 0
    xs[0, 0] = float("inf")
    status.zero_()
    y = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, src=src, top_k=2, status=status)
    z = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, src=src, top_k=2, status=status,
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert int(status) == moedc.ERR_EXPERT_RANGE
    assert (y[[7, 50]] == 0).all() and (z[[7, 50]] == 0).all()
    assert torch.equal(torch.nan_to_num(y.float()), torch.nan_to_num(z.float()))


def test_nan_stays_in_its_row_and_column():
    g = torch.Generator().manual_seed(6)
    w, ws = weights(g, 1, 256, 256, False)
    x, xs = rows_of(g, 140, 256)
    want = moedc.matmul_e4m3(x, xs, w[0], ws[0])
    x.view(torch.uint8)[130, 200] = 0x7f
    w.view(torch.uint8)[0, 200, 3] = 0xff
    got = moedc.matmul_e4m3(x, xs, w[0], ws[0])
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[130], nan[:, 200] = True, True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    codes, _ = moedc.matmul_e4m3(x, xs, w[0], ws[0], out_dtype=moedc.FP8_E4M3)
    assert torch.equal(torch.isnan(codes.float()), nan)


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,E,N,Kd", [(1, 1, 640, 2048), (3, 1, 7168, 7168), (16, 1, 256, 8192), (17, 1, 384, 2304),
                                         (64, 1, 512, 4096), (65, 1, 512, 4096), (128, 1, 256, 3200), (5, 3, 256, 2688),
                                         (2, 1, 128, 1920)])
def test_tiles_shared_by_a_cluster(rows, E, N, Kd, swiglu, out):
    """Few tiles: the channels are split among the blocks of a cluster, unevenly where their
    groups do not divide."""
    g = torch.Generator().manual_seed(rows + N)
    w, ws = weights(g, E, N, Kd, swiglu)
    x, xs = rows_of(g, rows, Kd)
    counts = [rows - 2 * (E // 2)] + [2 if i % 2 else 0 for i in range(E - 1)]
    offsets, cnt, _ = groups(counts)
    status = _status()
    got = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=swiglu, out_dtype=OUT[out], status=status)
    again = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=swiglu, out_dtype=OUT[out], status=status)
    assert int(status) == 0
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if not c:
            continue
        v, err = product(wide_x(x[a:a + c], xs[a:a + c]), wide_w(w[e], ws[e], swiglu), swiglu)
        check((got[0][a:a + c], got[1][a:a + c]) if out == "e4m3" else got[a:a + c], v, err, out)
    for p, q in zip(got if out == "e4m3" else [got], again if out == "e4m3" else [again]):
        assert torch.equal(p.float(), q.float())


def test_overlapping_groups_in_clusters():
    """Groups that share rows make more tiles than the call can know of; each is computed."""
    g = torch.Generator().manual_seed(13)
    w, ws = weights(g, 6, 256, 2048, False)
    x, xs = rows_of(g, 3, 2048)
    offsets = torch.zeros(7, dtype=torch.int32).cuda()
    cnt = torch.full((6,), 3, dtype=torch.int32).cuda()
    status = _status()
    y = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, status=status)
    # whichever expert came last
    best = torch.full((3, 256), float("inf"), dtype=torch.float64, device="cuda")
    for e in range(6):
        v, err = product(wide_x(x, xs), wide_w(w[e], ws[e], False), False)
        best = torch.minimum(best, (y.double() - v).abs() - err - rounding(v.abs() + err, torch.bfloat16))
    assert (best <= 0).all() and int(status) == 0


def test_large_scales_and_small_ones():
    """Scales far apart: the groups' sums are scaled one by one."""
    g = torch.Generator().manual_seed(7)
    w, ws = weights(g, 1, 128, 1024, False)
    x, xs = rows_of(g, 5, 1024)
    xs *= torch.exp2(torch.randint(-40, 40, xs.shape, generator=g).float()).cuda()
    ws *= torch.exp2(torch.randint(-20, 20, ws.shape, generator=g).float()).cuda()
    y = moedc.matmul_e4m3(x, xs, w[0], ws[0])
    v, err = product(wide_x(x, xs), wide_w(w[0], ws[0], False), False)
    check(y, v, err, "bf16")


def test_replays_as_a_graph_with_new_groups():
    g = torch.Generator().manual_seed(8)
    E, N, Kd, rows = 6, 256, 384, 700
    w, ws = weights(g, E, N, Kd, True)
    x, xs = rows_of(g, rows, Kd)
    offsets, cnt, _ = groups([100, 0, 300, 7, 200, 93])
    status = _status()

    def step():
        return moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=True,
                                 out_dtype=moedc.FP8_E4M3, status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    for counts in ([10, 300, 0, 1, 380, 9], [700, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 700]):
        o, c, _ = groups(counts)
        offsets.copy_(o)
        cnt.copy_(c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a.float(), b.float())
    assert int(status) == 0


def test_bounded_waits_end_the_call():
    g = torch.Generator().manual_seed(9)
    w, ws = weights(g, 2, 384, 1024, False)
    x, xs = rows_of(g, 320, 1024)
    offsets, cnt, _ = groups([300, 20])
    status = _status()

    def run():
        status.zero_()
        y = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, status=status)
        return y, int(status)

    want, code = run()
    assert code == moedc.OK
    moedc.load().moedc_test_set_wait_extra(1)
    try:
        assert run()[1] == moedc.ERR_TIMEOUT
    finally:
        moedc.load().moedc_test_set_wait_extra(0)
    got, code = run()
    assert code == moedc.OK and torch.equal(got, want)


def test_refusals():
    x = torch.zeros(4, 256, device="cuda").to(E4M3)
    xs = torch.ones(4, 2).cuda()
    w = torch.zeros(2, 128, 256, device="cuda").to(E4M3)
    ws = torch.ones(2, 1, 2).cuda()
    o = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    c = torch.tensor([2, 2], dtype=torch.int32).cuda()
    src = torch.arange(4, dtype=torch.int32).cuda()
    for change in (dict(x=x.float()), dict(x=x.cpu()), dict(w=w.float()), dict(xs=xs.half()), dict(xs=xs[:3]),
                   dict(ws=ws[:, :, :1]), dict(counts=None), dict(offsets=o.long()), dict(offsets=None),
                   dict(src=src.long()), dict(out_dtype=moedc.F32), dict(scale_layout=7), dict(x=x[:, :128]),
                   dict(scale_layout=moedc.SCALES_COL_MAJOR), dict(scale_layout=moedc.SCALES_PER_TOKEN),
                   dict(out=torch.zeros(4, 128).cuda()), dict(status=torch.zeros(1).cuda()),
                   dict(w=w[:, :96].contiguous(), out_dtype=moedc.FP8_E4M3), dict(w=w[:, :97].contiguous(), swiglu=True),
                   dict(offsets=None, src=src)):
        args = dict(x=x, xs=xs, w=w, ws=ws, offsets=o, counts=c) | change
        with pytest.raises(ValueError):
            moedc.matmul_e4m3(**args)
    for change in (dict(src=src, top_k=0), dict(offsets=None, counts=None)):
        args = dict(offsets=o, counts=c) | change
        with pytest.raises(moedc.MoedcError):
            moedc.matmul_e4m3(x, xs, w, ws, **args)
    off = torch.zeros(4 * 256 + 8, device="cuda").to(E4M3)[8:].view(4, 256)
    with pytest.raises(moedc.MoedcError):
        moedc.matmul_e4m3(off, xs, w, ws, offsets=o, counts=c)
