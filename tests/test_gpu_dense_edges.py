"""The dense layers at the edges of their arguments: offsets past 32 bits, the most experts,
two streams at once, workspaces of two graphs, waits that run out in every form."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import assert_within, rounding
from matmul_util import groups, product, randn
from test_gpu_matmul_e4m3 import check, rows_of, weights, wide_w, wide_x

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def _status():
    return torch.zeros(1, dtype=torch.int32).cuda()


def _need_bytes(n):
    free, _ = torch.cuda.mem_get_info()
    if free < n:
        pytest.skip("needs more device memory")


def _near(got, x, w, swiglu=False, dtype=torch.bfloat16):
    v, err = product(x, w, swiglu)
    assert_within(got, v, err + rounding(v.abs() + err, dtype))


def test_layers_past_32_bits():
    _need_bytes(40 << 30)
    g = torch.Generator().manual_seed(0)
    rows, N, Kd = 300000, 7168, 64
    counts = [4, rows - 1000, 996]
    offsets, cnt, _ = groups(counts)
    x = torch.zeros(rows, Kd, dtype=torch.bfloat16, device="cuda")
    x[-1000:] = randn(g, torch.bfloat16, 1000, Kd)
    w = randn(g, torch.bfloat16, 3, N, Kd)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    y = moedc.matmul(x, w, **maps)
    assert y.numel() > 2 ** 31
    _near(y[-996:], x[-996:], w[2])
    _near(y[-1000:-996], x[-1000:-996], w[1])
    dx, dw = moedc.matmul_grad(y, x, w, **maps)
    _near(dx[-996:], y[-996:], w[2].T.contiguous())
    _near(dw[2], y[-996:].T.contiguous(), x[-996:].T.contiguous())
    half = N // 2
    h, p = moedc.matmul(x, w, swiglu=True, keep=True, **maps)
    _near(h[-996:], x[-996:], w[2], True)
    assert torch.equal(p[-996:], y[-996:])
    d = moedc.swiglu_grad(h, p)
    alone = moedc.swiglu_grad(h[-996:], p[-996:])
    assert torch.equal(d[-996:], alone) and half * 2 == N
    assert int(maps["status"]) == 0


def test_weight_gradients_past_32_bits():
    _need_bytes(30 << 30)
    g = torch.Generator().manual_seed(1)
    E, N, Kd = 65, 8192, 4104
    counts = [2] * (E - 1) + [70]
    offsets, cnt, rows = groups(counts)
    x, d = randn(g, torch.float16, rows, Kd), randn(g, torch.float16, rows, N)
    _, dw = moedc.matmul_grad(d, x, None, offsets=offsets, counts=cnt, dw_dtype=torch.float32, status=_status())
    assert dw.numel() > 2 ** 31
    for e in (0, E - 1):
        a, c = int(offsets[e]), counts[e]
        _near(dw[e], d[a:a + c].T.contiguous(), x[a:a + c].T.contiguous(), dtype=torch.float32)


@pytest.mark.parametrize("form", ["packed", "gathered", "slots"])
def test_e4m3_past_32_bits(form):
    _need_bytes(30 << 30)
    g = torch.Generator().manual_seed(2)
    rows, N, Kd = 600000, 3712, 3712
    w, ws = weights(g, 2, N, Kd, False)
    last = rows_of(g, 200, Kd)
    if form == "gathered":
        x, xs = last
        src = torch.full((rows,), 0, dtype=torch.int32, device="cuda")
        src[-200:] = torch.arange(200, dtype=torch.int32).cuda()
        maps = dict(src=src)
    else:
        x = torch.zeros(rows, Kd, dtype=torch.uint8, device="cuda").view(E4M3)
        xs = torch.ones(rows, Kd // 128, device="cuda")
        x.view(torch.uint8)[-200:], xs[-200:] = last[0].view(torch.uint8), last[1]
        maps = {}
    status = _status()
    if form == "slots":
        counts = torch.tensor([3, rows // 2], dtype=torch.int32).cuda()
        y = moedc.matmul_e4m3(x.view(2, rows // 2, Kd), xs.view(2, rows // 2, -1), w, ws, counts=counts, status=status).view(rows, N)
    else:
        offsets, cnt, _ = groups([rows - 200, 200])
        y = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, status=status, **maps)
    assert y.numel() > 2 ** 31 and int(status) == 0
    v, err = product(wide_x(*last), wide_w(w[1], ws[1], False), False)
    check(y[-200:], v, err, "bf16")


def test_quant_past_32_bits():
    _need_bytes(20 << 30)
    g = torch.Generator().manual_seed(3)
    x = torch.zeros(300000, 7296, dtype=torch.bfloat16, device="cuda")
    x[-200:] = randn(g, torch.bfloat16, 200, 7296)
    for block_rows in (1, 128):
        codes, scales = moedc.quant_e4m3(x, block_rows=block_rows)
        tail = 200 if block_rows == 1 else 300000 % 128
        a, b = moedc.quant_e4m3(x[-tail:], block_rows=block_rows)
        assert torch.equal(codes[-tail:].view(torch.uint8), a.view(torch.uint8))
        assert torch.equal(scales[-b.shape[0]:], b)


def test_the_most_experts():
    g = torch.Generator().manual_seed(4)
    E, N, Kd = 1024, 40, 72
    counts = [(i * 7) % 5 for i in range(E)]
    offsets, cnt, rows = groups(counts)
    x, w = randn(g, torch.bfloat16, rows, Kd), randn(g, torch.bfloat16, E, N, Kd)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    y = moedc.matmul(x, w, **maps)
    dx, dw = moedc.matmul_grad(y, x, w, **maps)
    q, qs = rows_of(g, rows, 128)
    w8, s8 = weights(g, E, 24, 128, True)
    z = moedc.matmul_e4m3(q, qs, w8, s8, swiglu=True, **maps)
    assert int(maps["status"]) == 0
    for e in (0, 1, 511, 1022, 1023):
        a, c = int(offsets[e]), counts[e]
        if c:
            _near(y[a:a + c], x[a:a + c], w[e])
            _near(dx[a:a + c], y[a:a + c], w[e].T.contiguous())
            v, err = product(wide_x(q[a:a + c], qs[a:a + c]), wide_w(w8[e], s8[e], True), True)
            check(z[a:a + c], v, err, "bf16")
        else:
            assert (dw[e] == 0).all()


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(5)
    offsets, cnt, rows = groups([300, 7, 500])
    x, w = randn(g, torch.bfloat16, rows, 512), randn(g, torch.bfloat16, 3, 768, 512)
    q, qs = rows_of(g, 40, 1024)
    w8, s8 = weights(g, 1, 512, 1024, False)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    lone = _status()
    want = (moedc.matmul(x, w, **maps), moedc.matmul_e4m3(q, qs, w8, s8, status=lone))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got[0].append(moedc.matmul(x, w, **maps))
        with torch.cuda.stream(streams[1]):
            got[1].append(moedc.matmul_e4m3(q, qs, w8, s8, status=lone))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i]) for i in range(2) for a in got[i])
    assert int(maps["status"]) == 0 and int(lone) == 0


def test_two_graphs_with_workspaces_of_their_own():
    g = torch.Generator().manual_seed(6)
    T, E, K, N, Kd = 90, 2, 2, 256, 512
    w, ws = weights(g, E, N, Kd, False)
    tokens = [rows_of(g, T, Kd) for _ in range(2)]
    idx = torch.rand(T, E, generator=g).topk(K, dim=1).indices.to(torch.int32).cuda()
    m = moedc.sort(None, idx, E)
    assert moedc.moedc_matmul_e4m3_workspace_bytes(Kd, E, T * K) > 0

    def step(x, xs):
        return moedc.matmul_e4m3(x, xs, w, ws, offsets=m.offsets, counts=m.counts, src=m.src, top_k=K, status=m.status)

    want = [step(*t) for t in tokens]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, got = [], []
    for t in tokens:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got.append(step(*t))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and int(m.status) == 0


# few rows to an expert; a cluster's tile; many rows; rows copied first
@pytest.mark.parametrize("counts,N,Kd", [([3, 0, 9] * 60, 512, 1024), ([5], 512, 4096), ([300, 400], 512, 1024)])
@pytest.mark.parametrize("gather", [False, True])
def test_e4m3_waits_that_run_out_end_the_call(counts, N, Kd, gather):
    g = torch.Generator().manual_seed(7)
    w, ws = weights(g, len(counts), N, Kd, True)
    offsets, cnt, rows = groups(counts)
    x, xs = rows_of(g, rows, Kd)
    status = _status()
    maps = dict(src=torch.randperm(rows, generator=g).to(torch.int32).cuda()) if gather else {}

    def run():
        status.zero_()
        y, _ = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=True,
                                 out_dtype=moedc.FP8_E4M3, status=status, **maps)
        return y.view(torch.uint8), int(status)

    want, code = run()
    assert code == moedc.OK
    moedc.load().moedc_test_set_wait_extra(1)
    try:
        assert [run()[1] for _ in range(2)] == [moedc.ERR_TIMEOUT] * 2
    finally:
        moedc.load().moedc_test_set_wait_extra(0)
    got, code = run()
    assert code == moedc.OK and torch.equal(got, want)


def test_layers_with_overlapping_groups():
    """Groups that share rows: the gradients of each expert's weights count them all."""
    g = torch.Generator().manual_seed(8)
    x, w, d = (randn(g, torch.bfloat16, *s) for s in ((50, 64), (4, 72, 64), (50, 72)))
    offsets = torch.tensor([0, 10, 5, 0, 0], dtype=torch.int32).cuda()
    cnt = torch.tensor([50, 40, 20, 50], dtype=torch.int32).cuda()
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    moedc.matmul(x, w, **maps)
    _, dw = moedc.matmul_grad(d, x, w, **maps)
    assert int(maps["status"]) == 0
    for e in range(4):
        a, c = int(offsets[e]), int(cnt[e])
        _near(dw[e], d[a:a + c].T.contiguous(), x[a:a + c].T.contiguous())
