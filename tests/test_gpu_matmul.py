"""The experts' layers in training: products of packed rows with 16-bit weights, the gated
block, their gradients, against 64-bit forms at the edges of tiles, groups and stages."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from lm_util import DTYPES, ROUND, U32, assert_within, rounding
from matmul_util import groups, owned, product, randn

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32).cuda()


# rows around the tile's 256 and 128, none, one; columns and channels that end inside a tile,
# a box, a stage; groups that begin anywhere
CASES = [
    ([1], 8, 8, 1, "bf16"),
    ([3], 264, 72, 1, "f16"),
    ([0, 1, 127, 128, 129, 0, 2], 136, 64, 1, "bf16"),
    ([255, 256, 257, 0], 520, 200, 8, "bf16"),
    ([513, 31], 256, 1032, 16, "f16"),
    ([5] * 40, 384, 136, 1, "bf16"),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,Kd,align,dtype", CASES)
def test_forward(counts, N, Kd, align, dtype, swiglu):
    g = torch.Generator().manual_seed(len(counts) + N)
    dt = DTYPES[dtype]
    offsets, cnt, rows = groups(counts, align, tail=5)
    n = 2 * N if swiglu else N
    x, w = randn(g, dt, rows, Kd), randn(g, dt, len(counts), n, Kd, scale=Kd ** -0.5)
    mine = owned(offsets, cnt, rows)
    x[~mine] = float("nan")                  # rows of nobody
    out = torch.full((rows, N), 7.0, dtype=dt, device="cuda")
    kept = torch.full((rows, n), 7.0, dtype=dt, device="cuda")
    status = _status()
    args = dict(offsets=offsets, counts=cnt, swiglu=swiglu, status=status)
    if swiglu:
        moedc.matmul(x, w, keep=True, out=(out, kept), **args)
        alone = torch.full_like(out, 7.0)
        assert torch.equal(moedc.matmul(x, w, out=alone, **args), out)
        assert (kept[~mine] == 7.0).all()
    else:
        moedc.matmul(x, w, out=out, **args)
    assert int(status) == 0
    assert (out[~mine] == 7.0).all()
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if not c:
            continue
        v, err = product(x[a:a + c], w[e], swiglu)
        assert_within(out[a:a + c], v, err + rounding(v.abs() + err, dt))
        if swiglu:
            v, err = product(x[a:a + c], w[e], False)
            assert_within(kept[a:a + c], v, err + rounding(v.abs() + err, dt))


@pytest.mark.parametrize("dw_dtype", [None, torch.float32])
@pytest.mark.parametrize("counts,N,Kd,align,dtype", CASES + [
    ([0, 1, 15, 16, 17, 33, 63, 64, 65, 130], 24, 40, 1, "bf16"),
    ([16, 32, 0, 48], 264, 264, 16, "f16"),
])
def test_gradients(counts, N, Kd, align, dtype, dw_dtype):
    g = torch.Generator().manual_seed(len(counts) * 7 + N)
    dt = DTYPES[dtype]
    offsets, cnt, rows = groups(counts, align, tail=3)
    E = len(counts)
    x, w = randn(g, dt, rows, Kd), randn(g, dt, E, N, Kd, scale=Kd ** -0.5)
    d = randn(g, dt, rows, N)
    mine = owned(offsets, cnt, rows)
    x[~mine] = float("nan")
    d[~mine] = float("inf")
    dx = torch.full((rows, Kd), 7.0, dtype=dt, device="cuda")
    dw = torch.full((E, N, Kd), 7.0, dtype=dw_dtype or dt, device="cuda")
    status = _status()
    args = dict(offsets=offsets, counts=cnt, status=status)
    moedc.matmul_grad(d, x, w, out=(dx, dw), **args)
    assert int(status) == 0
    assert (dx[~mine] == 7.0).all()
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if not c:
            assert (dw[e] == 0).all()
            continue
        v, err = product(d[a:a + c], w[e].T.contiguous(), False)
        assert_within(dx[a:a + c], v, err + rounding(v.abs() + err, dt))
        v, err = product(d[a:a + c].T.contiguous(), x[a:a + c].T.contiguous(), False)
        assert_within(dw[e], v, err + rounding(v.abs() + err, dw.dtype))
    only = moedc.matmul_grad(d, None, w, **args)
    assert only[1] is None and torch.equal(only[0][mine], dx[mine])
    only = moedc.matmul_grad(d, x, None, dw_dtype=dw_dtype, **args)
    assert only[0] is None and torch.equal(only[1], dw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,N", [(1, 8), (33, 72), (300, 1032)])
def test_swiglu_grad(rows, N, dtype):
    g = torch.Generator().manual_seed(rows)
    dt = DTYPES[dtype]
    dh, p = randn(g, dt, rows, N), randn(g, dt, rows, 2 * N, scale=3.0)
    p[0, :4] = torch.tensor([0.0, -20.0, 20.0, -100.0])
    a, b = p[:, :N].double(), p[:, N:].double()
    s = torch.sigmoid(a)
    h = dh.double()
    ref = torch.cat([h * b * s * (1 + a * (1 - s)), h * a * s], 1)
    # eight roundings and expf's two ulps; 1 - s of an s near 1 is off by an ulp of 1, so is
    # 1 + a (1 - s) by |a| of them
    mag = torch.cat([(h * b * s).abs() * (2 + 2 * a.abs()), (h * a * s).abs()], 1)
    # below the smallest normal numbers a rounding is off by half the subnormal spacing: 2^-25 in
    # f16, 2^-134 in bf16, and 2^-150 for each binary32 one, whose factors here are below 2^9
    tiny = (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134) + 8 * 2.0 ** -150 * 2.0 ** 9
    bound = 16 * U32 * mag + rounding(ref, dt) + tiny
    got = moedc.swiglu_grad(dh, p)
    assert_within(got, ref, bound)
    wide = torch.zeros(rows, N + 8, dtype=dt, device="cuda")
    wide[:, :N] = dh
    assert torch.equal(moedc.swiglu_grad(wide[:, :N], p), got)
    assert moedc.swiglu_grad(dh, p, out=p) is p and torch.equal(p, got)


def test_block_gradients_against_differences():
    """(f(w + h d) - f(w - h d)) / 2h of the 64-bit block against the gradients' product with d:
    the difference's own error is h^2, the gradients' the roundings of their 16 bits."""
    g = torch.Generator().manual_seed(5)
    counts, N, Kd = [9, 0, 20], 24, 40
    offsets, cnt, rows = groups(counts)
    x, w = randn(g, torch.float16, rows, Kd), randn(g, torch.float16, 3, 2 * N, Kd, scale=Kd ** -0.5)
    c = randn(g, torch.float16, rows, N)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    _, p = moedc.matmul(x, w, swiglu=True, keep=True, **maps)
    dx, dw = moedc.matmul_grad(moedc.swiglu_grad(c, p), x, w, dw_dtype=torch.float32, **maps)

    def f(xx, ww):
        total = 0.0
        for e, n in enumerate(counts):
            a = int(offsets[e])
            v = xx[a:a + n] @ ww[e].T
            total = total + (v[:, :N] * torch.sigmoid(v[:, :N]) * v[:, N:] * c[a:a + n].double()).sum()
        return float(total)

    h = 1e-4
    for i in range(6):
        ex, ew = (torch.randn(t.shape, generator=g).double().cuda() for t in (x, w))
        by_x = (f(x.double() + h * ex, w.double()) - f(x.double() - h * ex, w.double())) / (2 * h)
        by_w = (f(x.double(), w.double() + h * ew) - f(x.double(), w.double() - h * ew)) / (2 * h)
        # products and their gradients are rounded to 11 bits, random signs: some 2^-10 of the norms
        assert abs(by_x - float((dx.double() * ex).sum())) <= 2.0 ** -9 * float(dx.double().norm() * 6)
        assert abs(by_w - float((dw.double() * ew).sum())) <= 2.0 ** -9 * float(dw.double().norm() * 6)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,E,N,Kd", [(1, 1, 4096, 4096), (33, 1, 2048, 1032), (128, 1, 520, 2048), (129, 1, 264, 4096),
                                         (256, 1, 264, 2048), (300, 1, 264, 1024), (5, 3, 256, 264), (7, 1, 8192, 512), (40, 1, 520, 4168),
                                         (128, 1, 264, 4168), (9, 4, 1544, 2056)])
def test_tiles_shared_by_a_cluster(rows, E, N, Kd, swiglu):
    """Few tiles: the contracted axis is split among pairs, unevenly where its stages do not
    divide.  The gradient of the rows contracts N."""
    g = torch.Generator().manual_seed(rows + N)
    counts = [rows - 2 * (E // 2)] + [2 if i % 2 else 0 for i in range(E - 1)]
    offsets, cnt, _ = groups(counts)
    n = 2 * N if swiglu else N
    x, w = randn(g, torch.bfloat16, rows, Kd), randn(g, torch.bfloat16, E, n, Kd, scale=Kd ** -0.5)
    d = randn(g, torch.bfloat16, rows, n)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    y = moedc.matmul(x, w, swiglu=swiglu, **maps)
    dx, _ = moedc.matmul_grad(d, None, w, **maps)
    assert int(maps["status"]) == 0
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if c:
            v, err = product(x[a:a + c], w[e], swiglu)
            assert_within(y[a:a + c], v, err + rounding(v.abs() + err, torch.bfloat16))
            v, err = product(d[a:a + c], w[e].T.contiguous(), False)
            assert_within(dx[a:a + c], v, err + rounding(v.abs() + err, torch.bfloat16))
    mine = owned(offsets, cnt, rows)
    assert torch.equal(moedc.matmul(x, w, swiglu=swiglu, **maps)[mine], y[mine])
    # groups that share rows: more tiles than the call can know of
    offsets.zero_()
    cnt.fill_(rows)
    moedc.matmul_grad(d, None, w, **maps)
    assert int(maps["status"]) == 0


@pytest.mark.parametrize("counts", [[8192], [1024, 1025, 2047, 0, 5000]])
def test_binary32_weight_gradients_of_many_tokens(counts):
    """The tensor core's sums lose up to an ulp (2^-23) with each product of 16 tokens, 48 of them in a
    piece of 768, the pieces' sums half an ulp each, 11 of them at most: less than 64 * 2^-23 of the
    sums, whose norms are at most the result's for values of random signs."""
    g = torch.Generator().manual_seed(12)
    offsets, cnt, rows = groups(counts, tail=3)
    x, d = randn(g, torch.bfloat16, rows, 264), randn(g, torch.bfloat16, rows, 328)
    _, dw = moedc.matmul_grad(d, x, None, offsets=offsets, counts=cnt, dw_dtype=torch.float32, status=_status())
    for e, c in enumerate(counts):
        a = int(offsets[e])
        ref = d[a:a + c].double().T @ x[a:a + c].double()
        assert (dw[e].double() - ref).norm() <= 64 * 2.0 ** -23 * ref.norm()


def test_slots_strides_and_capacity():
    g = torch.Generator().manual_seed(6)
    E, cap, N, Kd = 5, 40, 72, 104
    counts = torch.tensor([3, 40, 0, 45, 17], dtype=torch.int32).cuda()
    wide = randn(g, torch.bfloat16, E * cap, Kd + 24)
    x, w = wide[:, 8:8 + Kd], randn(g, torch.bfloat16, E, N, Kd)
    out = torch.full((E * cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = _status()
    moedc.matmul(x, w, counts=counts, status=status, out=out)
    assert int(status) == moedc.ERR_CAPACITY            # 45 of 40 slots: the rest is skipped
    for e, c in enumerate(counts.tolist()):
        c = min(c, cap)
        v, err = product(x[e * cap:e * cap + c], w[e], False)
        assert_within(out[e * cap:e * cap + c], v, err + rounding(v.abs() + err, torch.bfloat16))
        assert (out[e * cap + c:(e + 1) * cap] == 7.0).all()
    with pytest.raises(moedc.MoedcError) as err:
        moedc.matmul(x, w, counts=counts)
    assert err.value.code == moedc.ERR_CAPACITY
    # maps that point outside are clipped to the rows
    offsets = torch.tensor([-5, 10, 190, 500, 20, 60], dtype=torch.int32).cuda()
    status.zero_()
    moedc.matmul(x, w, offsets=offsets, counts=torch.tensor([2, -3, 90, 4, 2 ** 31 - 1], dtype=torch.int32).cuda(), status=status, out=out)
    assert int(status) == moedc.ERR_CAPACITY


def test_nan_and_infinities_stay_in_their_rows_and_experts():
    g = torch.Generator().manual_seed(7)
    counts, N, Kd = [70, 50], 136, 200
    offsets, cnt, rows = groups(counts)
    x, w = randn(g, torch.bfloat16, rows, Kd), randn(g, torch.bfloat16, 2, N, Kd)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    want = moedc.matmul(x, w, **maps)
    wantx, wantw = moedc.matmul_grad(want, x, w, **maps)
    x[3, 5], x[80, 9] = float("nan"), float("inf")
    got = moedc.matmul(x, w, **maps)
    same = torch.ones(rows, dtype=torch.bool)
    same[[3, 80]] = False
    assert torch.equal(got[same], want[same])
    assert torch.isnan(got[3]).all() and torch.isinf(got[80]).all()
    x[80, 9] = 1.0
    _, dw = moedc.matmul_grad(want, x, w, **maps)
    assert torch.isnan(dw[0][:, 5]).all() and not torch.isnan(dw[1]).any()
    w[1, 4, 6] = float("nan")                        # the other expert's first rows of 64 past N
    dx, _ = moedc.matmul_grad(want, x, w, **maps)
    assert torch.equal(dx[:70], wantx[:70])
    assert torch.isnan(dx[70:, 6]).all()


def test_replays_as_a_graph_on_another_stream_with_new_groups():
    g = torch.Generator().manual_seed(8)
    E, N, Kd, rows = 6, 264, 328, 700
    x, w = randn(g, torch.bfloat16, rows, Kd), randn(g, torch.bfloat16, E, 2 * N, Kd, scale=Kd ** -0.5)
    dh = randn(g, torch.bfloat16, rows, N)
    offsets, cnt, _ = groups([100, 0, 300, 7, 200, 93])
    status = _status()

    def step():
        h, p = moedc.matmul(x, w, offsets=offsets, counts=cnt, swiglu=True, keep=True, status=status)
        d = moedc.swiglu_grad(dh, p)
        return h, p, d, *moedc.matmul_grad(d, x, w, offsets=offsets, counts=cnt, status=status)

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
            assert torch.equal(a, b)
    assert int(status) == 0


def test_equal_bits_and_no_rows():
    g = torch.Generator().manual_seed(9)
    offsets, cnt, rows = groups([300, 20, 515])
    x, w = randn(g, torch.bfloat16, rows, 512), randn(g, torch.bfloat16, 3, 768, 512)
    d = randn(g, torch.bfloat16, rows, 768)
    maps = dict(offsets=offsets, counts=cnt, status=_status())
    first = (moedc.matmul(x, w, **maps), *moedc.matmul_grad(d, x, w, **maps))
    for _ in range(5):
        again = (moedc.matmul(x, w, **maps), *moedc.matmul_grad(d, x, w, **maps))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    none = torch.zeros(4, dtype=torch.int32).cuda()
    maps = dict(offsets=none, counts=none[:3], status=_status())
    assert moedc.matmul(x[:0], w, **maps).shape == (0, 768)
    dx, dw = moedc.matmul_grad(d[:0], x[:0], w, **maps)
    assert dx.shape == (0, 512) and (dw == 0).all()
    dx, dw = moedc.matmul_grad(d, x, w, **maps)        # rows that are nobody's
    assert (dw == 0).all()


def test_one_linear_layer():
    g = torch.Generator().manual_seed(10)
    for rows in (1, 129):
        x, w = randn(g, torch.float16, rows, 136), randn(g, torch.float16, 88, 136)
        y = moedc.matmul(x, w)
        v, err = product(x, w, False)
        assert_within(y, v, err + rounding(v.abs() + err, torch.float16))
        dx, dw = moedc.matmul_grad(y, x, w)
        assert dw.shape == w.shape and dx.shape == x.shape
        v, err = product(y, w.T.contiguous(), False)
        assert_within(dx, v, err + rounding(v.abs() + err, torch.float16))


def test_bounded_waits_end_the_calls():
    g = torch.Generator().manual_seed(11)
    offsets, cnt, rows = groups([300, 0, 40])
    x, w = randn(g, torch.bfloat16, rows, 512), randn(g, torch.bfloat16, 3, 768, 512)
    d = randn(g, torch.bfloat16, rows, 768)
    status = _status()
    maps = dict(offsets=offsets, counts=cnt, status=status)
    want = (moedc.matmul(x, w, **maps), *moedc.matmul_grad(d, x, w, **maps))
    lib = moedc.load()
    for call in (lambda: moedc.matmul(x, w, **maps), lambda: moedc.matmul_grad(d, None, w, **maps),
                 lambda: moedc.matmul_grad(d, x, None, **maps)):
        lib.moedc_test_set_wait_extra(1)
        try:
            status.zero_()
            call()
            assert int(status) == moedc.ERR_TIMEOUT
        finally:
            lib.moedc_test_set_wait_extra(0)
    status.zero_()
    got = (moedc.matmul(x, w, **maps), *moedc.matmul_grad(d, x, w, **maps))
    assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16).cuda()
    w = torch.zeros(2, 16, 64, dtype=torch.bfloat16).cuda()
    c = torch.tensor([2, 2], dtype=torch.int32).cuda()
    o = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    bad = [
        (dict(x=x.float(), w=w.float()), moedc.MoedcError), (dict(w=w.half()), ValueError),
        (dict(x=x.cpu()), ValueError), (dict(x=x[:, :56]), ValueError), (dict(counts=None), ValueError),
        (dict(offsets=None, counts=None), moedc.MoedcError), (dict(offsets=o[:2]), ValueError),
        (dict(counts=c.long()), ValueError), (dict(status=torch.zeros(1).cuda()), ValueError),
        (dict(keep=True), ValueError), (dict(w=w[:, :15], swiglu=True), ValueError),
        (dict(out=torch.zeros(4, 8).cuda()), ValueError), (dict(w=w[:, :, ::2].contiguous(), x=x[:, ::2]), ValueError),
        (dict(x=x.flatten()[4:228].view(4, 56), w=w[:, :, :56].contiguous()), moedc.MoedcError),   # 8 bytes off
        (dict(x=x.expand(4, 64)[:1].expand(4, 64)), ValueError),
        (dict(w=w[:, :12].contiguous()), moedc.MoedcError), (dict(w=w[:, :, :60].contiguous(), x=x[:, :60]), moedc.MoedcError),
    ]
    for change, error in bad:
        args = dict(x=x, w=w, offsets=o, counts=c) | change
        with pytest.raises(error):
            moedc.matmul(args.pop("x"), args.pop("w"), **args)
    with pytest.raises(moedc.MoedcError):
        moedc.matmul(x[:3], w, counts=c)             # slots that are not as many for each
    d = torch.zeros(4, 16, dtype=torch.bfloat16).cuda()
    for change in (dict(x=x[:3]), dict(w=w.half()), dict(x=None, w=None), dict(dw_dtype=torch.float16),
                   dict(out=(None, None)), dict(x=x.half())):
        args = dict(x=x, w=w, offsets=o, counts=c) | change
        with pytest.raises(ValueError):
            moedc.matmul_grad(d, args.pop("x"), args.pop("w"), **args)
    with pytest.raises(ValueError):
        moedc.swiglu_grad(d, d)
