"""e4m3 products whose tiles a cluster shares, up to the most tokens of a tile, against 64-bit
forms; rows gathered there."""
import pytest
import torch

from combine_moedc_layout_gb300 import moedc
from matmul_util import groups, product
from test_gpu_matmul_e4m3 import E4M3, OUT, check, rows_of, weights, wide_w, wide_x

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32).cuda()


def _near(got, x, xs, w, ws, offsets, counts, swiglu, out):
    for e, c in enumerate(counts):
        a = int(offsets[e])
        if c:
            v, err = product(wide_x(x[a:a + c], xs[a:a + c]), wide_w(w[e], ws[e], swiglu), swiglu)
            check((got[0][a:a + c], got[1][a:a + c]) if out == "e4m3" else got[a:a + c], v, err, out)


# both halves of the tokens and their edges; a whole tile of 64; two, four and eight parts
@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,Kd", [([31], 512, 4096), ([32], 512, 4096), ([33], 512, 4096), ([47], 256, 8192),
                                         ([48], 384, 2304), ([64, 4, 2], 256, 4096), ([2, 64, 0, 6], 128, 7168),
                                         ([63, 1, 1], 640, 2048), ([40], 7168, 1024)])
def test_up_to_a_whole_tile_of_tokens(counts, N, Kd, swiglu, out):
    g = torch.Generator().manual_seed(sum(counts) + N)
    w, ws = weights(g, len(counts), N, Kd, swiglu)
    offsets, cnt, rows = groups(counts)
    x, xs = rows_of(g, rows, Kd)
    status = _status()
    got = moedc.matmul_e4m3(x, xs, w, ws, offsets=offsets, counts=cnt, swiglu=swiglu, out_dtype=OUT[out], status=status)
    assert int(status) == 0
    _near(got, x, xs, w, ws, offsets, counts, swiglu, out)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,Kd", [([1], 256, 4096), ([40], 512, 4096), ([48], 256, 8192), ([64, 4, 2], 256, 4096)])
def test_gathered_rows(counts, N, Kd, swiglu):
    g = torch.Generator().manual_seed(sum(counts) + Kd)
    w, ws = weights(g, len(counts), N, Kd, swiglu)
    offsets, cnt, rows = groups(counts)
    tokens, scales = rows_of(g, 19, Kd)
    src = torch.randint(0, 19 * 3, (rows,), generator=g).to(torch.int32).cuda()
    t = src.long() // 3
    x, xs = tokens.view(torch.uint8)[t].view(E4M3), scales[t]
    maps = dict(offsets=offsets, counts=cnt, swiglu=swiglu, status=_status())
    flat = moedc.matmul_e4m3(x, xs, w, ws, **maps)
    for more in ({}, dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        got = moedc.matmul_e4m3(tokens, scales, w, ws, src=src, top_k=3, **maps, **more)
        assert torch.equal(got, flat)
    assert int(maps["status"]) == 0
    _near(flat, x, xs, w, ws, offsets, counts, swiglu, "bf16")
