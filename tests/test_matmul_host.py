"""Host-side checks of the dense layers' C entry points (no GPU needed): argument errors
come back before anything is launched."""
import ctypes

import pytest

from combine_moedc_layout_gb300 import build as mbuild
from combine_moedc_layout_gb300 import moedc

P = ctypes.c_void_p
F = P(256)                 # never dereferenced: validation fails first
ODD = P(257)
HALF = P(264)              # 8-byte aligned


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return moedc.load()


def test_quant_arguments(lib):
    def quant(x=F, ld=256, dt=moedc.BF16, E=1, rows=4, Kd=256, block=1, codes=F, scales=F):
        return lib.moedc_quant_e4m3(x, ld, dt, E, rows, Kd, block, codes, scales, None)

    for bad in (dict(ld=255), dict(ld=260), dict(dt=moedc.FP8_E4M3), dict(dt=9), dict(E=0), dict(rows=-1), dict(Kd=0),
                dict(Kd=64), dict(Kd=200), dict(block=0), dict(block=64), dict(x=None), dict(x=HALF), dict(codes=None),
                dict(codes=HALF), dict(scales=None), dict(scales=ODD), dict(dt=moedc.F32, ld=258)):
        assert quant(**bad) == moedc.ERR_ARG, bad
    assert quant(rows=0) == moedc.OK


def test_e4m3_arguments(lib):
    def mm(x=F, xr=8, Kd=256, xs=F, lay=0, w=F, ws=F, E=2, N=128, flags=0, o=F, c=F, src=None, k=1, rows=8,
           dt=moedc.BF16, out=F, outs=F, st=F, ws_=None):
        return lib.moedc_matmul_e4m3(x, xr, Kd, xs, lay, w, ws, E, N, flags, o, c, src, k, rows, dt, out, outs, ws_, 0, st, None)

    for bad in (dict(x=None), dict(x=HALF), dict(xr=-1), dict(xr=7), dict(Kd=0), dict(Kd=192), dict(xs=None),
                dict(xs=ODD), dict(lay=3), dict(lay=moedc.SCALES_COL_MAJOR), dict(w=None), dict(w=HALF), dict(ws=None),
                dict(ws=ODD), dict(E=0), dict(E=2000), dict(N=0), dict(flags=2), dict(c=None), dict(o=None, c=None),
                dict(o=ODD), dict(c=ODD), dict(src=ODD), dict(src=F, k=0), dict(rows=-1), dict(o=None, rows=9, xr=9),
                dict(dt=moedc.F32), dict(dt=9), dict(out=None), dict(out=ODD), dict(ws_=HALF), dict(st=None), dict(st=ODD),
                dict(dt=moedc.FP8_E4M3, N=120), dict(dt=moedc.FP8_E4M3, outs=None), dict(dt=moedc.FP8_E4M3, out=HALF),
                dict(o=None, lay=moedc.SCALES_COL_MAJOR, src=F), dict(N=2 ** 30), dict(rows=2 ** 31 - 1, xr=2 ** 31 - 1, N=2 ** 20)):
        assert mm(**bad) == moedc.ERR_ARG, bad
    assert mm(rows=0, xr=0, x=None, xs=None, out=None) == moedc.OK
    assert mm(xr=0, src=F, x=None) == moedc.OK
    bytes_ = moedc.moedc_matmul_e4m3_workspace_bytes
    assert bytes_(256, 2, 640) == 640 * 256 + 640 * 2 * 4
    assert bytes_(256, 64, 640) == bytes_(200, 2, 640) == bytes_(256, 0, 640) == bytes_(256, 2, 0) == 0


def test_layer_arguments(lib):
    def mm(x=F, ld=64, dt=moedc.BF16, Kd=64, w=F, E=2, N=16, flags=0, o=F, c=F, rows=8, out=F, keep=None, st=F):
        return lib.moedc_matmul(x, ld, dt, Kd, w, E, N, flags, o, c, rows, out, keep, st, None)

    for bad in (dict(x=None), dict(x=HALF), dict(ld=63), dict(ld=68), dict(dt=moedc.F32), dict(dt=1), dict(Kd=0),
                dict(Kd=60), dict(w=None), dict(w=HALF), dict(E=0), dict(E=2000), dict(N=0), dict(N=12), dict(flags=2),
                dict(c=None), dict(o=None, c=None), dict(o=ODD), dict(o=None, rows=9), dict(rows=-1), dict(out=None),
                dict(out=HALF), dict(keep=F), dict(flags=1, keep=HALF), dict(st=None), dict(st=ODD)):
        assert mm(**bad) == moedc.ERR_ARG, bad
    assert mm(rows=0, x=None, out=None) == moedc.OK

    def grad(d=F, ldd=16, x=F, ldx=64, w=F, dt=moedc.BF16, Kd=64, E=2, N=16, o=F, c=F, rows=8, dx=F, dw=F,
             dwt=moedc.BF16, st=F):
        return lib.moedc_matmul_grad(d, ldd, x, ldx, w, dt, Kd, E, N, o, c, rows, dx, dw, dwt, st, None)

    for bad in (dict(d=None), dict(d=HALF), dict(ldd=15), dict(ldd=20), dict(x=None), dict(x=HALF), dict(ldx=56),
                dict(ldx=66), dict(w=None), dict(w=HALF), dict(dt=moedc.F32), dict(Kd=4), dict(N=4), dict(E=0),
                dict(c=None), dict(rows=-1), dict(dx=HALF), dict(dw=HALF), dict(dwt=moedc.F16), dict(st=None)):
        assert grad(**bad) == moedc.ERR_ARG, bad
    assert grad(rows=0, dw=None, d=None) == moedc.OK
    assert grad(dx=None, dw=None) == moedc.OK

    def act(dh=F, ld=16, p=F, dt=moedc.F16, rows=4, N=16, out=F):
        return lib.moedc_swiglu_grad(dh, ld, p, dt, rows, N, out, None)

    for bad in (dict(dh=None), dict(dh=HALF), dict(ld=8), dict(ld=20), dict(p=None), dict(p=HALF), dict(dt=moedc.F32),
                dict(rows=-1), dict(N=4), dict(out=None), dict(out=HALF)):
        assert act(**bad) == moedc.ERR_ARG, bad
    assert act(rows=0) == moedc.OK
