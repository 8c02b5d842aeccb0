"""Host-side checks of the language-model operators' C entry points (no GPU
needed): argument errors come back before anything is launched, and the size
queries follow their formulas."""
import ctypes

import pytest

from combine_moedc_layout_gb300 import build as mbuild
from combine_moedc_layout_gb300 import moedc

P = ctypes.c_void_p
F = P(256)                 # never dereferenced: validation fails first
ODD = P(257)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return moedc.load()


def test_sizes(lib):
    assert moedc.moedc_sort_rows(16, 8, 128, 1) == 128
    assert moedc.moedc_sort_rows(16, 8, 128, 16) == 128 + 128 * 15
    assert moedc.moedc_sort_rows(4, 2, 128, 16) == 8 + 8 * 15       # at most 8 experts filled
    assert moedc.moedc_sort_rows(0, 8, 128, 16) == 0
    for bad in [(16, 0, 8, 1), (16, 33, 64, 1), (16, 2, 2000, 1), (16, 2, 8, 0), (16, 2, 8, 2048)]:
        assert moedc.moedc_sort_rows(*bad) == 0
    assert moedc.moedc_sort_rows((1 << 24) // 32, 32, 1024, 1024) == (1 << 24) + 1024 * 1023
    assert moedc.moedc_sort_workspace_bytes(16, 0, 8) == 0
    for T, K, E in [(0, 1, 1), (1, 1, 1), (16, 8, 128), (4096, 8, 256), (40000, 8, 128)]:
        assert moedc.moedc_sort_workspace_bytes(T, K, E) >= \
            4 * T * K + T + 4 + moedc.moedc_layout_workspace_bytes(T, K, E, 1)


def test_gate_arguments(lib):
    def gate(l=F, ld=16, dt=moedc.F32, T=4, E=16, K=2, bias=None, flags=0, idx=F, w=F):
        return lib.moedc_gate(l, ld, dt, T, E, K, bias, flags, 1.0, idx, w, None)

    for bad in (dict(ld=15), dict(dt=moedc.FP8_E4M3), dict(dt=9), dict(T=-1), dict(E=0),
                dict(E=2000, ld=2000), dict(K=0), dict(K=17), dict(K=33, E=64, ld=64),
                dict(flags=2), dict(flags=0x20), dict(l=None), dict(l=ODD), dict(idx=None),
                dict(w=ODD), dict(bias=ODD)):
        assert gate(**bad) == moedc.ERR_ARG, bad
    assert gate(T=0) == moedc.OK

    def grad(ld=16, dt=moedc.F32, T=4, E=16, K=2, idx=F, dw=F, dl=F):
        return lib.moedc_gate_grad(F, ld, dt, T, E, K, None, 0, 1.0, idx, dw, dl, None)

    for bad in (dict(ld=8), dict(dt=1), dict(K=0), dict(idx=None), dict(dw=None), dict(dl=None),
                dict(dl=P(258)), dict(dw=ODD)):
        assert grad(**bad) == moedc.ERR_ARG, bad


def test_sort_arguments(lib):
    def sort(x=F, ldx=64, dt=moedc.BF16, T=4, H=64, idx=F, K=2, E=8, align=1, rows=8, out=F,
             row=F, src=F, off=F, cnt=F, ws=F, wsb=1 << 20, st=F):
        return lib.moedc_sort(x, ldx, dt, T, H, idx, K, E, align, rows, out, row, src, off, cnt,
                              ws, wsb, st, None)

    for bad in (dict(dt=1), dict(H=0), dict(T=-1), dict(K=0), dict(K=33), dict(E=0), dict(E=1025),
                dict(align=0), dict(align=1025), dict(rows=-1), dict(ldx=63), dict(x=None),
                dict(out=None), dict(idx=None), dict(row=None), dict(src=None), dict(off=None),
                dict(cnt=None), dict(st=None), dict(ws=None), dict(wsb=16), dict(ws=P(264)),
                dict(x=ODD), dict(out=ODD), dict(row=P(258)), dict(dt=moedc.F32, x=P(258))):
        assert sort(**bad) == moedc.ERR_ARG, bad

    def unsort(s=F, dt=moedc.BF16, rows=8, H=64, row=F, w=F, T=4, K=2, y=F):
        return lib.moedc_unsort(s, dt, rows, H, row, w, T, K, y, None)

    for bad in (dict(s=None), dict(dt=1), dict(rows=-1), dict(H=0), dict(row=None), dict(T=-1),
                dict(K=0), dict(K=33), dict(y=None), dict(y=ODD), dict(w=P(258))):
        assert unsort(**bad) == moedc.ERR_ARG, bad
    assert unsort(T=0) == moedc.OK

    def grad(dy=F, ld=64, s=F, dt=moedc.BF16, T=4, H=64, K=2, row=F, src=F, w=F, rows=8, ds=F,
             dw=F):
        return lib.moedc_unsort_grad(dy, ld, s, dt, T, H, K, row, src, w, rows, ds, dw, None)

    for bad in (dict(dy=None), dict(ld=63), dict(s=None), dict(dt=7), dict(T=-1), dict(H=0),
                dict(K=0), dict(row=None), dict(src=None), dict(w=None), dict(rows=-1),
                dict(ds=None), dict(dw=P(258)), dict(ds=ODD)):
        assert grad(**bad) == moedc.ERR_ARG, bad
    assert grad(T=0, rows=0) == moedc.OK


def test_matvec_arguments(lib):
    def mv(x=F, ldx=256, dt=moedc.BF16, xr=4, Kd=256, wq=F, s=F, sdt=moedc.BF16, z=None, g=64,
           E=2, N=16, flags=0, off=F, cnt=F, src=None, k=1, rows=4, out=F, ws=F, wsb=1 << 20,
           st=F):
        return lib.moedc_matvec_int4(x, ldx, dt, xr, Kd, wq, s, sdt, z, g, E, N, flags, off, cnt,
                                     src, k, rows, out, ws, wsb, st, None)

    for bad in (dict(x=None), dict(ldx=255), dict(ldx=260), dict(dt=moedc.F32), dict(dt=1),
                dict(xr=-1), dict(Kd=0), dict(Kd=288), dict(wq=None), dict(wq=P(264)),
                dict(s=None), dict(s=ODD), dict(sdt=1), dict(g=16), dict(g=256), dict(g=0),
                dict(E=0), dict(E=1025), dict(N=0), dict(flags=2), dict(off=None),
                dict(cnt=None), dict(off=None, cnt=None), dict(src=F, k=0), dict(rows=-1),
                dict(out=None), dict(out=ODD), dict(st=None), dict(x=P(264)),
                dict(N=1 << 30, E=4)):
        assert mv(**bad) == moedc.ERR_ARG, bad
    # 8 experts of 65536 x 256 weights: beyond the form that needs no workspace
    big = dict(E=8, N=1 << 16, rows=8)
    for bad in (dict(ws=None), dict(ws=P(264)), dict(wsb=5 * 576 - 1)):
        assert mv(**big, **bad) == moedc.ERR_ARG, bad
    assert mv(rows=0) == moedc.OK
    # one record of 576 bytes per row and 256 channels, and a row of zeros
    size = moedc.moedc_matvec_int4_workspace_bytes
    assert size(4, 256, 8, 1 << 16, 0, 8) == 5 * 576
    assert size(1, 288, 8, 1 << 16, 1, 8) == 2 * 2 * 576
    assert size(4, 256, 2, 16, 0, 4) == 0                     # few weights: none
    assert size(-1, 256, 8, 1 << 16, 0, 8) == 0 and size(4, 256, 8, 1 << 16, 2, 8) == 0
