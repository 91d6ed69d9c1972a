"""Refusals of the router, the sum of the experts' outputs and the low-rank
adapters: every call below fails validation on the host (or has nothing to do),
so none reaches a device."""
from __future__ import annotations

import ctypes

import pytest
import torch

import packed_xor_popcount_amd as bnn

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_LAUNCH, E_ARG = range(7)
P = ctypes.c_void_p
FAKE = P(0x1000)
BIG = 2 ** 30


@pytest.fixture(scope="module")
def lib():
    return bnn.library()


def test_route_fwd_refusals(lib):
    need = lib.bnn_route_fwd_workspace(5000, 8, 2)  # few tokens need none
    assert need > 0 and lib.bnn_route_fwd_workspace(4, 8, 2) == 0
    assert all(lib.bnn_route_fwd_workspace(*s) == 0 for s in ((0, 8, 2), (-1, 8, 2), (5000, 0, 2), (5000, 1025, 2),
                                                              (BIG, 8, 2), (5000, 8, 0)))

    def f(z=FAKE, dt=0, ldz=8, valid=None, ex=FAKE, w=FAKE, pl=FAKE, rows=FAKE, off=FAKE, cnt=FAKE, st=FAKE, sl=FAKE,
          lo=FAKE, ws=FAKE, wb=need, T=5000, E=8, k=2, norm=1):
        return lib.bnn_route_fwd(z, dt, ldz, valid, ex, w, pl, rows, off, cnt, st, sl, lo, ws, wb, T, E, k, norm, None)
    assert f(dt=2) == E_DTYPE and f(norm=2) == E_ARG and f(norm=-1) == E_ARG
    for kw in (dict(T=-1), dict(T=BIG), dict(E=0, ldz=8), dict(E=1025, ldz=2000), dict(k=0), dict(k=9), dict(ldz=7),
               dict(ldz=BIG), dict(E=64, ldz=64, k=33), dict(T=BIG // 2, k=2), dict(wb=need - 1), dict(wb=-1)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("z", "ex", "w", "pl", "rows", "off", "cnt", "st", "sl", "lo", "ws"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(z=P(0x1002)), dict(dt=1, z=P(0x1001)), dict(ex=P(0x1002)), dict(w=P(0x1001)), dict(pl=P(0x1002)),
               dict(rows=P(0x1002)), dict(off=P(0x1002)), dict(cnt=P(0x1002)), dict(st=P(0x1002)), dict(sl=P(0x1002)),
               dict(lo=P(0x1002)), dict(ws=P(0x1008))):
        assert f(**kw) == E_ALIGN, kw


def test_route_bwd_refusals(lib):
    def f(z=FAKE, dt=0, ldz=8, ex=FAKE, w=FAKE, st=FAKE, sl=FAKE, dw=FAKE, dl=FAKE, dz=FAKE, lddz=8, T=4, E=8, k=2, norm=0):
        return lib.bnn_route_bwd(z, dt, ldz, ex, w, st, sl, dw, dl, dz, lddz, T, E, k, norm, None)
    assert f(dt=-1) == E_DTYPE and f(norm=3) == E_ARG
    for kw in (dict(T=-1), dict(T=BIG), dict(E=0), dict(E=1025, ldz=2000, lddz=2000), dict(k=0), dict(k=9), dict(ldz=7),
               dict(lddz=7), dict(ldz=BIG), dict(lddz=BIG)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("z", "ex", "w", "st", "sl", "dl", "dz"):
        assert f(**{k: None}) == E_NULL, k
    for k in ("z", "ex", "w", "st", "sl", "dw", "dl", "dz"):
        assert f(**{k: P(0x1002)}) == E_ALIGN, k
    none = dict(z=None, ex=None, w=None, st=None, sl=None, dw=None, dl=None, dz=None)
    assert f(T=0, **none) == OK


def test_combine_fwd_refusals(lib):
    def f(y=FAKE, dty=0, ldy=8, R=6, pl=FAKE, w=FAKE, res=FAKE, ldr=8, out=FAKE, dt=0, ldo=8, T=3, N=8, k=2):
        return lib.bnn_combine_fwd(y, dty, ldy, R, pl, w, res, ldr, out, dt, ldo, T, N, k, None)
    assert f(dt=2) == E_DTYPE and f(dty=2) == E_DTYPE and f(dty=-1) == E_DTYPE
    for kw in (dict(T=-1), dict(N=-1), dict(R=-1), dict(T=BIG), dict(R=BIG), dict(k=0), dict(ldy=7), dict(ldo=7),
               dict(ldr=7), dict(ldy=BIG), dict(T=2 ** 20, k=2 ** 10)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("y", "pl", "out"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(y=P(0x1002)), dict(out=P(0x1002)), dict(res=P(0x1002)), dict(pl=P(0x1002)), dict(w=P(0x1002)),
               dict(dty=1, y=P(0x1001)), dict(dt=1, out=P(0x1001)), dict(dt=1, res=P(0x1001))):
        assert f(**kw) == E_ALIGN, kw
    none = dict(y=None, pl=None, w=None, res=None, out=None)
    assert f(T=0, **none) == OK and f(N=0, **none) == OK


def test_combine_bwd_refusals(lib):
    def f(do=FAKE, dt=0, lddo=8, y=FAKE, ys=None, dty=0, ldy=8, R=6, pl=FAKE, w=FAKE, dy=FAKE, dtd=0, lddy=8, dw=FAKE, T=3,
          N=8, k=2):
        return lib.bnn_combine_bwd(do, dt, lddo, y, ys, dty, ldy, R, pl, w, dy, dtd, lddy, dw, T, N, k, None)
    assert f(dt=2) == E_DTYPE and f(dtd=2) == E_DTYPE and f(dty=3) == E_DTYPE
    for kw in (dict(T=-1), dict(N=-1), dict(R=-1), dict(R=BIG), dict(k=0), dict(lddo=7), dict(ldy=7), dict(lddy=7),
               dict(lddy=BIG), dict(T=2 ** 20, k=2 ** 10)):
        assert f(**kw) == E_SHAPE, kw
    for kw in (dict(do=None), dict(pl=None), dict(y=None), dict(dty=2, ys=None)):
        assert f(**kw) == E_NULL, kw
    for kw in (dict(do=P(0x1002)), dict(y=P(0x1002)), dict(pl=P(0x1002)), dict(w=P(0x1002)), dict(dy=P(0x1002)),
               dict(dw=P(0x1002)), dict(dty=2, ys=FAKE, y=P(0x1008)), dict(dty=2, ys=P(0x1002))):
        assert f(**kw) == E_ALIGN, kw
    assert f(T=0, do=None, pl=None, y=None, w=None, dy=None, dw=None) == OK
    assert f(dy=None, dw=None) == OK


def test_adapter_fwd_refusals(lib):
    need = lib.bnn_adapter_fwd_workspace(400, 4096, 8, 16, 2)  # few rows need none
    assert need > 0 and lib.bnn_adapter_fwd_workspace(4, 4096, 8, 16, 2) == 0
    assert all(lib.bnn_adapter_fwd_workspace(*s) == 0 for s in (
        (0, 4096, 8, 16, 2), (-1, 4096, 8, 16, 2), (400, -1, 8, 16, 2), (400, 4096, 8, 0, 2), (400, 4096, 8, 129, 2),
        (2 ** 27, 4096, 8, 16, 2), (400, 4096, -1, 16, 2), (400, 4096, 8, 16, 2 ** 20)))

    def f(x=FAKE, ldx=4096, ids=FAKE, a=FAKE, b=FAKE, sc=None, base=None, ldb=0, out=FAKE, ldo=8, dt=0, u=FAKE, ws=FAKE,
          wb=need, T=400, K=4096, N=8, r=16, L=2):
        return lib.bnn_adapter_fwd(x, ldx, ids, a, b, sc, base, ldb, out, ldo, dt, u, ws, wb, T, K, N, r, L, None)
    assert f(dt=2) == E_DTYPE
    for kw in (dict(T=-1), dict(K=-1), dict(N=-1), dict(T=2 ** 27), dict(N=BIG, ldo=BIG), dict(r=0), dict(r=129), dict(L=-1),
               dict(L=2 ** 20), dict(ldx=4095), dict(ldo=7), dict(base=FAKE, ldb=7), dict(wb=need - 1), dict(wb=-1),
               dict(base=FAKE, ldb=9), dict(ldx=BIG), dict(ldo=BIG)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("x", "ids", "a", "b", "out", "u", "ws"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(x=P(0x1001)), dict(ids=P(0x1002)), dict(a=P(0x1001)), dict(b=P(0x1001)), dict(sc=P(0x1002)),
               dict(base=P(0x1002), ldb=8), dict(out=P(0x1002)), dict(u=P(0x1002)), dict(ws=P(0x1008)),
               dict(dt=1, out=P(0x1001))):
        assert f(**kw) == E_ALIGN, kw
    none = dict(x=None, ids=None, a=None, b=None, out=None, u=None, ws=None, wb=0)
    assert f(T=0, **none) == OK


def test_adapter_bwd_refusals(lib):
    need = lib.bnn_adapter_bwd_workspace(4, 16, 8, 4, 2)
    assert need > 0
    assert all(lib.bnn_adapter_bwd_workspace(*s) == 0 for s in ((-1, 16, 8, 4, 2), (4, 16, 8, 0, 2), (4, 16, 8, 129, 2),
                                                                (4, 16, 8, 4, 1025), (2 ** 27, 16, 8, 4, 2)))

    def f(dy=FAKE, lddy=8, x=FAKE, xs=None, dtx=1, ldx=16, u=FAKE, ids=FAKE, a=FAKE, b=FAKE, sc=None, base=None, ldb=0,
          dx=FAKE, lddx=16, dt=0, da=FAKE, db=FAKE, ws=FAKE, wb=need, T=4, K=16, N=8, r=4, L=2):
        return lib.bnn_adapter_bwd(dy, lddy, x, xs, dtx, ldx, u, ids, a, b, sc, base, ldb, dx, lddx, dt, da, db, ws, wb, T,
                                   K, N, r, L, None)
    assert f(dt=2) == E_DTYPE and f(dtx=0) == E_DTYPE and f(dtx=3) == E_DTYPE
    for kw in (dict(T=-1), dict(K=-1), dict(N=-1), dict(T=2 ** 27), dict(r=0), dict(r=129), dict(L=-1), dict(L=1025),
               dict(lddy=7), dict(ldx=15), dict(lddx=15), dict(base=FAKE, ldb=15), dict(base=FAKE, ldb=17),
               dict(wb=need - 1)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("dy", "x", "u", "ids", "a", "b", "da", "db", "ws"):
        assert f(**{k: None}) == E_NULL, k
    assert f(dtx=2, xs=None) == E_NULL
    for kw in (dict(dy=P(0x1001)), dict(x=P(0x1001)), dict(u=P(0x1002)), dict(ids=P(0x1002)), dict(a=P(0x1001)),
               dict(b=P(0x1001)), dict(sc=P(0x1002)), dict(base=P(0x1002), ldb=16), dict(dx=P(0x1002)), dict(da=P(0x1002)),
               dict(db=P(0x1001)), dict(ws=P(0x1004)), dict(dtx=2, xs=FAKE, x=P(0x1008)), dict(dtx=2, xs=P(0x1002))):
        assert f(**kw) == E_ALIGN, kw
    assert f(dx=None, da=None, db=None) == OK
    assert f(T=0, da=None, db=None, dy=None, x=None, u=None, ids=None, a=None, b=None, dx=None) == OK


def test_bindings_refuse_cpu_tensors():
    z, i, f = torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    h, ids = torch.zeros(2, 4, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    w = torch.zeros(1, 3, 4, dtype=torch.bfloat16)
    for call in (lambda: bnn.route_fwd(z, 1), lambda: bnn.route_bwd(z, i, f, torch.zeros(2, 2)),
                 lambda: bnn.combine_fwd(z, i), lambda: bnn.combine_bwd(z, i, y=z),
                 lambda: bnn.adapter_fwd(h, ids, w, w), lambda: bnn.adapter_bwd(h, h, f, ids, w, w)):
        with pytest.raises(TypeError):
            call()


def test_combine_fwd_in_place_takes_one_stride(lib):
    """The output may be the residual with its own stride only: rows would be read after others were written."""
    def f(res, ldr, out, ldo, T=3):
        return lib.bnn_combine_fwd(FAKE, 0, 8, 6, FAKE, FAKE, res, ldr, out, 0, ldo, T, 8, 2, None)
    assert f(FAKE, 9, FAKE, 8) == E_SHAPE and f(FAKE, 8, FAKE, 9) == E_SHAPE
    assert f(FAKE, 8, FAKE, 8, T=0) == OK and f(FAKE, 8, P(0x2000), 9, T=0) == OK
    assert f(None, 8, FAKE, 9, T=0) == OK
