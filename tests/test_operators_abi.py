"""Refusals of the operators around the packed products: every call below
fails validation on the host (or has nothing to do), so none reaches a
device."""
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


def test_layernorm_fwd_refusals(lib):
    def f(x=FAKE, dt=0, ldx=8, g=None, b=None, y=FAKE, ldy=8, mu=None, r=None, M=2, N=8, eps=1e-5):
        return lib.bnn_layernorm_fwd(x, dt, ldx, g, b, y, ldy, mu, r, M, N, eps, None)
    assert f(dt=2) == E_DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(M=BIG), dict(N=BIG, ldx=BIG, ldy=BIG), dict(ldx=7), dict(ldy=7),
               dict(ldx=BIG), dict(N=0)):
        assert f(**kw) == E_SHAPE, kw
    for eps in (-1e-5, float("nan"), float("inf")):
        assert f(eps=eps) == E_ARG, eps
    assert f(x=None) == E_NULL and f(y=None) == E_NULL
    for kw in (dict(x=P(0x1002)), dict(y=P(0x1002)), dict(g=P(0x1002)), dict(b=P(0x1001)), dict(mu=P(0x1002)),
               dict(r=P(0x1001)), dict(dt=1, x=P(0x1001))):
        assert f(**kw) == E_ALIGN, kw
    assert f(x=None, y=None, M=0) == OK and f(x=None, y=None, M=0, N=0) == OK


def test_layernorm_bwd_refusals(lib):
    need = lib.bnn_layernorm_bwd_workspace(5000, 8)  # few rows need none
    assert need > 0
    assert all(lib.bnn_layernorm_bwd_workspace(m, n) == 0 for m, n in ((0, 8), (8, 0), (-1, 8), (BIG, 8), (8, BIG)))

    def f(dy=FAKE, lddy=8, x=FAKE, ldx=8, dt=0, g=None, mu=FAKE, r=FAKE, dx=FAKE, lddx=8, dg=FAKE, db=FAKE, ws=FAKE,
          wb=need, M=5000, N=8):
        return lib.bnn_layernorm_bwd(dy, lddy, x, ldx, dt, g, mu, r, dx, lddx, dg, db, ws, wb, M, N, None)
    assert f(dt=-1) == E_DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(M=BIG), dict(ldx=7), dict(lddy=7), dict(lddx=7), dict(lddx=BIG),
               dict(N=0), dict(wb=need - 1), dict(wb=-1)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("dy", "x", "mu", "r", "dx", "dg", "db", "ws"):
        assert f(**{k: None}) == E_NULL, k
    for k in ("dy", "x", "mu", "r", "dx", "dg", "db"):
        assert f(**{k: P(0x1002)}) == E_ALIGN, k
    assert f(ws=P(0x1008)) == E_ALIGN and f(g=P(0x1001)) == E_ALIGN
    assert f(dy=None, x=None, mu=None, r=None, dx=None, dg=None, db=None, ws=None, wb=0, M=0) == OK
    assert f(M=0, N=0, wb=0, ws=None) == OK


def test_bindings_refuse_cpu_tensors():
    x, v = torch.zeros(2, 3), torch.zeros(2)
    with pytest.raises(TypeError):
        bnn.layernorm_fwd(x)
    with pytest.raises(TypeError):
        bnn.layernorm_bwd(x, x, v, v)


def test_f8_sizes():
    for k in (-3, 0, 1, 127, 128, 129, 512, 513, 4096, 2 ** 29):
        nb = 0 if k <= 0 else -(-k // 128)
        assert bnn.f8_row_bytes(k) == 128 * nb
        assert bnn.f8_scale_bytes(k) == 4 * -(-nb // 4)
        assert bnn.library().bnn_f8_row_bytes(k) == 128 * nb
        assert bnn.library().bnn_f8_scale_bytes(k) == 4 * -(-nb // 4)


def test_quant_f8_refusals(lib):
    def f(x=FAKE, dt=0, rows=2, k=8, ld=8, t=0, q=FAKE, s=FAKE):
        return lib.bnn_quant_f8(x, dt, rows, k, ld, t, q, s, None)
    assert f(dt=2) == E_DTYPE
    assert f(t=2) == E_ARG and f(t=-1) == E_ARG
    for kw in (dict(rows=-1), dict(k=-1), dict(rows=BIG), dict(k=BIG, ld=BIG), dict(ld=7), dict(ld=BIG)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("x", "q", "s"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(x=P(0x1002)), dict(x=P(0x1001), dt=1), dict(q=P(0x1008)), dict(s=P(0x1002))):
        assert f(**kw) == E_ALIGN, kw
    assert f(x=None, q=None, s=None, rows=0) == OK and f(x=None, q=None, s=None, k=0) == OK


def test_gemm_f8_refusals(lib):
    def f(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, y=FAKE, dt=0, M=2, N=3, K=8):
        return lib.bnn_gemm_f8(xq, xs, wq, ws, y, dt, M, N, K, None)
    assert f(dt=3) == E_DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=BIG), dict(N=BIG), dict(K=BIG),
               dict(K=2 ** 24 + 1)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("xq", "xs", "wq", "ws", "y"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(xq=P(0x1008)), dict(wq=P(0x1004)), dict(xs=P(0x1002)), dict(ws=P(0x1001)), dict(y=P(0x1002)),
               dict(y=P(0x1001), dt=1)):
        assert f(**kw) == E_ALIGN, kw
    assert f(xq=None, xs=None, y=None, M=0) == OK and f(wq=None, ws=None, y=None, N=0) == OK


def test_f8_bindings_refuse():
    x = torch.zeros(2, 128)
    with pytest.raises(TypeError):
        bnn.quant_f8(x)
    with pytest.raises(TypeError):
        bnn.gemm_f8(x, x, x, x, 128)


def test_signw_grouped_refusals(lib):
    def f(x=FAKE, ldx=64, xrows=4, rows=None, off=FAKE, wp=FAKE, a=None, rs=None, y=FAKE, dt=0, R=4, E=2, N=3, K=64,
          algo=0):
        return lib.bnn_gemm_signw_grouped(x, ldx, xrows, rows, off, wp, a, rs, y, dt, R, E, N, K, algo, None)
    assert f(dt=5) == E_DTYPE
    assert f(algo=bnn.ALGO_TILED) == E_ARG and f(algo=9) == E_ARG
    for kw in (dict(R=-1), dict(E=-1), dict(N=-1), dict(K=-1), dict(xrows=-1), dict(R=BIG, xrows=4), dict(N=BIG),
               dict(K=BIG, ldx=BIG), dict(E=2 ** 20), dict(ldx=63), dict(ldx=BIG), dict(xrows=3),
               dict(xrows=0, rows=FAKE), dict(xrows=BIG)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("x", "off", "wp", "y"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(x=P(0x1001)), dict(rows=P(0x1002)), dict(off=P(0x1002)), dict(wp=P(0x1004)), dict(a=P(0x1002)),
               dict(rs=P(0x1001)), dict(y=P(0x1002)), dict(y=P(0x1001), dt=1)):
        assert f(**kw) == E_ALIGN, kw
    none = dict(x=None, off=None, wp=None, y=None)
    assert f(R=0, xrows=0, **none) == OK and f(E=0, **none) == OK and f(N=0, **none) == OK


def test_signw_grouped_binding_refuses():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bnn.gemm_signw_grouped(x, torch.zeros(1, 3, 1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32))
