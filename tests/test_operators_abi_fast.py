"""Refusals of the fast 8-bit product: every call below fails validation on the
host (or has nothing to do), so none reaches a device."""
from __future__ import annotations

import ctypes

import pytest
import torch

import packed_xor_popcount_amd as bnn

OK, E_NULL, E_SHAPE, E_ALIGN = 0, 1, 2, 4
P = ctypes.c_void_p
FAKE = P(0x1000)
BIG = 2 ** 30


def test_gemm_f8_fast_refusals():
    def f(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, y=FAKE, M=2, N=3, K=8):
        return bnn.library().bnn_gemm_f8_fast(xq, xs, wq, ws, y, M, N, K, None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=BIG), dict(N=BIG), dict(K=BIG), dict(K=2 ** 24 + 1)):
        assert f(**kw) == E_SHAPE, kw
    for k in ("xq", "xs", "wq", "ws", "y"):
        assert f(**{k: None}) == E_NULL, k
    for kw in (dict(xq=P(0x1008)), dict(wq=P(0x1004)), dict(xs=P(0x1002)), dict(ws=P(0x1001)), dict(y=P(0x1001))):
        assert f(**kw) == E_ALIGN, kw
    assert f(xq=None, xs=None, y=None, M=0) == OK and f(wq=None, ws=None, y=None, N=0) == OK


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 128)
    with pytest.raises(TypeError):
        bnn.gemm_f8(x, x, x, x, 128, dtype=torch.bfloat16, fast=True)
