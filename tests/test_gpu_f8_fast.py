"""The 8-bit product on the 8-bit matrix instructions (fast=True) on the GPU.

Against the float64 product of the decoded operands
  |y - y64| <= (tol + cut)(1 + 2^-8) + 2^-8 |y64|,
tol = gamma(K + 8) sum|x w| the bound of an fp32 sum (u = 2^-23), and cut what
the instruction drops: inside a group of eight consecutive k, less than 2^-13
of the group's largest product from each of the other seven.
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn
from tests.test_gpu_f8 import DEV, SHAPES, U, decode, operand, small_integers
from tests.test_gpu_f8_range import PLACES, cancelling

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def run(x, w, K):
    y = bnn.gemm_f8(*x, *w, K, dtype=BF, fast=True)
    assert y.dtype == BF
    return y


def within(x, w, K):
    a, b = decode(*x, K), decode(*w, K)
    M, N = a.shape[0], b.shape[0]
    ref = a @ b.t()
    n = K + 8
    tol = n * U / (1 - n * U) * (a.abs() @ b.abs().t()) + K * 2.0 ** -126
    tol = tol + 7 * 2.0 ** -13 * (a.abs().view(M, -1, 8).amax(2) @ b.abs().view(N, -1, 8).amax(2).t())
    y = run(x, w, K)
    assert ((y.double() - ref).abs() <= tol * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8).all()
    assert torch.equal(y, run(x, w, K)), "not the same bits twice"


@pytest.mark.parametrize("M,N,K", SHAPES + [(2900, 2999, 300)])
def test_exact_and_bounded(M, N, K):
    print("fast", M, N, K, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + 2 * N + K)
    x, w = small_integers(g, M, K), small_integers(g, N, K)
    assert torch.equal(run(x, w, K), (decode(*x, K) @ decode(*w, K).t()).to(BF))
    within(operand(g, M, K), operand(g, N, K), K)


@pytest.mark.parametrize("M,N", PLACES)
def test_cancelling_groups(M, N):
    """Few rows keep the small products; on the instructions they are lost
    within the stated cut."""
    K = 300
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    x, w = cancelling(g, M, K, False), cancelling(g, N, K, True)
    within(x, w, K)
    if M <= 32:
        assert torch.equal(run(x, w, K), bnn.gemm_f8(*x, *w, K, dtype=BF))


@pytest.mark.parametrize("M,N", [(33, 70), (2900, 2999)])
def test_what_a_group_keeps(M, N):
    """1 - 1 + 2^-j in one group: kept down to 2^-13, then off by less than
    that; kept at any size in another group."""
    K = 128
    s = torch.full((max(M, N), 4), 127, dtype=torch.uint8, device=DEV)

    def q(rows, values):
        v = torch.zeros(rows, K, device=DEV)
        for at, x in values.items():
            v[:, at] = x
        return v.to(torch.float8_e4m3fn).view(torch.uint8), s[:rows]

    for j in range(0, 19):
        small = (2.0 ** -(j // 2), 2.0 ** -(j - j // 2))
        for at in (2, 7, 8, 100):
            y = run(q(M, {0: 1.0, 1: 1.0, at: small[0]}), q(N, {0: 1.0, 1: -1.0, at: small[1]}), K).double()
            if at >= 8 or j <= 13:
                assert (y == 2.0 ** -j).all(), (j, at, y[0, 0])
            else:
                assert ((y - 2.0 ** -j).abs() <= 2.0 ** -13).all(), (j, at, y[0, 0])


@pytest.mark.parametrize("M,N", [(5, 24), (40, 24), (300, 70), (2900, 2999)])
def test_every_scale(M, N):
    for e in range(-126, 127, 7):
        q = torch.full((M, 128), 0x38, dtype=torch.uint8, device=DEV)  # 1.0
        w = torch.full((N, 128), 0x40, dtype=torch.uint8, device=DEV)  # 2.0
        xs = torch.full((M, 4), 127 + e, dtype=torch.uint8, device=DEV)
        ws = torch.full((N, 4), 127 - e, dtype=torch.uint8, device=DEV)
        assert (run((q, xs), (w, ws), 128) == 256.0).all(), e


@pytest.mark.parametrize("M,N", [(20, 70), (300, 70), (2900, 2999)])
def test_nan_reaches_its_row_and_column_only(M, N):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x, w = torch.randn(M, 300, generator=g, device=DEV), torch.randn(N, 300, generator=g, device=DEV)
    ref = run(bnn.quant_f8(x), bnn.quant_f8(w), 300)
    x[M - 1, 299] = float("nan")
    w[33, 7] = float("inf")
    w[34, 8] = -float("inf")
    y = run(bnn.quant_f8(x), bnn.quant_f8(w), 300)
    bad = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    bad[M - 1] = True
    bad[:, 33:35] = True
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], ref[~bad])


def test_weights_past_32_bit_offsets():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    N, K = 1100000, 4096
    wq = torch.randint(0, 0x70, (4096, K), generator=g, device=DEV, dtype=torch.uint8)
    wq = wq.repeat(-(-N // 4096), 1)[:N].contiguous()
    ws = torch.full((N, 32), 120, dtype=torch.uint8, device=DEV)
    x = operand(g, 70, K)
    y = run(x, (wq, ws), K)
    within(x, (wq[:4096].contiguous(), ws[:4096].contiguous()), K)
    ref = decode(*x, K) @ decode(wq[:4096], ws[:4096], K).t()
    size = decode(*x, K).abs() @ decode(wq[:4096], ws[:4096], K).abs().t()
    tail = N - N % 4096
    for got, want, tol in ((y[:, :4096], ref, size), (y[:, tail:], ref[:, :N - tail], size[:, :N - tail])):
        assert ((got.double() - want).abs() <= tol * 2.0 ** -7).all()
    assert torch.equal(y[:, 4096:8192], y[:, :4096])


def test_empty_products():
    e, es = (torch.empty(0, n, dtype=torch.uint8, device=DEV) for n in (128, 4))
    q, s = bnn.quant_f8(torch.ones(3, 5, device=DEV))
    assert run((e, es), (q, s), 5).shape == (0, 3) and run((q, s), (e, es), 5).shape == (3, 0)
    z = torch.empty(40, 0, dtype=torch.uint8, device=DEV)
    for m in (3, 40):
        y = bnn.gemm_f8(z[:m], z[:m], z, z, 0, out=torch.full((m, 40), 9.0, device=DEV, dtype=BF), fast=True)
        assert not y.any()


def test_refusals():
    q, s = bnn.quant_f8(torch.ones(3, 5, device=DEV))
    with pytest.raises(TypeError):
        bnn.gemm_f8(q, s, q, s, 5, fast=True)  # fp32 outputs
    with pytest.raises(TypeError):
        bnn.gemm_f8(q, s, q, s, 5, out=torch.empty(3, 3, device=DEV), fast=True)
    with pytest.raises(ValueError):
        bnn.gemm_f8(q, s, q, s, 200, dtype=BF, fast=True)
