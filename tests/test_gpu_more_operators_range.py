"""Router, sum of the experts' outputs and adapters at the ends of fp32's range:
magnitudes that overflow on the way only, infinities and NaN.

Every value below is a power of two (or a short sum of them), so that products
and sums are exact and results are equal."""
from __future__ import annotations

import math

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
INF = math.inf


# 1, 8 and 9 columns of a row, the last of a block, three blocks; few tokens (four waves
# each) and many (one wave each)
@pytest.mark.parametrize("T", [3, 4100])
@pytest.mark.parametrize("N", [1, 8, 9, 128, 300])
def test_sum_of_experts_from_8_bits_takes_large_gradients(T, N):
    y = torch.zeros(T, N, device=DEV)
    y[:, N - 1], y[:, N // 2] = 2.0 ** -20, -2.0 ** -19
    dout = torch.full((T, N), 2.0 ** 120, device=DEV)
    place = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).view(T, 1).contiguous()
    _, want = bnn.combine_bwd(dout, place, y=y)
    dy, dw = bnn.combine_bwd(dout, place, y=bnn.quant_f8(y))
    assert torch.isfinite(want).all()
    assert torch.equal(dw, want) and torch.equal(dy, dout)


@pytest.mark.parametrize("byte", [0, 1, 60, 127, 200, 245, 246, 247, 250, 255])
def test_sum_of_experts_from_8_bits_at_every_scale(byte):
    """448, its negative and the smallest value under a scale of 2^(byte - 127), each times the power
    of two that takes the product to about 1 (or as near as fp32's range lets it)."""
    q = torch.zeros(3, 128, dtype=torch.float8_e4m3fn, device=DEV)
    q[0, 5], q[1, 127], q[2, 64] = 448.0, -448.0, 2.0 ** -9
    s = torch.zeros(3, 4, dtype=torch.uint8, device=DEV)
    s[:, 0] = byte
    up = max(-126, min(127, 127 - byte - 8))
    dout = torch.zeros(3, 128, device=DEV)
    dout[:2] = 2.0 ** up
    up2 = max(-126, min(127, 127 - byte + 9))
    dout[2] = 2.0 ** up2
    place = torch.arange(3, dtype=torch.int32, device=DEV).view(3, 1)
    _, dw = bnn.combine_bwd(dout, place, y=(q.view(torch.uint8), s))
    want = [448 * 2.0 ** (byte - 127 + up), -448 * 2.0 ** (byte - 127 + up), 2.0 ** (byte - 127 - 9 + up2)]
    assert dw.flatten().tolist() == want
