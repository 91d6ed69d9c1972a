"""Block-scaled 8-bit quantiser and product on the GPU.

The quantiser is exact but for one rounding per value, so it is compared value
by value and scale by scale with a float64 reference on the e4m3 grid.

The product: 8-bit products are exact and the sums are fp32, so against the
float64 product of the decoded operands
  |y - y64| <= gamma(K + 8) sum|x w| + 2^-126 K,   gamma(n) = n u / (1 - n u), u = 2^-23
(any order of the sum; u doubled for units that do not round to nearest).
bf16 outputs add their rounding, 2^-8 |y|, and what the 8-bit matrix
instruction cuts off: inside a group of eight consecutive k, bits below 2^-13
of the group's largest product, at most 7 2^-13 max|x| max|w| per group (a
measured property of the unit).  The product is exact wherever every partial sum is
representable (small integers under scales a few powers of two apart).
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -23


def decode(q, s, k):
    """Values of a block-scaled matrix in float64 from its bytes: the e4m3
    fields spelled out."""
    q = q.to(torch.int64)
    sign, ex, man = 1 - 2 * (q >> 7), (q >> 3) & 15, q & 7
    v = torch.where(ex > 0, (8 + man).double() * torch.exp2((ex - 10).double()), man.double() * 2.0 ** -9)
    v = torch.where((q & 127) == 127, torch.full_like(v, float("nan")), v) * sign
    nb = -(-k // 128)
    e = s[:, :nb].double() - 127
    return (v.reshape(q.shape[0], nb, 128) * torch.exp2(e).unsqueeze(2)).reshape(q.shape[0], nb * 128)


def quant64(x):
    """Reference: values (R, 128 nb) and scale bytes (R, nb) of real rows."""
    x = x.double()
    rows, k = x.shape
    nb = -(-k // 128)
    v = torch.zeros(rows, nb * 128, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(rows, nb, 128)
    mag = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)).amax(2)
    e = torch.zeros(rows, nb, dtype=torch.int64, device=x.device)
    for b in range(-127, 128):  # the smallest power of two that suffices
        e = torch.where((mag > 448 * 2.0 ** (b - 1)) if b > -127 else (mag > 0), torch.full_like(e, b), e)
    e = torch.where(mag == 0, torch.zeros_like(e), e)
    u = v * torch.exp2(-e.double()).unsqueeze(2)
    _, ex = torch.frexp(torch.where(u.isfinite(), u, torch.zeros_like(u)))
    step = torch.exp2((ex.clamp(min=-5) - 4).double())
    r = torch.round(u / step) * step  # round half to even
    r = torch.where(v.isfinite(), r, torch.full_like(r, float("nan")))
    return (r * torch.exp2(e.double()).unsqueeze(2)).reshape(rows, nb * 128), e + 127


def check_quant(x, transpose):
    q, s = bnn.quant_f8(x, transpose)
    src = x.t() if transpose else x
    R, K = src.shape
    nb = -(-K // 128)
    assert q.shape == (R, bnn.f8_row_bytes(K)) and s.shape == (R, bnn.f8_scale_bytes(K))
    val, sc = quant64(src)
    assert torch.equal(s[:, :nb].long(), sc)
    assert not s[:, nb:].any()
    got = decode(q, s, K)
    assert torch.equal(got.isnan(), val.isnan())
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(val, nan=0.0))
    assert not q[:, K:].any()


def spread(g, rows, k, dtype, pad=0, shift=0):
    """Rows of very different size, some zeros, in a wider buffer of NaN."""
    ld = k + pad
    buf = torch.full((shift + rows * ld,), float("nan"), dtype=dtype, device=DEV)
    v = buf[shift:].view(rows, ld)[:, :k]
    x = torch.randn(rows, k, generator=g, device=DEV) * torch.exp2(
        torch.randint(-30, 30, (rows, k), generator=g, device=DEV).float() / 4)
    x[torch.rand(rows, k, generator=g, device=DEV) < 0.05] = 0
    v.copy_(x.to(dtype))
    return v


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 128), (3, 127), (2, 129), (65, 64), (127, 200), (128, 513),
                                    (129, 1000), (1000, 129), (513, 66), (300, 1100), (1, 5000), (5000, 1)])
def test_quant_sizes(rows, k, dtype, transpose):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows * 13 + k)
    check_quant(spread(g, rows, k, DT[dtype]), transpose)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (4, 2), (64, 8)])
def test_quant_strides(pad, shift, dtype, transpose):
    g = torch.Generator(device=DEV)
    g.manual_seed(pad * 5 + shift)
    check_quant(spread(g, 150, 392, DT[dtype], pad, shift), transpose)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_quant_special_values(dtype, transpose):
    """Zero blocks, negative zeros, ties, the limits 448 and 1.75 of a scale,
    the largest and the smallest magnitudes, infinities and NaN."""
    rows = torch.zeros(12, 256, device=DEV)
    rows[1, :4] = torch.tensor([448.0, -448.0, 1.0625, -0.0])      # the largest value; a tie
    rows[2, :3] = torch.tensor([449.0, 1.0, 17.0])                 # past it: the next scale
    rows[3, :2] = torch.tensor([float("inf"), 3.0])
    rows[4, :3] = torch.tensor([float("nan"), -2.0, -float("inf")])
    rows[5] = float("inf")
    rows[6, :3] = torch.tensor([3.3895e38, 1.0, -3.3895e38])
    rows[7, :3] = torch.tensor([1.1755e-38, 9.2e-41, -2e-38])      # least normal and subnormals
    rows[8, 130] = 5.0                                             # a zero block beside another
    rows[9, :6] = torch.tensor([448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -5 * 2.0 ** -10, 2.0 ** -11])
    rows[10, :5] = torch.tensor([448.0, 17.0, 19.0, 23.0, 27.0])   # ties in a binade
    rows[11, :2] = torch.tensor([1e-45, -1e-45])
    x = rows.to(DT[dtype])
    check_quant(x.t().contiguous() if transpose else x, transpose)


def test_quant_rows_past_32_bit_offsets():
    ld, M = (1 << 20) + 8, 2100
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    x = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV).view(M, ld)[:, :200]
    x.copy_(torch.randn(M, 200, generator=g, device=DEV))
    for transpose in (False, True):
        a, b = bnn.quant_f8(x, transpose), bnn.quant_f8(x.contiguous(), transpose)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_quant_nothing():
    for shape in ((0, 5), (5, 0)):
        for transpose in (False, True):
            q, s = bnn.quant_f8(torch.empty(*shape, device=DEV), transpose)
            assert q.numel() == 0 and s.numel() == 0


# ---------------------------------------------------------------------------

def operand(g, rows, k):
    return bnn.quant_f8(torch.randn(rows, k, generator=g, device=DEV)
                        * torch.exp2(torch.randint(-3, 4, (rows, k), generator=g, device=DEV).float()))


def small_integers(g, rows, k):
    """q in {-4 .. 4}, scales 2^-1 .. 2^1: every partial sum of a product is a
    multiple of 1/4 below 64 K, exact in fp32 for K < 2^16."""
    nb = -(-k // 128)
    v = torch.randint(-4, 5, (rows, nb * 128), generator=g, device=DEV).float()
    v[:, k:] = 0
    q = v.to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.zeros(rows, bnn.f8_scale_bytes(k), dtype=torch.uint8, device=DEV)
    s[:, :nb] = torch.randint(126, 129, (rows, nb), generator=g, device=DEV).to(torch.uint8)
    s[:, nb:] = 255  # unused
    return q, s


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 4096, 4096), (1, 1501, 1000), (2, 33, 200), (3, 100, 129), (7, 65, 640),
          (8, 512, 512), (9, 300, 1100), (16, 128, 384), (17, 129, 256), (31, 257, 700), (33, 64, 1000),
          (64, 1000, 1000), (65, 63, 4096), (100, 513, 385), (128, 128, 8192), (130, 700, 896), (201, 1501, 1000),
          (256, 256, 1024), (257, 255, 1025), (300, 2049, 64), (512, 700, 512), (777, 1030, 2000), (1024, 1024, 1024),
          (1, 3, 20000), (40, 20000, 130), (2049, 40, 130)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact(M, N, K):
    print("gemm_f8 exact", M, N, K, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(M * 3 + N * 5 + K)
    xq, xs = small_integers(g, M, K)
    wq, ws = small_integers(g, N, K)
    ref = decode(xq, xs, K) @ decode(wq, ws, K).t()
    y = bnn.gemm_f8(xq, xs, wq, ws, K)
    assert y.dtype == torch.float32
    assert torch.equal(y.double(), ref)
    yb = bnn.gemm_f8(xq, xs, wq, ws, K, dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_rounding(M, N, K):
    print("gemm_f8", M, N, K, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    xq, xs = operand(g, M, K)
    wq, ws = operand(g, N, K)
    x, w = decode(xq, xs, K), decode(wq, ws, K)
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    n = K + 8
    tol = n * U / (1 - n * U) * size + K * 2.0 ** -126
    y = bnn.gemm_f8(xq, xs, wq, ws, K)
    assert ((y.double() - ref).abs() <= tol).all(), float(((y.double() - ref).abs() / tol).max())
    assert torch.equal(y, bnn.gemm_f8(xq, xs, wq, ws, K)), "not the same bits twice"
    yb = bnn.gemm_f8(xq, xs, wq, ws, K, dtype=torch.bfloat16)
    cut = 7 * 2.0 ** -13 * (x.abs().view(M, -1, 8).amax(2) @ w.abs().view(N, -1, 8).amax(2).t())
    assert ((yb.double() - ref).abs() <= tol + cut + (ref.abs() + cut) * 2.0 ** -8 * 1.01).all()


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_every_scale(M):
    """One block per scale byte: x scale 2^e, w scale 2^-e."""
    K = 128
    for e in range(-126, 127, 7):
        q = torch.full((M, 128), 0x38, dtype=torch.uint8, device=DEV)  # 1.0
        w = torch.full((24, 128), 0x40, dtype=torch.uint8, device=DEV)  # 2.0
        xs = torch.full((M, 4), 127 + e, dtype=torch.uint8, device=DEV)
        ws = torch.full((24, 4), 127 - e, dtype=torch.uint8, device=DEV)
        assert (bnn.gemm_f8(q, xs, w, ws, K) == 256.0).all(), e


@pytest.mark.parametrize("M", [1, 20, 300])
def test_nan_reaches_its_row_and_column_only(M):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x, w = torch.randn(M, 300, generator=g, device=DEV), torch.randn(70, 300, generator=g, device=DEV)
    ref = bnn.gemm_f8(*bnn.quant_f8(x), *bnn.quant_f8(w), 300)
    x2, w2 = x.clone(), w.clone()
    x2[M - 1, 299] = float("nan")
    w2[33, 7] = float("inf")
    y = bnn.gemm_f8(*bnn.quant_f8(x2), *bnn.quant_f8(w2), 300)
    bad = torch.zeros(M, 70, dtype=torch.bool, device=DEV)
    bad[M - 1] = True
    bad[:, 33] = True
    assert torch.equal(y.isnan(), bad)
    # a block that holds the bad value keeps the scale of its other values
    assert torch.equal(y[~bad], ref[~bad])


def test_empty_products():
    e = torch.empty(0, 128, dtype=torch.uint8, device=DEV)
    es = torch.empty(0, 4, dtype=torch.uint8, device=DEV)
    q, s = bnn.quant_f8(torch.ones(3, 5, device=DEV))
    assert bnn.gemm_f8(e, es, q, s, 5).shape == (0, 3)
    assert bnn.gemm_f8(q, s, e, es, 5).shape == (3, 0)
    z = torch.empty(3, 0, dtype=torch.uint8, device=DEV)
    for m in (1, 3):
        y = bnn.gemm_f8(z[:m], z[:m], z, z, 0, out=torch.full((m, 3), 9.0, device=DEV))
        assert not y.any()


def test_gradient_products():
    """The transposed quantiser gives the operands of both gradients: dX =
    dY W and dW = dY^T X, within the products' bound on the quantised values
    and (differences of the bilinear form are the products themselves) equal
    to the float64 products of the decoded operands."""
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    T, N, K = 190, 260, 390
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device=DEV)
    dy = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    for a, b, red in ((bnn.quant_f8(dy), bnn.quant_f8(w, transpose=True), N),
                      (bnn.quant_f8(dy, transpose=True), bnn.quant_f8(x, transpose=True), T)):
        p, q = decode(*a, red), decode(*b, red)
        y = bnn.gemm_f8(*a, *b, red)
        tol = (red + 8) * U / (1 - (red + 8) * U) * (p.abs() @ q.abs().t()) + red * 2.0 ** -126
        assert ((y.double() - p @ q.t()).abs() <= tol).all()
    assert torch.equal(decode(*bnn.quant_f8(w, transpose=True), N)[:, :N],
                       decode(*bnn.quant_f8(w.t().contiguous()), N)[:, :N])


def test_weights_past_32_bit_offsets():
    """A weight of more than 2^32 bytes; one token and a few rows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    N, K = 1100000, 4096
    wq = torch.randint(0, 0x70, (4096, K), generator=g, device=DEV, dtype=torch.uint8)
    wq = wq.repeat(-(-N // 4096), 1)[:N].contiguous()
    ws = torch.full((N, 32), 120, dtype=torch.uint8, device=DEV)
    for M in (1, 70):
        xq, xs = operand(g, M, K)
        y = bnn.gemm_f8(xq, xs, wq, ws, K)
        ref = bnn.gemm_f8(xq, xs, wq[:4096].contiguous(), ws[:4096].contiguous(), K)
        tail = N - N % 4096
        bound = 2 * (K + 8) * U / (1 - (K + 8) * U) * (decode(xq, xs, K).abs() @ decode(wq[:4096], ws[:4096], K).abs().t())
        assert ((y[:, :4096].double() - ref.double()).abs() <= bound).all()
        assert torch.equal(y[:, 4096:8192], y[:, :4096])
        assert ((y[:, tail:].double() - ref[:, :N - tail].double()).abs() <= bound[:, :N - tail]).all()
        del y


def test_side_stream():
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    x, w = torch.randn(300, 777, generator=g, device=DEV), torch.randn(200, 777, generator=g, device=DEV)
    ref = bnn.gemm_f8(*bnn.quant_f8(x), *bnn.quant_f8(w), 777)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = bnn.gemm_f8(*bnn.quant_f8(x), *bnn.quant_f8(w), 777)
    s.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("rows,k", [(2100, 2001), (2100, 2048), (4097, 1030), (257, 20001)])
def test_quant_many_tiles(rows, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + k)
    for dtype in DT.values():
        for pad in (0, 1):
            x = spread(g, rows, k, dtype, pad)
            for transpose in (False, True):
                check_quant(x, transpose)


@pytest.mark.parametrize("M,N,K", [(2900, 2999, 300), (3073, 2817, 1024), (5000, 2000, 129)])
def test_product_large(M, N, K):
    test_product_exact(M, N, K)
    test_product_rounding(M, N, K)
