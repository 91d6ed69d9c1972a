"""Sign-weight products grouped by expert on the GPU, against float64.

  * exact regime: integer activations, every partial sum exact in fp32, so the
    output is fp32(fp32(s * alpha) * row_scale) bit for bit (rounded once more
    for bf16 outputs);
  * general inputs: |y - y64| <= |alpha rs| (gamma(K + 4) sum|x| + K 2^-125)
    + 2^-22 |y64|, gamma(n) = n u / (1 - n u), u = 2^-23 (any order of the sum,
    u doubled for units that do not round to nearest; two multiplies), plus
    2^-8 |y64| for bf16 outputs.
Places that must not be used hold NaN (activations) or random bits (pads).
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -23
ALGOS = {"auto": bnn.ALGO_AUTO, "gemv": bnn.ALGO_GEMV, "mfma": bnn.ALGO_MFMA}


def signs(wp, k):
    at = torch.arange(k, device=wp.device)
    return (1 - 2 * ((wp[..., at // 64] >> (at % 64)) & 1)).double()


class Case:
    """Inputs of one call.  `counts`: rows of each expert; `lead`, `tail`:
    rows outside the groups; `gather`: rows come from a table."""

    def __init__(self, seed, counts, N, K, gather=False, pad=0, shift=0, integers=False, lead=0, tail=0,
                 alpha=True, row_scale=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        E, R = len(counts), lead + sum(counts) + tail
        self.N, self.K, self.E, self.R = N, K, E, R
        off = [lead]
        for c in counts:
            off.append(off[-1] + c)
        self.off = off
        self.offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        xrows = R // 2 + 3 if gather else R
        ld = K + pad
        buf = torch.full((shift + xrows * ld + 1,), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.x = buf[shift:shift + xrows * ld].view(xrows, ld)
        v = (torch.randint(-64, 65, (xrows, K), generator=g, device=DEV).float() if integers
             else torch.randn(xrows, K, generator=g, device=DEV))
        self.x[:, :K] = v.to(torch.bfloat16)
        self.rows = None
        self.src = torch.arange(R, device=DEV)
        if gather:
            used = max(1, xrows - 2)  # the last rows are never named: all NaN
            self.x[used:] = float("nan")
            self.src = torch.randint(0, used, (R,), generator=g, device=DEV)
            self.rows = self.src.to(torch.int32)
        self.wp = torch.empty(E, N, bnn.words(K), dtype=torch.int64, device=DEV)
        if K > 0:
            self.wp.view(torch.uint8).random_(0, 256, generator=g)
        self.alpha = torch.randn(E, N, generator=g, device=DEV) if alpha else None
        self.row_scale = torch.rand(R, generator=g, device=DEV) - 0.3 if row_scale else None

    def run(self, algo, dtype, out=None):
        return bnn.gemm_signw_grouped(self.x, self.wp, self.offsets, self.K, alpha=self.alpha, rows=self.rows,
                                      row_scale=self.row_scale, dtype=dtype, algo=algo, out=out)

    def sums(self):
        """Exact sums (R, N) and sums of magnitudes (R,) in float64."""
        x = self.x[self.src][:, :self.K].double()
        s = torch.zeros(self.R, self.N, dtype=torch.float64, device=DEV)
        for e in range(self.E):
            lo, hi = self.off[e], self.off[e + 1]
            if hi > lo:
                s[lo:hi] = x[lo:hi] @ signs(self.wp[e], self.K).t()
        return s, x.abs().sum(1, keepdim=True)

    def factors(self):
        a = torch.ones(self.R, self.N, device=DEV)
        for e in range(self.E):
            if self.alpha is not None:
                a[self.off[e]:self.off[e + 1]] = self.alpha[e]
        r = torch.ones(self.R, 1, device=DEV) if self.row_scale is None else self.row_scale[:, None]
        return a, r

    def inside(self):
        m = torch.zeros(self.R, dtype=torch.bool, device=DEV)
        m[self.off[0]:self.off[-1]] = True
        return m


def check(case, algo, dtype, integers):
    print("grouped", case.R, case.E, case.N, case.K, algo, dtype, flush=True)
    out = torch.full((case.R, case.N), 7.0, dtype=dtype, device=DEV)
    y = case.run(algo, dtype, out)
    assert y is out
    use = case.inside()
    assert (y[~use] == 7.0).all(), "rows outside the groups were written"
    s, size = case.sums()
    a, r = case.factors()
    if integers:
        ref = (s.float() * a) * r
        assert torch.equal(y[use], ref.to(dtype)[use])
    else:
        ref = s * a.double() * r.double()
        n = case.K + 4
        tol = (a * r).double().abs() * 1.0001 * (n * U / (1 - n * U) * size + case.K * 2.0 ** -125) \
            + 2.0 ** -22 * ref.abs()
        if dtype == torch.bfloat16:
            tol = tol * 1.01 + 2.0 ** -8 * ref.abs() + 2.0 ** -134
        bad = ~((y.double() - ref).abs() <= tol)[use]
        assert not bad.any(), (int(bad.sum()), float((y.double() - ref).abs()[use].max()))
    assert torch.equal(case.run(algo, dtype)[use], y[use]), "not the same bits twice"


SETS = {
    "one": [1], "lonely": [0, 0, 1, 0], "empty": [0, 0, 0], "small": [1, 2, 0, 3, 8, 9, 1],
    "tiles": [31, 32, 33, 0, 64, 65, 127, 128, 129], "skewed": [0, 700, 1, 0, 2, 0, 257, 0],
    "many": [i % 3 for i in range(130)], "wide": [300],
}


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("groups", list(SETS))
@pytest.mark.parametrize("N,K", [(1, 1), (33, 64), (64, 65), (100, 130), (257, 1000), (130, 2048)])
def test_groups(groups, N, K, algo):
    for integers in (True, False):
        c = Case(len(groups) + N + K, SETS[groups], N, K, gather=(N + K) % 2 == 0, integers=integers)
        for dtype in DT.values():
            check(c, ALGOS[algo], dtype, integers)


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (1, 1), (4, 2), (24, 8)])
@pytest.mark.parametrize("K", [7, 72, 300, 1088])
def test_strides_and_alignment(K, pad, shift, gather, algo):
    c = Case(K + pad + shift, [5, 0, 40, 140, 1], 70, K, gather, pad, shift, integers=True)
    check(c, ALGOS[algo], torch.float32, True)


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("alpha,row_scale", [(False, False), (True, False), (False, True)])
def test_optional_factors(alpha, row_scale, algo):
    for integers in (True, False):
        c = Case(5, [3, 0, 9, 70], 90, 200, integers=integers, alpha=alpha, row_scale=row_scale)
        for dtype in DT.values():
            check(c, ALGOS[algo], dtype, integers)


@pytest.mark.parametrize("algo", list(ALGOS))
def test_rows_outside_the_groups_stay(algo):
    for gather in (False, True):
        check(Case(6, [4, 0, 66], 65, 129, gather, lead=5, tail=37, integers=True), ALGOS[algo], torch.float32, True)


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("N,K,counts", [(1024, 4096, [1, 0, 1, 1, 0, 2]), (700, 1000, [60, 61, 90, 0, 100]),
                                        (520, 4160, [256, 300, 5]), (1100, 512, [513, 0, 255, 1])])
def test_larger(N, K, counts, algo):
    for integers in (True, False):
        c = Case(7, counts, N, K, gather=True, integers=integers, row_scale=False)
        for dtype in DT.values():
            check(c, ALGOS[algo], dtype, integers)


@pytest.mark.parametrize("algo", list(ALGOS))
def test_no_k(algo):
    c = Case(8, [2, 0, 3], 33, 0, lead=1)
    y = c.run(ALGOS[algo], torch.float32, torch.full((6, 33), 7.0, device=DEV))
    assert not y[1:].any() and (y[0] == 7.0).all()


def test_nothing():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(3, 5, 1, dtype=torch.int64, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert bnn.gemm_signw_grouped(x, w, off).shape == (0, 5)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    y = bnn.gemm_signw_grouped(x, w[:0].contiguous(), off[:1], out=torch.full((2, 5), 7.0, device=DEV))
    assert (y == 7.0).all()
    assert bnn.gemm_signw_grouped(x, torch.zeros(3, 0, 1, dtype=torch.int64, device=DEV), off).shape == (2, 0)


@pytest.mark.parametrize("algo", list(ALGOS))
def test_one_group_is_the_plain_product(algo):
    """One group over all rows: the same values as gemm_signw_bf16 (integers,
    so both are exact)."""
    c = Case(9, [77], 150, 777, integers=True, row_scale=False)
    ref = bnn.gemm_signw_bf16(c.x, c.wp[0], c.K, c.alpha[0].contiguous())
    assert torch.equal(c.run(ALGOS[algo], torch.float32), ref)


@pytest.mark.parametrize("algo", list(ALGOS))
def test_a_bad_row_stays_alone(algo):
    c = Case(10, [3, 40, 1, 9], 66, 200)
    ref = c.run(ALGOS[algo], torch.float32)
    c.x[17, 199] = float("nan")
    c.x[44, 0] = float("inf")
    y = c.run(ALGOS[algo], torch.float32)
    keep = [r for r in range(c.R) if r not in (17, 44)]
    assert torch.equal(y[keep], ref[keep])
    assert y[17].isnan().all() and not y[44].isfinite().any()


@pytest.mark.parametrize("algo", list(ALGOS))
def test_offsets_and_rows_out_of_range_touch_nothing_else(algo):
    """Clamped in the kernel: guard rows around the output and the table stay
    as they were, and the rows named properly are right."""
    c = Case(11, [4, 6, 5], 40, 100, integers=True, gather=True)
    ref = c.run(ALGOS[algo], torch.float32)
    guard = torch.full((c.R + 20, 40), 7.0, device=DEV)
    bad_rows = c.rows.clone()
    bad_rows[0], bad_rows[14] = -5, 2 ** 31 - 1
    c.rows = bad_rows
    y = c.run(ALGOS[algo], torch.float32, guard[10:10 + c.R])
    assert torch.equal(y[1:14], ref[1:14])
    for off in ([-7, 4, 10, 15], [0, 4, 10, 2 ** 31 - 1], [-2 ** 31, 4, 10, 99]):
        c.offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        y = c.run(ALGOS[algo], torch.float32, guard[10:10 + c.R])
        assert torch.equal(y[1:14], ref[1:14])
    for off in ([15, 10, 4, 0], [9, 2, 30, -1]):  # decreasing: any rows, but inside y
        c.offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        c.run(ALGOS[algo], torch.float32, guard[10:10 + c.R])
    assert (guard[:10] == 7.0).all() and (guard[10 + c.R:] == 7.0).all()


def test_weights_past_32_bit_offsets():
    """Experts whose packed words lie past 2^32 bytes."""
    E, N, K = 70, 16384, 32768
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    words = torch.randint(-2 ** 62, 2 ** 62, (1, N, K // 64), generator=g, device=DEV)
    wp = words.expand(E, N, K // 64).clone()
    wp[E - 1] = ~words[0]
    assert wp.numel() * 8 > 2 ** 32
    x = torch.randint(-8, 9, (40, K), generator=g, device=DEV).to(torch.bfloat16)
    for algo in ALGOS.values():
        for first in (2, 38):
            off = torch.tensor([0] + [first] * (E - 1) + [40], dtype=torch.int32, device=DEV)
            y = bnn.gemm_signw_grouped(x, wp, off, K, algo=algo)
            ref = bnn.gemm_signw_bf16(x, words[0].contiguous(), K)
            assert torch.equal(y[:first], ref[:first]) and torch.equal(y[first:], -ref[first:])


@pytest.mark.parametrize("algo", list(ALGOS))
def test_activations_past_32_bit_offsets(algo):
    ld, M, K = (1 << 20) + 8, 2100, 136
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    x = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV).view(M, ld)[:, :K]
    x.copy_(torch.randint(-8, 9, (M, K), generator=g, device=DEV))
    wp = torch.randint(-2 ** 62, 2 ** 62, (2, 70, 3), generator=g, device=DEV)
    off = torch.tensor([0, 900, M], dtype=torch.int32, device=DEV)
    a = bnn.gemm_signw_grouped(x, wp, off, K, algo=ALGOS[algo])
    b = bnn.gemm_signw_grouped(x.contiguous(), wp, off, K, algo=ALGOS[algo])
    assert torch.equal(a, b)


@pytest.mark.parametrize("algo", list(ALGOS))
def test_side_stream(algo):
    c = Case(12, [3, 40, 1, 9], 66, 200)
    ref = c.run(ALGOS[algo], torch.float32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = c.run(ALGOS[algo], torch.float32)
    s.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("counts,N,K", [([9000, 0, 4100], 2561, 130), ([140, 300, 17, 190], 1000, 1100),
                                        ([20, 9, 0, 30] * 20, 500, 600), ([1, 0, 7, 2] * 40, 300, 1030)])
def test_every_tile(counts, N, K, algo):
    """Groupings that reach each tile of both kernels."""
    for integers in (True, False):
        c = Case(13, counts, N, K, gather=True, pad=1, integers=integers)
        for dtype in DT.values():
            check(c, ALGOS[algo], dtype, integers)
