// gemm_f8.hip -- product of two block-scaled 8-bit matrices (see f8.h):
//
//   y[m][n] = sum_b 2^(xs[m][b] + ws[n][b] - 254) sum_{k in block b} xq[m][k] wq[n][k]
//
// Two ways through the matrix cores, the second only where the caller asks for
// it (bnn_gemm_f8_fast):
//
//  * the values are widened to bf16 with their scale applied
//    (v_cvt_scalef32_pk_bf16_fp8: exact, an e4m3 significand has 4 bits) and
//    multiplied by v_mfma_f32_32x32x16_bf16, which keeps fp32 precision
//    throughout (products down to 2^-23 of the largest were measured to
//    count), at half the 8-bit rate.
//  * v_mfma_scale_f32_32x32x64_f8f6f4 takes the 8-bit values and the scale byte
//    of each operand row as they are.  Measured on this unit: the sum over
//    groups of eight consecutive k and onto the accumulator keeps fp32
//    precision, but inside a group the products are cut below 2^-13 of the
//    group's largest.  For normally distributed operands that is an error of
//    1.6e-5 of the result, a hundredth of a bf16 rounding; where the large
//    products of a group cancel, the small ones are lost.
//
// Lane l supplies row / column l % 32 and half of the k values of an
// instruction (which half is free as long as both operands agree).  Output
// layout of a 32 x 32 tile: lane l, register v -> row 8(v/4) + 4(l/32) + v%4,
// column l%32.
#include "bnn_internal.h"
#include "f8.h"

namespace bnn {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16_t;

__device__ __forceinline__ v16f mfma_f8(v8i a, v8i b, v16f c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Scale byte as the fp32 power of two.
__device__ __forceinline__ float pow2_of(int s) { return __uint_as_float((uint32_t)s << 23); }

// Eight e4m3 bytes times 2^(s - 127) as bf16, s given as pow2_of(s).
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Under scale byte 247 (2^120) and larger ones a value can decode to 2^128, past
// bf16's range (the quantiser makes it of magnitudes from 1.9375 * 2^127 on).
// The kernels note the largest scale byte that a wave meets, and a wave that met
// such a one computes its sums again here, with operands in two parts: twice the
// half of such a block's values, once those of other blocks and then zeros.
// Rare, so nothing is staged, and one copy of the arithmetic keeps the registers
// of the ordinary path: 4096 x 11008 x 4096 with 2^128 in one row of x 2.4 ms, in
// every row 4.4 ms (0.3 ms without).  The 8-bit instructions need none of this:
// they apply the scales past bf16's range.
constexpr uint32_t kF8Split = 247;

// Sums of 16 x 16 outputs over blocks b0, b0 + step, ...: xr, wr the lane's
// operand rows + 32 (lane / 16), xs, ws their scale bytes; lanes, instruction
// and output as in the few-row kernel.
__device__ __forceinline__ v4f split_16x16(const uint8_t *xr, const uint8_t *xs, const uint8_t *wr,
                                           const uint8_t *ws, int b0, int step, int nb) {
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = b0; b < nb; b += step) {
    const int64_t o = (int64_t)b * kF8Block;
    const uint32_t sx = xs[b], sw = ws[b];
    const bool bx = sx >= kF8Split, bw = sw >= kF8Split;
    const float fx = pow2_of(bx ? sx - 1 : sx), fw = pow2_of(bw ? sw - 1 : sw);
    const bool any_x = __any(bx), any_w = __any(bw);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // halves of the block, up to four times each
      if (((i & 1) && !any_x) || ((i & 2) && !any_w)) continue;
      const v4u x = *reinterpret_cast<const v4u *>(xr + o + 16 * (i >> 2));
      const v4u w = *reinterpret_cast<const v4u *>(wr + o + 16 * (i >> 2));
      const v4u p = x & (bx || !(i & 1) ? ~0u : 0u), q = w & (bw || !(i & 2) ? ~0u : 0u);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(p.x, p.y, fx), widen8(q.x, q.y, fw), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(p.z, p.w, fx), widen8(q.z, q.w, fw), acc, 0, 0, 0);
    }
  }
  return acc;
}

// ---------------------------------------------------------------------------
// Tiled kernel: WR x WC = 8 waves, each RB x CB tiles of 32 x 32.  Per step of
// 128 elements of K (one scale) the tile's rows of both operands and their
// scale bytes go straight from memory into one of NBUF LDS buffers (the
// format keeps rows 16-byte aligned); NBUF - 1 steps are in flight ahead of
// the one that is multiplied.  The 16-byte pieces of a row are swapped by half
// the row's number, so that 16 neighbouring rows meet all 64 banks (by the whole
// number, rows 8 apart collided; the conflict counter now reads 0).
//
// 4096 x 11008 x 4096, bf16 out, a launch among others: 293-302 us, 1.2 PFLOP/s (a
// large library product of bf16 matrices: 1.38); FAST 177 us, 2.09 PFLOP/s (a
// library product of one scale: 189 us).  The widening product's matrix cores
// are busy 56 % of the cycles (2.1 GHz); the rest goes to the widening between
// them and to a last round of 176 of 256 blocks.  256 x 4096 x 4096: 22 and 17 us.
// Bands of row tiles (below) took the large FAST product from 250 us.  Under
// about 100 tiles the steps' latency bounds it, 0.5 us each.

constexpr int kF8Threads = 512;

// 16 bytes per lane from base + off to LDS at lds + 16 * lane, past the
// registers (lds: a wave-uniform LDS byte address), or 4 bytes.  Counted by
// vmcnt, in order.
__device__ __forceinline__ void load_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}
__device__ __forceinline__ void load4_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}
// Waits until at most LEFT of this wave's loads are outstanding.
template <int LEFT>
__device__ __forceinline__ void lds_loads_done() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

template <int WR, int WC, int RB, int CB, int NBUF, bool FAST, typename T>
__global__ void __launch_bounds__(kF8Threads, 2)
    gemm_f8_kernel(const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs,
                   const uint8_t *__restrict__ wq, const uint8_t *__restrict__ ws,
                   T *__restrict__ y, int M, int N, int nb, int sb, int tiles_m, int64_t tiles) {
  static_assert(WR * WC == 8, "eight waves");
  constexpr int BM = WR * RB * 32, BN = WC * CB * 32;
  constexpr int PA = BM * 8 / kF8Threads, PB = BN * 8 / kF8Threads;  // loads of a thread per step
  static_assert(PA >= 1 && PB >= 1, "every thread stages");
  // Scale words (four steps' bytes) of the tile's BM + BN rows: a load of 64
  // rows per wave, the waves past the last row repeating others' loads, so
  // that every wave has the same number of loads in a step.
  constexpr int SROWS = BM + BN, SCHUNKS = SROWS / 64, LOADS = PA + PB + 1;
  static_assert(SROWS % 64 == 0 && SCHUNKS <= 8, "scale rows per wave");
  constexpr int A0 = 0, B0 = BM * 128, S0 = B0 + BN * 128, STEP = S0 + SROWS * 4;
  __shared__ __attribute__((aligned(16))) unsigned char lds[NBUF * STEP];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, h = lane >> 5;
  const int wm = (wave / WC) * (RB * 32), wn = (wave % WC) * (CB * 32);
  const int64_t ldq = (int64_t)nb * kF8Block;

  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    // Block b runs on XCD b % 8: each XCD takes a contiguous range of tiles (the
    // first tiles % 8 XCDs one more), in bands of eight row tiles, so that the
    // 32 blocks it runs at a time share 8 row and 4 column slabs in its L2.
    const int xcd = (int)(b & 7), extra = (int)(tiles & 7);
    const int64_t tile = xcd * (tiles >> 3) + (xcd < extra ? xcd : extra) + (b >> 3);
    const int64_t tiles_n = tiles / tiles_m;
    const int band = (int)(tile / (8 * tiles_n));
    const int high = tiles_m - 8 * band < 8 ? tiles_m - 8 * band : 8;
    const int64_t in = tile - 8 * tiles_n * band;
    const int m0 = (8 * band + (int)(in % high)) * BM, n0 = (int)(in / high) * BN;

    // Row offsets inside a tile fit 32 bits: 256 rows of at most 2^24 bytes.
    // Thread tid fills place tid + 512 i of the tile's pieces: row tid / 8 + 64 i,
    // place tid % 8, which holds piece (tid % 8) ^ (row / 2 % 8).
    const uint8_t *xt = xq + m0 * ldq, *wt = wq + n0 * ldq;
    const uint32_t piece = 16 * ((tid & 7) ^ ((tid >> 4) & 7));
    uint32_t ox[PA], ow[PB], os;
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = (tid >> 3) + i * (kF8Threads / 8);
      ox[i] = (uint32_t)(m0 + r < M ? r : M - 1 - m0) * (uint32_t)ldq + piece;
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int r = (tid >> 3) + i * (kF8Threads / 8);
      ow[i] = (uint32_t)(n0 + r < N ? r : N - 1 - n0) * (uint32_t)ldq + piece;
    }
    const int schunk = wave % SCHUNKS;  // scale rows 64 schunk .. + 63 of (X's, then W's)
    const bool sx = schunk < BM / 64;
    const uint8_t *st = sx ? xs + (int64_t)m0 * sb : ws + (int64_t)n0 * sb;
    {
      const int r = (sx ? schunk : schunk - BM / 64) * 64 + lane;
      const int most = sx ? M - 1 - m0 : N - 1 - n0;
      os = (uint32_t)(r < most ? r : most) * (uint32_t)sb;
    }
    const uint32_t lds0 = lds_address(lds);
    auto load = [&](int s, int buf) __attribute__((always_inline)) {
      const uint32_t l = lds0 + buf * STEP;
      const uint8_t *xb = xt + (int64_t)s * kF8Block, *wb = wt + (int64_t)s * kF8Block;
#pragma unroll
      for (int i = 0; i < PA; ++i)
        load_to_lds(xb, ox[i], l + A0 + wave * 1024 + i * (kF8Threads * 16));
#pragma unroll
      for (int i = 0; i < PB; ++i)
        load_to_lds(wb, ow[i], l + B0 + wave * 1024 + i * (kF8Threads * 16));
      load4_to_lds(st + (s & ~3), os, l + S0 + schunk * 256);
    };
    auto frag = [&](const unsigned char *buf, int row, int t) __attribute__((always_inline)) {
      const int p0 = ((4 * t + 2 * h) ^ (li >> 1 & 7)) << 4, p1 = ((4 * t + 2 * h + 1) ^ (li >> 1 & 7)) << 4;
      const uint4 lo = *reinterpret_cast<const uint4 *>(buf + row * 128 + p0);
      const uint4 hi = *reinterpret_cast<const uint4 *>(buf + row * 128 + p1);
      return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
                 (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    v16f acc[RB][CB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    uint32_t top = 0;  // largest scale byte met
    auto compute = [&](int s, int buf) __attribute__((always_inline)) {
      const unsigned char *as = lds + buf * STEP + A0, *bs = lds + buf * STEP + B0;
      const unsigned char *sc = lds + buf * STEP + S0 + (s & 3);
      uint32_t ca[RB], cw[CB];
#pragma unroll
      for (int i = 0; i < RB; ++i) ca[i] = sc[(wm + i * 32 + li) * 4];
#pragma unroll
      for (int i = 0; i < CB; ++i) cw[i] = sc[(BM + wn + i * 32 + li) * 4];
      if (!FAST) {
#pragma unroll
        for (int i = 0; i < RB; ++i) top = ca[i] > top ? ca[i] : top;
#pragma unroll
        for (int i = 0; i < CB; ++i) top = cw[i] > top ? cw[i] : top;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v8i fa[RB], fb[CB];
#pragma unroll
        for (int j = 0; j < CB; ++j) fb[j] = frag(bs, wn + j * 32 + li, t);
#pragma unroll
        for (int i = 0; i < RB; ++i) fa[i] = frag(as, wm + i * 32 + li, t);
        if (FAST) {
#pragma unroll
          for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j)
              acc[i][j] = mfma_f8(fa[i], fb[j], acc[i][j], (int)ca[i], (int)cw[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bf16x8 va[RB], vb[CB];
#pragma unroll
            for (int j = 0; j < CB; ++j)
              vb[j] = widen8(fb[j][2 * k], fb[j][2 * k + 1], pow2_of(cw[j]));
#pragma unroll
            for (int i = 0; i < RB; ++i)
              va[i] = widen8(fa[i][2 * k], fa[i][2 * k + 1], pow2_of(ca[i]));
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
              for (int j = 0; j < CB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[i], vb[j], acc[i][j], 0, 0, 0);
          }
        }
      }
    };
    // Loads past the last step read it again (in bounds, into a buffer that
    // nobody reads), so that the waits' counts stay exact.
    __syncthreads();  // the last tile's reads of LDS are done
    if (nb > 0) {
      const int last = nb - 1;
#pragma unroll
      for (int d = 0; d < NBUF - 1; ++d) load(d < last ? d : last, d);
      int buf = 0;
      for (int s = 0; s < nb; ++s) {
        lds_loads_done<LOADS *(NBUF - 2)>();
        __syncthreads();  // step s has arrived; everyone is done with step s - 1
        const int into = buf == 0 ? NBUF - 1 : buf - 1;
        load(s + NBUF - 1 < last ? s + NBUF - 1 : last, into);
        compute(s, buf);
        buf = buf == NBUF - 1 ? 0 : buf + 1;
      }
      lds_loads_done<0>();
    }

    if (!FAST && __any(top >= kF8Split)) {
      const int l16 = lane & 15, g = lane >> 4;
#pragma unroll 1
      for (int t = 0; t < RB * CB * 4; ++t) {
        const int mt = m0 + wm + 16 * (t / (2 * CB)), nt = n0 + wn + 16 * (t % (2 * CB));
        const int m = mt + l16 < M ? mt + l16 : M - 1, n = nt + l16 < N ? nt + l16 : N - 1;
        const v4f sum = split_16x16(xq + m * ldq + 32 * g, xs + (int64_t)m * sb,
                                    wq + n * ldq + 32 * g, ws + (int64_t)n * sb, 0, 1, nb);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (mt + 4 * g + v < M && nt + l16 < N)
            y[(int64_t)(mt + 4 * g + v) * N + nt + l16] = (T)sum[v];
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + wm + i * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m >= M) continue;
        T *yr = y + (int64_t)m * N + n0 + wn + li;
#pragma unroll
        for (int j = 0; j < CB; ++j)
          if (n0 + wn + j * 32 + li < N) yr[j * 32] = (T)acc[i][j][v];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// ---------------------------------------------------------------------------
// Few-row kernel: 16 columns x 16 RM rows per block, the blocks of K dealt out
// to the block's waves and their sums joined through LDS in a fixed order.
// Every wave streams its part of the weight rows from memory exactly once, so
// small products keep the whole card busy.  1 x 4096 x 4096: 7.4 us, two blocks of K
// a wave one after the other; 1 x 65536 x 4096: 60 us, 4.5 TB/s, the weights' bytes.
// Always on bf16 instructions: the matrix rate does not matter here.
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row / column l % 16; lane group
// l / 16 takes bytes 32 (l / 16) .. + 31 of a block of 128, eight per
// instruction.  Output: register v -> row 4 (l / 16) + v, column l % 16.

template <int RM, typename T>
__global__ void __launch_bounds__(1024)
    gemm_f8_rows_kernel(const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs,
                        const uint8_t *__restrict__ wq, const uint8_t *__restrict__ ws,
                        T *__restrict__ y, int M, int N, int nb, int sb, int64_t tiles_n,
                        int64_t tiles) {
  __shared__ float join[16][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int li = lane & 15, g = lane >> 4;
  const int64_t ldq = (int64_t)nb * kF8Block;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n0 = (int)(tile % tiles_n) * 16, m0 = (int)(tile / tiles_n) * (16 * RM);
    const int n = n0 + li < N ? n0 + li : N - 1;
    const uint8_t *wr = wq + n * ldq + 32 * g, *wsr = ws + (int64_t)n * sb;
    const uint8_t *xr[RM], *xsr[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int m = m0 + i * 16 + li < M ? m0 + i * 16 + li : M - 1;
      xr[i] = xq + m * ldq + 32 * g;
      xsr[i] = xs + (int64_t)m * sb;
    }
    v4f acc[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t top = 0;  // largest scale byte met
    for (int b = wave; b < nb; b += waves) {
      const int64_t o = (int64_t)b * kF8Block;
      const v4u w0 = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wr + o));
      const v4u w1 = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(wr + o + 16));
      const uint32_t cw = wsr[b];
      top = cw > top ? cw : top;
      const float sw = pow2_of(cw);
      const bf16x8 vb[4] = {widen8(w0.x, w0.y, sw), widen8(w0.z, w0.w, sw),
                            widen8(w1.x, w1.y, sw), widen8(w1.z, w1.w, sw)};
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const v4u a0 = *reinterpret_cast<const v4u *>(xr[i] + o);
        const v4u a1 = *reinterpret_cast<const v4u *>(xr[i] + o + 16);
        const uint32_t cx = xsr[i][b];
        top = cx > top ? cx : top;
        const float sx = pow2_of(cx);
        const bf16x8 va[4] = {widen8(a0.x, a0.y, sx), widen8(a0.z, a0.w, sx),
                              widen8(a1.x, a1.y, sx), widen8(a1.z, a1.w, sx)};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va[k], vb[k], acc[i], 0, 0, 0);
      }
    }
    if (__any(top >= kF8Split)) {
#pragma unroll
      for (int i = 0; i < RM; ++i) acc[i] = split_16x16(xr[i], xsr[i], wr, wsr, wave, waves, nb);
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      __syncthreads();  // join is free
#pragma unroll
      for (int v = 0; v < 4; ++v) join[wave][(4 * g + v) * 16 + li] = acc[i][v];
      __syncthreads();
      for (int e = threadIdx.x; e < 256; e += blockDim.x) {
        float sum = 0.0f;
        for (int w = 0; w < waves; ++w) sum += join[w][e];
        const int m = m0 + i * 16 + (e >> 4), c = n0 + (e & 15);
        if (m < M && c < N) y[(int64_t)m * N + c] = (T)sum;
      }
    }
  }
}

template <int RM, typename T>
void launch_rows(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                 void *y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const int64_t tiles_n = (N + 15) / 16, tiles = tiles_n * ((M + 16 * RM - 1) / (16 * RM));
  const int64_t blocks = tiles < (1 << 20) ? tiles : (1 << 20);
  const int64_t nb = f8_blocks(K);
  const int waves = nb >= 16 ? 16 : (nb < 1 ? 1 : (int)nb);
  hipLaunchKernelGGL((gemm_f8_rows_kernel<RM, T>), dim3((unsigned)blocks), dim3(64 * waves), 0, s,
                     xq, xs, wq, ws, static_cast<T *>(y), (int)M, (int)N, (int)nb,
                     (int)f8_scale_bytes(K), tiles_n, tiles);
}

template <int WR, int WC, int RB, int CB, int NBUF, bool FAST, typename T>
void launch_tile(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                 void *y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  constexpr int BM = WR * RB * 32, BN = WC * CB * 32;
  const int64_t tiles_m = (M + BM - 1) / BM, tiles = tiles_m * ((N + BN - 1) / BN);
  const int64_t blocks = tiles < (1 << 20) ? tiles : (1 << 20);
  hipLaunchKernelGGL((gemm_f8_kernel<WR, WC, RB, CB, NBUF, FAST, T>), dim3((unsigned)blocks),
                     dim3(kF8Threads), 0, s, xq, xs, wq, ws, static_cast<T *>(y), (int)M, (int)N,
                     (int)f8_blocks(K), (int)f8_scale_bytes(K), (int)tiles_m, tiles);
}

template <bool FAST, typename T>
void launch(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, void *y,
            int64_t M, int64_t N, int64_t K, hipStream_t s) {
  // Large tiles once the outputs fill enough of them, whole or not; measured
  // (device, bf16 out, small against large tiles, and the same FAST):
  //   2048 x 4096 x 4096 (128 of them)  77 / 89 us    62 / 54 us
  //   300 x 30000 x 2048 (137)          49 / 55       36 / 34
  //   3000 x 5000 x 1000 (229)          45 / 33       33 / 23
  //   4096 x 4096 x 4096 (256)         154 / 105     124 / 60
  //   33 x 65536 x 1024 (33, of 256)    15 / 29       13 / 19
  // Few-row kernel against small tiles: 33 x 4096 x 4096 18 / 21 us, 64 rows 22 /
  // 21, 33 x 65536 x 1024 48 / 15.
  const int64_t filled = M * N / (256 * 256);
  auto run = launch_tile<2, 4, 4, 2, 2, FAST, T>;
  if (M <= 16) run = launch_rows<1, T>;
  else if (M <= 32) run = launch_rows<2, T>;
  else if (filled < (FAST ? 128 : 160)) run = launch_tile<2, 4, 1, 1, 3, FAST, T>;
  run(xq, xs, wq, ws, y, M, N, K, s);
}

}  // namespace

hipError_t launch_gemm_f8(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                          const uint8_t *ws, void *y, int dtype, bool fast, int64_t M, int64_t N,
                          int64_t K, hipStream_t s) {
  const auto run = dtype == BNN_FP32 ? launch<false, float>
                   : fast            ? launch<true, bf16_t>
                                     : launch<false, bf16_t>;
  run(xq, xs, wq, ws, y, M, N, K, s);
  return hipGetLastError();
}

}  // namespace bnn
