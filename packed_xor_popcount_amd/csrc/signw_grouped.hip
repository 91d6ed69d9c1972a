// signw_grouped.hip -- sign-weight products grouped by expert:
//
//   y[r][n] = rs[r] * alpha[e][n] * sum_k x[src(r)][k] * w_e,n[k],   off[e] <= r < off[e + 1]
//
// with x real bf16 rows (src(r) = rows[r], or r itself), w_e,n[k] = +1 (bit 0)
// or -1 (bit 1) from packed rows, the groups' row ranges on the device.
//
// A packed bit becomes a bf16 +-0.5, whose lower byte is zero (0x3F00 /
// 0xBF00): for a 32-bit chunk c, register S_p = ((c << (7 - p)) & 0x80808080)
// | 0x3F3F3F3F holds in byte q the upper byte of element 8q + p, and one byte
// permute of (S_2i, S_2i+1) makes the operand pair (8q + 2i, 8q + 2i + 1). That
// is one VALU operation per element (8 + 8 + 16 for 32), and the activations
// stay in their natural order.  The factor 2 is applied to the sum, exactly.
//
// v_mfma_f32_32x32x16_bf16: lane l supplies row / column l % 32; lanes 0-31
// take the first 32 elements of a 64-element step, lanes 32-63 the last 32,
// eight per instruction.  Output layout of a 32 x 32 tile: lane l, register v
// -> row 8(v/4) + 4(l/32) + v%4, column l%32.
#include "bnn_internal.h"

namespace bnn {
namespace {

typedef __bf16 bf16_t;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// The upper bytes of a 32-bit chunk's 32 operands: byte q of s[p] belongs to
// element 8q + p.
__device__ __forceinline__ void sign_bytes(uint32_t c, uint32_t s[8]) {
#pragma unroll
  for (int p = 0; p < 8; ++p) s[p] = ((c << (7 - p)) & 0x80808080u) | 0x3F3F3F3Fu;
}

// Operands (+-0.5) of elements 8q .. 8q + 7.
__device__ __forceinline__ bf16x8 sign_operand(const uint32_t s[8], int q) {
  const uint32_t sel = 0x040C000Cu + (uint32_t)q * 0x01000100u;
  uint4 r;
  r.x = __builtin_amdgcn_perm(s[1], s[0], sel);
  r.y = __builtin_amdgcn_perm(s[3], s[2], sel);
  r.z = __builtin_amdgcn_perm(s[5], s[4], sel);
  r.w = __builtin_amdgcn_perm(s[7], s[6], sel);
  return __builtin_bit_cast(bf16x8, r);
}

// Row range of group e, whatever the offsets hold: 0 <= lo <= hi <= T.
__device__ __forceinline__ void group_range(const int32_t *off, int e, int T, int &lo, int &hi) {
  const int a = off[e], b = off[e + 1];
  lo = a < 0 ? 0 : (a > T ? T : a);
  hi = b < lo ? lo : (b > T ? T : b);
}

// Group and first row of the idx-th row tile (tiles of BM rows, counted group
// by group); false past the last.  Called by whole waves.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t *off, int E, int T, int64_t idx, int &e,
                                          int &r0, int &hi) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int a = 0, b = 0;
    if (e0 + lane < E) group_range(off, e0 + lane, T, a, b);
    const int n = (b - a + BM - 1) / BM;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const int total = __shfl(sum, 63, 64);
    if (idx < before + total) {
      const uint64_t past = __ballot(before + sum > idx);
      const int l = __ffsll((unsigned long long)past) - 1;
      e = e0 + l;
      const int first = (int)(idx - before) - __shfl(sum - n, l, 64);
      r0 = __shfl(a, l, 64) + first * BM;
      hi = __shfl(b, l, 64);
      return true;
    }
    before += total;
  }
  return false;
}

// ---------------------------------------------------------------------------
// Matrix-core kernel.  Eight waves side by side along N, each RB x CB tiles of
// 32 x 32: one wave's sign operands are made while another's matrix
// instructions run.  The weights need next to no bytes, so the tile is wide
// (every activation row read from L2 serves 256 columns) and low (few rows are
// wasted at a group's end); two blocks share a CU and hide each other's
// barriers.  Tiles of 128 x 512, one block a CU, read the activations half as
// often, but lose more at the groups' ends: 16384 routed rows on 32 experts of
// 4096 x 4096 622-652 us against 587-615 us, on 64 experts 701-709 against
// 625-628, one group of them all 523 against 532; 16384 x 1024 x 1024 on 8
// experts at 128 x 256 71 against 47.
//
// Per 64-element step the block's activation rows (128 bytes each, their
// 16-byte pieces swapped by row so that the reads spread over the banks) pass
// through one of two LDS buffers; the step after is on its way through
// registers, loaded at any alignment, zero past K.  The columns' weight words
// go the same way, eight steps at a time: one word of a column per step would
// move a cache line for eight of its bytes.
//
// 16384 routed rows on 32 experts of 4096 x 4096, bf16 out: 547 us, 1.0 PFLOP/s
// (a launch among others; single launches under a profiler 585-620 us); one group
// of them all 499 us, 1.1 PFLOP/s (a dense library product of bf16 weights:
// 355 us).  The matrix cores are busy 47 % of the cycles, the VALU, which makes the
// operands and addresses, about as long; 6 % of the instructions are for rows
// past a group's end.

constexpr int kGroupThreads = 512;
constexpr int kGroupRB = 2, kGroupCB = 1;  // a wave's tiles

template <typename T>
__global__ void __launch_bounds__(kGroupThreads, 2)
    signw_grouped_kernel(const uint16_t *__restrict__ x, int64_t ldx, int xrows,
                         const int32_t *__restrict__ rows, const int32_t *__restrict__ off,
                         const uint64_t *__restrict__ wp, const float *__restrict__ alpha,
                         const float *__restrict__ row_scale, T *__restrict__ y, int R, int E,
                         int N, int K, int tiles_n, int64_t most) {
  constexpr int RB = kGroupRB, CB = kGroupCB, BM = RB * 32, BN = 8 * CB * 32;
  constexpr int PIECES = BM * 8 / kGroupThreads;  // 16-byte pieces a thread stages
  static_assert(PIECES >= 1 && BN <= kGroupThreads, "every thread stages");
  __shared__ __attribute__((aligned(16))) unsigned char as[2][BM * 128];
  __shared__ __attribute__((aligned(16))) uint64_t ws[2][8][BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, h = lane >> 5;
  const int kw = (K + 63) / 64, nfull = K / 64;

  // Tiles: consecutive blocks go to the eight XCDs in turn, so block b takes a
  // row tile of its XCD's own (b % 8) and walks along N first: an XCD's L2
  // then reads an activation row once.
  for (int64_t b = blockIdx.x; b < most; b += gridDim.x) {
    const int64_t u = b >> 3;
    const int tn = (int)(u % tiles_n);
    int e, r0, hi;
    if (!find_tile<BM>(off, E, R, (u / tiles_n) * 8 + (b & 7), e, r0, hi)) continue;
    const int n0 = tn * BN + wave * (CB * 32);

    const uint16_t *xr[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      int r = r0 + (tid >> 3) + i * (kGroupThreads / 8);
      r = r < hi ? r : hi - 1;
      int src = rows ? rows[r] : r;
      src = src < 0 ? 0 : (src < xrows ? src : xrows - 1);
      xr[i] = x + src * ldx + 8 * (tid & 7);
    }
    const uint64_t *wr;
    {
      int n = tn * BN + (tid < BN ? tid : BN - 1);
      n = n < N ? n : N - 1;
      wr = wp + ((int64_t)e * N + n) * kw;
    }
    struct Stage {
      uint4 a[PIECES];
    };
    auto load = [&](int s, Stage &st) __attribute__((always_inline)) {  // a whole step
#pragma unroll
      for (int i = 0; i < PIECES; ++i) __builtin_memcpy(&st.a[i], xr[i] + 64 * (int64_t)s, 16);
    };
    auto load_tail = [&](Stage &st) __attribute__((always_inline)) {  // the last, partial one
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (64 * nfull + 8 * (tid & 7) + j < K)
            v[j / 2] |= (uint32_t)xr[i][64 * (int64_t)nfull + j] << (16 * (j & 1));
        st.a[i] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    };
    auto stage = [&](const Stage &st, int buf) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int row = (tid >> 3) + i * (kGroupThreads / 8);
        *reinterpret_cast<uint4 *>(as[buf] + row * 128 + (((tid & 7) ^ (row >> 1 & 7)) << 4)) = st.a[i];
      }
    };
    uint64_t wn[8];  // this thread's column's words of the next eight steps
    auto load_words = [&](int q) __attribute__((always_inline)) {
      if (8 * q + 8 <= kw) {
        __builtin_memcpy(wn, wr + 8 * q, 64);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) wn[j] = wr[8 * q + j < kw ? 8 * q + j : kw - 1];
      }
    };
    auto stage_words = [&](int q) __attribute__((always_inline)) {
      if (BN == kGroupThreads || tid < BN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ws[q & 1][j][tid] = wn[j];
      }
    };
    v16f acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[rb][cb][v] = 0.0f;
    auto compute = [&](int s, int buf) __attribute__((always_inline)) {
      const uint32_t *w = reinterpret_cast<const uint32_t *>(ws[(s >> 3) & 1][s & 7]);
      uint32_t sg[CB][8];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        sign_bytes(w[2 * (wave * CB * 32 + cb * 32 + li) + h], sg[cb]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        bf16x8 a[RB], bo[CB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
          a[rb] = __builtin_bit_cast(
              bf16x8, *reinterpret_cast<const uint4 *>(as[buf] + (rb * 32 + li) * 128 +
                                                       (((4 * h + t) ^ (li >> 1 & 7)) << 4)));
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) bo[cb] = sign_operand(sg[cb], t);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int cb = 0; cb < CB; ++cb)
            acc[rb][cb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[rb], bo[cb], acc[rb][cb], 0, 0, 0);
      }
    };

    // Loads past the last whole step read it again (in bounds, not used), so
    // that the loop has no branches and its waits are exact.
    Stage sa, sb;
    __syncthreads();  // the last tile's reads of LDS are done
    if (kw > 0) {
      load_words(0);
      stage_words(0);
    }
    if (nfull > 0) {
      const int last = nfull - 1;
      load(0, sa);
      load(last < 1 ? last : 1, sb);
      stage(sa, 0);
      __syncthreads();
      for (int s = 0; s + 1 < nfull; s += 2) {
        const int q = (s >> 3) + 1;
        const bool more = 8 * q < kw;
        if ((s & 7) == 0 && more) load_words(q);
        stage(sb, 1);
        load(s + 2 < last ? s + 2 : last, sa);
        __builtin_amdgcn_sched_barrier(0);
        compute(s, 0);
        __syncthreads();
        if ((s & 7) == 6 && more) stage_words(q);
        stage(sa, 0);
        load(s + 3 < last ? s + 3 : last, sb);
        __builtin_amdgcn_sched_barrier(0);
        compute(s + 1, 1);
        __syncthreads();
      }
      if (nfull & 1) compute(last, 0);
    }
    if (nfull < kw) {
      load_tail(sa);
      __syncthreads();
      stage(sa, 0);
      __syncthreads();
      compute(nfull, 0);
    }

    float al[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      int n = n0 + cb * 32 + li;
      n = n < N ? n : N - 1;
      al[cb] = alpha ? alpha[(int64_t)e * N + n] : 1.0f;
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int r = r0 + rb * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (r >= hi) continue;
        const float rs = row_scale ? row_scale[r] : 1.0f;
        T *yr = y + (int64_t)r * N + n0 + li;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          if (n0 + cb * 32 + li < N) yr[cb * 32] = (T)(2.0f * acc[rb][cb][v] * al[cb] * rs);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// ---------------------------------------------------------------------------
// Few-row kernel: 16 RC columns x 16 RM rows of a group per block, steps of
// 512 elements of K dealt out to the block's waves, their sums joined through
// LDS in a fixed order.  Each weight word is read once per 16 RM rows of its
// group, by 16-byte loads of 16 columns at a time, and groups without rows are
// not touched.  Bound by the launch for one token (RC = 1: many blocks), by the
// activation rows' way from L2 where many groups are active (RC = 4: one
// reading of a row serves 64 columns).
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row / column l % 16; lane group
// g = l / 16 takes elements 128 g .. 128 g + 127 of a step, eight per
// instruction.  Output: register v -> row 4 g + v, column l % 16.

typedef float v4f __attribute__((ext_vector_type(4)));

template <int RM, int RC, typename T>
__global__ void __launch_bounds__(512)
    signw_grouped_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int xrows,
                              const int32_t *__restrict__ rows, const int32_t *__restrict__ off,
                              const uint64_t *__restrict__ wp, const float *__restrict__ alpha,
                              const float *__restrict__ row_scale, T *__restrict__ y, int R, int E,
                              int N, int K, int tiles_n, int64_t most) {
  __shared__ float join[8][256 * RC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int li = lane & 15, g = lane >> 4;
  const int kw = (K + 63) / 64, steps = (K + 511) / 512;
  for (int64_t tile = blockIdx.x; tile < most; tile += gridDim.x) {
    int e, r0, hi;
    if (!find_tile<16 * RM>(off, E, R, tile / tiles_n, e, r0, hi)) return;
    const int n0 = (int)(tile % tiles_n) * (16 * RC);
    const uint64_t *wr[RC];
#pragma unroll
    for (int c = 0; c < RC; ++c) {
      const int n = n0 + c * 16 + li < N ? n0 + c * 16 + li : N - 1;
      wr[c] = wp + ((int64_t)e * N + n) * kw;
    }
    const uint16_t *xr[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = r0 + i * 16 + li < hi ? r0 + i * 16 + li : hi - 1;
      int src = rows ? rows[r] : r;
      src = src < 0 ? 0 : (src < xrows ? src : xrows - 1);
      xr[i] = x + src * ldx;
    }
    v4f acc[RM][RC];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int c = 0; c < RC; ++c) acc[i][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int st = wave; st < steps; st += waves) {
      const int k0 = 512 * st + 128 * g;
      uint32_t w[RC][4];
#pragma unroll
      for (int c = 0; c < RC; ++c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[c][j] = 0;
        if (k0 + 128 <= K) {
          __builtin_memcpy(w[c], wr[c] + k0 / 64, 16);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (k0 + 64 * j < K) __builtin_memcpy(w[c] + 2 * j, wr[c] + k0 / 64 + j, 8);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = k0 + 32 * t;
        uint4 a[RM][4];
        if (k + 32 <= K) {
#pragma unroll
          for (int i = 0; i < RM; ++i) __builtin_memcpy(a[i], xr[i] + k, 64);
        } else {  // zero past K
#pragma unroll
          for (int i = 0; i < RM; ++i) {
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[j] = k + 2 * j < K ? xr[i][k + 2 * j] : 0u;
              v[j] |= k + 2 * j + 1 < K ? (uint32_t)xr[i][k + 2 * j + 1] << 16 : 0u;
            }
            __builtin_memcpy(a[i], v, 64);
          }
        }
#pragma unroll
        for (int c = 0; c < RC; ++c) {
          uint32_t sg[8];
          sign_bytes(w[c][t], sg);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bf16x8 b = sign_operand(sg, q);
#pragma unroll
            for (int i = 0; i < RM; ++i)
              acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, a[i][q]), b, acc[i][c], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      __syncthreads();  // join is free
#pragma unroll
      for (int c = 0; c < RC; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          join[wave][(4 * g + v) * (16 * RC) + c * 16 + li] = acc[i][c][v];
      __syncthreads();
      for (int q = threadIdx.x; q < 256 * RC; q += blockDim.x) {
        float sum = 0.0f;
        for (int w = 0; w < waves; ++w) sum += join[w][q];
        const int r = r0 + i * 16 + q / (16 * RC), c = n0 + q % (16 * RC);
        if (r < hi && c < N) {
          float o = 2.0f * sum * (alpha ? alpha[(int64_t)e * N + c] : 1.0f);
          if (row_scale) o *= row_scale[r];
          y[(int64_t)r * N + c] = (T)o;
        }
      }
    }
  }
}

template <int RM, int RC, typename T>
void launch_rows(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows,
                 const int32_t *off, const uint64_t *wp, const float *alpha,
                 const float *row_scale, void *y, int64_t R, int64_t E, int64_t N, int64_t K,
                 hipStream_t s) {
  const int64_t tiles_n = (N + 16 * RC - 1) / (16 * RC);
  const int64_t most = tiles_n * (R / (16 * RM) + (E < R ? E : R));
  const int64_t blocks = most < (1 << 20) ? most : (1 << 20);
  const int64_t steps = (K + 511) / 512;
  const int waves = steps >= 8 ? 8 : (steps < 1 ? 1 : (int)steps);
  hipLaunchKernelGGL((signw_grouped_rows_kernel<RM, RC, T>), dim3((unsigned)blocks),
                     dim3(64 * waves), 0, s, x, ldx, (int)xrows, rows, off, wp, alpha, row_scale,
                     static_cast<T *>(y), (int)R, (int)E, (int)N, (int)K, (int)tiles_n, most);
}

template <typename T>
void launch_tile(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows,
                 const int32_t *off, const uint64_t *wp, const float *alpha,
                 const float *row_scale, void *y, int64_t R, int64_t E, int64_t N, int64_t K,
                 hipStream_t s) {
  constexpr int BM = kGroupRB * 32, BN = 8 * kGroupCB * 32;
  const int64_t tiles_n = (N + BN - 1) / BN;
  // Row tiles of any grouping of R rows: the whole ones and one partial tile
  // for each group that has rows; a multiple of the eight XCDs.
  const int64_t tiles_m = (R / BM + (E < R ? E : R) + 7) / 8 * 8;
  const int64_t most = tiles_m * tiles_n;
  const int64_t blocks = most < (1 << 20) ? most : (1 << 20);
  hipLaunchKernelGGL((signw_grouped_kernel<T>), dim3((unsigned)blocks),
                     dim3(kGroupThreads), 0, s, x, ldx, (int)xrows, rows, off, wp, alpha, row_scale,
                     static_cast<T *>(y), (int)R, (int)E, (int)N, (int)K, (int)tiles_n, most);
}

template <typename T>
void launch(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows, const int32_t *off,
            const uint64_t *wp, const float *alpha, const float *row_scale, void *y, int64_t R,
            int64_t E, int64_t N, int64_t K, int algo, hipStream_t s) {
  // All the host knows of the groups is R and E.  The few-row kernel serves
  // small groups and products with too few tiles to fill the card; measured
  // (device, bf16 out, N x K): 256 rows on 64 experts of 1024 x 4096 25 us
  // against 44 us on tiles, 602 on 10 of 700 x 1000 12 against 17; 2000 on 128
  // of 1024 x 512 27 against 15.  A small mean can hide a large group: 640 rows
  // on 64 experts of 1024 x 4096, 577 of them on one, 62 us against 61; 1280 on
  // 128 of 4096 x 4096, 1153 on one, 449 against 319 (a caller who knows of such
  // a router names BNN_ALGO_MFMA).
  const int64_t mean = R / E, active = E < R ? E : R;
  const int64_t tiles = (R / 64 + active / 2) * ((N + 255) / 256);  // half a tile lost per group
  if (algo == BNN_ALGO_AUTO) algo = mean <= 12 || tiles < 64 ? BNN_ALGO_GEMV : BNN_ALGO_MFMA;
  auto run = launch_tile<T>;
  if (algo == BNN_ALGO_GEMV) {
    // 16 columns a block while 64 would leave CUs idle (8 rows on 8 of 64 experts
    // of 1024 x 4096: 7 us against 9); 64 beyond (256 rows on 64: 45 -> 25 us).
    run = active * ((N + 63) / 64) < 512 ? launch_rows<1, 1, T>
          : mean <= 8                    ? launch_rows<1, 4, T>
                                         : launch_rows<2, 4, T>;
  }
  run(x, ldx, xrows, rows, off, wp, alpha, row_scale, y, R, E, N, K, s);
}

}  // namespace

hipError_t launch_signw_grouped(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows,
                                const int32_t *off, const uint64_t *wp, const float *alpha,
                                const float *row_scale, void *y, int dtype, int64_t R, int64_t E,
                                int64_t N, int64_t K, int algo, hipStream_t s) {
  const auto run = dtype == BNN_FP32 ? launch<float> : launch<bf16_t>;
  run(x, ldx, xrows, rows, off, wp, alpha, row_scale, y, R, E, N, K, algo, s);
  return hipGetLastError();
}

}  // namespace bnn
