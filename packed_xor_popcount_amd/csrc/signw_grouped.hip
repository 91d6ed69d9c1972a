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
// stay in their natural order.  The factor 2 is applied with alpha, exactly.
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

// The 32 operands (+-0.5, natural order) of a 32-bit chunk: op[q] holds
// elements 8q .. 8q + 7.
__device__ __forceinline__ void half_signs(uint32_t c, bf16x8 op[4]) {
  uint32_t s[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) s[p] = ((c << (7 - p)) & 0x80808080u) | 0x3F3F3F3Fu;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t sel = 0x040C000Cu + (uint32_t)q * 0x01000100u;
    uint4 r;
    r.x = __builtin_amdgcn_perm(s[1], s[0], sel);
    r.y = __builtin_amdgcn_perm(s[3], s[2], sel);
    r.z = __builtin_amdgcn_perm(s[5], s[4], sel);
    r.w = __builtin_amdgcn_perm(s[7], s[6], sel);
    op[q] = __builtin_bit_cast(bf16x8, r);
  }
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

// One 32 x 32 tile per wave, operands straight from memory.
template <typename T>
__global__ void __launch_bounds__(256)
    signw_grouped_kernel(const uint16_t *__restrict__ x, int64_t ldx, int xrows,
                         const int32_t *__restrict__ rows, const int32_t *__restrict__ off,
                         const uint64_t *__restrict__ wp, const float *__restrict__ alpha,
                         const float *__restrict__ row_scale, T *__restrict__ y, int R, int E,
                         int N, int K) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 31, h = lane >> 5;
  const int kw = (K + 63) / 64;
  const int tiles_n = (N + 63) / 64;
  for (int64_t tile = blockIdx.x;; tile += gridDim.x) {
    int e, r0, hi;
    if (!find_tile<64>(off, E, R, tile / tiles_n, e, r0, hi)) return;
    r0 += (wave >> 1) * 32;
    const int n0 = (int)(tile % tiles_n) * 64 + (wave & 1) * 32;
    const int r = r0 + li < hi ? r0 + li : hi - 1, n = n0 + li < N ? n0 + li : N - 1;
    int src = rows ? rows[r] : r;
    src = src < 0 ? 0 : (src < xrows ? src : xrows - 1);
    const uint16_t *xr = x + src * ldx + 32 * h;
    const uint64_t *wr = wp + ((int64_t)e * N + n) * kw;
    v16f acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    for (int w = 0; w < kw; ++w) {
      bf16x8 b[4];
      half_signs((uint32_t)(wr[w] >> (32 * h)), b);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint16_t a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = 64 * w + 8 * t + j;
          a[j] = k + 32 * h < K ? xr[k] : (uint16_t)0;
        }
        bf16x8 av;
        __builtin_memcpy(&av, a, 16);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, b[t], acc, 0, 0, 0);
      }
    }
    if (n0 + li < N) {
      const float al = 2.0f * (alpha ? alpha[(int64_t)e * N + n] : 1.0f);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int rr = r0 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (rr < hi) {
          float o = acc[v] * al;
          if (row_scale) o *= row_scale[rr];
          y[(int64_t)rr * N + n] = (T)o;
        }
      }
    }
  }
}

template <typename T>
void launch(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows, const int32_t *off,
            const uint64_t *wp, const float *alpha, const float *row_scale, void *y, int64_t R,
            int64_t E, int64_t N, int64_t K, hipStream_t s) {
  const int64_t tiles = (R / 64 + (E < R ? E : R)) * ((N + 63) / 64);
  const int64_t blocks = tiles < (1 << 16) ? tiles : (1 << 16);
  hipLaunchKernelGGL((signw_grouped_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, s, x, ldx,
                     (int)xrows, rows, off, wp, alpha, row_scale, static_cast<T *>(y), (int)R,
                     (int)E, (int)N, (int)K);
}

}  // namespace

hipError_t launch_signw_grouped(const uint16_t *x, int64_t ldx, int64_t xrows, const int32_t *rows,
                                const int32_t *off, const uint64_t *wp, const float *alpha,
                                const float *row_scale, void *y, int dtype, int64_t R, int64_t E,
                                int64_t N, int64_t K, int algo, hipStream_t s) {
  (void)algo;
  if (dtype == BNN_FP32) launch<float>(x, ldx, xrows, rows, off, wp, alpha, row_scale, y, R, E, N, K, s);
  else launch<bf16_t>(x, ldx, xrows, rows, off, wp, alpha, row_scale, y, R, E, N, K, s);
  return hipGetLastError();
}

}  // namespace bnn
