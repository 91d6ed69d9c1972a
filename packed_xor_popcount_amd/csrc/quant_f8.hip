// quant_f8.hip -- fp32 / bf16 rows to the block-scaled 8-bit form (see f8.h).
//
// Per block of 128 elements with largest finite magnitude a = 1.f * 2^E:
//   e = E - 8, one more if 1.f > 1.75 (448 = 1.75 * 2^8), at least -127;
//   q = e4m3(v * 2^-e) to nearest even;  scale byte e + 127 (127 if a = 0).
// The scaling is exact, so q is the only rounding.  Infinities and NaN become
// NaN and do not enter a.
//
// Both forms are bound by HBM: one read of the source, one byte written per
// element.  4096 x 4096 bf16 (inputs that fit the Infinity Cache): rows 11.7 us
// (4.3 TB/s), transposed 13.8 us; 11008 x 4096 fp32: rows 39 us (5.8 TB/s),
// transposed 47 us (4.8 TB/s; its writes are pieces of 32 bytes).
#include "bnn_internal.h"
#include "f8.h"

namespace bnn {
namespace {

typedef __bf16 bf16_t;

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }

// |v| as an ordered integer, 0 for infinities and NaN.
__device__ __forceinline__ uint32_t finite_mag(float v) {
  const uint32_t a = bits_of(v) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// Biased scale exponent for the largest magnitude's bits.
__device__ __forceinline__ int scale_byte(uint32_t a) {
  int s = (int)(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  s = s < 0 ? 0 : s;
  return a == 0 ? 127 : s;
}

// 2^-e for scale byte e + 127.
__device__ __forceinline__ float inv_scale(int s) {
  return __uint_as_float((uint32_t)(254 - s) << 23);
}

__device__ __forceinline__ float scaled(float v, float inv) {
  const float p = v * inv;
  return (bits_of(v) & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FC00000u) : p;
}

__device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(a, inv), scaled(b, inv), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(c, inv), scaled(d, inv), r, true);
  return (uint32_t)r;
}

// Largest of a value over aligned groups of 16 lanes.
__device__ __forceinline__ uint32_t max16(uint32_t a) {
#define BNN_MAX(CTRL)                                                                    \
  {                                                                                      \
    const uint32_t m = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, CTRL, 0xF, 0xF, false); \
    a = a > m ? a : m;                                                                   \
  }
  BNN_MAX(0xB1)   // quad_perm 1,0,3,2
  BNN_MAX(0x4E)   // quad_perm 2,3,0,1
  BNN_MAX(0x141)  // row_half_mirror
  BNN_MAX(0x140)  // row_mirror
#undef BNN_MAX
  return a;
}

// Rows: 16 lanes per block of 128, eight consecutive elements a lane (16-byte
// loads at any alignment), kRowsInFlight blocks a lane on their way before any
// is used.
constexpr int kRowsInFlight = 2;

template <typename T>
__global__ void __launch_bounds__(256)
    quant_rows_kernel(const T *__restrict__ src, int64_t rows, int64_t k, int64_t ld,
                      uint8_t *__restrict__ q, uint8_t *__restrict__ s) {
  const int64_t nb = f8_blocks(k), sb = f8_scale_bytes(k);
  const int t = threadIdx.x & 15;
  const int64_t total = rows * sb;  // scale bytes, the pads of a row's last four among them
  constexpr int U = kRowsInFlight;
  for (int64_t g0 = (int64_t)blockIdx.x * (16 * U); g0 < total; g0 += (int64_t)gridDim.x * (16 * U)) {
    uint32_t raw[U][2 * sizeof(T)];  // packed until used: the loads stay in flight
    int64_t row[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * 16 + (threadIdx.x >> 4);
      // both fit 32 bits in all but huge matrices: a 32-bit division is a third of the work
      if (total < (int64_t(1) << 31)) {
        row[u] = (uint32_t)g / (uint32_t)sb;
      } else {
        row[u] = g / sb;
      }
      b[u] = g - row[u] * sb;
      const int64_t e = b[u] * kF8Block + t * 8;
#pragma unroll
      for (unsigned i = 0; i < 2 * sizeof(T); ++i) raw[u][i] = 0;
      if (g < total && e + 8 <= k) {
        __builtin_memcpy(raw[u], src + row[u] * ld + e, sizeof(raw[u]));
      } else if (g < total && e < k) {
#pragma unroll
        for (int j = 0; j < 7; ++j) {
          if (e + j < k) {
            const uint32_t w = bits_of((float)src[row[u] * ld + e + j]);
            if (sizeof(T) == 4) raw[u][j] = w;
            else raw[u][j / 2] |= (j & 1) ? w : w >> 16;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * 16 + (threadIdx.x >> 4);
      float v[8];
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = sizeof(T) == 4 ? __uint_as_float(raw[u][j])
               : (j & 1)      ? __uint_as_float(raw[u][j / 2] & 0xFFFF0000u)
                              : __uint_as_float(raw[u][j / 2] << 16);
        const uint32_t m = finite_mag(v[j]);
        a = a > m ? a : m;
      }
      const int sc = scale_byte(max16(a));
      if (g >= total) continue;
      if (b[u] < nb) {
        const float inv = inv_scale(sc);
        uint2 o;
        o.x = to_f8x4(v[0], v[1], v[2], v[3], inv);
        o.y = to_f8x4(v[4], v[5], v[6], v[7], inv);
        *reinterpret_cast<uint2 *>(q + (row[u] * nb + b[u]) * kF8Block + t * 8) = o;
      }
      if (t == 0) s[g] = b[u] < nb ? (uint8_t)sc : 0;
    }
  }
}

// Columns: a block takes 128 source rows x 64 C columns; a thread holds 32 rows
// of C neighbouring columns (C = 2: bf16 pairs, so that a wave's load is not a
// half-used line), four threads share a column's scale through LDS.  Loads
// come from clamped places, so that all of a thread's are in flight at once;
// rows past the end count as zero.
template <typename T, int C>
__global__ void __launch_bounds__(256)
    quant_cols_kernel(const T *__restrict__ src, int64_t rows, int64_t k, int64_t ld,
                      uint8_t *__restrict__ q, uint8_t *__restrict__ s) {
  static_assert(C == 1 || sizeof(T) == 2, "pairs of bf16");
  __shared__ uint32_t top[4][64][C];
  const int64_t nb = f8_blocks(rows), sb = f8_scale_bytes(rows);
  const int c = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t ctiles = (k + 64 * C - 1) / (64 * C);
  for (int64_t tile = blockIdx.x; tile < ctiles * sb; tile += gridDim.x) {
    const int64_t b = tile / ctiles, col = ((tile - b * ctiles) * 64 + c) * C;
    const int64_t r0 = b * kF8Block + part * 32;
    const int64_t from = col + C <= k ? col : k - C;  // the pair that ends the row, for a last odd one
    const bool second = C == 2 && col + 1 == k;       // whose upper half it is
    uint32_t raw[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int64_t r = r0 + j < rows ? r0 + j : rows - 1;
      raw[j] = 0;
      __builtin_memcpy(&raw[j], src + r * ld + from, C * sizeof(T));
    }
    uint32_t a[C];
#pragma unroll
    for (int i = 0; i < C; ++i) a[i] = 0;
    auto value = [&](int j, int i) __attribute__((always_inline)) {
      if (sizeof(T) == 4) return __uint_as_float(raw[j]);
      return __uint_as_float(i ? raw[j] & 0xFFFF0000u : raw[j] << 16);
    };
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (second) raw[j] >>= 16;
      if (r0 + j >= rows) raw[j] = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const uint32_t m = finite_mag(value(j, i));
        a[i] = a[i] > m ? a[i] : m;
      }
    }
    __syncthreads();  // the last tile's maxima have been read
#pragma unroll
    for (int i = 0; i < C; ++i) top[part][c][i] = a[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (col + i >= k) continue;
#pragma unroll
      for (int p = 0; p < 4; ++p) a[i] = a[i] > top[p][c][i] ? a[i] : top[p][c][i];
      const int sc = scale_byte(a[i]);
      if (b < nb) {
        const float inv = inv_scale(sc);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = to_f8x4(value(4 * j, i), value(4 * j + 1, i), value(4 * j + 2, i),
                         value(4 * j + 3, i), inv);
        uint4 *o = reinterpret_cast<uint4 *>(q + (col + i) * nb * kF8Block + r0);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (part == 0) s[(col + i) * sb + b] = b < nb ? (uint8_t)sc : 0;
    }
  }
}

template <typename T>
void launch(const void *src, int64_t rows, int64_t k, int64_t ld, bool transpose, uint8_t *q,
            uint8_t *s, hipStream_t st) {
  const T *p = static_cast<const T *>(src);
  if (!transpose) {
    const int64_t groups = rows * f8_scale_bytes(k);
    int64_t blocks = (groups + 16 * kRowsInFlight - 1) / (16 * kRowsInFlight);
    if (blocks > 256 * 16) blocks = 256 * 16;
    hipLaunchKernelGGL((quant_rows_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, st, p, rows, k,
                       ld, q, s);
  } else {
    // Pairs need two columns; with few tiles single columns fill more CUs.
    constexpr int P = sizeof(T) == 2 ? 2 : 1;
    const bool pairs = P == 2 && k >= 2 && (k + 127) / 128 * f8_blocks(rows) >= 256;
    const int64_t wide = pairs ? 128 : 64, tiles = (k + wide - 1) / wide * f8_scale_bytes(rows);
    const int64_t blocks = tiles < (1 << 20) ? tiles : (1 << 20);
    const auto run = pairs ? quant_cols_kernel<T, P> : quant_cols_kernel<T, 1>;
    hipLaunchKernelGGL(run, dim3((unsigned)blocks), dim3(256), 0, st, p, rows, k, ld, q, s);
  }
}

}  // namespace

hipError_t launch_quant_f8(const void *src, int dtype, int64_t rows, int64_t k, int64_t ld,
                           bool transpose, uint8_t *q, uint8_t *s, hipStream_t st) {
  if (dtype == BNN_FP32) launch<float>(src, rows, k, ld, transpose, q, s, st);
  else launch<bf16_t>(src, rows, k, ld, transpose, q, s, st);
  return hipGetLastError();
}

}  // namespace bnn
