// quant_f8.hip -- fp32 / bf16 rows to the block-scaled 8-bit form (see f8.h).
//
// Per block of 128 elements with largest finite magnitude a = 1.f * 2^E:
//   e = E - 8, one more if 1.f > 1.75 (448 = 1.75 * 2^8), at least -127;
//   q = e4m3(v * 2^-e) to nearest even;  scale byte e + 127 (127 if a = 0).
// The scaling is exact, so q is the only rounding.  Infinities and NaN become
// NaN and do not enter a.
//
// Both forms are bound by HBM: one read of the source, one byte written per
// element.
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

// Rows: 16 lanes per block of 128, eight consecutive elements a lane.
template <typename T>
__global__ void __launch_bounds__(256)
    quant_rows_kernel(const T *__restrict__ src, int64_t rows, int64_t k, int64_t ld,
                      uint8_t *__restrict__ q, uint8_t *__restrict__ s) {
  const int64_t nb = f8_blocks(k), sb = f8_scale_bytes(k);
  const int t = threadIdx.x & 15;
  const int64_t total = rows * sb;  // scale bytes, the pads of a row's last four among them
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < total;
       g += (int64_t)gridDim.x * 16) {
    const int64_t row = g / sb, b = g - row * sb;
    float v[8];
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = b * kF8Block + t * 8 + j;
      v[j] = e < k ? (float)src[row * ld + e] : 0.0f;
      const uint32_t m = finite_mag(v[j]);
      a = a > m ? a : m;
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      const uint32_t m = (uint32_t)__shfl_xor((int)a, o, 64);
      a = a > m ? a : m;
    }
    const int sc = scale_byte(a);
    if (b < nb) {
      const float inv = inv_scale(sc);
      uint2 o;
      o.x = to_f8x4(v[0], v[1], v[2], v[3], inv);
      o.y = to_f8x4(v[4], v[5], v[6], v[7], inv);
      *reinterpret_cast<uint2 *>(q + row * nb * kF8Block + b * kF8Block + t * 8) = o;
    }
    if (t == 0) s[g] = b < nb ? (uint8_t)sc : 0;
  }
}

// Columns: a block takes 128 source rows x 64 columns; a thread holds 32
// rows of one column, four threads share a column's scale through LDS.
template <typename T>
__global__ void __launch_bounds__(256)
    quant_cols_kernel(const T *__restrict__ src, int64_t rows, int64_t k, int64_t ld,
                      uint8_t *__restrict__ q, uint8_t *__restrict__ s) {
  __shared__ uint32_t top[4][64];
  const int64_t nb = f8_blocks(rows), sb = f8_scale_bytes(rows);
  const int c = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t ctiles = (k + 63) / 64;
  for (int64_t tile = blockIdx.x; tile < ctiles * sb; tile += gridDim.x) {
    const int64_t b = tile / ctiles, col = (tile - b * ctiles) * 64 + c;
    const int64_t r0 = b * kF8Block + part * 32;
    float v[32];
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = (col < k && r0 + j < rows) ? (float)src[(r0 + j) * ld + col] : 0.0f;
      const uint32_t m = finite_mag(v[j]);
      a = a > m ? a : m;
    }
    __syncthreads();  // the last tile's maxima have been read
    top[part][c] = a;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) a = a > top[p][c] ? a : top[p][c];
    if (col < k) {
      const int sc = scale_byte(a);
      if (b < nb) {
        const float inv = inv_scale(sc);
        uint8_t *o = q + col * nb * kF8Block + r0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float *u = v + 16 * h;
          uint4 w;
          w.x = to_f8x4(u[0], u[1], u[2], u[3], inv);
          w.y = to_f8x4(u[4], u[5], u[6], u[7], inv);
          w.z = to_f8x4(u[8], u[9], u[10], u[11], inv);
          w.w = to_f8x4(u[12], u[13], u[14], u[15], inv);
          *reinterpret_cast<uint4 *>(o + 16 * h) = w;
        }
      }
      if (part == 0) s[col * sb + b] = b < nb ? (uint8_t)sc : 0;
    }
  }
}

template <typename T>
void launch(const void *src, int64_t rows, int64_t k, int64_t ld, bool transpose, uint8_t *q,
            uint8_t *s, hipStream_t st) {
  const T *p = static_cast<const T *>(src);
  if (!transpose) {
    const int64_t groups = rows * f8_scale_bytes(k);
    int64_t blocks = (groups + 15) / 16;
    if (blocks > 256 * 16) blocks = 256 * 16;
    hipLaunchKernelGGL((quant_rows_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, st, p, rows, k,
                       ld, q, s);
  } else {
    const int64_t tiles = (k + 63) / 64 * f8_scale_bytes(rows);
    const int64_t blocks = tiles < (1 << 20) ? tiles : (1 << 20);
    hipLaunchKernelGGL((quant_cols_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, st, p, rows, k,
                       ld, q, s);
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
