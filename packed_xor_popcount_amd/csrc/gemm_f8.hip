// gemm_f8.hip -- product of two block-scaled 8-bit matrices (see f8.h):
//
//   y[m][n] = sum_b 2^(xs[m][b] + ws[n][b] - 254) sum_{k in block b} xq[m][k] wq[n][k]
//
// Two ways through the matrix cores, chosen by the output's precision:
//
//  * bf16 outputs: v_mfma_scale_f32_32x32x64_f8f6f4 takes the 8-bit values and
//    the scale byte of each operand row as they are, so a block boundary costs
//    nothing.  Measured on this unit: the sum over groups of eight consecutive
//    k and onto the accumulator keeps fp32 precision, but inside a group the
//    products are cut below 2^-13 of the group's largest.  For normally
//    distributed operands that is an error of 1.6e-5 of the result, a
//    hundredth of the bf16 rounding that follows.
//  * fp32 outputs: the values are widened to bf16 with their scale applied
//    (v_cvt_scalef32_pk_bf16_fp8: exact, an e4m3 significand has 4 bits) and
//    multiplied by v_mfma_f32_32x32x16_bf16, which keeps fp32 precision
//    throughout (products down to 2^-23 of the largest were measured to
//    count), at half the rate.
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

__device__ __forceinline__ v8i load32(const uint8_t *p) {
  const int4 a = reinterpret_cast<const int4 *>(p)[0], b = reinterpret_cast<const int4 *>(p)[1];
  v8i r;
  r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
  r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
  return r;
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

// acc += the products of 32 bytes of A and B per lane.
template <bool WIDE>
__device__ __forceinline__ v16f step(v8i a, v8i b, v16f acc, int sa, int sb) {
  if (!WIDE) return mfma_f8(a, b, acc, sa, sb);
  const float fa = pow2_of(sa), fb = pow2_of(sb);
#pragma unroll
  for (int t = 0; t < 4; ++t)
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(a[2 * t], a[2 * t + 1], fa),
                                                  widen8(b[2 * t], b[2 * t + 1], fb), acc, 0, 0, 0);
  return acc;
}

// One 32 x 32 tile per wave, operands straight from memory.
template <typename T>
__global__ void __launch_bounds__(256)
    gemm_f8_kernel(const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs,
                   const uint8_t *__restrict__ wq, const uint8_t *__restrict__ ws,
                   T *__restrict__ y, int M, int N, int nb, int sb) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 31, h = lane >> 5;
  const int64_t tiles_m = (M + 63) / 64, tiles = tiles_m * ((N + 63) / 64);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int m0 = (int)(tile % tiles_m) * 64 + (wave >> 1) * 32;
    const int n0 = (int)(tile / tiles_m) * 64 + (wave & 1) * 32;
    const int m = m0 + li < M ? m0 + li : M - 1, n = n0 + li < N ? n0 + li : N - 1;
    const uint8_t *xr = xq + (int64_t)m * nb * kF8Block + 32 * h;
    const uint8_t *wr = wq + (int64_t)n * nb * kF8Block + 32 * h;
    const uint8_t *xsr = xs + (int64_t)m * sb, *wsr = ws + (int64_t)n * sb;
    v16f acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    for (int b = 0; b < nb; ++b) {
      const int sa = xsr[b], sw = wsr[b];
      const int64_t o = (int64_t)b * kF8Block;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc = step<sizeof(T) == 4>(load32(xr + o + 64 * t), load32(wr + o + 64 * t), acc, sa, sw);
    }
    if (n0 + li < N) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int mm = m0 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (mm < M) y[(int64_t)mm * N + n0 + li] = (T)acc[v];
      }
    }
  }
}

template <typename T>
void launch(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, void *y,
            int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
  const int64_t blocks = tiles < (1 << 20) ? tiles : (1 << 20);
  hipLaunchKernelGGL((gemm_f8_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, s, xq, xs, wq,
                     ws, static_cast<T *>(y), (int)M, (int)N, (int)f8_blocks(K),
                     (int)f8_scale_bytes(K));
}

}  // namespace

hipError_t launch_gemm_f8(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                          const uint8_t *ws, void *y, int dtype, int64_t M, int64_t N, int64_t K,
                          hipStream_t s) {
  if (dtype == BNN_FP32) launch<float>(xq, xs, wq, ws, y, M, N, K, s);
  else launch<bf16_t>(xq, xs, wq, ws, y, M, N, K, s);
  return hipGetLastError();
}

}  // namespace bnn
