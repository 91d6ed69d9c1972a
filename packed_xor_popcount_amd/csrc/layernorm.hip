// layernorm.hip -- layer norm over rows and its gradient.
//
//   mu = 1/N sum_n x_n      v = 1/N sum_n (x_n - mu)^2      r = 1/sqrt(v + eps)
//   y_n = (x_n - mu) r gamma_n + beta_n
//
// and, for an output gradient dy with xh_n = (x_n - mu) r and g_n = dy_n gamma_n,
//
//   dx_n = r (g_n - 1/N sum g - xh_n 1/N sum g xh)
//   dgamma_n = sum_m dy xh        dbeta_n = sum_m dy      (over the rows m)
//
// Everything is computed in fp32; bf16 values are widened exactly on load and
// the stored y / dx are rounded once (to nearest even).
#include "bnn_internal.h"

namespace bnn {
namespace {

typedef __bf16 bf16_t;

template <typename T>
__device__ __forceinline__ float load_f32(const T *p) { return (float)*p; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the block's 256 threads; every thread receives it.
__device__ __forceinline__ float block_sum(float v, float *lds) {
  v = wave_sum(v);
  __syncthreads();  // lds is free
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// One block per row, the row read three times (from the caches after the
// first): mean, centred second moment, output.
template <typename T>
__global__ void __launch_bounds__(256)
    ln_fwd_kernel(const T *__restrict__ x, int64_t ldx, const float *__restrict__ gamma,
                  const float *__restrict__ beta, T *__restrict__ y, int64_t ldy,
                  float *__restrict__ mean, float *__restrict__ rstd, int64_t M, int N, float eps) {
  __shared__ float lds[4];
  const float inv_n = 1.0f / (float)N;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const T *xr = x + m * ldx;
    float s = 0.0f;
    for (int n = threadIdx.x; n < N; n += 256) s += load_f32(xr + n);
    const float mu = block_sum(s, lds) * inv_n;
    float q = 0.0f;
    for (int n = threadIdx.x; n < N; n += 256) {
      const float d = load_f32(xr + n) - mu;
      q += d * d;
    }
    const float r = 1.0f / sqrtf(block_sum(q, lds) * inv_n + eps);
    for (int n = threadIdx.x; n < N; n += 256) {
      float v = (load_f32(xr + n) - mu) * r;
      if (gamma) v *= gamma[n];
      if (beta) v += beta[n];
      y[m * ldy + n] = (T)v;
    }
    if (threadIdx.x == 0) {
      if (mean) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
}

// Block b takes rows b, b + P, ... and keeps its part of the columns' sums in
// row b of `part` (P x 2 x N: dgamma, then dbeta).
template <typename T>
__global__ void __launch_bounds__(256)
    ln_bwd_kernel(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                  const float *__restrict__ gamma, const float *__restrict__ mean,
                  const float *__restrict__ rstd, T *__restrict__ dx, int64_t lddx,
                  float *__restrict__ part, int64_t M, int N) {
  __shared__ float lds[4];
  const float inv_n = 1.0f / (float)N;
  float *pg = part ? part + (int64_t)blockIdx.x * 2 * N : nullptr;
  bool first = true;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const T *xr = x + m * ldx, *dr = dy + m * lddy;
    const float mu = mean[m], r = rstd[m];
    float s1 = 0.0f, s2 = 0.0f;
    for (int n = threadIdx.x; n < N; n += 256) {
      const float d = load_f32(dr + n), xh = (load_f32(xr + n) - mu) * r;
      const float g = gamma ? d * gamma[n] : d;
      s1 += g;
      s2 += g * xh;
      if (pg) {
        pg[n] = first ? d * xh : pg[n] + d * xh;
        pg[N + n] = first ? d : pg[N + n] + d;
      }
    }
    const float c1 = block_sum(s1, lds) * inv_n, c2 = block_sum(s2, lds) * inv_n;
    for (int n = threadIdx.x; n < N; n += 256) {
      const float d = load_f32(dr + n), xh = (load_f32(xr + n) - mu) * r;
      const float g = gamma ? d * gamma[n] : d;
      dx[m * lddx + n] = (T)((g - c1 - xh * c2) * r);
    }
    first = false;
  }
}

// Columns' sums over the P partial rows, in a fixed order.
__global__ void __launch_bounds__(256)
    ln_bwd_finish_kernel(const float *__restrict__ part, int P, int N, float *__restrict__ dgamma,
                         float *__restrict__ dbeta) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * (int64_t)N) return;
  float s = 0.0f;
  for (int p = 0; p < P; ++p) s += part[(int64_t)p * 2 * N + i];
  if (i < N) dgamma[i] = s;
  else dbeta[i - N] = s;
}

constexpr int64_t kBwdBlocks = 512;  // blocks (and partial rows) of the gradient

template <typename T>
void fwd(const void *x, int64_t ldx, const float *gamma, const float *beta, void *y, int64_t ldy,
         float *mean, float *rstd, int64_t M, int64_t N, float eps, hipStream_t s) {
  const int64_t blocks = M < 65536 ? M : 65536;
  hipLaunchKernelGGL((ln_fwd_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, s,
                     static_cast<const T *>(x), ldx, gamma, beta, static_cast<T *>(y), ldy, mean,
                     rstd, M, (int)N, eps);
}

template <typename T>
void bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, const float *gamma,
         const float *mean, const float *rstd, void *dx, int64_t lddx, float *part, int64_t M,
         int64_t N, int64_t P, hipStream_t s) {
  hipLaunchKernelGGL((ln_bwd_kernel<T>), dim3((unsigned)P), dim3(256), 0, s,
                     static_cast<const T *>(dy), lddy, static_cast<const T *>(x), ldx, gamma, mean,
                     rstd, static_cast<T *>(dx), lddx, part, M, (int)N);
}

}  // namespace

int64_t layernorm_bwd_partials(int64_t M, int64_t N) {
  (void)N;
  return M < kBwdBlocks ? M : kBwdBlocks;
}

hipError_t launch_layernorm_fwd(const void *x, int dtype, int64_t ldx, const float *gamma,
                                const float *beta, void *y, int64_t ldy, float *mean, float *rstd,
                                int64_t M, int64_t N, float eps, hipStream_t s) {
  if (dtype == BNN_FP32) fwd<float>(x, ldx, gamma, beta, y, ldy, mean, rstd, M, N, eps, s);
  else fwd<bf16_t>(x, ldx, gamma, beta, y, ldy, mean, rstd, M, N, eps, s);
  return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                int dtype, const float *gamma, const float *mean,
                                const float *rstd, void *dx, int64_t lddx, float *dgamma,
                                float *dbeta, float *part, int64_t M, int64_t N, hipStream_t s) {
  const int64_t P = layernorm_bwd_partials(M, N);
  float *p = dgamma ? part : nullptr;
  if (P > 0) {
    if (dtype == BNN_FP32) bwd<float>(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, p, M, N, P, s);
    else bwd<bf16_t>(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, p, M, N, P, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dgamma) {
    hipLaunchKernelGGL(ln_bwd_finish_kernel, dim3((unsigned)((2 * N + 255) / 256)), dim3(256), 0, s,
                       part, (int)P, (int)N, dgamma, dbeta);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace bnn
