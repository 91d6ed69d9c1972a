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

// ---------------------------------------------------------------------------
// A row in registers.  TPR threads share a row; a thread holds C chunks of
// eight neighbours, chunk c of thread t from element 8 (c TPR + t) on.  A
// chunk wholly inside the row is one or two 16-byte accesses, whatever the
// row's alignment (gfx950 serves unaligned vector accesses); the row's last
// elements are accessed one by one.

template <typename T>
__device__ __forceinline__ void load8(const T *row, int n, int N, float v[8]) {
  if (n + 8 <= N) {
    T r[8];
    __builtin_memcpy(r, row + n, sizeof(r));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)r[j];
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = n + j < N ? (float)row[n + j] : 0.0f;
}

template <typename T>
__device__ __forceinline__ void store8(T *row, int n, int N, const float v[8]) {
  if (n + 8 <= N) {
    T r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (T)v[j];
    __builtin_memcpy(row + n, r, sizeof(r));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (n + j < N) row[n + j] = (T)v[j];
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);   // quad_perm 1,0,3,2
  v += dpp<0x4E>(v);   // quad_perm 2,3,0,1
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));  // lane ^ 16
  return v + __shfl_xor(v, 32, 64);
}

// Sums of A values over the TPR threads of a row; every thread receives
// them.  With one wave per row nothing is shared.  `lds`: A * TPR / 64 floats,
// one of two buffers that alternate from call to call (`flip`), so that one
// barrier a call is enough.
template <int TPR, int A>
__device__ __forceinline__ void row_sum(float (&v)[A], float *lds, int &flip) {
#pragma unroll
  for (int a = 0; a < A; ++a) v[a] = wave_sum(v[a]);
  if (TPR == 64) return;
  constexpr int W = TPR / 64;
  float *l = lds + flip * A * W;
  flip ^= 1;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int a = 0; a < A; ++a) l[a * W + (threadIdx.x >> 6)] = v[a];
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < A; ++a) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += l[a * W + w];
    v[a] = s;
  }
}

constexpr int block_of(int tpr) { return tpr < 256 ? 256 : tpr; }

// Bound by HBM: x is read and y written once, gamma and beta stay in the
// registers of a block that walks over rows.
template <typename T, int TPR, int C>
__global__ void __launch_bounds__(block_of(TPR))
    ln_fwd_kernel(const T *__restrict__ x, int64_t ldx, const float *__restrict__ gamma,
                  const float *__restrict__ beta, T *__restrict__ y, int64_t ldy,
                  float *__restrict__ mean, float *__restrict__ rstd, int64_t M, int N, float eps) {
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float lds[2 * (TPR / 64)];
  int flip = 0;
  const int t = threadIdx.x % TPR;
  const float inv_n = 1.0f / (float)N;
  float g[C][8], b[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = 8 * (c * TPR + t);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[c][j] = 1.0f;
      b[c][j] = 0.0f;
    }
    if (gamma) load8(gamma, n, N, g[c]);
    if (beta) load8(beta, n, N, b[c]);
  }
  for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < M;
       m += (int64_t)gridDim.x * RPB) {
    float v[C][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) load8(x + m * ldx, 8 * (c * TPR + t), N, v[c]);
#pragma unroll
    for (int c = 0; c < C; ++c)
      s[0] += ((v[c][0] + v[c][1]) + (v[c][2] + v[c][3])) +
              ((v[c][4] + v[c][5]) + (v[c][6] + v[c][7]));
    row_sum<TPR, 1>(s, lds, flip);
    const float mu = s[0] * inv_n;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[c][j] = 8 * (c * TPR + t) + j < N ? v[c][j] - mu : 0.0f;
        s[0] = fmaf(v[c][j], v[c][j], s[0]);
      }
    row_sum<TPR, 1>(s, lds, flip);
    const float r = 1.0f / sqrtf(s[0] * inv_n + eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = fmaf(v[c][j] * r, g[c][j], b[c][j]);
      store8(y + m * ldy, 8 * (c * TPR + t), N, v[c]);
    }
    if (t == 0) {
      if (mean) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
}

// The gradient, bound by HBM as well: x and dy are read and dx written once;
// gamma and the block's column sums stay in registers.  A block takes every
// gridDim.x-th group of rows and leaves its sums in row blockIdx.x of `part`
// (2 x N: dgamma, then dbeta); rows of one block's waves (TPR = 64) are joined
// through LDS, wave after wave.
template <typename T, int TPR, int C>
__global__ void __launch_bounds__(block_of(TPR))
    ln_bwd_kernel(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                  const float *__restrict__ gamma, const float *__restrict__ mean,
                  const float *__restrict__ rstd, T *__restrict__ dx, int64_t lddx,
                  float *__restrict__ part, int64_t M, int N) {
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float lds[4 * (TPR / 64)];
  __shared__ float join[RPB > 1 ? 2 * C * 8 * TPR : 1];
  int flip = 0;
  const int t = threadIdx.x % TPR;
  const float inv_n = 1.0f / (float)N;
  float g[C][8], ag[C][8], ab[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int n = 8 * (c * TPR + t) + j;
      g[c][j] = gamma ? (n < N ? gamma[n] : 0.0f) : 1.0f;
      ag[c][j] = ab[c][j] = 0.0f;
    }
  for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < M;
       m += (int64_t)gridDim.x * RPB) {
    float xh[C][8], d[C][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load8(x + m * ldx, 8 * (c * TPR + t), N, xh[c]);
      load8(dy + m * lddy, 8 * (c * TPR + t), N, d[c]);  // zero past N: no part of any sum
    }
    const float mu = mean[m], r = rstd[m];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[c][j] = 8 * (c * TPR + t) + j < N ? (xh[c][j] - mu) * r : 0.0f;
        ag[c][j] = fmaf(d[c][j], xh[c][j], ag[c][j]);
        ab[c][j] += d[c][j];
        d[c][j] *= g[c][j];
        s[0] += d[c][j];
        s[1] = fmaf(d[c][j], xh[c][j], s[1]);
      }
    row_sum<TPR, 2>(s, lds, flip);
    const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[c][j] = (d[c][j] - c1 - xh[c][j] * c2) * r;
      store8(dx + m * lddx, 8 * (c * TPR + t), N, d[c]);
    }
  }
  if (!part) return;
  if (RPB > 1) {
    const int w = threadIdx.x / TPR;
#pragma unroll 1
    for (int k = 0; k < RPB; ++k) {
      if (w == k) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float *p = join + (c * 8 + j) * TPR + t;
            if (k > 0) {
              ag[c][j] += p[0];
              ab[c][j] += p[C * 8 * TPR];
            }
            p[0] = ag[c][j];
            p[C * 8 * TPR] = ab[c][j];
          }
      }
      __syncthreads();
    }
    if (w != RPB - 1) return;
  }
  float *pg = part + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int n = 8 * (c * TPR + t) + j;
      if (n < N) {
        pg[n] = ag[c][j];
        pg[N + n] = ab[c][j];
      }
    }
}

// Rows too long for registers: one block per row, the row read again from
// the caches for each pass; the gradient's column sums are kept in `part`.
constexpr int kLongThreads = 1024;

template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    ln_fwd_long_kernel(const T *__restrict__ x, int64_t ldx, const float *__restrict__ gamma,
                       const float *__restrict__ beta, T *__restrict__ y, int64_t ldy,
                       float *__restrict__ mean, float *__restrict__ rstd, int64_t M, int N,
                       float eps) {
  __shared__ float lds[2 * (kLongThreads / 64)];
  int flip = 0;
  const float inv_n = 1.0f / (float)N;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const T *xr = x + m * ldx;
    float s[1] = {0.0f};
    for (int n = threadIdx.x; n < N; n += kLongThreads) s[0] += (float)xr[n];
    row_sum<kLongThreads, 1>(s, lds, flip);
    const float mu = s[0] * inv_n;
    s[0] = 0.0f;
    for (int n = threadIdx.x; n < N; n += kLongThreads) {
      const float d = (float)xr[n] - mu;
      s[0] = fmaf(d, d, s[0]);
    }
    row_sum<kLongThreads, 1>(s, lds, flip);
    const float r = 1.0f / sqrtf(s[0] * inv_n + eps);
    for (int n = threadIdx.x; n < N; n += kLongThreads) {
      const float v = ((float)xr[n] - mu) * r;
      y[m * ldy + n] = (T)fmaf(v, gamma ? gamma[n] : 1.0f, beta ? beta[n] : 0.0f);
    }
    if (threadIdx.x == 0) {
      if (mean) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    ln_bwd_long_kernel(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                       const float *__restrict__ gamma, const float *__restrict__ mean,
                       const float *__restrict__ rstd, T *__restrict__ dx, int64_t lddx,
                       float *__restrict__ part, int64_t M, int N) {
  __shared__ float lds[4 * (kLongThreads / 64)];
  int flip = 0;
  const float inv_n = 1.0f / (float)N;
  float *pg = part ? part + (int64_t)blockIdx.x * 2 * N : nullptr;
  bool first = true;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const T *xr = x + m * ldx, *dr = dy + m * lddy;
    const float mu = mean[m], r = rstd[m];
    float s[2] = {0.0f, 0.0f};
    for (int n = threadIdx.x; n < N; n += kLongThreads) {
      const float d = (float)dr[n], xh = ((float)xr[n] - mu) * r;
      const float g = gamma ? d * gamma[n] : d;
      s[0] += g;
      s[1] = fmaf(g, xh, s[1]);
      if (pg) {
        pg[n] = first ? d * xh : fmaf(d, xh, pg[n]);
        pg[N + n] = first ? d : pg[N + n] + d;
      }
    }
    row_sum<kLongThreads, 2>(s, lds, flip);
    const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
    for (int n = threadIdx.x; n < N; n += kLongThreads) {
      const float d = (float)dr[n], xh = ((float)xr[n] - mu) * r;
      const float g = gamma ? d * gamma[n] : d;
      dx[m * lddx + n] = (T)((g - c1 - xh * c2) * r);
    }
    first = false;
  }
}

// Columns' sums over the P partial rows, in a fixed order: 16 columns x 16
// parts of the rows per block, the parts joined through LDS.
__global__ void __launch_bounds__(256)
    ln_bwd_finish_kernel(const float *__restrict__ part, int P, int N, float *__restrict__ dgamma,
                         float *__restrict__ dbeta) {
  __shared__ float lds[16][17];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t i = (int64_t)blockIdx.x * 16 + c;
  float s = 0.0f;
  if (i < 2 * (int64_t)N) {
#pragma unroll 8
    for (int p = q; p < P; p += 16) s += part[(int64_t)p * 2 * N + i];
  }
  lds[q][c] = s;
  __syncthreads();
  if (q != 0 || i >= 2 * (int64_t)N) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += lds[k][c];
  if (i < N) dgamma[i] = s;
  else dbeta[i - N] = s;
}

// Threads per row and chunks per thread by the row's length: a wave holds up
// to 2048 values (no barrier), a block of up to 1024 threads two chunks each.
struct Shape {
  int tpr, c;  // tpr 0: the row is read again for each pass
};
Shape shape_of(int64_t N) {
  if (N <= 512) return {64, 1};
  if (N <= 1024) return {64, 2};
  if (N <= 2048) return {64, 4};
  if (N <= 4096) return {256, 2};
  if (N <= 8192) return {512, 2};
  if (N <= 16384) return {1024, 2};
  return {0, 0};
}

constexpr int64_t kBwdBlocks = 512;  // partial rows of the gradient at most

template <typename T>
void fwd(const void *xv, int64_t ldx, const float *gamma, const float *beta, void *yv, int64_t ldy,
         float *mean, float *rstd, int64_t M, int64_t N, float eps, hipStream_t s) {
  const T *x = static_cast<const T *>(xv);
  T *y = static_cast<T *>(yv);
  const Shape sh = shape_of(N);
#define BNN_LN(TPR, C)                                                                          \
  if (sh.tpr == TPR && sh.c == C) {                                                             \
    constexpr int B = block_of(TPR);                                                            \
    const int64_t want = (M + B / TPR - 1) / (B / TPR), cap = 256 * (2048 / B);                 \
    hipLaunchKernelGGL((ln_fwd_kernel<T, TPR, C>), dim3((unsigned)(want < cap ? want : cap)), \
                       dim3(B), 0, s, x, ldx, gamma, beta, y, ldy, mean, rstd, M, (int)N, eps); \
    return;                                                                                     \
  }
  BNN_LN(64, 1) BNN_LN(64, 2) BNN_LN(64, 4) BNN_LN(256, 2) BNN_LN(512, 2) BNN_LN(1024, 2)
#undef BNN_LN
  hipLaunchKernelGGL((ln_fwd_long_kernel<T>), dim3((unsigned)(M < 512 ? M : 512)),
                     dim3(kLongThreads), 0, s, x, ldx, gamma, beta, y, ldy, mean, rstd, M, (int)N,
                     eps);
}

template <typename T>
void bwd(const void *dyv, int64_t lddy, const void *xv, int64_t ldx, const float *gamma,
         const float *mean, const float *rstd, void *dxv, int64_t lddx, float *part, int64_t M,
         int64_t N, int64_t P, hipStream_t s) {
  const T *dy = static_cast<const T *>(dyv), *x = static_cast<const T *>(xv);
  T *dx = static_cast<T *>(dxv);
  const Shape sh = shape_of(N);
#define BNN_LN(TPR, C)                                                                         \
  if (sh.tpr == TPR && sh.c == C) {                                                            \
    hipLaunchKernelGGL((ln_bwd_kernel<T, TPR, C>), dim3((unsigned)P), dim3(block_of(TPR)), \
                       0, s, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, part, M, (int)N);  \
    return;                                                                                    \
  }
  BNN_LN(64, 1) BNN_LN(64, 2) BNN_LN(64, 4) BNN_LN(256, 2) BNN_LN(512, 2) BNN_LN(1024, 2)
#undef BNN_LN
  hipLaunchKernelGGL((ln_bwd_long_kernel<T>), dim3((unsigned)P), dim3(kLongThreads), 0, s, dy, lddy,
                     x, ldx, gamma, mean, rstd, dx, lddx, part, M, (int)N);
}

}  // namespace

int64_t layernorm_bwd_partials(int64_t M, int64_t N) {
  const Shape sh = shape_of(N);
  const int64_t rpb = sh.tpr == 64 ? 4 : 1;
  const int64_t groups = (M + rpb - 1) / rpb;
  return groups < kBwdBlocks ? groups : kBwdBlocks;
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
    if (dtype == BNN_FP32)
      bwd<float>(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, p, M, N, P, s);
    else
      bwd<bf16_t>(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, p, M, N, P, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dgamma) {
    hipLaunchKernelGGL(ln_bwd_finish_kernel, dim3((unsigned)((2 * N + 15) / 16)), dim3(256), 0, s,
                       part, (int)P, (int)N, dgamma, dbeta);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace bnn
