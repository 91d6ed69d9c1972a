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
// row's alignment (gfx950 serves unaligned vector accesses); a row's last
// elements are accessed one by one (EVEN: N is a multiple of 8, there are
// none).  The bits stay packed until they are used, so that a load can be in
// flight across other work, and are zero past N.

template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};

template <bool EVEN, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *row, int n, int N) {
  Raw<T> r;
#pragma unroll
  for (unsigned i = 0; i < 2 * sizeof(T); ++i) r.w[i] = 0;
  if (EVEN ? n < N : n + 8 <= N) {
    __builtin_memcpy(r.w, row + n, sizeof(r.w));
  } else if (!EVEN && n < N) {
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      if (n + j < N) {
        if (sizeof(T) == 4) r.w[j] = __builtin_bit_cast(uint32_t, (float)row[n + j]);
        else r.w[j / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, (bf16_t)row[n + j]) << (16 * (j & 1));
      }
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ float value(const Raw<T> &r, int j) {
  if (sizeof(T) == 4) return __uint_as_float(r.w[j]);
  return __uint_as_float((j & 1) ? r.w[j / 2] & 0xFFFF0000u : r.w[j / 2] << 16);
}

template <bool EVEN, typename T>
__device__ __forceinline__ void store8(T *row, int n, int N, const float v[8]) {
  if (EVEN ? n < N : n + 8 <= N) {
    T r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (T)v[j];
    __builtin_memcpy(row + n, r, sizeof(r));
  } else if (!EVEN) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (n + j < N) row[n + j] = (T)v[j];
  }
}

// `v` where element n + j exists, else 0.
template <bool EVEN>
__device__ __forceinline__ float where_in(float v, int n, int j, int N) {
  return n + (EVEN ? 0 : j) < N ? v : 0.0f;
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
// registers of a block that walks over rows.  16384 x 4096: bf16 49 us, 5.4 TB/s,
// fp32 104 us, 5.1 TB/s (a large copy reaches 5.1); one row of 4096: 2.5 us, the
// launch and two joins of the block's sums.
template <typename T, int TPR, int C, bool EVEN>
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
    const Raw<float> rg = gamma ? load_raw<EVEN>(gamma, n, N) : Raw<float>();
    const Raw<float> rb = beta ? load_raw<EVEN>(beta, n, N) : Raw<float>();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[c][j] = gamma ? value(rg, j) : 1.0f;
      b[c][j] = beta ? value(rb, j) : 0.0f;
    }
  }
  for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < M;
       m += (int64_t)gridDim.x * RPB) {
    Raw<T> raw[C];
    float v[C][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = load_raw<EVEN>(x + m * ldx, 8 * (c * TPR + t), N);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = value(raw[c], j);
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
        v[c][j] -= where_in<EVEN>(mu, 8 * (c * TPR + t), j, N);
        s[0] = fmaf(v[c][j], v[c][j], s[0]);
      }
    row_sum<TPR, 1>(s, lds, flip);
    const float r = 1.0f / sqrtf(s[0] * inv_n + eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = fmaf(v[c][j] * r, g[c][j], b[c][j]);
      store8<EVEN>(y + m * ldy, 8 * (c * TPR + t), N, v[c]);
    }
    if (t == 0) {
      if (mean) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
}

// Column sums of 64 columns over all rows, by a whole block, when there are so
// few rows that reading them a second time (from the caches) is cheaper than
// a second launch: the sums need only the forward pass's statistics.
template <typename T>
__device__ void column_sums(const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *mean,
                            const float *rstd, float *dgamma, float *dbeta, int M, int N,
                            int n0, float *lds) {
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6, W = blockDim.x >> 6;
  const int n = n0 + c < N ? n0 + c : N - 1;
  float sg = 0.0f, sb = 0.0f;
#pragma unroll 4
  for (int m = w; m < M; m += W) {
    const float d = (float)dy[m * lddy + n];
    sg = fmaf(d, ((float)x[m * ldx + n] - mean[m]) * rstd[m], sg);
    sb += d;
  }
  lds[w * 64 + c] = sg;
  lds[(W + w) * 64 + c] = sb;
  __syncthreads();
  if (w < 2 && n0 + c < N) {
    float s = 0.0f;
    for (int k = 0; k < W; ++k) s += lds[(w * W + k) * 64 + c];
    (w == 0 ? dgamma : dbeta)[n0 + c] = s;
  }
}

// The gradient, bound by HBM as well: x and dy are read and dx written once
// (16384 x 4096 bf16: 80 us + 7 us for the finish, 4.6 TB/s in all);
// gamma and the block's column sums stay in registers.  A block takes every
// gridDim.x-th group of rows and leaves its sums in row blockIdx.x of `part`
// (2 x N: dgamma, then dbeta); rows of one block's waves (TPR = 64) are joined
// through LDS, wave after wave.  DIRECT: blocks from `row_blocks` on take 64
// columns each instead and write dgamma (`part`) and dbeta themselves.
template <typename T, int TPR, int C, bool EVEN, bool DIRECT>
__global__ void __launch_bounds__(block_of(TPR))
    ln_bwd_kernel(const T *__restrict__ dy, int64_t lddy, const T *__restrict__ x, int64_t ldx,
                  const float *__restrict__ gamma, const float *__restrict__ mean,
                  const float *__restrict__ rstd, T *__restrict__ dx, int64_t lddx,
                  float *__restrict__ part, float *__restrict__ dbeta, int64_t M, int N,
                  int row_blocks) {
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float lds[4 * (TPR / 64)];
  __shared__ float join[DIRECT ? 2 * block_of(TPR) : (RPB > 1 ? 2 * C * 8 * TPR : 1)];
  if (DIRECT && (int)blockIdx.x >= row_blocks) {
    column_sums(dy, lddy, x, ldx, mean, rstd, part, dbeta, (int)M, N,
                ((int)blockIdx.x - row_blocks) * 64, join);
    return;
  }
  int flip = 0;
  const int t = threadIdx.x % TPR;
  const float inv_n = 1.0f / (float)N;
  float g[C][8], ag[C][8], ab[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Raw<float> rg = gamma ? load_raw<EVEN>(gamma, 8 * (c * TPR + t), N) : Raw<float>();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[c][j] = gamma ? value(rg, j) : 1.0f;
      ag[c][j] = ab[c][j] = 0.0f;
    }
  }
  // The next row's values are loaded before this row's sums are joined: few
  // blocks keep `part` small, and each keeps two rows in flight.
  Raw<T> nx[C], nd[C];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](int64_t m) {
    nmu = mean[m];
    nr = rstd[m];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      nx[c] = load_raw<EVEN>(x + m * ldx, 8 * (c * TPR + t), N);
      nd[c] = load_raw<EVEN>(dy + m * lddy, 8 * (c * TPR + t), N);
    }
  };
  const int64_t step = (int64_t)row_blocks * RPB;
  int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (m < M) fetch(m);
  for (; m < M; m += step) {
    float xh[C][8], d[C][8], s[2] = {0.0f, 0.0f};
    const float mu = nmu, r = nr;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // zero past N: no part of any sum
        xh[c][j] = value(nx[c], j) - where_in<EVEN>(mu, 8 * (c * TPR + t), j, N);
        d[c][j] = value(nd[c], j);
      }
    fetch(m + step < M ? m + step : m);  // the last row again: in bounds, unused
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[c][j] *= r;
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
      store8<EVEN>(dx + m * lddx, 8 * (c * TPR + t), N, d[c]);
    }
  }
  if (DIRECT || !part) return;
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
  for (int c = 0; c < C; ++c) {
    store8<EVEN>(pg, 8 * (c * TPR + t), N, ag[c]);
    store8<EVEN>(pg + N, 8 * (c * TPR + t), N, ab[c]);
  }
}

// Rows too long for registers: one block per row, the row read again from
// the caches for each pass; the gradient's column sums are kept in `part`.
// 2048 x 20000 bf16: forward 97 us (1.7 TB/s of x and y), gradient 342 + 14 us:
// element by element, three dependent passes with a block's join between them.
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
// parts of the rows per block and turn, the parts joined through LDS.
__global__ void __launch_bounds__(256)
    ln_bwd_finish_kernel(const float *__restrict__ part, int P, int N, float *__restrict__ dgamma,
                         float *__restrict__ dbeta) {
  __shared__ float lds[16][17];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t columns = 2 * (int64_t)N;
  for (int64_t i0 = (int64_t)blockIdx.x * 16; i0 < columns; i0 += (int64_t)gridDim.x * 16) {
    const int64_t i = i0 + c;
    float s = 0.0f;
    if (i < columns) {
#pragma unroll 8
      for (int p = q; p < P; p += 16) s += part[p * columns + i];
    }
    __syncthreads();  // the last turn's parts have been read
    lds[q][c] = s;
    __syncthreads();
    if (q != 0 || i >= columns) continue;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += lds[k][c];
    if (i < N) dgamma[i] = s;
    else dbeta[i - N] = s;
  }
}

// Threads per row and chunks per thread by the row's length: a wave holds up
// to 1024 values (no barrier), a block of up to 1024 threads two chunks each.
struct Shape {
  int tpr, c;  // tpr 0: the row is read again for each pass
};
Shape shape_of(int64_t N) {
  if (N <= 512) return {64, 1};
  if (N <= 1024) return {64, 2};
  if (N <= 2048) return {256, 1};
  if (N <= 4096) return {256, 2};
  if (N <= 8192) return {512, 2};
  if (N <= 16384) return {1024, 2};
  return {0, 0};
}

template <typename T, bool EVEN>
void fwd(const void *xv, int64_t ldx, const float *gamma, const float *beta, void *yv, int64_t ldy,
         float *mean, float *rstd, int64_t M, int64_t N, float eps, hipStream_t s) {
  const T *x = static_cast<const T *>(xv);
  T *y = static_cast<T *>(yv);
  const Shape sh = shape_of(N);
#define BNN_LN(TPR, C)                                                                          \
  if (sh.tpr == TPR && sh.c == C) {                                                             \
    constexpr int B = block_of(TPR);                                                            \
    const int64_t want = (M + B / TPR - 1) / (B / TPR), cap = 256 * (2048 / B);                 \
    hipLaunchKernelGGL((ln_fwd_kernel<T, TPR, C, EVEN>), dim3((unsigned)(want < cap ? want : cap)), \
                       dim3(B), 0, s, x, ldx, gamma, beta, y, ldy, mean, rstd, M, (int)N, eps); \
    return;                                                                                     \
  }
  BNN_LN(64, 1) BNN_LN(64, 2) BNN_LN(256, 1) BNN_LN(256, 2) BNN_LN(512, 2) BNN_LN(1024, 2)
#undef BNN_LN
  hipLaunchKernelGGL((ln_fwd_long_kernel<T>), dim3((unsigned)(M < 512 ? M : 512)),
                     dim3(kLongThreads), 0, s, x, ldx, gamma, beta, y, ldy, mean, rstd, M, (int)N,
                     eps);
}

// Up to 64 rows for each wave of a block (and no longer rows than a block
// holds) the column sums are taken straight from the inputs, in the same
// launch: 256 x 4096 bf16 7.7 us against 13.2, 1024 x 16384 37 against 55;
// beyond that the partial rows win (1024 x 4096: 20 us against 49).
bool direct_sums(int64_t M, int64_t N) {
  const Shape sh = shape_of(N);
  return sh.tpr != 0 && M <= block_of(sh.tpr);
}

template <typename T, bool EVEN>
void bwd(const void *dyv, int64_t lddy, const void *xv, int64_t ldx, const float *gamma,
         const float *mean, const float *rstd, void *dxv, int64_t lddx, float *dgamma, float *dbeta,
         float *part, int64_t M, int64_t N, int64_t P, hipStream_t s) {
  const T *dy = static_cast<const T *>(dyv), *x = static_cast<const T *>(xv);
  T *dx = static_cast<T *>(dxv);
  const Shape sh = shape_of(N);
  const bool direct = dgamma && direct_sums(M, N);
#define BNN_LN(TPR, C)                                                                            \
  if (sh.tpr == TPR && sh.c == C) {                                                               \
    if (direct) {                                                                                 \
      const int rb = (int)((M + block_of(TPR) / TPR - 1) / (block_of(TPR) / TPR));                \
      hipLaunchKernelGGL((ln_bwd_kernel<T, TPR, C, EVEN, true>),                                  \
                         dim3((unsigned)(rb + (N + 63) / 64)), dim3(block_of(TPR)), 0, s, dy,     \
                         lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, M, (int)N, rb); \
    } else {                                                                                      \
      hipLaunchKernelGGL((ln_bwd_kernel<T, TPR, C, EVEN, false>), dim3((unsigned)P),              \
                         dim3(block_of(TPR)), 0, s, dy, lddy, x, ldx, gamma, mean, rstd, dx,      \
                         lddx, dgamma ? part : nullptr, nullptr, M, (int)N, (int)P);              \
    }                                                                                             \
    return;                                                                                       \
  }
  BNN_LN(64, 1) BNN_LN(64, 2) BNN_LN(256, 1) BNN_LN(256, 2) BNN_LN(512, 2) BNN_LN(1024, 2)
#undef BNN_LN
  hipLaunchKernelGGL((ln_bwd_long_kernel<T>), dim3((unsigned)P), dim3(kLongThreads), 0, s, dy, lddy,
                     x, ldx, gamma, mean, rstd, dx, lddx, dgamma ? part : nullptr, M, (int)N);
}

}  // namespace

// Blocks of the gradient, equal turns for each: enough to fill the card with
// two (256 threads) or one (more) per CU, few so that `part` stays small.
static int64_t row_blocks(int64_t M, int64_t N) {
  const Shape sh = shape_of(N);
  const int64_t rpb = sh.tpr == 64 ? 4 : 1, cap = sh.tpr <= 256 && sh.tpr > 0 ? 512 : 256;
  const int64_t groups = (M + rpb - 1) / rpb;
  if (groups <= 0) return 0;
  const int64_t turns = (groups + cap - 1) / cap;
  return (groups + turns - 1) / turns;
}

int64_t layernorm_bwd_partials(int64_t M, int64_t N) {
  return direct_sums(M, N) ? 0 : row_blocks(M, N);
}

hipError_t launch_layernorm_fwd(const void *x, int dtype, int64_t ldx, const float *gamma,
                                const float *beta, void *y, int64_t ldy, float *mean, float *rstd,
                                int64_t M, int64_t N, float eps, hipStream_t s) {
  const auto run = dtype == BNN_FP32 ? (N % 8 == 0 ? fwd<float, true> : fwd<float, false>)
                                     : (N % 8 == 0 ? fwd<bf16_t, true> : fwd<bf16_t, false>);
  run(x, ldx, gamma, beta, y, ldy, mean, rstd, M, N, eps, s);
  return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                int dtype, const float *gamma, const float *mean,
                                const float *rstd, void *dx, int64_t lddx, float *dgamma,
                                float *dbeta, float *part, int64_t M, int64_t N, hipStream_t s) {
  const int64_t P = row_blocks(M, N);
  if (P > 0) {
    const auto run = dtype == BNN_FP32 ? (N % 8 == 0 ? bwd<float, true> : bwd<float, false>)
                                       : (N % 8 == 0 ? bwd<bf16_t, true> : bwd<bf16_t, false>);
    run(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, part, M, N, P, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dgamma && (M == 0 || layernorm_bwd_partials(M, N) > 0)) {
    // A launch takes less than 2^32 threads: wider rows go round in turns.
    const int64_t want = (2 * N + 15) / 16, blocks = want < (1 << 20) ? want : (1 << 20);
    hipLaunchKernelGGL(ln_bwd_finish_kernel, dim3((unsigned)blocks), dim3(256), 0, s, part, (int)P,
                       (int)N, dgamma, dbeta);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace bnn
