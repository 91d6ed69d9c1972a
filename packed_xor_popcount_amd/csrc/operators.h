// operators.h -- declarations of the operators beside the grouped sign-weight
// products (router, sum of the experts' outputs, low-rank adapters) and the
// device helpers that they share.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bnn.h"

namespace bnn {

// Router and its gradient (arguments as in the C-ABI; already validated).
constexpr int64_t kRouteMaxExperts = 1024;
constexpr int64_t kRouteMaxK = 32;
int64_t route_fwd_workspace(int64_t T, int64_t E, int64_t k);
struct RouteOut {
  int32_t *experts;
  float *weights;
  int32_t *place, *rows, *offsets, *counts;
  float *stats, *slope, *loss;
};
hipError_t launch_route_fwd(const void *z, int dtype, int64_t ldz, const uint8_t *valid,
                            const RouteOut &out, void *workspace, int64_t T, int E, int k,
                            bool normalise, hipStream_t s);
hipError_t launch_route_bwd(const void *z, int dtype, int64_t ldz, const int32_t *experts,
                            const float *weights, const float *stats, const float *slope,
                            const float *dweights, const float *dloss, void *dz, int64_t lddz,
                            int64_t T, int E, int k, bool normalise, hipStream_t s);

// Indices 0 .. n - 1 sorted by ids[i] in [0, G), stable, with -1 for those of
// other ids behind them; offsets: G + 1 group bounds.  G <= kRouteMaxExperts.
int64_t group_rows_workspace(int64_t n, int64_t G);
hipError_t launch_group_rows(const int32_t *ids, int32_t *rows, int32_t *offsets, void *workspace,
                             int64_t n, int G, hipStream_t s);

// Sum of the experts' outputs and its gradient.  `y` is fp32, bf16 or (ydtype
// BNN_F8) the block-scaled 8-bit form with scale bytes ys.
hipError_t launch_combine_fwd(const void *y, int ydtype, int64_t ldy, int64_t R,
                              const int32_t *place, const float *weights, const void *residual,
                              int64_t ldr, void *out, int dtype, int64_t ldo, int64_t T, int64_t N,
                              int k, hipStream_t s);
hipError_t launch_combine_bwd(const void *dout, int dtype, int64_t lddo, const void *y,
                              const uint8_t *ys, int ydtype, int64_t ldy, int64_t R,
                              const int32_t *place, const float *weights, void *dy, int dydtype,
                              int64_t lddy, float *dweights, int64_t T, int64_t N, int k,
                              hipStream_t s);

// Low-rank adapters and their gradient.
constexpr int64_t kAdapterMaxRank = 128;
constexpr int64_t kAdapterMaxRows = int64_t(1) << 27;
int64_t adapter_fwd_workspace(int64_t T, int64_t N, int64_t r, int64_t L);
hipError_t launch_adapter_fwd(const uint16_t *x, int64_t ldx, const int32_t *ids,
                              const uint16_t *a, const uint16_t *b, const float *scale,
                              const void *base, int64_t ldb, void *out, int64_t ldo, int dtype,
                              float *u, void *workspace, int64_t T, int64_t K, int64_t N, int r,
                              int L, hipStream_t s);
int64_t adapter_bwd_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L);
struct AdapterGrad {
  const uint16_t *dy;
  int64_t lddy;
  const void *x;  // bf16 rows, or with xs the block-scaled 8-bit form
  const uint8_t *xs;
  int64_t ldx;
  const float *u;
  const int32_t *ids;
  const uint16_t *a, *b;
  const float *scale;
  const void *base;
  int64_t ldb;
  void *dx;
  int64_t lddx;
  int dtype;
  bool sums;  // da and db are wanted
  float *da, *db;
};
hipError_t launch_adapter_bwd(const AdapterGrad &g, void *workspace, int64_t T, int64_t K,
                              int64_t N, int r, int L, hipStream_t s);

// Eight neighbours of a row, from element n on (a multiple of 8), as they are
// in memory.  gfx950 serves vector accesses at any alignment, so a row of N >= 8
// is read by whole vectors only: the last one ends with the row, and
// settle_chunk, called when the value is used, moves its elements into place
// (zeros past N).  Shorter rows are read element by element.
template <typename T>
struct Chunk {
  uint32_t w[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Chunk<T> raw_chunk_long(const T *row, int n, int N) {  // N >= 8
  Chunk<T> c;
  __builtin_memcpy(c.w, row + (n < N - 8 ? n : N - 8), sizeof(c.w));
  return c;
}

template <typename T>
__device__ __forceinline__ Chunk<T> raw_chunk(const T *row, int n, int N) {
  if (N >= 8) return raw_chunk_long(row, n, N);
  Chunk<T> c;
#pragma unroll
  for (unsigned i = 0; i < 2 * sizeof(T); ++i) c.w[i] = 0;
#pragma unroll
  for (int j = 0; j < 7; ++j) {
    if (n + j < N) {
      if (sizeof(T) == 4) {
        __builtin_memcpy(&c.w[j], row + n + j, 4);
      } else {
        uint16_t h;
        __builtin_memcpy(&h, row + n + j, 2);
        c.w[j / 2] |= (uint32_t)h << (16 * (j & 1));
      }
    }
  }
  return c;
}

template <typename T>
__device__ __forceinline__ void settle_chunk(Chunk<T> &c, int n, int N) {
  if (N < 8 || n + 8 <= N) return;
  constexpr int W = 2 * sizeof(T), PER = 4 / sizeof(T);  // words, elements of one
  const int by = n - (N - 8);
#pragma unroll
  for (int d = 4; d >= PER; d /= 2) {  // by d elements
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t from = i + d / PER < W ? c.w[i + d / PER] : 0u;
      c.w[i] = (by & d) ? from : c.w[i];
    }
  }
  if (PER == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t up = i + 1 < W ? c.w[i + 1] : 0u;
      c.w[i] = (by & 1) ? __builtin_amdgcn_alignbit(up, c.w[i], 16) : c.w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) c.w[i] = by < 8 ? c.w[i] : 0u;
}

template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T *row, int n, int N) {
  Chunk<T> c = raw_chunk(row, n, N);
  settle_chunk(c, n, N);
  return c;
}

template <typename T>
__device__ __forceinline__ float chunk_value(const Chunk<T> &c, int j) {
  if (sizeof(T) == 4) return __uint_as_float(c.w[j]);
  return __uint_as_float((j & 1) ? c.w[j / 2] & 0xFFFF0000u : c.w[j / 2] << 16);
}

template <typename T>
__device__ __forceinline__ void store_chunk(T *row, int n, int N, const float (&v)[8]) {
  T r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = (T)v[j];
  if (n + 8 <= N) {
    __builtin_memcpy(row + n, r, sizeof(r));
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (n + j < N) row[n + j] = r[j];
}

// Sums over the 64 lanes and the largest of them in VALU instructions alone:
// within rows of 16 lanes by shifts, across them by the row broadcasts; lane
// 63 holds the result, which every lane receives.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float x, float other) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(x), CTRL,
                                                    ROWS, 0xF, false));
}
__device__ __forceinline__ float lane63(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_add(float v) {
  v += dpp_or<0x111, 0xF>(v, 0.0f);  // row_shr 1
  v += dpp_or<0x112, 0xF>(v, 0.0f);  // row_shr 2
  v += dpp_or<0x114, 0xF>(v, 0.0f);  // row_shr 4
  v += dpp_or<0x118, 0xF>(v, 0.0f);  // row_shr 8
  v += dpp_or<0x142, 0xA>(v, 0.0f);  // row_bcast 15, into rows 1 and 3
  v += dpp_or<0x143, 0xC>(v, 0.0f);  // row_bcast 31, into rows 2 and 3
  return lane63(v);
}
__device__ __forceinline__ float wave_max(float v) {  // of numbers and -inf
  v = fmaxf(v, dpp_or<0x111, 0xF>(v, v));
  v = fmaxf(v, dpp_or<0x112, 0xF>(v, v));
  v = fmaxf(v, dpp_or<0x114, 0xF>(v, v));
  v = fmaxf(v, dpp_or<0x118, 0xF>(v, v));
  v = fmaxf(v, dpp_or<0x142, 0xA>(v, v));
  v = fmaxf(v, dpp_or<0x143, 0xC>(v, v));
  return lane63(v);
}

}  // namespace bnn
