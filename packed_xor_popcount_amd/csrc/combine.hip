// combine.hip -- the sum of the experts' outputs at each token, and its gradient.
//
//   out_t = residual_t + sum_j w_tj y[place_tj]          (slots in order j)
//   dy[place_tj] = w_tj dout_t        dw_tj = <dout_t, y[place_tj]>
//
// A slot whose place is negative has no expert and adds nothing; place = -2 - r
// names the row r of y that belongs to it, whose gradient is written as zeros.
// Sums are fp32; each output is rounded once.
#include "f8.h"
#include "operators.h"

namespace bnn {
namespace {

typedef __bf16 bf16_t;
typedef float v2f __attribute__((ext_vector_type(2)));

// Bound by HBM: k rows of y and the residual are read, a row is written.  A
// thread has eight columns of one token; all its rows' loads are in flight at
// once (K slots at a time).  8192 x 4096 bf16, 2 experts 45 us (5.9 TB/s: the
// last-level cache holds part of it); 4096 x 4096, 8 experts in fp32 113 us (5.3
// TB/s); 4 tokens 4.2 us.
template <typename Y, typename O, int K>
__global__ void __launch_bounds__(256)
    combine_fwd_kernel(const Y *__restrict__ y, int64_t ldy, int R,
                       const int32_t *__restrict__ place, const float *__restrict__ weights,
                       const O *residual, int64_t ldr, O *out,
                       int64_t ldo, int64_t T, int N, int k, int parts) {
  const int64_t t = blockIdx.x / (unsigned)parts;
  const int n = 8 * ((int)(blockIdx.x % (unsigned)parts) * (int)blockDim.x + (int)threadIdx.x);
  if (n >= N) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  Chunk<O> first;
  if (residual) first = raw_chunk(residual + t * ldr, n, N);
  for (int j0 = 0; j0 < k; j0 += K) {
    Chunk<Y> c[K];
    float w[K];
    bool has[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int p = j0 + j < k ? place[t * k + j0 + j] : -1;
      has[j] = p >= 0 && p < R;
      w[j] = !has[j] ? 0.0f : weights ? weights[t * k + j0 + j] : 1.0f;
      if (has[j]) c[j] = raw_chunk(y + p * ldy, n, N);
    }
    if (residual && j0 == 0) {
      settle_chunk(first, n, N);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = chunk_value(first, i);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (has[j]) {
        settle_chunk(c[j], n, N);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], chunk_value(c[j], i), acc[i]);
      }
    }
  }
  store_chunk(out + t * ldo, n, N, acc);
}

// Eight values of y: <d, y> over them.
template <typename Y>
struct Rows {
  const Y *y;
  int64_t ld;
  typedef Chunk<Y> Piece;
  __device__ __forceinline__ Piece load(int64_t row, int n, int N) const {
    return raw_chunk(y + row * ld, n, N);
  }
  static __device__ __forceinline__ float dot(Piece &c, const float (&d)[8], int n, int N, float s) {
    settle_chunk(c, n, N);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(d[i], chunk_value(c, i), s);
    return s;
  }
};

// The 8-bit form.  Eight neighbours share a block's scale, which each is multiplied
// by before its product (exactly: 448 * 2^119 and 2^-9 * 2^-127 are fp32 values), so
// that a sum leaves fp32's range only where the rows' own values take it there.  Of a
// scale byte over 246 the rest of the power of two multiplies the sum: a value of
// 2^128 (what magnitudes from 1.9375 * 2^127 on decode to) is never formed.
struct Rows8 {
  const uint8_t *q, *s;
  int64_t ldq, lds;
  struct Piece {
    uint32_t lo, hi, e;
  };
  __device__ __forceinline__ Piece load(int64_t row, int n, int) const {
    Piece p;
    uint2 v;
    __builtin_memcpy(&v, q + row * ldq + n, 8);  // rows are padded to whole blocks
    p.lo = v.x;
    p.hi = v.y;
    p.e = s[row * lds + n / kF8Block];
    return p;
  }
  static __device__ __forceinline__ float dot(const Piece &p, const float (&d)[8], int n, int N,
                                              float s) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(p.lo, false);
    const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8(p.lo, true);
    const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8(p.hi, false);
    const v2f e = __builtin_amdgcn_cvt_pk_f32_fp8(p.hi, true);
    const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
    const uint32_t held = p.e < 246 ? p.e : 246;
    const float scale = __uint_as_float(held ? held << 23 : 0x00400000u);
    const float rest = __uint_as_float((127 + p.e - held) << 23);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(d[i], n + i < N ? v[i] * scale : 0.0f, sum);
    return fmaf(sum, rest, s);
  }
};

struct None {  // no y: only dy is wanted
  struct Piece {};
  __device__ __forceinline__ Piece load(int64_t, int, int) const { return {}; }
  static __device__ __forceinline__ float dot(const Piece &, const float (&)[8], int, int, float s) {
    return s;
  }
};

// Bound by HBM: dout is read once, y's rows once, dy's rows are written once.
// W waves share a token; the K products of a group of slots are summed over the
// lanes, then over the waves in their order.  8192 x 4096, 4 experts, y in 8 bits:
// 97 us, 4.8 TB/s (four waves a token 89 us; while the scale multiplied a sum of eight,
// one wave took 104, four 112, non-temporal stores 115); 301 x 1000 fp32 5 us.
template <typename D, typename Y, typename G, int K, int W>
__global__ void __launch_bounds__(256)
    combine_bwd_kernel(const D *__restrict__ dout, int64_t lddo, Y y, int R,
                       const int32_t *__restrict__ place, const float *__restrict__ weights,
                       G *__restrict__ dy, int64_t lddy, float *__restrict__ dweights, int64_t T,
                       int N, int k) {
  __shared__ float join[4][K];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (4 / W) + wave / W;
  if (W == 1 && t >= T) return;  // W > 1: the grid is exact
  for (int j0 = 0; j0 < k; j0 += K) {
    int64_t row[K];
    float w[K], acc[K];
    bool has[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int p = j0 + j < k ? place[t * k + j0 + j] : -1;
      has[j] = p >= 0 && p < R;
      const int r = p >= 0 ? p : -2 - p;
      row[j] = r >= 0 && r < R ? r : -1;
      w[j] = has[j] ? (weights ? weights[t * k + j0 + j] : 1.0f) : 0.0f;
      acc[j] = 0.0f;
    }
    for (int n = 8 * (lane + 64 * (wave % W)); n < N; n += 512 * W) {
      Chunk<D> c = raw_chunk(dout + t * lddo, n, N);
      typename Y::Piece p[K];
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (has[j]) p[j] = y.load(row[j], n, N);
      float d[8];
      settle_chunk(c, n, N);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = chunk_value(c, i);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (has[j]) acc[j] = Y::dot(p[j], d, n, N, acc[j]);
        if (dy && row[j] >= 0) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = has[j] ? w[j] * d[i] : 0.0f;
          store_chunk(dy + row[j] * lddy, n, N, v);
        }
      }
    }
    if (!dweights) continue;
#pragma unroll
    for (int j = 0; j < K; ++j) acc[j] = wave_add(acc[j]);
    if (W == 1) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (lane == j && j0 + j < k) dweights[t * k + j0 + j] = acc[j];
    } else {
      __syncthreads();  // the group before has been read
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < K; ++j) join[wave][j] = acc[j];
      }
      __syncthreads();
      if (wave % W == 0 && lane < K && j0 + lane < k) {
        float s = 0.0f;
        for (int i = 0; i < W; ++i) s += join[wave + i][lane];
        dweights[t * k + j0 + lane] = s;
      }
    }
  }
}

template <typename Y, typename O>
hipError_t fwd(const void *y, int64_t ldy, int R, const int32_t *place, const float *weights,
               const void *residual, int64_t ldr, void *out, int64_t ldo, int64_t T, int N, int k,
               hipStream_t s) {
  int threads = 64;  // few tokens: more, smaller blocks
  if (T * ((N + 511) / 512) > 2048)
    while (threads < 256 && threads * 8 < N) threads *= 2;
  const int parts = (N + threads * 8 - 1) / (threads * 8);
  // a launch takes less than 2^32 threads
  const int64_t most = parts < (1 << 23) ? (int64_t(1) << 23) / parts : 1;
  for (int64_t t = 0; t < T; t += most) {
    const int64_t n = T - t < most ? T - t : most;
    const dim3 grid((unsigned)(n * parts));
    const Y *yt = static_cast<const Y *>(y);
    const O *r = residual ? static_cast<const O *>(residual) + t * ldr : nullptr;
    O *o = static_cast<O *>(out) + t * ldo;
    const float *w = weights ? weights + t * k : nullptr;
    const int32_t *p = place + t * k;
#define BNN_FWD(K) \
  combine_fwd_kernel<Y, O, K><<<grid, threads, 0, s>>>(yt, ldy, R, p, w, r, ldr, o, ldo, n, N, k, parts)
    if (k == 1) BNN_FWD(1);
    else if (k == 2) BNN_FWD(2);
    else if (k <= 4) BNN_FWD(4);
    else BNN_FWD(8);
#undef BNN_FWD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename D, typename Y, typename G, int K>
hipError_t bwd_k(const D *dout, int64_t lddo, const Y &y, int R, const int32_t *place,
                 const float *weights, G *dy, int64_t lddy, float *dweights, int64_t T, int N,
                 int k, hipStream_t s) {
  // Four waves a token while there are few of them.  (The bound stands as it was measured
  // before the 8-bit form's scale went to the values; since then four are faster at 8192
  // tokens too, see the kernel.)
  if (T < 4096) {
    combine_bwd_kernel<D, Y, G, K, 4><<<(unsigned)T, 256, 0, s>>>(
        dout, lddo, y, R, place, weights, dy, lddy, dweights, T, N, k);
    return hipGetLastError();
  }
  constexpr int64_t most = int64_t(1) << 24;  // a launch takes less than 2^32 threads
  for (int64_t t = 0; t < T; t += most) {
    const int64_t n = T - t < most ? T - t : most;
    combine_bwd_kernel<D, Y, G, K, 1><<<(unsigned)((n + 3) / 4), 256, 0, s>>>(
        dout + t * lddo, lddo, y, R, place + t * k, weights ? weights + t * k : nullptr, dy, lddy,
        dweights ? dweights + t * k : nullptr, n, N, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename D, typename Y, typename G>
hipError_t bwd_y(const void *dout, int64_t lddo, const Y &y, int R, const int32_t *place,
                 const float *weights, void *dy, int64_t lddy, float *dweights, int64_t T, int N,
                 int k, hipStream_t s) {
  const D *d = static_cast<const D *>(dout);
  G *g = static_cast<G *>(dy);
  if (k == 1) return bwd_k<D, Y, G, 1>(d, lddo, y, R, place, weights, g, lddy, dweights, T, N, k, s);
  if (k == 2) return bwd_k<D, Y, G, 2>(d, lddo, y, R, place, weights, g, lddy, dweights, T, N, k, s);
  if (k <= 4) return bwd_k<D, Y, G, 4>(d, lddo, y, R, place, weights, g, lddy, dweights, T, N, k, s);
  return bwd_k<D, Y, G, 8>(d, lddo, y, R, place, weights, g, lddy, dweights, T, N, k, s);
}

template <typename D, typename G>
hipError_t bwd(const void *dout, int64_t lddo, const void *y, const uint8_t *ys, int ydtype,
               int64_t ldy, int R, const int32_t *place, const float *weights, void *dy,
               int64_t lddy, float *dweights, int64_t T, int N, int k, hipStream_t s) {
  if (!dweights)
    return bwd_y<D, None, G>(dout, lddo, None{}, R, place, weights, dy, lddy, dweights, T, N, k, s);
  if (ydtype == BNN_F8)
    return bwd_y<D, Rows8, G>(dout, lddo,
                              Rows8{static_cast<const uint8_t *>(y), ys, f8_row_bytes(N),
                                    f8_scale_bytes(N)},
                              R, place, weights, dy, lddy, dweights, T, N, k, s);
  if (ydtype == BNN_FP32)
    return bwd_y<D, Rows<float>, G>(dout, lddo, Rows<float>{static_cast<const float *>(y), ldy}, R,
                                    place, weights, dy, lddy, dweights, T, N, k, s);
  return bwd_y<D, Rows<bf16_t>, G>(dout, lddo, Rows<bf16_t>{static_cast<const bf16_t *>(y), ldy}, R,
                                   place, weights, dy, lddy, dweights, T, N, k, s);
}

}  // namespace

hipError_t launch_combine_fwd(const void *y, int ydtype, int64_t ldy, int64_t R,
                              const int32_t *place, const float *weights, const void *residual,
                              int64_t ldr, void *out, int dtype, int64_t ldo, int64_t T, int64_t N,
                              int k, hipStream_t s) {
#define BNN_COMBINE(Y, O)                                                                          \
  fwd<Y, O>(y, ldy, (int)R, place, weights, residual, ldr, out, ldo, T, (int)N, k, s)
  if (ydtype == BNN_FP32)
    return dtype == BNN_FP32 ? BNN_COMBINE(float, float) : BNN_COMBINE(float, bf16_t);
  return dtype == BNN_FP32 ? BNN_COMBINE(bf16_t, float) : BNN_COMBINE(bf16_t, bf16_t);
#undef BNN_COMBINE
}

hipError_t launch_combine_bwd(const void *dout, int dtype, int64_t lddo, const void *y,
                              const uint8_t *ys, int ydtype, int64_t ldy, int64_t R,
                              const int32_t *place, const float *weights, void *dy, int dydtype,
                              int64_t lddy, float *dweights, int64_t T, int64_t N, int k,
                              hipStream_t s) {
#define BNN_COMBINE(D, G)                                                                          \
  bwd<D, G>(dout, lddo, y, ys, ydtype, ldy, (int)R, place, weights, dy, lddy, dweights, T, (int)N, \
            k, s)
  if (dtype == BNN_FP32)
    return dydtype == BNN_FP32 ? BNN_COMBINE(float, float) : BNN_COMBINE(float, bf16_t);
  return dydtype == BNN_FP32 ? BNN_COMBINE(bf16_t, float) : BNN_COMBINE(bf16_t, bf16_t);
#undef BNN_COMBINE
}

}  // namespace bnn
