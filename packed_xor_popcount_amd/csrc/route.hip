// route.hip -- the router of a mixture of experts and its gradient.
//
// Token t has E logits z; an expert is open to it where its logit is above
// -inf (and the token is valid).  With m = max z and p = exp(z - m) / sum exp(z - m):
//   choices   the k largest open logits, ties to the lowest index
//   weights   p of the choices, or (normalised) exp(z - m) over its sum over
//             the token's choices
//   place     slots (t, j) sorted by expert, stable: slot (t, j) is row
//             place[t][j] and rows[place] = t; slots without an expert follow
//             the last group (place = -2 - row, rows = -1)
//   loss      E sum_e f_e P_e with f_e = counts_e / (k Tv), P_e = sum_t p_te / Tv
//             over the Tv tokens that have an expert; slope_e = E f_e / Tv
// and, with the choices held fixed, for gradients dw and dl of weights and loss
//   g_e = dl slope_e (+ dw_j at the choices when not normalised)
//   dz_e = p_e (g_e - sum_i p_i g_i)  (+ w_j (dw_j - sum_i w_i dw_i) when normalised)
//
// Everything is fp32; the order of every sum goes by the sizes alone.
#include "operators.h"

#include <math.h>

namespace bnn {
namespace {

typedef __bf16 bf16_t;

// A wave per token: lane l holds the logits l + 64 i.
constexpr int threads_of(int vpl) { return vpl >= 16 ? 512 : 1024; }
constexpr int64_t kRouteBlocks = 256;  // most blocks: each leaves one row of partial sums

// Tokens of a block: a multiple of its waves, so that there are at most
// kRouteBlocks of them.
inline int64_t tokens_per_block(int64_t T, int threads) {
  const int64_t w = threads / 64;
  const int64_t c = (T + kRouteBlocks - 1) / kRouteBlocks;
  const int64_t least = 4 * w;
  return c < least ? least : (c + w - 1) / w * w;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_logits(const T *z, int E, float (&v)[VPL]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? (float)z[e] : -INFINITY;
  }
}

// The block's LDS.  `join` holds the waves' sums of p first, later the slots
// counted by wave and expert.
template <int THREADS>
struct Shared {
  int hist[kRouteMaxExperts + 1];    // this block's slots per expert
  int first[kRouteMaxExperts + 1];   // row of the block's next slot per expert
  int total[kRouteMaxExperts + 1];
  union {
    float sums[8192];                // waves x E
    uint16_t seen[8192 + 16];        // waves x (E + 1)
    int seg[2 * THREADS];
  } join;
  int wave[THREADS / 64];
  float fwave[THREADS / 64];
  int routed;
};

// Choices, weights and statistics of the block's tokens, their counts in
// sh.hist, the number of tokens with an expert in sh.routed and the sums of p
// in psum (E floats, or null).
template <typename T, int VPL>
__device__ void choose(const T *z, int64_t ldz, const uint8_t *valid, const RouteOut &o, int64_t t0,
                       int64_t t1, int E, int k, bool normalise, float *psum,
                       Shared<threads_of(VPL)> &sh) {
  constexpr int W = threads_of(VPL) / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < E; e += 64 * W) sh.hist[e] = 0;
  if (threadIdx.x == 0) sh.routed = 0;
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int routed = 0;
  for (int64_t t = t0 + wave; t < t1; t += W) {
    float v[VPL], key[VPL], ex[VPL];
    load_logits<T, VPL>(z + t * ldz, E, v);
    if (valid && !valid[t]) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = -INFINITY;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = v[i] > -INFINITY ? v[i] : -INFINITY;  // NaN is never chosen
      m = fmaxf(m, key[i]);
    }
    m = wave_max(m);
    const float mz = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      ex[i] = expf(v[i] - mz);
      sum += ex[i];
    }
    sum = wave_add(sum);
    const float rsum = sum == 0.0f ? 0.0f : 1.0f / sum;  // NaN where a logit is NaN or +inf
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = fmaf(ex[i], rsum, acc[i]);
    routed += m > -INFINITY;
    // the k largest, one after the other; lane j keeps choice j
    float best = -INFINITY, top = m;
    int chosen = -1;
    for (int j = 0; j < k && top > -INFINITY; ++j) {
      int at = VPL;  // this lane's lowest i that holds the largest value
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == top) at = i;
      uint64_t has = __ballot(at < VPL);
      int i0 = __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)has) - 1);
      if (VPL > 1 && (has & (has - 1))) {  // a tie: the lowest i, then the lowest lane
        for (i0 = 0; i0 < VPL; ++i0) {
          has = __ballot(at == i0);
          if (has) break;
        }
      }
      const int l0 = __ffsll((unsigned long long)has) - 1;
      if (lane == j) {
        best = top;
        chosen = l0 + 64 * i0;
      }
      float next = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (lane == l0 && i == i0) key[i] = -INFINITY;
        next = fmaxf(next, key[i]);
      }
      top = wave_max(next);
    }
    float w = chosen >= 0 ? expf(best - mz) : 0.0f;
    if (normalise) {
      const float s = wave_add(w);
      w = chosen >= 0 ? w / s + 0.0f * rsum : 0.0f;  // NaN where the statistics are
    } else if (chosen >= 0) {
      w *= rsum;
    }
    if (lane < k) {
      o.experts[t * k + lane] = chosen;
      o.weights[t * k + lane] = w;
      if (chosen >= 0) atomicAdd(&sh.hist[chosen], 1);
    }
    if (lane == 0) {
      o.stats[2 * t] = mz;
      o.stats[2 * t + 1] = rsum;
    }
  }
  if (lane == 0 && routed) atomicAdd(&sh.routed, routed);
  if (psum) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < E) sh.join.sums[wave * E + lane + 64 * i] = acc[i];
  }
  __syncthreads();
  if (psum) {
    for (int e = threadIdx.x; e < E; e += 64 * W) {
      float s = 0.0f;
      for (int w = 0; w < W; ++w) s += sh.join.sums[w * E + e];
      psum[e] = s;
    }
  }
}

// sh.total (slots of each expert over all blocks) -> sh.first: the expert's
// first row plus what the blocks before this one hold (sh.first on entry).
// Returns the number of rows that have an expert.
template <int THREADS>
__device__ int scan_experts(int E, Shared<THREADS> &sh, int32_t *offsets) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    const int n = e < E ? sh.total[e] : 0;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(inc, d, 64);
      if (lane >= d) inc += up;
    }
    if (lane == 63) sh.wave[wave] = inc;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < wave) before += sh.wave[w];
      all += sh.wave[w];
    }
    if (e < E) {
      sh.first[e] += before + inc - n;
      if (offsets) offsets[e] = before + inc - n;
    }
    carry += all;
    __syncthreads();
  }
  if (offsets && threadIdx.x == 0) offsets[E] = carry;
  return carry;
}

// Rows of the block's slots, in their order: sh.first holds the row of the
// next slot of each expert (index E: of the slots without one).
template <int THREADS>
__device__ void place_slots(const RouteOut &o, int64_t s0, int64_t s1, int E, int k,
                            Shared<THREADS> &sh) {
  constexpr int W = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t b = s0; b < s1; b += THREADS) {
    for (int i = threadIdx.x; i < W * (E + 1); i += THREADS) sh.join.seen[i] = 0;
    __syncthreads();
    const int64_t s = b + threadIdx.x;
    int e = s < s1 ? o.experts[s] : E;
    if (e < 0 || e >= E) e = E;
    uint64_t same = __ballot(s < s1);  // lanes of this wave with the same expert
    for (int bit = 1; bit <= E; bit <<= 1) {
      const uint64_t set = __ballot((e & bit) != 0);
      same &= (e & bit) ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (s < s1 && rank == 0) sh.join.seen[wave * (E + 1) + e] = (uint16_t)__popcll(same);
    __syncthreads();
    int row = 0;
    if (s < s1) {
      row = sh.first[e] + rank;
      for (int w = 0; w < wave; ++w) row += sh.join.seen[w * (E + 1) + e];
      if (o.place) o.place[s] = e < E ? row : -2 - row;
      o.rows[row] = e < E ? (int32_t)(s / k) : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += THREADS) {
      int n = 0;
      for (int w = 0; w < W; ++w) n += sh.join.seen[w * (E + 1) + i];
      sh.first[i] += n;
    }
    __syncthreads();
  }
}

// Counts, slope and loss from the experts' totals and sums of p.
template <int THREADS>
__device__ void finish(const RouteOut &o, const float *sums, int routed, int E, int k,
                       Shared<THREADS> &sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const double per = routed > 0 ? (double)E / ((double)k * (double)routed * (double)routed) : 0.0;
  float part = 0.0f;
  for (int e = threadIdx.x; e < E; e += THREADS) {
    const int n = sh.total[e];
    if (o.counts) o.counts[e] = n;
    if (o.slope) {
      const float sl = (float)((double)n * per);
      o.slope[e] = sl;
      part = fmaf(sl, sums[e], part);
    }
  }
  if (!o.slope) return;
  part = wave_add(part);
  if (lane == 0) sh.fwave[wave] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < THREADS / 64; ++w) s += sh.fwave[w];
    o.loss[0] = s;
  }
}

// All of it in one launch of one block.
template <typename T, int VPL>
__global__ void __launch_bounds__(threads_of(VPL))
    route_one_kernel(const T *__restrict__ z, int64_t ldz, const uint8_t *__restrict__ valid,
                     RouteOut o, int64_t Tn, int E, int k, bool normalise) {
  constexpr int THREADS = threads_of(VPL);
  __shared__ Shared<THREADS> sh;
  __shared__ float sums[kRouteMaxExperts];
  choose<T, VPL>(z, ldz, valid, o, 0, Tn, E, k, normalise, o.slope ? sums : nullptr, sh);
  for (int e = threadIdx.x; e < E; e += THREADS) {
    sh.total[e] = sh.hist[e];
    sh.first[e] = 0;
  }
  __syncthreads();
  const int all = scan_experts<THREADS>(E, sh, o.offsets);
  if (threadIdx.x == 0) sh.first[E] = all;
  finish<THREADS>(o, sums, sh.routed, E, k, sh);
  __syncthreads();
  place_slots<THREADS>(o, 0, Tn * k, E, k, sh);
}

// Two launches: the blocks' choices, with their counts and sums of p in the
// workspace (a row of `table`: E counts, then the tokens with an expert) ...
template <typename T, int VPL>
__global__ void __launch_bounds__(threads_of(VPL))
    route_choose_kernel(const T *__restrict__ z, int64_t ldz, const uint8_t *__restrict__ valid,
                        RouteOut o, int64_t Tn, int E, int k, bool normalise, int64_t C,
                        int *__restrict__ table, float *__restrict__ psum) {
  __shared__ Shared<threads_of(VPL)> sh;
  const int64_t t0 = (int64_t)blockIdx.x * C, t1 = t0 + C < Tn ? t0 + C : Tn;
  choose<T, VPL>(z, ldz, valid, o, t0, t1, E, k, normalise,
                 psum ? psum + (int64_t)blockIdx.x * E : nullptr, sh);
  int *row = table + (int64_t)blockIdx.x * (E + 1);
  for (int e = threadIdx.x; e < E; e += threads_of(VPL)) row[e] = sh.hist[e];
  if (threadIdx.x == 0) row[E] = sh.routed;
}

// ... and the rows: every block sums the whole table itself (a launch less),
// the first one takes the loss too.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    route_place_kernel(RouteOut o, int64_t Tn, int E, int k, int64_t C,
                       const int *__restrict__ table, const float *__restrict__ psum) {
  __shared__ Shared<THREADS> sh;
  __shared__ float sums[kRouteMaxExperts];
  const int B = gridDim.x, me = blockIdx.x;
  // thread (segment, expert): the segment's share of the table's rows
  int wide = 64;
  while (wide < E) wide <<= 1;
  const int segs = wide <= THREADS ? THREADS / wide : 1;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + threadIdx.x % wide, seg = threadIdx.x / wide;
    const int per = (B + segs - 1) / segs;
    int before = 0, total = 0;
    if (e < E && seg < segs) {
      const int b1 = (seg + 1) * per < B ? (seg + 1) * per : B;
#pragma unroll 16
      for (int b = seg * per; b < b1; ++b) {
        const int n = table[(int64_t)b * (E + 1) + e];
        total += n;
        before += b < me ? n : 0;
      }
    }
    sh.join.seg[threadIdx.x] = before;
    sh.join.seg[THREADS + threadIdx.x] = total;
    __syncthreads();
    if (seg == 0 && e < E) {
      for (int s = 1; s < segs; ++s) {
        before += sh.join.seg[s * wide + threadIdx.x];
        total += sh.join.seg[THREADS + s * wide + threadIdx.x];
      }
      sh.first[e] = before;
      sh.total[e] = total;
    }
    __syncthreads();
    if (psum && me == 0) {  // the sums of p in the same segments
      float *part = reinterpret_cast<float *>(sh.join.seg);
      float sum = 0.0f;
      if (e < E && seg < segs) {
        const int b1 = (seg + 1) * per < B ? (seg + 1) * per : B;
#pragma unroll 16
        for (int b = seg * per; b < b1; ++b) sum += psum[(int64_t)b * E + e];
      }
      part[threadIdx.x] = sum;
      __syncthreads();
      if (seg == 0 && e < E) {
        for (int s = 1; s < segs; ++s) sum += part[s * wide + threadIdx.x];
        sums[e] = sum;
      }
      __syncthreads();
    }
  }
  // slots of the blocks before this one that have no expert
  int mine = 0;
  for (int e = threadIdx.x; e < E; e += THREADS) mine += sh.first[e];
  for (int d = 32; d > 0; d >>= 1) mine += __shfl_xor(mine, d, 64);
  if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = mine;
  __syncthreads();
  const int64_t s0 = (int64_t)me * C * k;
  const int64_t s1 = s0 + C * k < Tn * k ? s0 + C * k : Tn * k;
  int tail = (int)s0;
  for (int w = 0; w < THREADS / 64; ++w) tail -= sh.wave[w];
  __syncthreads();
  const int all = scan_experts<THREADS>(E, sh, me == 0 ? o.offsets : nullptr);
  if (threadIdx.x == 0) sh.first[E] = all + tail;
  if (me == 0) {
    int routed = 0;
    for (int b = threadIdx.x; b < B; b += THREADS) routed += table[(int64_t)b * (E + 1) + E];
    for (int d = 32; d > 0; d >>= 1) routed += __shfl_xor(routed, d, 64);
    if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = routed;
    __syncthreads();
    routed = 0;
    for (int w = 0; w < THREADS / 64; ++w) routed += sh.wave[w];
    finish<THREADS>(o, sums, routed, E, k, sh);
  }
  __syncthreads();
  place_slots<THREADS>(o, s0, s1, E, k, sh);
}

// Rows by group: counts of the block's ids for route_place_kernel.
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    group_count_kernel(const int32_t *__restrict__ ids, int64_t n, int G, int64_t C,
                       int *__restrict__ table) {
  __shared__ int hist[kRouteMaxExperts];
  for (int g = threadIdx.x; g < G; g += THREADS) hist[g] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * C, i1 = i0 + C < n ? i0 + C : n;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += THREADS) {
    const int g = ids[i];
    if (g >= 0 && g < G) atomicAdd(&hist[g], 1);
  }
  __syncthreads();
  int *row = table + (int64_t)blockIdx.x * (G + 1);
  for (int g = threadIdx.x; g < G; g += THREADS) row[g] = hist[g];
  if (threadIdx.x == 0) row[G] = 0;
}

// dz of a token, by one wave.
template <typename T, int VPL>
__global__ void __launch_bounds__(256)
    route_bwd_kernel(const T *__restrict__ z, int64_t ldz, const int32_t *__restrict__ experts,
                     const float *__restrict__ weights, const float *__restrict__ stats,
                     const float *__restrict__ slope, const float *__restrict__ dweights,
                     const float *__restrict__ dloss, T *__restrict__ dz, int64_t lddz, int64_t Tn,
                     int E, int k, bool normalise) {
  const int lane = threadIdx.x & 63;
  float gl[VPL];  // the loss's share of g
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    gl[i] = slope && e < E ? dloss[0] * slope[e] : 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < Tn;
       t += (int64_t)gridDim.x * 4) {
    float v[VPL];
    load_logits<T, VPL>(z + t * ldz, E, v);
    const float m = stats[2 * t], rsum = stats[2 * t + 1];
    int mine = -1;
    float w = 0.0f, d = 0.0f;
    if (dweights && lane < k) {
      mine = experts[t * k + lane];
      w = weights[t * k + lane];
      d = dweights[t * k + lane];
      if (mine < 0 || mine >= E) {
        mine = -1;
        w = d = 0.0f;
      }
    }
    const float inner = wave_add(w * d);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = rsum == 0.0f ? 0.0f : expf(v[i] - m) * rsum;
      s = fmaf(v[i], gl[i], s);
    }
    s = wave_add(s);
    if (!normalise) s += inner;
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= gl[i] - s;
    const float add = w * (normalise ? d - inner : d);
    if (dweights) {
      for (int j = 0; j < k; ++j) {
        const int e = __builtin_amdgcn_readlane(mine, j);
        const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(add), j));
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane + 64 * i == e) v[i] += a;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < E) dz[t * lddz + lane + 64 * i] = (T)v[i];
  }
}

template <typename T, int VPL>
hipError_t fwd(const void *z, int64_t ldz, const uint8_t *valid, const RouteOut &o, void *ws,
               int64_t Tn, int E, int k, bool normalise, hipStream_t s) {
  constexpr int THREADS = threads_of(VPL);
  const T *zt = static_cast<const T *>(z);
  const int64_t C = tokens_per_block(Tn, THREADS), B = (Tn + C - 1) / C;
  if (B <= 1) {
    route_one_kernel<T, VPL><<<1, THREADS, 0, s>>>(zt, ldz, valid, o, Tn, E, k, normalise);
    return hipGetLastError();
  }
  int *table = static_cast<int *>(ws);
  float *psum = o.slope ? reinterpret_cast<float *>(table + B * (E + 1)) : nullptr;
  route_choose_kernel<T, VPL><<<(unsigned)B, THREADS, 0, s>>>(zt, ldz, valid, o, Tn, E, k,
                                                              normalise, C, table, psum);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place_kernel<THREADS><<<(unsigned)B, THREADS, 0, s>>>(o, Tn, E, k, C, table, psum);
  return hipGetLastError();
}

template <typename T, int VPL>
hipError_t bwd(const void *z, int64_t ldz, const int32_t *experts, const float *weights,
               const float *stats, const float *slope, const float *dweights, const float *dloss,
               void *dz, int64_t lddz, int64_t Tn, int E, int k, bool normalise, hipStream_t s) {
  const int64_t need = (Tn + 3) / 4, most = 2048;
  route_bwd_kernel<T, VPL><<<(unsigned)(need < most ? need : most), 256, 0, s>>>(
      static_cast<const T *>(z), ldz, experts, weights, stats, slope, dweights, dloss,
      static_cast<T *>(dz), lddz, Tn, E, k, normalise);
  return hipGetLastError();
}

// Calls F<T, VPL> for the logits' type and number.
#define BNN_ROUTE(F, ...)                                                             \
  (dtype == BNN_FP32 ? (E <= 64    ? F<float, 1>(__VA_ARGS__)                         \
                        : E <= 128 ? F<float, 2>(__VA_ARGS__)                         \
                        : E <= 256 ? F<float, 4>(__VA_ARGS__)                         \
                        : E <= 512 ? F<float, 8>(__VA_ARGS__)                         \
                                   : F<float, 16>(__VA_ARGS__))                       \
                     : (E <= 64    ? F<bf16_t, 1>(__VA_ARGS__)                        \
                        : E <= 128 ? F<bf16_t, 2>(__VA_ARGS__)                        \
                        : E <= 256 ? F<bf16_t, 4>(__VA_ARGS__)                        \
                        : E <= 512 ? F<bf16_t, 8>(__VA_ARGS__)                        \
                                   : F<bf16_t, 16>(__VA_ARGS__)))

}  // namespace

int64_t route_fwd_workspace(int64_t T, int64_t E, int64_t k) {
  const int64_t C = tokens_per_block(T, E > 512 ? 512 : 1024), B = (T + C - 1) / C;
  return B <= 1 ? 0 : B * (2 * E + 1) * 4;
}

static int64_t group_chunk(int64_t n) {
  const int64_t c = (n + kRouteBlocks - 1) / kRouteBlocks;
  return c < 1024 ? 1024 : (c + 63) / 64 * 64;
}

int64_t group_rows_workspace(int64_t n, int64_t G) {
  const int64_t C = group_chunk(n), B = (n + C - 1) / C;
  return (B > 0 ? B : 1) * (G + 1) * 4;
}

hipError_t launch_group_rows(const int32_t *ids, int32_t *rows, int32_t *offsets, void *workspace,
                             int64_t n, int G, hipStream_t s) {
  const int64_t C = group_chunk(n);
  const unsigned B = n > 0 ? (unsigned)((n + C - 1) / C) : 1;
  int *table = static_cast<int *>(workspace);
  RouteOut o = {};
  o.experts = const_cast<int32_t *>(ids);
  o.rows = rows;
  o.offsets = offsets;
  if (G <= 512) {
    group_count_kernel<1024><<<B, 1024, 0, s>>>(ids, n, G, C, table);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<1024><<<B, 1024, 0, s>>>(o, n, G, 1, C, table, nullptr);
  } else {
    group_count_kernel<512><<<B, 512, 0, s>>>(ids, n, G, C, table);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<512><<<B, 512, 0, s>>>(o, n, G, 1, C, table, nullptr);
  }
  return hipGetLastError();
}

hipError_t launch_route_fwd(const void *z, int dtype, int64_t ldz, const uint8_t *valid,
                            const RouteOut &out, void *workspace, int64_t T, int E, int k,
                            bool normalise, hipStream_t s) {
  return BNN_ROUTE(fwd, z, ldz, valid, out, workspace, T, E, k, normalise, s);
}

hipError_t launch_route_bwd(const void *z, int dtype, int64_t ldz, const int32_t *experts,
                            const float *weights, const float *stats, const float *slope,
                            const float *dweights, const float *dloss, void *dz, int64_t lddz,
                            int64_t T, int E, int k, bool normalise, hipStream_t s) {
  return BNN_ROUTE(bwd, z, ldz, experts, weights, stats, slope, dweights, dloss, dz, lddz, T, E, k,
                   normalise, s);
}

}  // namespace bnn
