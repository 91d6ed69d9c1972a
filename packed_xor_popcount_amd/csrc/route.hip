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

// LPT lanes share a token (16: a DPP row, four tokens a wave); lane l of them holds
// the V neighbouring logits from V l on, so that ties go to the lowest lane and
// then to the lowest place.
constexpr int threads_of(int lpt, int v) { return lpt == 64 && v > 8 ? 512 : 1024; }

template <int LPT, int V>
struct Shape {
  static constexpr int kThreads = threads_of(LPT, V);
  static constexpr int kWaves = kThreads / 64, kTokens = 64 / LPT;
};

template <int CTRL>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// Of the token's lanes; every one receives it.  (Rotations by 8, 4, 2, 1: the
// lanes add the same pairs, so their sums are equal bit for bit.)
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  if (LPT == 64) return wave_max(v);
  v = fmaxf(v, rotated<0x128>(v));
  v = fmaxf(v, rotated<0x124>(v));
  v = fmaxf(v, rotated<0x122>(v));
  return fmaxf(v, rotated<0x121>(v));
}
template <int LPT>
__device__ __forceinline__ float token_add(float v) {
  if (LPT == 64) return wave_add(v);
  v += rotated<0x128>(v);
  v += rotated<0x124>(v);
  v += rotated<0x122>(v);
  return v + rotated<0x121>(v);
}

template <int V>
__device__ __forceinline__ float largest(const float (&v)[V]) {
  float m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) m[i] = v[i];
#pragma unroll
  for (int d = V / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < d; ++i) m[i] = fmaxf(m[i], m[i + d]);
  return m[0];
}

constexpr int64_t kRouteBlocks = 256;  // most blocks: each leaves a row of partial sums

// Tokens of a block: a multiple of those that it takes at once.
inline int64_t tokens_per_block(int64_t T, int at_once) {
  const int64_t c = (T + kRouteBlocks - 1) / kRouteBlocks;
  return c < at_once ? at_once : (c + at_once - 1) / at_once * at_once;
}

// A lane's elements of a row of E >= V; `past` behind its end.  One vector access,
// whatever E: the last one ends with the row, and its elements move into place.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *z, int e0, int E, float past, float (&v)[V]) {
  T r[V];
  const int at = e0 < E - V ? e0 : E - V;
  __builtin_memcpy(r, z + at, sizeof(r));
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = (float)r[i];
  const int by = e0 - at;
#pragma unroll
  for (int d = V / 2; d > 0; d /= 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float from = i + d < V ? v[i + d] : past;
      v[i] = (by & d) ? from : v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = by < V ? v[i] : past;
}

// The block's LDS.  `join` holds the tokens' choices and the waves' sums of p
// first, later partial sums of the table or the slots counted by wave and expert.
template <int THREADS>
struct Shared {
  int hist[kRouteMaxExperts + 1];   // this block's slots per expert
  int first[kRouteMaxExperts + 1];  // row of the block's next slot per expert
  int total[kRouteMaxExperts + 1];
  union {
    float2 slots[THREADS / 16][kRouteMaxK];  // (logit, expert) by token
    float sums[8192];                        // waves x E
    uint16_t seen[8192 + 16];                // waves x (E + 1)
    int seg[8 * THREADS];
    float fseg[4 * THREADS];
  } join;
  int wave[THREADS / 64];
  float fwave[THREADS / 64];
  int routed;
};

// A token's logits stay in registers: the largest is found k times over (rotations
// within 16 lanes, four tokens a wave at once), its lane takes it out, without a
// branch.  Bound by that chain of dependent instructions, not by the 2 us that the
// logits' bytes take: 16384 x 128 fp32, 8 choices 11 to 12 us (a wave a token 19 us;
// with a branch for the lane that wins 11.8 where this took 10.9), 8192 x 256 bf16 15.9 us.
//
// Choices, weights and statistics of the block's tokens, their counts in
// sh.hist, the number of tokens with an expert in sh.routed and the sums of p
// in psum (E floats, or null).
template <typename T, int LPT, int V>
__device__ void choose(const T *z, int64_t ldz, const uint8_t *valid, const RouteOut &o, int64_t t0,
                       int64_t t1, int E, int k, bool normalise, float *psum,
                       Shared<Shape<LPT, V>::kThreads> &sh) {
  constexpr int W = Shape<LPT, V>::kWaves, TOKENS = Shape<LPT, V>::kTokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LPT, grp = lane / LPT, e0 = V * sub;
  // lanes of the same token before this one
  const uint64_t before = ((uint64_t(1) << lane) - 1) & ~((uint64_t(1) << (grp * LPT)) - 1);
  for (int e = threadIdx.x; e < E; e += 64 * W) sh.hist[e] = 0;
  if (threadIdx.x == 0) sh.routed = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  int routed = 0;
  float2 *slots = sh.join.slots[wave * TOKENS + grp];
  for (int64_t tw = t0 + wave * TOKENS; tw < t1; tw += W * TOKENS) {
    const int64_t t = tw + grp;
    const bool in = t < t1;
    float v[V], key[V], ex[V];
    load_row<T, V>(z + (in ? t : t1 - 1) * ldz, e0, E, -INFINITY, v);
    const bool on = in && !(valid && !valid[t]);
    for (int j = sub; j < k; j += LPT) slots[j] = make_float2(0.0f, __int_as_float(-1));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!on) v[i] = -INFINITY;
      key[i] = v[i] > -INFINITY ? v[i] : -INFINITY;  // NaN is never chosen
    }
    float best = largest<V>(key);
    float top = token_max<LPT>(best);
    const bool some = top > -INFINITY;  // an expert is open
    const float mz = some ? top : 0.0f;
    routed += some && sub == 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // the k largest, one after the other
    for (int j = 0; j < k; ++j) {
      const bool has = best == top && top > -INFINITY;
      const uint64_t lanes = __ballot(has);
      if (lanes == 0) break;
      const bool wins = has && (lanes & before) == 0;
      int at = V;  // the lane's lowest place that holds its largest value
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == best ? i : at;
      if (wins) slots[j] = make_float2(top, __int_as_float(e0 + at));
      at = wins ? at : -1;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = at == i ? -INFINITY : key[i];
      best = largest<V>(key);
      top = token_max<LPT>(best);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = expf(v[i] - mz);
      sum += ex[i];
    }
    sum = token_add<LPT>(sum);
    const float rsum = sum == 0.0f ? 0.0f : 1.0f / sum;  // NaN where a logit is NaN or +inf
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(ex[i], rsum, acc[i]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // lane `sub` finishes choices sub, sub + LPT
    constexpr int PER = LPT == 16 ? 2 : 1;
    float w[PER], wsum = 0.0f;
    int e[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = sub + LPT * i;
      const float2 c = j < k ? slots[j] : make_float2(0.0f, __int_as_float(-1));
      e[i] = __float_as_int(c.y);
      w[i] = e[i] >= 0 ? expf(c.x - mz) : 0.0f;
      wsum += w[i];
    }
    if (normalise) wsum = token_add<LPT>(wsum);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = sub + LPT * i;
      if (e[i] >= 0)  // NaN where the statistics are
        w[i] = normalise ? w[i] / wsum + 0.0f * rsum : w[i] * rsum;
      if (in && j < k) {
        o.experts[t * k + j] = e[i];
        o.weights[t * k + j] = w[i];
        if (e[i] >= 0) atomicAdd(&sh.hist[e[i]], 1);
      }
    }
    if (in && sub == 0) {
      o.stats[2 * t] = mz;
      o.stats[2 * t + 1] = some ? rsum : 0.0f;  // 0 for NaN alone too: no gradient
    }
  }
  if (routed) atomicAdd(&sh.routed, routed);
  __syncthreads();  // the choices have been read, the counts are complete
  if (!psum) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    for (int d = LPT; d < 64; d *= 2) acc[i] += __shfl_xor(acc[i], d, 64);
    if (lane < LPT && e0 + i < E) sh.join.sums[wave * E + e0 + i] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 64 * W) {
    float s = 0.0f;
    for (int w = 0; w < W; ++w) s += sh.join.sums[w * E + e];
    psum[e] = s;
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

// All of it in one launch of one block, for as many tokens as it takes at once: 4
// tokens of 64 experts 6.2 us.
template <typename T, int LPT, int V>
__global__ void __launch_bounds__(threads_of(LPT, V))
    route_one_kernel(const T *__restrict__ z, int64_t ldz, const uint8_t *__restrict__ valid,
                     RouteOut o, int64_t Tn, int E, int k, bool normalise) {
  constexpr int THREADS = Shape<LPT, V>::kThreads;
  __shared__ Shared<THREADS> sh;
  __shared__ float sums[kRouteMaxExperts];
  choose<T, LPT, V>(z, ldz, valid, o, 0, Tn, E, k, normalise, o.slope ? sums : nullptr, sh);
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

// Two launches: the blocks' choices, with their counts (a row of `table`: counts,
// zeros up to a multiple of four), tokens with an expert and sums of p (`psum`,
// rows as the table's) in the workspace ...
__host__ __device__ inline int table_row(int E) { return (E + 3) / 4 * 4; }

template <typename T, int LPT, int V>
__global__ void __launch_bounds__(threads_of(LPT, V))
    route_choose_kernel(const T *__restrict__ z, int64_t ldz, const uint8_t *__restrict__ valid,
                        RouteOut o, int64_t Tn, int E, int k, bool normalise, int64_t C,
                        int *__restrict__ table, int *__restrict__ routed,
                        float *__restrict__ psum) {
  __shared__ Shared<Shape<LPT, V>::kThreads> sh;
  const int64_t t0 = (int64_t)blockIdx.x * C, t1 = t0 + C < Tn ? t0 + C : Tn;
  const int row = table_row(E);
  choose<T, LPT, V>(z, ldz, valid, o, t0, t1, E, k, normalise,
                    psum ? psum + (int64_t)blockIdx.x * row : nullptr, sh);
  for (int e = threadIdx.x; e < row; e += Shape<LPT, V>::kThreads)
    table[(int64_t)blockIdx.x * row + e] = e < E ? sh.hist[e] : 0;
  if (threadIdx.x == 0) routed[blockIdx.x] = sh.routed;
}

// ... and the rows: every block sums the whole table itself (a launch less), four
// experts a thread with eight rows in flight, and the first one takes the loss too.
// 16384 x 128, 8 choices: 8.7 us (with 1024 threads 10.6, with 256 10.0; one expert a
// thread 22.8); the launch, the table's latency and about ten barriers.
constexpr int kPlaceThreads = 512;

__global__ void __launch_bounds__(kPlaceThreads)
    route_place_kernel(RouteOut o, int64_t Tn, int E, int k, int64_t C,
                       const int *__restrict__ table, const int *__restrict__ block_routed,
                       const float *__restrict__ psum) {
  constexpr int THREADS = kPlaceThreads;
  __shared__ Shared<THREADS> sh;
  __shared__ float sums[kRouteMaxExperts];
  const int B = gridDim.x, me = blockIdx.x, row = table_row(E);
  // thread (segment, four experts): the segment's share of the table's rows
  int wide = 16;
  while (4 * wide < E) wide <<= 1;
  const int segs = THREADS / wide, per = (B + segs - 1) / segs;
  const int quad = threadIdx.x % wide, seg = threadIdx.x / wide;
  const int b0 = seg * per, b1 = b0 + per < B ? b0 + per : B;
  int4 before = {0, 0, 0, 0}, total = {0, 0, 0, 0};
  if (4 * quad < E) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
      const int4 n = *reinterpret_cast<const int4 *>(table + (int64_t)b * row + 4 * quad);
      const int m = b < me ? -1 : 0;
      total.x += n.x;
      total.y += n.y;
      total.z += n.z;
      total.w += n.w;
      before.x += n.x & m;
      before.y += n.y & m;
      before.z += n.z & m;
      before.w += n.w & m;
    }
  }
  reinterpret_cast<int4 *>(sh.join.seg)[threadIdx.x] = before;
  reinterpret_cast<int4 *>(sh.join.seg)[THREADS + threadIdx.x] = total;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int first = 0, all = 0;
#pragma unroll 4
    for (int i = 0; i < segs; ++i) {
      first += sh.join.seg[4 * wide * i + e];
      all += sh.join.seg[4 * THREADS + 4 * wide * i + e];
    }
    sh.first[e] = first;
    sh.total[e] = all;
  }
  __syncthreads();
  if (psum && me == 0) {  // the sums of p, in the same segments
    float4 p = {0.0f, 0.0f, 0.0f, 0.0f};
    if (4 * quad < E) {
#pragma unroll 8
      for (int b = b0; b < b1; ++b) {
        const float4 n = *reinterpret_cast<const float4 *>(psum + (int64_t)b * row + 4 * quad);
        p.x += n.x;
        p.y += n.y;
        p.z += n.z;
        p.w += n.w;
      }
    }
    reinterpret_cast<float4 *>(sh.join.fseg)[threadIdx.x] = p;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) {
      float s = 0.0f;
#pragma unroll 4
      for (int i = 0; i < segs; ++i) s += sh.join.fseg[4 * wide * i + e];
      sums[e] = s;
    }
    __syncthreads();
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
    if (block_routed)
      for (int b = threadIdx.x; b < B; b += THREADS) routed += block_routed[b];
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
__global__ void __launch_bounds__(1024)
    group_count_kernel(const int32_t *__restrict__ ids, int64_t n, int G, int64_t C,
                       int *__restrict__ table) {
  constexpr int THREADS = 1024;
  __shared__ int hist[kRouteMaxExperts];
  for (int g = threadIdx.x; g < G; g += THREADS) hist[g] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * C, i1 = i0 + C < n ? i0 + C : n;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += THREADS) {
    const int g = ids[i];
    if (g >= 0 && g < G) atomicAdd(&hist[g], 1);
  }
  __syncthreads();
  const int row = table_row(G);
  for (int g = threadIdx.x; g < row; g += THREADS)
    table[(int64_t)blockIdx.x * row + g] = g < G ? hist[g] : 0;
}

// dz of TOKENS tokens by a wave, lanes as in the forward pass.  What the choices
// add goes to its lanes through LDS.  16384 x 128 fp32: 6.9 us (2.4 TB/s; 10.2 us with
// the loss's slopes loaded one by one); one pass of a wave, bound by its latency.
template <typename T, int LPT, int V>
__global__ void __launch_bounds__(256)
    route_bwd_kernel(const T *__restrict__ z, int64_t ldz, const int32_t *__restrict__ experts,
                     const float *__restrict__ weights, const float *__restrict__ stats,
                     const float *__restrict__ slope, const float *__restrict__ dweights,
                     const float *__restrict__ dloss, T *__restrict__ dz, int64_t lddz, int64_t Tn,
                     int E, int k, bool normalise) {
  constexpr int TOKENS = Shape<LPT, V>::kTokens, PER = LPT == 16 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float adds[4][TOKENS][LPT * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LPT, grp = lane / LPT, e0 = V * sub;
  float *mine = adds[wave][grp];
  float gl[V];  // the loss's share of g
#pragma unroll
  for (int i = 0; i < V; ++i) gl[i] = 0.0f;
  if (slope) {
    const float dl = dloss[0];
    load_row<float, V>(slope, e0, E, 0.0f, gl);
#pragma unroll
    for (int i = 0; i < V; ++i) gl[i] = e0 + i < E ? gl[i] * dl : 0.0f;
  }
  for (int64_t tw = ((int64_t)blockIdx.x * 4 + wave) * TOKENS; tw < Tn;
       tw += (int64_t)gridDim.x * 4 * TOKENS) {
    const bool in = tw + grp < Tn;
    const int64_t t = in ? tw + grp : Tn - 1;
    float v[V];
    load_row<T, V>(z + t * ldz, e0, E, -INFINITY, v);
    const float m = stats[2 * t], rsum = stats[2 * t + 1];
    int e[PER];
    float w[PER], d[PER], inner = 0.0f;
    if (dweights) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = sub + LPT * i;
        const int64_t at = t * k + (j < k ? j : k - 1);
        e[i] = experts[at];
        w[i] = weights[at];
        d[i] = dweights[at];
        if (j >= k || e[i] < 0 || e[i] >= E) {
          e[i] = -1;
          w[i] = d[i] = 0.0f;
        }
        inner = fmaf(w[i], d[i], inner);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) mine[e0 + i] = 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = rsum == 0.0f ? 0.0f : expf(v[i] - m) * rsum;
      s = fmaf(v[i], gl[i], s);
    }
    s = token_add<LPT>(s);
    if (dweights) {
      inner = token_add<LPT>(inner);
      if (!normalise) s += inner;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e[i] >= 0) atomicAdd(&mine[e[i]], w[i] * (normalise ? d[i] - inner : d[i]));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = rsum == 0.0f ? 0.0f : v[i] * (gl[i] - s);
    if (dweights) {
      float add[V];
      __builtin_memcpy(add, __builtin_assume_aligned(mine + e0, 4 * (V < 4 ? V : 4)), sizeof(add));
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += add[i];
    }
    if (!in) continue;
    T *row = dz + t * lddz;
    if (e0 + V <= E) {
      T r[V];
#pragma unroll
      for (int i = 0; i < V; ++i) r[i] = (T)v[i];
      __builtin_memcpy(row + e0, r, sizeof(r));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) row[e0 + i] = (T)v[i];
    }
  }
}

template <typename T, int LPT, int V>
hipError_t fwd(const void *z, int64_t ldz, const uint8_t *valid, const RouteOut &o, void *ws,
               int64_t Tn, int E, int k, bool normalise, hipStream_t s) {
  constexpr int THREADS = Shape<LPT, V>::kThreads;
  const T *zt = static_cast<const T *>(z);
  const int64_t C = tokens_per_block(Tn, THREADS / LPT), B = (Tn + C - 1) / C;
  if (B <= 1) {
    route_one_kernel<T, LPT, V><<<1, THREADS, 0, s>>>(zt, ldz, valid, o, Tn, E, k, normalise);
    return hipGetLastError();
  }
  int *table = static_cast<int *>(ws), *routed = table + 2 * B * table_row(E);
  float *psum = o.slope ? reinterpret_cast<float *>(table + B * table_row(E)) : nullptr;
  route_choose_kernel<T, LPT, V><<<(unsigned)B, THREADS, 0, s>>>(zt, ldz, valid, o, Tn, E, k,
                                                                 normalise, C, table, routed, psum);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place_kernel<<<(unsigned)B, kPlaceThreads, 0, s>>>(o, Tn, E, k, C, table, routed, psum);
  return hipGetLastError();
}

template <typename T, int LPT, int V>
hipError_t bwd(const void *z, int64_t ldz, const int32_t *experts, const float *weights,
               const float *stats, const float *slope, const float *dweights, const float *dloss,
               void *dz, int64_t lddz, int64_t Tn, int E, int k, bool normalise, hipStream_t s) {
  constexpr int64_t kAtOnce = 4 * Shape<LPT, V>::kTokens, most = 2048;
  const int64_t need = (Tn + kAtOnce - 1) / kAtOnce;
  route_bwd_kernel<T, LPT, V><<<(unsigned)(need < most ? need : most), 256, 0, s>>>(
      static_cast<const T *>(z), ldz, experts, weights, stats, slope, dweights, dloss,
      static_cast<T *>(dz), lddz, Tn, E, k, normalise);
  return hipGetLastError();
}

// Calls F<T, LPT, V> for the logits' type and number.
#define BNN_ROUTE_AS(F, T, ...)              \
  (E <= 16    ? F<T, 16, 1>(__VA_ARGS__)     \
   : E <= 32  ? F<T, 16, 2>(__VA_ARGS__)     \
   : E <= 64  ? F<T, 16, 4>(__VA_ARGS__)     \
   : E <= 128 ? F<T, 16, 8>(__VA_ARGS__)     \
   : E <= 256 ? F<T, 16, 16>(__VA_ARGS__)    \
   : E <= 512 ? F<T, 64, 8>(__VA_ARGS__)     \
              : F<T, 64, 16>(__VA_ARGS__))
#define BNN_ROUTE(F, ...) \
  (dtype == BNN_FP32 ? BNN_ROUTE_AS(F, float, __VA_ARGS__) : BNN_ROUTE_AS(F, bf16_t, __VA_ARGS__))

}  // namespace

int64_t route_fwd_workspace(int64_t T, int64_t E, int64_t k) {
  const int64_t C = tokens_per_block(T, E <= 256 ? 64 : E <= 512 ? 16 : 8), B = (T + C - 1) / C;
  return B <= 1 ? 0 : B * (2 * table_row((int)E) + 1) * 4;
}

static int64_t group_chunk(int64_t n) {
  const int64_t c = (n + kRouteBlocks - 1) / kRouteBlocks;
  return c < 1024 ? 1024 : (c + 63) / 64 * 64;
}

int64_t group_rows_workspace(int64_t n, int64_t G) {
  const int64_t C = group_chunk(n), B = (n + C - 1) / C;
  return (B > 0 ? B : 1) * table_row((int)G) * 4;
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
  group_count_kernel<<<B, 1024, 0, s>>>(ids, n, G, C, table);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place_kernel<<<B, kPlaceThreads, 0, s>>>(o, n, G, 1, C, table, nullptr, nullptr);
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
