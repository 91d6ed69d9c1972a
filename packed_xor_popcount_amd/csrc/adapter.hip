// adapter.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradient.  Row t uses adapter l = id_t (none outside [0, L)), of
// scale s_l and factors A_l (r x K), B_l (r x N), both bf16 with the rank as
// the slow dimension:
//
//   u_t = A_l x_t             out_t = base_t + s_l sum_j u_t[j] B_l[j]
//   v_t = B_l dy_t            dx_t = base_t + s_l sum_j v_t[j] A_l[j]
//   dA_l = s_l sum_t v_t x_t'            dB_l = s_l sum_t u_t dy_t'
//
// Three kernels: shrink (u, v: sums over the long side), expand (out, dx: sums
// over the rank) and outer (dA, dB: sums over an adapter's rows); a gradient runs
// the last two side by side in one launch.  All sums are
// fp32 on the matrix cores from exact products of bf16 values: u and v, which
// are fp32, are split into three bf16 parts (8 + 8 + 8 significant bits), so that
// no rounding comes between the two factors.  The order of every sum goes by
// the sizes and the rows' ids alone.
//
// v_mfma_f32_16x16x32_bf16: lane l supplies row / column l % 16 and eight
// elements of k, those of index 8 (l / 16) ...; output register v of lane l is
// row 4 (l / 16) + v, column l % 16.  The sum does not depend on which k an
// index stands for, as long as both operands agree.
#include "f8.h"
#include "operators.h"

#include <type_traits>

namespace bnn {
namespace {

typedef __bf16 bf16_t;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma(const uint4 &a, const uint4 &b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint4 words(const Chunk<bf16_t> &c) {
  return make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
}
// Eight elements of a row of C; LONG: C >= 8, so that no choice comes between the
// loads of a kernel.
template <bool LONG, typename T>
__device__ __forceinline__ Chunk<T> raw8(const T *row, int64_t c, int64_t C) {
  return LONG ? raw_chunk_long(row, (int)c, (int)C) : raw_chunk(row, (int)c, (int)C);
}
template <bool LONG>
__device__ __forceinline__ Chunk<bf16_t> raw8(const uint16_t *row, int64_t c, int64_t C) {
  return raw8<LONG>(reinterpret_cast<const bf16_t *>(row), c, C);
}

// Three bf16 parts whose sum is v exactly (bits below 2^-133 aside); an
// infinity or NaN is its own first part.
struct Parts {
  uint32_t hi, mid, lo;  // in the upper halves
};
__device__ __forceinline__ Parts parts_of(float v) {
  Parts p;
  p.hi = __float_as_uint(v) & 0xFFFF0000u;
  const bool finite = (p.hi & 0x7F800000u) != 0x7F800000u;
  const float r1 = finite ? v - __uint_as_float(p.hi) : 0.0f;
  p.mid = __float_as_uint(r1) & 0xFFFF0000u;
  p.lo = __float_as_uint(r1 - __uint_as_float(p.mid));
  return p;
}

// Operands of eight fp32 values, one for each part.
__device__ __forceinline__ void split8(const float (&v)[8], uint4 (&o)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const Parts p = parts_of(v[2 * m]), q = parts_of(v[2 * m + 1]);
    w[0][m] = __builtin_amdgcn_perm(q.hi, p.hi, 0x07060302u);
    w[1][m] = __builtin_amdgcn_perm(q.mid, p.mid, 0x07060302u);
    w[2][m] = __builtin_amdgcn_perm(q.lo, p.lo, 0x07060302u);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) o[i] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
}

// A middle or low part is often 0 where v is not, and 0 times an infinity is NaN where v
// times it is an infinity.  A sum that holds a product of an infinity or NaN is one of
// these itself, which one the high parts' products alone tell: they replace a NaN.
__device__ __forceinline__ float unless_nan(float sum, float high) {
  return sum != sum && !(fabsf(high) <= 3.402823466e38f) ? high : sum;
}

// Operands of eight columns from eight rows of them (rows r[0..7], columns
// two to a register): f[j] holds column j's eight rows.
__device__ __forceinline__ void transpose8(const uint4 (&r)[8], uint4 (&f)[8]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = d == 0 ? r[i].x : d == 1 ? r[i].y : d == 2 ? r[i].z : r[i].w;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      lo[m] = __builtin_amdgcn_perm(w[2 * m + 1], w[2 * m], 0x05040100u);
      hi[m] = __builtin_amdgcn_perm(w[2 * m + 1], w[2 * m], 0x07060302u);
    }
    f[2 * d] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    f[2 * d + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// ---------------------------------------------------------------------------
// The rows of a chunk in tiles of one adapter each.  A block puts up to kChunk
// neighbouring rows in the order of their ids, where these change often (a rank
// by comparison, in LDS), and cuts that order at every change and every 16th
// place.  So rows of one adapter share its factors wherever they stand in the
// chunk, and nothing has to be sorted or looked up by the caller.

constexpr int kChunk = 256;

struct Plan {
  int row[kChunk];              // 256 id + place in the chunk (id L: none); by tile in `sorted`
  int sorted[kChunk];
  uint16_t start[kChunk + 1];
  int waves[kChunk / 64];
  int tiles;

  // row `i` of tile `at`'s `len` ones (the last again past them), and the id
  __device__ __forceinline__ int place(int at, int len, int i) const {
    return sorted[at + (i < len ? i : len - 1)] & (kChunk - 1);
  }
  __device__ __forceinline__ int id(int at) const { return sorted[at] / kChunk; }
};

// By at least kChunk threads, all of the block's.
__device__ __forceinline__ void make_plan(Plan &p, const int32_t *ids, int64_t t0, int64_t T,
                                          int L) {
  const int i = threadIdx.x;
  const int n = T - t0 < kChunk ? (int)(T - t0) : kChunk;
  int mine = 0x7FFFFFFF;
  if (i < n) {
    int id = ids[t0 + i];
    if (id < 0 || id >= L) id = L;
    mine = id * kChunk + i;
  }
  if (i < kChunk) p.row[i] = mine;
  __syncthreads();
  const bool change = i > 0 && i < n && mine / kChunk != p.row[i - 1] / kChunk;
  int at = i;
  if (__syncthreads_count(change) > 8) {
    at = 0;
    if (i < n) {
#pragma unroll 4
      for (int j = 0; j < n; j += 4) {  // places past n hold the largest value
        const int4 k = *reinterpret_cast<const int4 *>(p.row + j);
        at += k.x < mine;
        at += k.y < mine;
        at += k.z < mine;
        at += k.w < mine;
      }
    }
  }
  if (i < n) p.sorted[at] = mine;
  __syncthreads();
  const bool begin = i < n && ((i & 15) == 0 || p.id(i) != p.id(i - 1));
  const uint64_t all = __ballot(begin);
  if ((i & 63) == 0 && i < kChunk) p.waves[i >> 6] = __popcll(all);
  __syncthreads();
  if (i < kChunk) {
    int before = __popcll(all & ((uint64_t(1) << (i & 63)) - 1)), total = 0;
    for (int w = 0; w < kChunk / 64; ++w) {
      if (w < (i >> 6)) before += p.waves[w];
      total += p.waves[w];
    }
    if (begin) p.start[before] = (uint16_t)i;
    if (i == 0) {
      p.start[total] = (uint16_t)n;
      p.tiles = total;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// shrink: u_t[j] = sum_c x_t[c] w_id,j[c], and the parts of u_t for expand.
// The eight waves of a block take every eighth step of 128 columns of a tile and
// join their sums in LDS.  blockIdx: chunk, share of the chunk's tiles.
//
// 4096 rows of 4096, rank 16: 15 us; 8192 of 4096, rank 32: 29 us (x's bytes take 6.5
// and 13; ranks over 64 spill 95 registers).  Without any load it would still take 9 and 15 us (the plan 5 us, then each
// tile's exchange, sums and join), on top of which come the loads; tiles in one
// pipeline, four waves a block, two blocks a CU and more or fewer shares were no
// faster.
//
// A row's parts are 16 RP bf16 values a part: for ranks up to 16 (RP = 1) four of
// them -- high, middle, low, zeros -- so that two neighbouring ones make one operand
// of 32; for larger ranks (RP even) three.

constexpr int kShrinkWaves = 8;
constexpr int parts_kept(int rp) { return rp == 1 ? 4 : 3; }

// A step's 16 rows of 128 columns are loaded 256 bytes a row (16 lanes each) and
// change to the operands' lanes through the wave's own 4 KiB of LDS, the 16-byte
// pieces swapped by row so that neither side meets a bank twice.  Loaded as
// operands at once, four neighbouring lanes read four rows, and a CU took in 16
// bytes a cycle instead of 64 (8192 rows of 4096, rank 32: 37 us).
typedef uint4 StepRows[16][16];

__device__ __forceinline__ void fence_wave() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// In: v[m] is piece lane % 16 of row 4 m + lane / 16.  Out: piece 4 k + lane / 16 of
// row lane % 16 in v[k].
__device__ __forceinline__ void to_operands(StepRows &buf, uint4 (&v)[4]) {
  const int lane = threadIdx.x & 63, low = lane & 15, g = lane >> 4;
  fence_wave();
#pragma unroll
  for (int m = 0; m < 4; ++m) buf[4 * m + g][low ^ (4 * m + g)] = v[m];
  fence_wave();
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = buf[low][(4 * k + g) ^ low];
}

template <int RT>
constexpr int kJoined = RT < 4 ? RT : 4;  // rank tiles joined at a time

template <int RT>
union ShrinkLds {
  StepRows rows[kShrinkWaves];
  v4f join[kShrinkWaves][kJoined<RT>][64];
};

// The columns past the last whole step.
template <int RT, bool LONG>
__device__ __forceinline__ void last_columns(StepRows &buf, const uint16_t *const (&xr)[4],
                                             const uint16_t *const (&wr)[RT][4], int64_t st,
                                             int64_t C, v4f (&acc)[RT]) {
  const int lane = threadIdx.x & 63;
  const int c = (int)(st * 128) + 8 * (lane & 15);
  uint4 xv[4];
#pragma unroll
  for (int q0 = 0; q0 < RT; q0 += kJoined<RT>) {
    Chunk<bf16_t> xc[4], wc[kJoined<RT>][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (q0 == 0) xc[m] = raw8<LONG>(xr[m], c, C);
#pragma unroll
      for (int q = 0; q < kJoined<RT>; ++q) wc[q][m] = raw8<LONG>(wr[q0 + q][m], c, C);
    }
    if (q0 == 0) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        settle_chunk(xc[m], c, (int)C);
        xv[m] = words(xc[m]);
      }
      to_operands(buf, xv);
    }
#pragma unroll
    for (int q = 0; q < kJoined<RT>; ++q) {
      uint4 wv[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        settle_chunk(wc[q][m], c, (int)C);
        wv[m] = words(wc[q][m]);
      }
      to_operands(buf, wv);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[q0 + q] = mfma(wv[m], xv[m], acc[q0 + q]);
    }
    if (RT > 4) __builtin_amdgcn_sched_barrier(0);
  }
}

// The waves' sums of a tile.  done(j, t, sum) is called with the sums of ranks
// j .. j + 3 of row t (zeros past r) by the lanes that hold them; the block is
// synchronised afterwards.
template <int RT, typename Done>
__device__ __forceinline__ void join_tile(ShrinkLds<RT> &lds, const v4f (&acc)[RT], int64_t t,
                                          bool mine, int r, Done done) {
  constexpr int JT = kJoined<RT>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
#pragma unroll
  for (int q0 = 0; q0 < RT; q0 += JT) {
    __syncthreads();  // rows and sums before have been read
#pragma unroll
    for (int q = 0; q < JT; ++q) lds.join[wave][q][lane] = acc[q0 + q];
    __syncthreads();
    if (wave < JT && mine) {
      v4f sum = lds.join[0][wave][lane];
#pragma unroll
      for (int k = 1; k < kShrinkWaves; ++k) sum += lds.join[k][wave][lane];
      const int j = 16 * (q0 + wave) + 4 * g;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (j + v >= r) sum[v] = 0.0f;  // rank r - 1 again
      done(j, t, sum);
    }
  }
  __syncthreads();  // the sums have been read
}

// Sums of tile i by all eight waves, up to STEPS of a wave's steps in flight.
template <int RT, int STEPS, bool LONG, typename Done>
__device__ __forceinline__ void contract_tile(ShrinkLds<RT> &lds, const Plan &plan, int i,
                                              int64_t t0, const uint16_t *x, int64_t ldx,
                                              const uint16_t *w, int64_t C, int r, int L,
                                              Done done) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int64_t steps = (C + 127) / 128, whole = C / 128;
  const int s0 = plan.start[i], len = plan.start[i + 1] - s0;
  const int l = plan.id(s0);
  const bool mine = (lane & 15) < len;
  const int64_t t = t0 + plan.place(s0, len, lane & 15);
  v4f acc[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) acc[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (l < L) {
    const uint16_t *xr[4], *wr[RT][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      xr[m] = x + (t0 + plan.place(s0, len, 4 * m + g)) * ldx;
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int j = 16 * q + 4 * m + g;
        wr[q][m] = w + ((int64_t)l * r + (j < r ? j : r - 1)) * C;
      }
    }
    int64_t st = wave;
    auto several = [&](auto n) {  // n steps, the loads of up to four rank tiles in flight
      uint4 xv[n][4];
#pragma unroll
      for (int q0 = 0; q0 < RT; q0 += kJoined<RT>) {
        uint4 wv[n][kJoined<RT>][4];
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const int64_t c = (st + k * kShrinkWaves) * 128 + 8 * (lane & 15);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (q0 == 0) __builtin_memcpy(&xv[k][m], xr[m] + c, 16);
#pragma unroll
            for (int q = 0; q < kJoined<RT>; ++q)
              __builtin_memcpy(&wv[k][q][m], wr[q0 + q][m] + c, 16);
          }
        }
#pragma unroll
        for (int k = 0; k < n; ++k) {
          if (q0 == 0) to_operands(lds.rows[wave], xv[k]);
#pragma unroll
          for (int q = 0; q < kJoined<RT>; ++q) {
            to_operands(lds.rows[wave], wv[k][q]);
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[q0 + q] = mfma(wv[k][q][m], xv[k][m], acc[q0 + q]);
          }
        }
        if (RT > 4) __builtin_amdgcn_sched_barrier(0);
      }
      st += n * kShrinkWaves;
    };
    while (st + (STEPS - 1) * kShrinkWaves < whole)
      several(std::integral_constant<int, STEPS>());
    if (STEPS > 1)
      while (st < whole) several(std::integral_constant<int, 1>());
    if (st < steps) last_columns<RT, LONG>(lds.rows[wave], xr, wr, st, C, acc);
  }
  join_tile<RT>(lds, acc, t, mine, r, done);
}

// The parts of sum in a row of parts, from rank j on.
template <int RT>
__device__ __forceinline__ void store_parts(uint16_t *row, int j, const v4f &sum) {
  const Parts a = parts_of(sum[0]), b = parts_of(sum[1]);
  const Parts c = parts_of(sum[2]), d = parts_of(sum[3]);
  *reinterpret_cast<uint2 *>(row + j) = make_uint2(
      __builtin_amdgcn_perm(b.hi, a.hi, 0x07060302u), __builtin_amdgcn_perm(d.hi, c.hi, 0x07060302u));
  *reinterpret_cast<uint2 *>(row + j + 16 * RT) =
      make_uint2(__builtin_amdgcn_perm(b.mid, a.mid, 0x07060302u),
                 __builtin_amdgcn_perm(d.mid, c.mid, 0x07060302u));
  *reinterpret_cast<uint2 *>(row + j + 32 * RT) = make_uint2(
      __builtin_amdgcn_perm(b.lo, a.lo, 0x07060302u), __builtin_amdgcn_perm(d.lo, c.lo, 0x07060302u));
  if (RT == 1) *reinterpret_cast<uint2 *>(row + j + 48) = make_uint2(0, 0);
}

__device__ __forceinline__ void store_sums(float *u, int j, int r, const v4f &sum) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (j + v < r) u[j + v] = sum[v];
}

// The outer sums take an adapter's rows in tiles of `chunk`; an adapter with one
// tile is written at once, the others' tiles leave their sums in slots that
// adapter_join_kernel adds up.
struct Grouping {
  int32_t *rows, *off;  // rows by adapter (null: none wanted); bounds (launch_group_rows)
  int4 *tiles;          // (adapter, first row, end, slot or -1); adapter -1 past the last
  int2 *sums;           // of each adapter: tiles, first slot
  int most, chunk;      // entries of `tiles`
};

// Tiles and slots of the adapters, 64 at a time, by one wave: `at` and `m` are the
// first row and the number of rows of adapter l (m = 0 past the last).
struct TileMaker {
  int tiles = 0, slots = 0;
  __device__ __forceinline__ void add(const Grouping &gr, int l, int L, int at, int m) {
    const int lane = threadIdx.x & 63;
    const int n = (m + gr.chunk - 1) / gr.chunk, k = n > 1 ? n : 0;
    int tn = n, tk = k;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int un = __shfl_up(tn, d, 64), uk = __shfl_up(tk, d, 64);
      if (lane >= d) {
        tn += un;
        tk += uk;
      }
    }
    const int first = tiles + tn - n, slot = slots + tk - k;
    if (l < L) gr.sums[l] = make_int2(n, slot);
    for (int i = 0; i < n; ++i) {
      const int r0 = at + i * gr.chunk, r1 = r0 + gr.chunk;
      gr.tiles[first + i] = make_int4(l, r0, r1 < at + m ? r1 : at + m, n > 1 ? slot + i : -1);
    }
    tiles += __shfl(tn, 63, 64);
    slots += __shfl(tk, 63, 64);
  }
  __device__ __forceinline__ void finish(const Grouping &gr) {
    for (int i = tiles + (threadIdx.x & 63); i < gr.most; i += 64)
      gr.tiles[i] = make_int4(-1, 0, 0, -1);
  }
};

__global__ void __launch_bounds__(64) adapter_tiles_kernel(Grouping gr, int L) {
  TileMaker tm;
  for (int l0 = 0; l0 < L; l0 += 64) {
    const int l = l0 + threadIdx.x;
    const int at = l < L ? gr.off[l] : 0;
    tm.add(gr, l, L, at, l < L ? gr.off[l + 1] - at : 0);
  }
  tm.finish(gr);
}

// Rows by adapter for the outer sums (what launch_group_rows makes), by one block
// beside the contraction: 8192 rows make that 28 -> 29 us, where three launches
// take 13 us and 10 us of the host's time.  Each wave counts and then places a stretch of the rows; `start`, its
// next row of each id (L: none), holds kShrinkWaves x (L + 1).
constexpr int64_t kGroupedRows = 8192;  // more would outlast the contraction
constexpr int kGroupedMost = 1000;      // adapters

__device__ __forceinline__ void group_block(const int32_t *ids, int n, int L, const Grouping &gr,
                                            int *start) {
  constexpr int W = kShrinkWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int k = threadIdx.x; k < W * (L + 1); k += 64 * W) start[k] = 0;
  __syncthreads();
  int *mine = start + wave * (L + 1);
  const int per = (n + 64 * W - 1) / (64 * W) * 64;
  const int i0 = wave * per, i1 = i0 + per < n ? i0 + per : n;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 64) {
    const int l = ids[i];
    atomicAdd(&mine[l >= 0 && l < L ? l : L], 1);
  }
  __syncthreads();
  if (wave == 0) {  // counts -> first rows
    int carry = 0;
    TileMaker tm;
    for (int l0 = 0; l0 <= L; l0 += 64) {
      const int l = l0 + lane <= L ? l0 + lane : L;
      int m[W], all = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        m[w] = start[w * (L + 1) + l];
        all += m[w];
      }
      int inc = l0 + lane <= L ? all : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(inc, d, 64);
        if (lane >= d) inc += up;
      }
      int at = carry + inc - all;
      tm.add(gr, l0 + lane, L, at, l0 + lane < L ? all : 0);
      if (l0 + lane <= L) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          start[w * (L + 1) + l] = at;
          at += m[w];
        }
      }
      carry += __shfl(inc, 63, 64);
    }
    tm.finish(gr);
  }
  __syncthreads();
  int next = i0 < i1 ? ids[i0 + lane < i1 ? i0 + lane : i1 - 1] : 0;
  for (int i = i0 + lane; i - lane < i1; i += 64) {
    int l = i < i1 ? next : L;
    if (l < 0 || l >= L) l = L;
    next = ids[i + 64 < i1 ? i + 64 : i1 - 1];
    uint64_t same = __ballot(i < i1);  // lanes with the same id
    for (int bit = 1; bit <= L; bit <<= 1) {
      const uint64_t set = __ballot((l & bit) != 0);
      same &= (l & bit) ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    fence_wave();
    const int row = mine[l] + rank;
    fence_wave();
    if (i < i1) {
      if (rank == 0) mine[l] = row + __popcll(same);
      gr.rows[row] = l < L ? i : -1;
    }
  }
}

// gridDim.y counts the shares of a chunk, and one more where `gr` is wanted: its
// first block groups the rows.
template <int RT, bool LONG>
__global__ void __launch_bounds__(64 * kShrinkWaves)
    adapter_shrink_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                          const int32_t *__restrict__ ids, const uint16_t *__restrict__ w,
                          float *__restrict__ u, uint16_t *__restrict__ parts, int64_t T, int64_t C,
                          int r, int L, Grouping gr) {
  __shared__ Plan plan;
  __shared__ ShrinkLds<RT> lds;
  int shares = gridDim.y, share = blockIdx.y;
  if (gr.rows) {  // dispatched first, as it takes longest
    if (share == 0) {
      static_assert(sizeof(lds) >= 4 * kShrinkWaves * (kGroupedMost + 1), "room for the counts");
      if (blockIdx.x == 0) group_block(ids, (int)T, L, gr, reinterpret_cast<int *>(&lds));
      return;
    }
    --shares;
    --share;
  }
  const int64_t t0 = (int64_t)blockIdx.x * kChunk;
  make_plan(plan, ids, t0, T, L);
  const int lo = (int)((int64_t)plan.tiles * share / shares);
  const int hi = (int)((int64_t)plan.tiles * (share + 1) / shares);
  for (int i = lo; i < hi; ++i)
    contract_tile<RT, (RT == 1 ? 4 : RT == 2 ? 2 : 1), LONG>(
        lds, plan, i, t0, x, ldx, w, C, r, L, [&](int j, int64_t t, const v4f &sum) {
          store_sums(u + t * r, j, r, sum);
          if (parts) store_parts<RT>(parts + t * (parts_kept(RT) * 16 * RT), j, sum);
        });
}

// ---------------------------------------------------------------------------
// expand: out_t[c] = base_t[c] + s sum_j u_t[j] w_id,j[c], u from the parts that shrink
// left.  (s multiplies the sum, not u: s u may leave fp32's range where out does not.)
// A wave has 128 columns; the operand of its adapter's factor stays in registers while
// the adapter does not change.  A lane ends up with eight neighbouring columns of four
// rows.  The next tile's operands and base are on their way while a tile is computed.
// blockIdx: 512 columns, chunk, share of the chunk's tiles.
//
// Bound by HBM: 4096 rows of 11008 bf16, rank 16, 38 us, 4.9 TB/s (48 us with the two
// blocks a CU that the compiler's own choice of registers allows; 127 us for the
// first form, which loaded u one value at a time); 8192 of 4096, rank 32, 31 us;
// 4096 of 4096 fp32 on 16 adapters in random order 43 us.  The blocks a CU are those
// whose registers hold a type and rank, to within a few spills: at ranks 33 .. 64 in
// fp32, where two leave 8 spilled, 2048 of 4096 take 20.8 us, with one 24.0 (bf16, none
// spilled: the call 28 us, with one 34); from 65 on one.

constexpr int operands(int rp) { return (rp + 1) / 2; }     // of 32 ranks
constexpr int parts_of_operand(int rp) { return rp == 1 ? 2 : 3; }

// A row's operands, for lane group g.
template <int RP>
struct RowParts {
  uint4 v[operands(RP)][parts_of_operand(RP)];
  __device__ __forceinline__ void load(const uint16_t *row, int g) {
#pragma unroll
    for (int q = 0; q < operands(RP); ++q)
#pragma unroll
      for (int p = 0; p < parts_of_operand(RP); ++p)
        v[q][p] = *reinterpret_cast<const uint4 *>(row + 8 * g + 32 * q +
                                                   p * (RP == 1 ? 32 : 16 * RP));
  }
};

// Eight columns of 32 ranks (operand q) of an adapter's factor (r x C) from column
// c on.
template <int RP, bool LONG>
struct Factor {
  Chunk<bf16_t> raw[8];
  __device__ __forceinline__ static int rank(int q, int g, int k) {
    return (RP == 1 ? 8 * (g & 1) : 32 * q + 8 * g) + k;
  }
  __device__ __forceinline__ void load(const uint16_t *w, int q, int64_t c, int64_t C, int r,
                                       int g) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = rank(q, g, k);
      raw[k] = raw8<LONG>(w + (int64_t)(j < r ? j : r - 1) * C, c, C);
    }
  }
  __device__ __forceinline__ void operand(int q, int64_t c, int64_t C, int r, int g, bool edge,
                                          uint4 (&f)[8]) {
    uint4 rows[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (edge) settle_chunk(raw[k], (int)c, (int)C);
      rows[k] = words(raw[k]);
    }
    if (r < 16 * RP) {  // ranks past r: no value, not even an infinite one
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (rank(q, g, k) >= r) rows[k] = make_uint4(0, 0, 0, 0);
    }
    transpose8(rows, f);
  }
};

// An adapter's scale, l the same in all lanes: a scalar load, beside the vector loads in
// flight instead of behind them, and without a choice ahead of it (`ids`, of at least one
// row, is read where there is no scale).
__device__ __forceinline__ float scale_of(const float *scale, int l, bool has,
                                          const int32_t *ids) {
  typedef const __attribute__((address_space(4))) uint32_t constant_t;
  has = has && scale;
  const uintptr_t at = has ? (uintptr_t)(scale + l) : (uintptr_t)ids;
  const uint32_t v = *(constant_t *)at;
  return has ? __uint_as_float(v) : 1.0f;
}

// base + s times the products of a tile: lane g holds rows 4 g .. 4 g + 3 of it, eight
// columns.
template <typename O, int RP, bool LONG>
__device__ __forceinline__ void finish_tile(const Plan &plan, int s0, int len, bool has, float s,
                                            const RowParts<RP> &u,
                                            const uint4 (&f)[operands(RP)][8], Chunk<O> (&b)[4],
                                            bool base, O *out, int64_t ldo, int64_t t0, int64_t c,
                                            int64_t C, bool edge, int g) {
  v4f acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (has) {
#pragma unroll
    for (int p = parts_of_operand(RP) - 1; p >= 0; --p)
#pragma unroll
      for (int q = 0; q < operands(RP); ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = mfma(u.v[q][p], f[q][j], acc[j]);
    bool nan = false;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float all = acc[0][v];
#pragma unroll
      for (int j = 1; j < 8; ++j) all += acc[j][v];
      nan |= 4 * g + v < len && all != all;
    }
    if (__any(nan)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v4f high = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < operands(RP); ++q) {
          const bool lower = RP == 1 && g >= 2;  // the operand's other half: middle parts
          high = mfma(u.v[q][0], lower ? make_uint4(0, 0, 0, 0) : f[q][j], high);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][v] = unless_nan(acc[j][v], high[v]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (4 * g + v >= len) continue;
    if (edge && base) settle_chunk(b[v], (int)c, (int)C);
    float val[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float from = base ? chunk_value(b[v], j) : 0.0f;
      val[j] = has ? fmaf(acc[j][v], s, from) : from;
    }
    store_chunk(out + (t0 + plan.place(s0, len, 4 * g + v)) * ldo, (int)c, (int)C, val);
  }
}

template <typename O>
struct Expand {
  const uint16_t *parts;  // of w's side, T x parts_kept x 16 RP
  const int32_t *ids;
  const uint16_t *w;
  const float *scale;
  const O *base;
  O *out;
  int64_t ldb, ldo, T, C;
  int r, L;
};

// Block: 512 columns, a chunk of rows, a share of its tiles.
template <typename O, int RP, bool LONG>
__device__ __forceinline__ void expand_block(const Expand<O> &e, Plan &plan, dim3 block,
                                             int shares) {
  const uint16_t *__restrict__ parts = e.parts, *__restrict__ w = e.w;
  const O *base = e.base;
  O *out = e.out;
  const int64_t ldb = e.ldb, ldo = e.ldo, T = e.T, C = e.C;
  const int r = e.r, L = e.L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int64_t t0 = (int64_t)block.y * kChunk;
  make_plan(plan, e.ids, t0, T, L);
  const int lo = (int)((int64_t)plan.tiles * block.z / shares);
  const int hi = (int)((int64_t)plan.tiles * (block.z + 1) / shares);
  const int64_t c0 = ((int64_t)block.x * 4 + wave) * 128;
  if (c0 >= C || lo >= hi) return;
  const int64_t c = c0 + 8 * (lane & 15);
  const bool edge = c0 + 128 > C;

  struct Fetch {
    RowParts<RP> u;
    Chunk<O> b[4];
  };
  auto fetch = [&](int i, Fetch &f) {
    i = i < hi ? i : hi - 1;  // past the last: again, unused
    const int s0 = plan.start[i], len = plan.start[i + 1] - s0;
    f.u.load(parts + (t0 + plan.place(s0, len, lane & 15)) * (parts_kept(RP) * 16 * RP), g);
    if (base) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        f.b[v] = raw8<LONG>(base + (t0 + plan.place(s0, len, 4 * g + v)) * ldb, c, C);
    }
  };
  int now = -1;  // the adapter whose factor is in wf, and its scale
  float s = 1.0f;
  uint4 wf[operands(RP)][8];
  auto tile = [&](int i, Fetch &f) {
    const int s0 = plan.start[i], len = plan.start[i + 1] - s0;
    const int l = __builtin_amdgcn_readfirstlane(plan.id(s0));  // the tile's: of all lanes
    const bool has = l < L;
    if (!has && base == out) return;  // in place, rows without an adapter stay as they are
    if (has && l != now) {
      now = l;
      s = scale_of(e.scale, l, true, e.ids);
#pragma unroll
      for (int q = 0; q < operands(RP); ++q) {
        Factor<RP, LONG> w8;
        w8.load(w + (int64_t)l * r * C, q, c, C, r, g);
        w8.operand(q, c, C, r, g, edge, wf[q]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    finish_tile<O, RP, LONG>(plan, s0, len, has, s, f.u, wf, f.b, base != nullptr, out, ldo, t0, c,
                             C, edge, g);
  };
  Fetch one, two;
  fetch(lo, one);
  for (int i = lo; i < hi; i += 2) {
    fetch(i + 1, two);
    __builtin_amdgcn_sched_barrier(0);
    tile(i, one);
    if (i + 1 >= hi) return;
    fetch(i + 2, one);
    __builtin_amdgcn_sched_barrier(0);
    tile(i + 1, two);
  }
}

template <typename O, int RP, bool LONG>
__global__ void __launch_bounds__(256, RP <= 2 ? (sizeof(O) == 2 ? 3 : 2) : RP == 4 ? 2 : 1)
    adapter_expand_kernel(Expand<O> e) {
  __shared__ Plan plan;
  expand_block<O, RP, LONG>(e, plan, blockIdx, gridDim.z);
}

// Few rows: both products in one launch.  Every block of 1024 columns sums u
// again for its tiles, from the caches, which costs less than a second launch
// waiting for the first: 32 rows on 24 adapters, 4096 x 4096 rank 16, 10.3 us (the
// two kernels 7.2 + 5.2 us, and 3.5 us more on the host); one row 8.6 us from HBM,
// 5.3 from the caches.  Bound by the chain ids -> plan -> columns -> join -> factor.
// More steps in flight, or the factor asked for ahead of the sums, need registers
// that are not there (12.7 us with spills).
template <typename O, int RT, bool LONG>
__global__ void __launch_bounds__(64 * kShrinkWaves)
    adapter_small_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                         const int32_t *__restrict__ ids, const uint16_t *__restrict__ a,
                         const uint16_t *__restrict__ b, const float *__restrict__ scale,
                         const O *base, int64_t ldb, O *out, int64_t ldo, float *__restrict__ u,
                         int64_t T, int64_t K, int64_t N, int r, int L) {
  static_assert(operands(RT) == 1, "one operand of ranks");
  constexpr int kRow = parts_kept(RT) * 16 * RT;
  __shared__ Plan plan;
  __shared__ ShrinkLds<RT> lds;
  __shared__ uint16_t parts[16][kRow] __attribute__((aligned(16)));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  make_plan(plan, ids, 0, T, L);
  const int lo = (int)((int64_t)plan.tiles * blockIdx.y / gridDim.y);
  const int hi = (int)((int64_t)plan.tiles * (blockIdx.y + 1) / gridDim.y);
  const int64_t c0 = ((int64_t)blockIdx.x * kShrinkWaves + wave) * 128;
  const int64_t c = c0 + 8 * (lane & 15);
  const bool edge = c0 + 128 > N;
  for (int i = lo; i < hi; ++i) {
    const int s0 = plan.start[i], len = plan.start[i + 1] - s0;
    const int l = __builtin_amdgcn_readfirstlane(plan.id(s0));
    const bool has = l < L, mine = c0 < N && (has || base != out);
    Chunk<O> bs[4];
    if (mine && base) {  // under way during the first product
#pragma unroll
      for (int v = 0; v < 4; ++v)
        bs[v] = raw8<LONG>(base + (int64_t)plan.place(s0, len, 4 * g + v) * ldb, c, N);
    }
    contract_tile<RT, 1, LONG>(lds, plan, i, 0, x, ldx, a, K, r, L,
                               [&](int j, int64_t t, const v4f &sum) {
                                 if (blockIdx.x == 0) store_sums(u + t * r, j, r, sum);
                                 store_parts<RT>(parts[lane & 15], j, sum);
                               });
    if (!mine) continue;
    const float s = scale_of(scale, l, has, ids);
    RowParts<RT> rp;
    rp.load(parts[lane & 15], g);
    uint4 f[operands(RT)][8];
    if (has) {
      Factor<RT, LONG> w8;
      w8.load(b + (int64_t)l * r * N, 0, c, N, r, g);
      w8.operand(0, c, N, r, g, edge, f[0]);
    }
    finish_tile<O, RT, LONG>(plan, s0, len, has, s, rp, f, bs, base != nullptr, out, ldo, 0, c, N,
                             edge, g);
  }
}

// ---------------------------------------------------------------------------
// outer: d_l[j][c] = s_l sum over the rows t of adapter l of w_t[j] y_t[c], tile by
// tile.  A wave has 128 columns; 32 rows of them and of w are loaded while the 32
// before are multiplied.  8192 rows, 4096 columns bf16 and 4096 in 8 bits, rank 32:
// 36 us (bytes: 20); without y's loads 26, w's 32, two thirds of the matrix
// instructions 29: no one part of a step holds it up, the steps' latency does.

// One side of the gradient: d += w y'.
struct Side {
  const float *w;     // T x r
  const void *y;      // T x C, bf16 or 8 bits
  const uint8_t *ys;  // scale bytes of the 8-bit form
  int64_t ldy, C;
  float *d;     // L x r x C
  float *slot;  // slots of r x C
};

__device__ __forceinline__ bf16x2 widen2(uint32_t v, float scale, bool high) {
  return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false);
}

// Scale bytes that a bf16 operand takes as they are; the rest of the power of
// two goes to w, so that no value leaves bf16's range on either side.
__device__ __forceinline__ int held_scale(int s) { return s < 27 ? 27 : s > 245 ? 245 : s; }

// A finite w that the rest 2^(e - 245) of a scale byte e > 245 would take out of fp32's
// range (what is not zero in the block is at least 2^109, and overflows beside it): the
// largest that it does not, so that the block's zeros give zeros.
__device__ __forceinline__ float held_factor(float w, int e) {
  if (e <= 245 || (__float_as_uint(w) & 0x7F800000u) == 0x7F800000u) return w;
  const float most = __uint_as_float(0x7F7FFFFFu - ((uint32_t)(e - 245) << 23));
  return fminf(fmaxf(w, -most), most);
}

// Rows, values of y and of w for 32 rows of a tile, as they are in memory.
template <int RT, bool F8>
struct Step {
  uint4 y[8];  // 8 bits: x, y the bytes, z the scale byte
  float w[RT][8];
};

// The high parts' sums of a tile, where a sum in `out` is NaN.  In little code, a column
// at a time: what a kernel holds beside its way costs it too (all eight columns at once,
// 777 rows, rank 12: 0.7 us).
__device__ __forceinline__ void outer_high(const Side &sd, const int32_t *rows, int r0, int r1,
                                           float s, int64_t c0, int j0, int tiles, int r,
                                           float *out) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll 1
  for (int n = 0; n < 8 * tiles; ++n) {
    const int64_t c = c0 + 8 * (lane & 15) + (n & 7);
    const uint16_t *y = static_cast<const uint16_t *>(sd.y) + (c < sd.C ? c : 0);
    const int first = j0 + 16 * (n >> 3), j = first + (lane & 15);
    const float *w = sd.w + (j < r ? j : r - 1);
    v4f high = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int i0 = r0; i0 < r1; i0 += 32) {
      uint32_t a[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + 8 * g + k;
        const int64_t t = rows[i < r1 ? i : r1 - 1];
        a[k] = __float_as_uint(w[t * r]);
        b[k] = y[t * sd.ldy];
        if (i >= r1) a[k] = b[k] = 0;
      }
      uint32_t o[4], f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        o[m] = __builtin_amdgcn_perm(a[2 * m + 1], a[2 * m], 0x07060302u);
        f[m] = __builtin_amdgcn_perm(b[2 * m + 1], b[2 * m], 0x05040100u);
      }
      high = mfma(make_uint4(o[0], o[1], o[2], o[3]), make_uint4(f[0], f[1], f[2], f[3]), high);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (c < sd.C && first + 4 * g + v < r) {
        float *at = out + (int64_t)(first + 4 * g + v) * sd.C + c;
        *at = unless_nan(*at, high[v] * s);
      }
    }
  }
}

template <int RT, bool F8, bool LONG>
__device__ __forceinline__ void outer_tile(const Side &sd, const int32_t *rows, int r0, int r1,
                                           float s, int64_t c0, int j0, int r, float *out) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int64_t c = c0 + 8 * (lane & 15), C = sd.C;
  const bool edge = c0 + 128 > C;
  const int last = rows[r1 - 1];
  struct Rows {
    int t[8];
  };
  // the buffer behind rows allows reading past the tile's end
  auto rows_of = [&](int i0) {
    Rows q;
    __builtin_memcpy(q.t, rows + i0 + 8 * g, 32);
    return q;
  };
  auto fetch = [&](int i0, const Rows &q, Step<RT, F8> &st) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t t = i0 + 8 * g + k < r1 ? q.t[k] : last;
      if (F8) {
        uint2 v;
        const int64_t at = c < C ? c : 0;  // columns past C are not stored
        __builtin_memcpy(&v, static_cast<const uint8_t *>(sd.y) + t * f8_row_bytes(C) + at, 8);
        st.y[k].x = v.x;
        st.y[k].y = v.y;
        st.y[k].z = sd.ys[t * f8_scale_bytes(C) + c0 / kF8Block];
      } else {
        st.y[k] = words(raw8<LONG>(static_cast<const uint16_t *>(sd.y) + t * sd.ldy, c, C));
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int j = j0 + 16 * q + (lane & 15);
        st.w[q][k] = sd.w[t * r + (j < r ? j : r - 1)];
      }
    }
  };
  v4f acc[RT][8];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[q][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  Step<RT, F8> cur, next;
  Rows ahead = rows_of(r0);
  fetch(r0, ahead, cur);
  if (r0 + 32 < r1) ahead = rows_of(r0 + 32);
  for (int i0 = r0; i0 < r1; i0 += 32) {
    if (i0 + 32 < r1) {
      fetch(i0 + 32, ahead, next);
      if (i0 + 64 < r1) ahead = rows_of(i0 + 64);
    }
    __builtin_amdgcn_sched_barrier(0);
    uint4 y[8], f[8];
    float rest[8];
    if (F8) {
      int e = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) e = (int)cur.y[k].z > e ? (int)cur.y[k].z : e;
      if (__any(e > 245)) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int q = 0; q < RT; ++q) cur.w[q][k] = held_factor(cur.w[q][k], (int)cur.y[k].z);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] = cur.y[k];
      rest[k] = 1.0f;
      if (F8) {
        const int e = (int)cur.y[k].z, h = held_scale(e);
        const float p = __uint_as_float((uint32_t)h << 23);
        rest[k] = __uint_as_float((uint32_t)(127 + e - h) << 23);
        y[k].x = __builtin_bit_cast(uint32_t, widen2(cur.y[k].x, p, false));
        y[k].y = __builtin_bit_cast(uint32_t, widen2(cur.y[k].x, p, true));
        y[k].z = __builtin_bit_cast(uint32_t, widen2(cur.y[k].y, p, false));
        y[k].w = __builtin_bit_cast(uint32_t, widen2(cur.y[k].y, p, true));
      } else if (edge) {
        Chunk<bf16_t> h = {{y[k].x, y[k].y, y[k].z, y[k].w}};
        settle_chunk(h, (int)c, (int)C);
        y[k] = words(h);
      }
    }
    if (i0 + 32 > r1) {  // rows past the tile's end: zeros on both sides
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + 8 * g + k >= r1) {
          y[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < RT; ++q) cur.w[q][k] = 0.0f;
        }
    }
    transpose8(y, f);
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const bool in = j0 + 16 * q + (lane & 15) < r;
      float w[8];
      uint4 o[3];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = in ? (F8 ? cur.w[q][k] * rest[k] : cur.w[q][k]) : 0.0f;
      split8(w, o);
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[q][j] = mfma(o[p], f[j], acc[q][j]);
    }
    cur = next;
  }
  bool nan = false;
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int j = j0 + 16 * q + 4 * g + v;
      if (j >= r) continue;
      float val[8], all = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        val[k] = acc[q][k][v] * s;
        all += acc[q][k][v];
      }
      nan |= all != all;
      store_chunk(out + (int64_t)j * C, (int)c, (int)C, val);
    }
  // infinities in y's rows (8 bits hold none)
  if (!F8 && __any(nan)) outer_high(sd, rows, r0, r1, s, c0, j0, RT, r, out);
}

struct Outer {
  Side first, second;
  const int32_t *rows;
  const int4 *tiles;
  const float *scale;
  int split, most, r;
};

// Block: 512 columns of the first or (from `split` on) the second side, a tile,
// RT x 16 of the ranks.
template <int RT, bool F8, bool LONG>
__device__ __forceinline__ void outer_block(const Outer &o, dim3 block, int step) {
  const bool two = (int)block.x >= o.split;
  const int wave = threadIdx.x >> 6, r = o.r;
  const Side &sd = two ? o.second : o.first;
  const int64_t c0 = ((int64_t)(two ? block.x - o.split : block.x) * 4 + wave) * 128;
  if (c0 >= sd.C) return;
  for (int i = block.y; i < o.most; i += step) {
    const int4 t = o.tiles[i];
    if (t.x < 0) return;
    const float s = o.scale ? o.scale[t.x] : 1.0f;
    float *out = t.w < 0 ? sd.d + (int64_t)t.x * r * sd.C : sd.slot + (int64_t)t.w * r * sd.C;
    const int j0 = block.z * RT * 16;
    if (two || !F8) outer_tile<RT, false, LONG>(sd, o.rows, t.y, t.z, s, c0, j0, r, out);
    else outer_tile<RT, F8, LONG>(sd, o.rows, t.y, t.z, s, c0, j0, r, out);
  }
}

template <int RT, bool F8, bool LONG>
__global__ void __launch_bounds__(256) adapter_outer_kernel(Outer o) {
  outer_block<RT, F8, LONG>(o, blockIdx, gridDim.y);
}

// The input's gradient and the outer sums in one launch: neither waits for the
// other, the first is bound by memory, the second by its steps' latency.  Their
// blocks alternate, so that a CU has one of each: 8192 rows, 4096 bf16 and 4096 in 8
// bits, rank 32: the call 94 us, as two launches 102; 20000 rows, rank 16: 186 us
// (outer sums first 201, last 209, two launches 227).  Two blocks a CU, although that
// spills 6 to 26 registers at ranks 17 .. 32 with x in 8 bits and at 33 .. 64 with that or
// fp32 outputs: the first case with one 117 us, 4096 rows, rank 64, x in bf16 85 (one
// 105), in 8 bits with fp32 outputs 107 (one 110).
struct Grid {
  unsigned x, y, z;
  __host__ __device__ unsigned blocks() const { return x * y * z; }
  __device__ dim3 at(unsigned i) const { return dim3(i % x, i / x % y, i / x / y); }
};

template <typename O, int RP, bool F8, bool LONG>
__global__ void __launch_bounds__(256, 2)
    adapter_both_kernel(Expand<O> e, Grid ge, Outer o, Grid go) {
  __shared__ Plan plan;
  const uint64_t i = blockIdx.x, no = go.blocks(), n = no + ge.blocks();
  const unsigned k = (unsigned)(i * no / n);  // outer sums before this block
  if ((unsigned)((i + 1) * no / n) > k)
    outer_block<RP == 1 ? 1 : 2, F8, LONG>(o, go.at(k), go.y);
  else
    expand_block<O, RP, LONG>(e, plan, ge.at((unsigned)i - k), ge.z);
}

// The sums of adapters with several tiles, and zeros for those without rows.  A
// thread has four neighbours (the last ones end with the matrix) of eight slots at
// a time, without a choice between the loads; blockIdx.y and gridDim.y deal out
// the adapters.  20 slots of 32 x 8192: 5.3 us (17 us with branches).
__global__ void __launch_bounds__(256)
    adapter_join_kernel(Side first, Side second, int split, const int2 *__restrict__ sums, int r,
                        int L) {
  constexpr int V = 4, IN_FLIGHT = 8;
  const bool two = (int)blockIdx.x >= split;
  const int64_t n = (int64_t)r * (two ? second.C : first.C);
  const float *slots = two ? second.slot : first.slot;
  float *d = two ? second.d : first.d;
  const int64_t i0 = V * ((int64_t)((int)blockIdx.x - (two ? split : 0)) * 256 + threadIdx.x);
  const int64_t step = (int64_t)(two ? gridDim.x - split : split) * 256 * V;
  for (int l = blockIdx.y; l < L; l += gridDim.y) {
    const int2 e = sums[l];
    const int tiles = e.x;
    if (tiles == 1) continue;
    if (n < V) {
      for (int64_t i = i0 / V; i < n; i += step / V) {
        float sum = 0.0f;
        for (int k = 0; k < tiles; ++k) sum += slots[(e.y + k) * n + i];
        d[l * n + i] = sum;
      }
      continue;
    }
    for (int64_t i = i0; i < n; i += step) {
      float s[V];
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] = 0.0f;
      const float *at = slots + e.y * n + (i + V <= n ? i : n - V);
      for (int k0 = 0; k0 < tiles; k0 += IN_FLIGHT) {
        float v[IN_FLIGHT][V];
#pragma unroll
        for (int k = 0; k < IN_FLIGHT; ++k)
          __builtin_memcpy(v[k], at + (k0 + k < tiles ? k0 + k : tiles - 1) * n, 4 * V);
#pragma unroll
        for (int k = 0; k < IN_FLIGHT; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) s[j] += k0 + k < tiles ? v[k][j] : 0.0f;
      }
      __builtin_memcpy(d + l * n + (i + V <= n ? i : n - V), s, 4 * V);
    }
  }
}

// ---------------------------------------------------------------------------

// Ranks in tiles of 16, as the kernels are made for them.
int rank_tiles(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

int64_t parts_bytes(int64_t T, int64_t r) {
  const int rp = rank_tiles(r);
  return T * parts_kept(rp) * 32 * rp;
}

// Shares of a chunk's tiles: `want` blocks in all, no more than tiles there can be.
unsigned tile_shares(int64_t T, int L, int64_t blocks, int64_t want) {
  const int64_t n = T < kChunk ? T : kChunk;
  const int64_t most = n / 16 + 1 + (L + 1 < n ? L + 1 : n);
  int64_t z = (want + blocks - 1) / blocks;
  return (unsigned)(z < 1 ? 1 : z > most ? most : z);
}

hipError_t shrink(const uint16_t *x, int64_t ldx, const int32_t *ids, const uint16_t *w,
                  float *u, uint16_t *parts, int64_t T, int64_t C, int r, int L,
                  const Grouping &gr, hipStream_t s) {
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  // a block a CU, and a few CUs left for the one that groups the rows: 8192 rows in
  // 224 blocks 29 us, in 256 (one more round then) 33
  const dim3 grid((unsigned)chunks, tile_shares(T, L, chunks, 224) + (gr.rows ? 1 : 0));
#define BNN_SHRINK_AS(RT, LONG)                                                                 \
  adapter_shrink_kernel<RT, LONG><<<grid, 64 * kShrinkWaves, 0, s>>>(x, ldx, ids, w, u, parts,  \
                                                                     T, C, r, L, gr)
#define BNN_SHRINK(RT)                    \
  do {                                    \
    if (C >= 8) BNN_SHRINK_AS(RT, true);  \
    else BNN_SHRINK_AS(RT, false);        \
  } while (0)
  switch (rank_tiles(r)) {
    case 1: BNN_SHRINK(1); break;
    case 2: BNN_SHRINK(2); break;
    case 4: BNN_SHRINK(4); break;
    default: BNN_SHRINK(8);
  }
#undef BNN_SHRINK
#undef BNN_SHRINK_AS
  return hipGetLastError();
}

constexpr int64_t kMostChunks = 65535;  // of a launch

template <typename O>
hipError_t expand(const uint16_t *parts, const int32_t *ids, const uint16_t *w, const float *scale,
                  const void *base, int64_t ldb, void *out, int64_t ldo, int64_t T, int64_t C, int r,
                  int L, hipStream_t s) {
  const int64_t all = (T + kChunk - 1) / kChunk, cols = (C + 511) / 512;
  const O *bt = static_cast<const O *>(base);
  O *ot = static_cast<O *>(out);
  for (int64_t k = 0; k < all; k += kMostChunks) {
    const int64_t chunks = all - k < kMostChunks ? all - k : kMostChunks, t = k * kChunk;
    const int64_t n = T - t < chunks * kChunk ? T - t : chunks * kChunk;
    const dim3 grid((unsigned)cols, (unsigned)chunks, tile_shares(n, L, cols * chunks, 384));
    const uint16_t *pt = parts + parts_bytes(t, r) / 2;
    const Expand<O> e = {pt,  ids + t, w, scale, bt ? bt + t * ldb : nullptr, ot + t * ldo,
                         ldb, ldo,     n, C,     r,                           L};
#define BNN_EXPAND_AS(RP, LONG) adapter_expand_kernel<O, RP, LONG><<<grid, 256, 0, s>>>(e)
#define BNN_EXPAND(RP)                    \
  do {                                    \
    if (C >= 8) BNN_EXPAND_AS(RP, true);  \
    else BNN_EXPAND_AS(RP, false);        \
  } while (0)
    switch (rank_tiles(r)) {
      case 1: BNN_EXPAND(1); break;
      case 2: BNN_EXPAND(2); break;
      case 4: BNN_EXPAND(4); break;
      default: BNN_EXPAND(8);
    }
#undef BNN_EXPAND
#undef BNN_EXPAND_AS
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

hipError_t expand_as(int dtype, const uint16_t *parts, const int32_t *ids, const uint16_t *w,
                     const float *scale, const void *base, int64_t ldb, void *out, int64_t ldo,
                     int64_t T, int64_t C, int r, int L, hipStream_t s) {
  if (dtype == BNN_FP32)
    return expand<float>(parts, ids, w, scale, base, ldb, out, ldo, T, C, r, L, s);
  return expand<bf16_t>(parts, ids, w, scale, base, ldb, out, ldo, T, C, r, L, s);
}

// Rows of a tile of the outer sums: about 16 tiles, which with the columns' blocks
// fill the chip (8192 rows, rank 32, 2 x 4096 columns: 37 us of 512 each, 43 of 256;
// 1024 rows, rank 16: 10.6 us of 128, 13.2 of 256), and at most 64.
int64_t outer_chunk(int64_t T) {
  int64_t c = (T + 15) / 16;
  c = c < 128 ? 128 : c > 512 ? 512 : c;
  if (c < (T + 63) / 64) c = (T + 63) / 64;
  return (c + 31) / 32 * 32;
}

struct BwdLayout {
  int64_t v, parts, rows, off, tiles, sums, group, slot_a, slot_b, bytes, chunk, most;
};

BwdLayout bwd_layout(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  BwdLayout b;
  b.chunk = outer_chunk(T);
  b.most = (T < L ? T : L) + T / b.chunk;
  const int64_t slots = T <= b.chunk ? 0 : 2 * (T / b.chunk);
  b.v = 0;
  b.parts = b.v + align16(T * r * 4);
  b.rows = b.parts + parts_bytes(T, r);
  b.off = b.rows + align16(T * 4 + 256);  // read a step past a tile's end
  b.tiles = b.off + align16((L + 1) * 4);
  b.sums = b.tiles + b.most * 16;
  b.group = b.sums + align16(L * 8);
  b.slot_a = b.group + align16(group_rows_workspace(T, L));
  b.slot_b = b.slot_a + align16(slots * r * K * 4);
  b.bytes = b.slot_b + align16(slots * r * N * 4);
  return b;
}

template <typename O>
hipError_t both(Expand<O> e, const Grid &ge, const Outer &o, const Grid &go, hipStream_t s) {
  const unsigned blocks = ge.blocks() + go.blocks();
  const bool f8 = o.first.ys != nullptr;
  const bool wide = (o.first.C >= 8 || o.first.C == 0) && (o.second.C >= 8 || o.second.C == 0);
#define BNN_BOTH_AS(RP, F8, LONG) \
  adapter_both_kernel<O, RP, F8, LONG><<<blocks, 256, 0, s>>>(e, ge, o, go)
#define BNN_BOTH(RP)                                  \
  do {                                                \
    if (wide && f8) BNN_BOTH_AS(RP, true, true);      \
    else if (wide) BNN_BOTH_AS(RP, false, true);      \
    else if (f8) BNN_BOTH_AS(RP, true, false);        \
    else BNN_BOTH_AS(RP, false, false);               \
  } while (0)
  switch (rank_tiles(o.r)) {
    case 1: BNN_BOTH(1); break;
    case 2: BNN_BOTH(2); break;
    default: BNN_BOTH(4);
  }
#undef BNN_BOTH
#undef BNN_BOTH_AS
  return hipGetLastError();
}

bool adapter_small(int64_t T, int64_t N, int64_t r, int64_t L) {
  return T <= kChunk && r <= 32 && (T / 16 + 1 + (L + 1 < T ? L + 1 : T)) * ((N + 1023) / 1024) <= 256;
}

// No more tiles than blocks that run at once, in one chunk.
template <typename O>
hipError_t small(const uint16_t *x, int64_t ldx, const int32_t *ids, const uint16_t *a,
                 const uint16_t *b, const float *scale, const void *base, int64_t ldb, void *out,
                 int64_t ldo, float *u, int64_t T, int64_t K, int64_t N, int r, int L,
                 hipStream_t s) {
  const dim3 grid((unsigned)((N + 1023) / 1024), tile_shares(T, (int)L, 1, kChunk));
#define BNN_SMALL_AS(RT, LONG)                                                               \
  adapter_small_kernel<O, RT, LONG><<<grid, 64 * kShrinkWaves, 0, s>>>(                      \
      x, ldx, ids, a, b, scale, static_cast<const O *>(base), ldb, static_cast<O *>(out), ldo, \
      u, T, K, N, r, L)
#define BNN_SMALL(RT)                              \
  do {                                             \
    if (K >= 8 && N >= 8) BNN_SMALL_AS(RT, true);  \
    else BNN_SMALL_AS(RT, false);                  \
  } while (0)
  if (r <= 16) BNN_SMALL(1);
  else BNN_SMALL(2);
#undef BNN_SMALL
#undef BNN_SMALL_AS
  return hipGetLastError();
}

}  // namespace

int64_t adapter_fwd_workspace(int64_t T, int64_t N, int64_t r, int64_t L) {
  return N == 0 || adapter_small(T, N, r, L) ? 0 : parts_bytes(T, r);
}

hipError_t launch_adapter_fwd(const uint16_t *x, int64_t ldx, const int32_t *ids,
                              const uint16_t *a, const uint16_t *b, const float *scale,
                              const void *base, int64_t ldb, void *out, int64_t ldo, int dtype,
                              float *u, void *workspace, int64_t T, int64_t K, int64_t N, int r,
                              int L, hipStream_t s) {
  if (N > 0 && adapter_small(T, N, r, L)) {
    if (dtype == BNN_FP32)
      return small<float>(x, ldx, ids, a, b, scale, base, ldb, out, ldo, u, T, K, N, r, L, s);
    return small<bf16_t>(x, ldx, ids, a, b, scale, base, ldb, out, ldo, u, T, K, N, r, L, s);
  }
  uint16_t *parts = static_cast<uint16_t *>(workspace);
  const hipError_t e = shrink(x, ldx, ids, a, u, N > 0 ? parts : nullptr, T, K, r, L, Grouping{}, s);
  if (e != hipSuccess || N == 0) return e;
  return expand_as(dtype, parts, ids, b, scale, base, ldb, out, ldo, T, N, r, L, s);
}

int64_t adapter_bwd_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  return bwd_layout(T, K, N, r, L).bytes;
}

hipError_t launch_adapter_bwd(const AdapterGrad &q, void *workspace, int64_t T, int64_t K,
                              int64_t N, int r, int L, hipStream_t s) {
  const BwdLayout b = bwd_layout(T, K, N, r, L);
  char *ws = static_cast<char *>(workspace);
  float *v = reinterpret_cast<float *>(ws + b.v);
  const Grouping gr = {reinterpret_cast<int32_t *>(ws + b.rows),
                       reinterpret_cast<int32_t *>(ws + b.off),
                       reinterpret_cast<int4 *>(ws + b.tiles),
                       reinterpret_cast<int2 *>(ws + b.sums), (int)b.most, (int)b.chunk};
  uint16_t *parts = reinterpret_cast<uint16_t *>(ws + b.parts);
  const bool beside = q.sums && T > 0 && T <= kGroupedRows && L <= kGroupedMost;
  const int split = (int)((K + 511) / 512), cols = split + (int)((N + 511) / 512);
  const Side sa = {v, q.x, q.xs, q.ldx, K, q.da, reinterpret_cast<float *>(ws + b.slot_a)};
  const Side sb = {q.u, q.dy, nullptr, q.lddy, N, q.db, reinterpret_cast<float *>(ws + b.slot_b)};
  const Outer o = {sa, sb, gr.rows, gr.tiles, q.scale, split, gr.most, r};
  const Grid go = {(unsigned)cols, (unsigned)(b.most < 65535 ? b.most : 65535),
                   (unsigned)((r + (r <= 16 ? 15 : 31)) / (r <= 16 ? 16 : 32))};
  const int64_t kc = (K + 511) / 512, chunks = (T + kChunk - 1) / kChunk;
  // one launch for both, unless its blocks are too many for one line of them
  const bool joined = q.sums && q.dx && T > 0 && K > 0 && r <= 64 && kc * chunks <= (1 << 20) &&
                      cols * b.most <= (1 << 20);
  hipError_t e = hipSuccess;
  if (T > 0) {
    e = shrink(q.dy, q.lddy, q.ids, q.b, v, q.dx ? parts : nullptr, T, N, r, L,
               beside ? gr : Grouping{}, s);
    if (e != hipSuccess) return e;
    if (q.dx && !joined) {
      e = expand_as(q.dtype, parts, q.ids, q.a, q.scale, q.base, q.ldb, q.dx, q.lddx, T, K, r, L, s);
      if (e != hipSuccess) return e;
    }
  }
  if (!q.sums) return hipSuccess;
  if (!beside) {
    e = launch_group_rows(q.ids, gr.rows, gr.off, ws + b.group, T, L, s);
    if (e != hipSuccess) return e;
    adapter_tiles_kernel<<<1, 64, 0, s>>>(gr, L);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (joined) {
    // 640 shorter blocks of dx beside the sums' (384: 4096 rows on 16 adapters in random
    // order, rank 16, 72 us, here 68; 8192 in order 91, here 93)
    const Grid ge = {(unsigned)kc, (unsigned)chunks, tile_shares(T, L, kc * chunks, 640)};
    if (q.dtype == BNN_FP32)
      e = both<float>({parts, q.ids, q.a, q.scale, static_cast<const float *>(q.base),
                       static_cast<float *>(q.dx), q.ldb, q.lddx, T, K, r, L},
                      ge, o, go, s);
    else
      e = both<bf16_t>({parts, q.ids, q.a, q.scale, static_cast<const bf16_t *>(q.base),
                        static_cast<bf16_t *>(q.dx), q.ldb, q.lddx, T, K, r, L},
                       ge, o, go, s);
    if (e != hipSuccess) return e;
  } else if (b.most > 0) {
    const dim3 grid(go.x, go.y, go.z);
#define BNN_OUTER(RT, F8, LONG) adapter_outer_kernel<RT, F8, LONG><<<grid, 256, 0, s>>>(o)
#define BNN_OUTER_AS(RT)                                             \
  do {                                                               \
    if ((K < 8 && K > 0) || (N < 8 && N > 0)) {                      \
      if (q.xs) BNN_OUTER(RT, true, false);                          \
      else BNN_OUTER(RT, false, false);                              \
    } else {                                                         \
      if (q.xs) BNN_OUTER(RT, true, true);                           \
      else BNN_OUTER(RT, false, true);                               \
    }                                                                \
  } while (0)
    if (r <= 16) BNN_OUTER_AS(1);
    else BNN_OUTER_AS(2);
#undef BNN_OUTER_AS
#undef BNN_OUTER
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t na = ((int64_t)r * K + 1023) / 1024, nb = ((int64_t)r * N + 1023) / 1024;
  const int ja = (int)(na < 1024 ? na : 1024), jb = (int)(nb < 1024 ? nb : 1024);
  adapter_join_kernel<<<dim3(ja + jb, L < 16 ? L : 16), 256, 0, s>>>(sa, sb, ja, gr.sums, r,
                                                                     L);
  return hipGetLastError();
}

}  // namespace bnn
