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
// over the rank) and outer (dA, dB: sums over an adapter's rows).  All sums are
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

// Eight bf16 values of a row of n from element c on; zero past n.
__device__ __forceinline__ uint4 load8(const uint16_t *row, int64_t c, int64_t n) {
  uint4 v = {0, 0, 0, 0};
  if (c + 8 <= n) {
    __builtin_memcpy(&v, row + c, 16);
    return v;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (c + j < n) w[j / 2] |= (uint32_t)row[c + j] << (16 * (j & 1));
  v.x = w[0];
  v.y = w[1];
  v.z = w[2];
  v.w = w[3];
  return v;
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

// The adapters met among the 16 rows of a tile: lane l < 16 is told row l's id
// (-1: none, -2: no such row); the s-th distinct one, in the order of its first
// row.  False past the last.
__device__ __forceinline__ uint64_t leaders_of(int id) {
  const int lane = threadIdx.x & 63;
  bool first = lane < 16 && id > -2;
#pragma unroll
  for (int i = 0; i < 15; ++i) {
    const int other = __builtin_amdgcn_readlane(id, i);
    first = first && !(i < lane && other == id);
  }
  return __ballot(first);
}
__device__ __forceinline__ int nth_bit(uint64_t m, int s) {  // -1 past the last
  for (; s > 0 && m; --s) m &= m - 1;
  return m ? __ffsll((unsigned long long)m) - 1 : -1;
}

__device__ __forceinline__ int tile_id(const int32_t *ids, int64_t t0, int64_t T, int L) {
  const int64_t t = t0 + (threadIdx.x & 15);
  if (t >= T) return -2;
  const int id = ids[t];
  return id >= 0 && id < L ? id : -1;
}

// ---------------------------------------------------------------------------
// shrink: part[s][t][j] = sum over split s of the columns of x_t[c] w_id,j[c].
// A block has 16 rows; its four waves take every fourth step of 128 columns
// (a lane: 32 neighbours, 64 bytes) of the block's split and join their sums in
// LDS.  blockIdx.z and gridDim.z deal out the tile's adapters.

template <int RT>
__global__ void __launch_bounds__(256)
    adapter_shrink_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                          const int32_t *__restrict__ ids, const uint16_t *__restrict__ w,
                          float *__restrict__ part, int64_t T, int64_t C, int r, int L) {
  __shared__ v4f join[4][RT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int id = tile_id(ids, t0, T, L);
  const uint64_t leaders = leaders_of(id);
  const int64_t t = t0 + (lane & 15);
  const uint16_t *xr = x + (t < T ? t : T - 1) * ldx;
  float *out = part + ((int64_t)blockIdx.y * T + t) * r;
  const int64_t steps = (C + 127) / 128, whole = C / 128;
  const int units = 4 * gridDim.y, unit = 4 * blockIdx.y + wave;
  for (int z = blockIdx.z;; z += gridDim.z) {
    const int lead = nth_bit(leaders, z);
    if (lead < 0) return;
    const int l = __builtin_amdgcn_readlane(id, lead);
    v4f acc[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (l >= 0) {
      const uint16_t *wr[RT];
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int j = 16 * q + (lane & 15);
        wr[q] = w + ((int64_t)l * r + (j < r ? j : r - 1)) * C;
      }
      int64_t st = unit;
      for (; st < whole; st += units) {
        const int64_t c = st * 128 + 32 * g;
        uint4 xv[4], wv[RT][4];
        __builtin_memcpy(xv, xr + c, 64);
#pragma unroll
        for (int q = 0; q < RT; ++q) __builtin_memcpy(wv[q], wr[q] + c, 64);
#pragma unroll
        for (int q = 0; q < RT; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[q] = mfma(wv[q][i], xv[i], acc[q]);
      }
      if (st < steps) {  // the last columns
        const int64_t c = st * 128 + 32 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 xv = load8(xr, c + 8 * i, C);
#pragma unroll
          for (int q = 0; q < RT; ++q) acc[q] = mfma(load8(wr[q], c + 8 * i, C), xv, acc[q]);
        }
      }
    }
    __syncthreads();  // the sums of the adapter before have been read
#pragma unroll
    for (int q = 0; q < RT; ++q) join[wave][q][lane] = acc[q];
    __syncthreads();
    const bool mine = t < T && id == l;
    for (int q = wave; q < RT; q += 4) {
      v4f s = join[0][q][lane];
#pragma unroll
      for (int i = 1; i < 4; ++i) s += join[i][q][lane];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int j = 16 * q + 4 * g + v;
        if (mine && j < r) out[j] = s[v];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// expand: out_t[c] = base_t[c] + s sum_j u_t[j] w_id,j[c], u_t the sum of S parts.
// A wave has 128 columns; the operand of its adapter's factor stays in registers
// while the adapter does not change.  A lane ends up with eight neighbouring
// columns of four rows.

template <typename O, int RQ>
__global__ void __launch_bounds__(256)
    adapter_expand_kernel(const float *__restrict__ part, int S, const int32_t *__restrict__ ids,
                          const uint16_t *__restrict__ w, const float *__restrict__ scale,
                          const O *base, int64_t ldb, O *out, int64_t ldo, float *__restrict__ u,
                          int64_t T, int64_t C, int r, int L, int tiles) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + wave) * 128;
  const bool store_u = u && c0 == 0;
  if (c0 >= C) return;
  const int64_t c = c0 + 8 * (lane & 15);
  int now = -1;  // the adapter whose factor is in f
  uint4 f[RQ][8];
  float s = 0.0f;
  for (int i = 0; i < tiles; ++i) {
    const int64_t t0 = ((int64_t)blockIdx.y * tiles + i) * 16;
    if (t0 >= T) return;
    const int id = tile_id(ids, t0, T, L);
    const uint64_t leaders = leaders_of(id);
    const int64_t tu = t0 + (lane & 15);
    for (int z = blockIdx.z;; z += gridDim.z) {
      const int lead = nth_bit(leaders, z);
      if (lead < 0) break;
      const int l = __builtin_amdgcn_readlane(id, lead);
      if (l < 0) {  // rows without an adapter
        if (store_u && id == -1)
          for (int j = g; j < r; j += 4) u[tu * r + j] = 0.0f;
        if (base == out) continue;  // in place (the strides are the same then)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t t = t0 + 4 * g + v;
          if (__shfl(id, 4 * g + v, 64) != -1) continue;
          float val[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) val[j] = 0.0f;
          if (base) {
            const Chunk<O> b = load_chunk(base + t * ldb, (int)c, (int)C);
#pragma unroll
            for (int j = 0; j < 8; ++j) val[j] = chunk_value(b, j);
          }
          store_chunk(out + t * ldo, (int)c, (int)C, val);
        }
        continue;
      }
      if (l != now) {
        now = l;
        s = scale ? scale[l] : 1.0f;
#pragma unroll
        for (int q = 0; q < RQ; ++q) {
          uint4 rows[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = 32 * q + 8 * g + k;
            rows[k] = make_uint4(0, 0, 0, 0);
            if (j < r) rows[k] = load8(w + ((int64_t)l * r + j) * C, c, C);
          }
          transpose8(rows, f[q]);
        }
      }
      bool on[4];
      Chunk<O> b[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        on[v] = __shfl(id, 4 * g + v, 64) == l;
        if (base && on[v]) b[v] = load_chunk(base + (t0 + 4 * g + v) * ldb, (int)c, (int)C);
      }
      v4f acc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      const bool mine = id == l;  // of row lane % 16
#pragma unroll
      for (int q = 0; q < RQ; ++q) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = 32 * q + 8 * g + k;
          v[k] = 0.0f;
          if (mine && j < r) {
            for (int p = 0; p < S; ++p) v[k] += part[((int64_t)p * T + tu) * r + j];
            if (store_u) u[tu * r + j] = v[k];
          }
          v[k] *= s;
        }
        uint4 o[3];
        split8(v, o);
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = mfma(o[p], f[q][j], acc[j]);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (!on[v]) continue;
        float val[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) val[j] = base ? chunk_value(b[v], j) + acc[j][v] : acc[j][v];
        store_chunk(out + (t0 + 4 * g + v) * ldo, (int)c, (int)C, val);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// outer: d_l[j][c] = s_l sum over the rows t of adapter l of w_t[j] y_t[c].  Rows are
// sorted by adapter and cut into tiles of `chunk`; an adapter with one tile is
// written at once, the others' tiles leave their sums in slots that
// adapter_join_kernel adds up.

// Tile of an adapter's rows: which adapter, its rows, how many tiles it has and
// the slot of its first one (slots count the tiles of adapters with several).
struct Tile {
  int l, r0, r1, tiles, slot;
};

// The idx-th tile; false past the last.  By whole waves.
__device__ __forceinline__ bool find_tile(const int32_t *off, int L, int chunk, int64_t idx,
                                          Tile &t) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  int slots = 0;
  for (int l0 = 0; l0 < L; l0 += 64) {
    int a = 0, b = 0;
    if (l0 + lane < L) {
      a = off[l0 + lane];
      b = off[l0 + lane + 1];
    }
    const int n = (b - a + chunk - 1) / chunk, m = n > 1 ? n : 0;
    int sum = n, msum = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64), k = __shfl_up(msum, o, 64);
      if (lane >= o) {
        sum += v;
        msum += k;
      }
    }
    const int total = __shfl(sum, 63, 64);
    if (idx < before + total) {
      const uint64_t past = __ballot(before + sum > idx);
      const int at = __ffsll((unsigned long long)past) - 1;
      const int i = (int)(idx - before) - __shfl(sum - n, at, 64);
      t.l = l0 + at;
      t.r0 = __shfl(a, at, 64) + i * chunk;
      const int end = __shfl(b, at, 64);
      t.r1 = t.r0 + chunk < end ? t.r0 + chunk : end;
      t.tiles = __shfl(n, at, 64);
      t.slot = slots + __shfl(msum - m, at, 64) + i;
      return true;
    }
    before += total;
    slots += __shfl(msum, 63, 64);
  }
  return false;
}

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

template <int RT, bool F8>
__device__ __forceinline__ void outer_tile(const Side &sd, const int32_t *rows, const Tile &tile,
                                           float s, int64_t c0, int j0, int r, float *out) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int64_t c = c0 + 8 * (lane & 15), C = sd.C;
  v4f acc[RT][8];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[q][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = tile.r0; i0 < tile.r1; i0 += 32) {
    uint4 y[8], f[8], o[RT][3];
    float w[RT][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + 8 * g + k;
      const bool in = i < tile.r1;
      const int64_t t = rows[in ? i : tile.r1 - 1];
      float rest = 1.0f;
      y[k] = make_uint4(0, 0, 0, 0);
      if (F8) {
        if (in && c < C) {
          uint2 q;
          __builtin_memcpy(&q, static_cast<const uint8_t *>(sd.y) + t * f8_row_bytes(C) + c, 8);
          const int e = sd.ys[t * f8_scale_bytes(C) + c0 / kF8Block], h = held_scale(e);
          const float p = __uint_as_float((uint32_t)h << 23);
          rest = __uint_as_float((uint32_t)(127 + e - h) << 23);
          y[k].x = __builtin_bit_cast(uint32_t, widen2(q.x, p, false));
          y[k].y = __builtin_bit_cast(uint32_t, widen2(q.x, p, true));
          y[k].z = __builtin_bit_cast(uint32_t, widen2(q.y, p, false));
          y[k].w = __builtin_bit_cast(uint32_t, widen2(q.y, p, true));
        }
      } else if (in) {
        y[k] = load8(static_cast<const uint16_t *>(sd.y) + t * sd.ldy, c, C);
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int j = j0 + 16 * q + (lane & 15);
        w[q][k] = in && j < r ? sd.w[t * r + j] * rest : 0.0f;
      }
    }
    transpose8(y, f);
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      split8(w[q], o[q]);
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[q][j] = mfma(o[q][p], f[j], acc[q][j]);
    }
  }
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int j = j0 + 16 * q + 4 * g + v;
      if (j >= r) continue;
      float val[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) val[k] = acc[q][k][v] * s;
      store_chunk(out + (int64_t)j * C, (int)c, (int)C, val);
    }
}

// blockIdx.x: 512 columns of the first or (from `split` on) the second side;
// blockIdx.y: a tile; blockIdx.z: RT x 16 of the ranks.
template <int RT, bool F8>
__global__ void __launch_bounds__(256)
    adapter_outer_kernel(Side first, Side second, int split, const int32_t *__restrict__ rows,
                         const int32_t *__restrict__ off, const float *__restrict__ scale, int r,
                         int L, int chunk) {
  const bool two = (int)blockIdx.x >= split;
  const int wave = threadIdx.x >> 6;
  const Side &sd = two ? second : first;
  const int64_t c0 = ((int64_t)(two ? blockIdx.x - split : blockIdx.x) * 4 + wave) * 128;
  if (c0 >= sd.C) return;
  for (int64_t idx = blockIdx.y;; idx += gridDim.y) {
    Tile t;
    if (!find_tile(off, L, chunk, idx, t)) return;
    const bool whole = t.tiles == 1;
    const float s = scale ? scale[t.l] : 1.0f;
    float *out = whole ? sd.d + (int64_t)t.l * r * sd.C : sd.slot + (int64_t)t.slot * r * sd.C;
    const int j0 = blockIdx.z * RT * 16;
    if (two || !F8) outer_tile<RT, false>(sd, rows, t, s, c0, j0, r, out);
    else outer_tile<RT, F8>(sd, rows, t, s, c0, j0, r, out);
  }
}

// The sums of adapters with several tiles, and zeros for those without rows.
__global__ void __launch_bounds__(256)
    adapter_join_kernel(Side first, Side second, int split, const int32_t *__restrict__ off, int r,
                        int L, int chunk) {
  const bool two = (int)blockIdx.x >= split;
  const Side &sd = two ? second : first;
  const int64_t n = (int64_t)r * sd.C;
  const int64_t i0 = (int64_t)(two ? blockIdx.x - split : blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = (int64_t)(two ? gridDim.x - split : split) * 256;
  int slot = 0;
  for (int l = 0; l < L; ++l) {
    const int tiles = (off[l + 1] - off[l] + chunk - 1) / chunk;
    if (tiles != 1 && (int)blockIdx.y == l % (int)gridDim.y) {
      for (int64_t i = i0; i < n; i += step) {
        float s = 0.0f;
#pragma unroll 4
        for (int k = 0; k < tiles; ++k) s += sd.slot[(int64_t)(slot + k) * n + i];
        sd.d[(int64_t)l * n + i] = s;
      }
    }
    if (tiles > 1) slot += tiles;
  }
}

// ---------------------------------------------------------------------------

int64_t shrink_splits(int64_t T, int64_t C) {
  // at least a step of 128 columns for each wave, and no more waves than fill
  // the chip twice
  const int64_t tiles = T > 0 ? (T + 15) / 16 : 1, steps = (C + 127) / 128;
  int64_t s = 512 / tiles;
  if (s > (steps + 3) / 4) s = (steps + 3) / 4;
  return s < 1 ? 1 : s > 16 ? 16 : s;
}

// Few rows: a tile's adapters go to blocks of their own.
unsigned adapter_slots(int64_t T, int L) {
  return T <= 512 ? (unsigned)(L < 15 ? L + 1 : 16) : 1;
}

hipError_t shrink(const uint16_t *x, int64_t ldx, const int32_t *ids, const uint16_t *w,
                  float *part, int64_t T, int64_t C, int r, int L, int64_t S, hipStream_t s) {
  const dim3 grid((unsigned)((T + 15) / 16), (unsigned)S, adapter_slots(T, L));
#define BNN_SHRINK(RT) \
  adapter_shrink_kernel<RT><<<grid, 256, 0, s>>>(x, ldx, ids, w, part, T, C, r, L)
  if (r <= 16) BNN_SHRINK(1);
  else if (r <= 32) BNN_SHRINK(2);
  else if (r <= 64) BNN_SHRINK(4);
  else BNN_SHRINK(8);
#undef BNN_SHRINK
  return hipGetLastError();
}

template <typename O>
hipError_t expand(const float *part, int64_t S, const int32_t *ids, const uint16_t *w,
                  const float *scale, const void *base, int64_t ldb, void *out, int64_t ldo,
                  float *u, int64_t T, int64_t C, int r, int L, hipStream_t s) {
  const int64_t all = (T + 15) / 16, cols = (C + 511) / 512;
  int64_t tiles = all * cols / 2048;
  tiles = tiles < 1 ? 1 : tiles > 8 ? 8 : tiles;
  while ((all + tiles - 1) / tiles > 65535) tiles *= 2;
  const dim3 grid((unsigned)cols, (unsigned)((all + tiles - 1) / tiles), adapter_slots(T, L));
#define BNN_EXPAND(RQ)                                                                           \
  adapter_expand_kernel<O, RQ><<<grid, 256, 0, s>>>(part, (int)S, ids, w, scale,                 \
                                                    static_cast<const O *>(base), ldb,           \
                                                    static_cast<O *>(out), ldo, u, T, C, r, L,   \
                                                    (int)tiles)
  if (r <= 32) BNN_EXPAND(1);
  else if (r <= 64) BNN_EXPAND(2);
  else BNN_EXPAND(4);
#undef BNN_EXPAND
  return hipGetLastError();
}

hipError_t expand_as(int dtype, const float *part, int64_t S, const int32_t *ids,
                     const uint16_t *w, const float *scale, const void *base, int64_t ldb,
                     void *out, int64_t ldo, float *u, int64_t T, int64_t C, int r, int L,
                     hipStream_t s) {
  if (dtype == BNN_FP32)
    return expand<float>(part, S, ids, w, scale, base, ldb, out, ldo, u, T, C, r, L, s);
  return expand<bf16_t>(part, S, ids, w, scale, base, ldb, out, ldo, u, T, C, r, L, s);
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

// Rows of a tile of the outer sums: few enough tiles that the slots stay small.
int64_t outer_chunk(int64_t T) {
  const int64_t c = ((T + 63) / 64 + 31) / 32 * 32;
  return c < 256 ? 256 : c;
}

struct BwdLayout {
  int64_t v, part, rows, off, group, slot_a, slot_b, bytes, chunk;
};

BwdLayout bwd_layout(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  BwdLayout b;
  const int64_t S = shrink_splits(T, N);
  b.chunk = outer_chunk(T);
  const int64_t slots = T <= b.chunk ? 0 : 2 * (T / b.chunk);
  b.v = 0;
  b.part = b.v + align16(T * r * 4);
  b.rows = b.part + (S > 1 ? align16(S * T * r * 4) : 0);
  b.off = b.rows + align16(T * 4);
  b.group = b.off + align16((L + 1) * 4);
  b.slot_a = b.group + align16(group_rows_workspace(T, L));
  b.slot_b = b.slot_a + align16(slots * r * K * 4);
  b.bytes = b.slot_b + align16(slots * r * N * 4);
  return b;
}

}  // namespace

int64_t adapter_fwd_workspace(int64_t T, int64_t K, int64_t r) {
  const int64_t S = shrink_splits(T, K);
  return S > 1 ? S * T * r * 4 : 0;
}

hipError_t launch_adapter_fwd(const uint16_t *x, int64_t ldx, const int32_t *ids,
                              const uint16_t *a, const uint16_t *b, const float *scale,
                              const void *base, int64_t ldb, void *out, int64_t ldo, int dtype,
                              float *u, void *workspace, int64_t T, int64_t K, int64_t N, int r,
                              int L, hipStream_t s) {
  const int64_t S = N > 0 ? shrink_splits(T, K) : 1;
  float *part = S > 1 ? static_cast<float *>(workspace) : u;
  const hipError_t e = shrink(x, ldx, ids, a, part, T, K, r, L, S, s);
  if (e != hipSuccess) return e;
  if (N == 0) return hipSuccess;
  return expand_as(dtype, part, S, ids, b, scale, base, ldb, out, ldo, S > 1 ? u : nullptr, T, N,
                   r, L, s);
}

int64_t adapter_bwd_workspace(int64_t T, int64_t K, int64_t N, int64_t r, int64_t L) {
  return bwd_layout(T, K, N, r, L).bytes;
}

hipError_t launch_adapter_bwd(const AdapterGrad &q, void *workspace, int64_t T, int64_t K,
                              int64_t N, int r, int L, hipStream_t s) {
  const BwdLayout b = bwd_layout(T, K, N, r, L);
  char *ws = static_cast<char *>(workspace);
  float *v = reinterpret_cast<float *>(ws + b.v);
  int32_t *rows = reinterpret_cast<int32_t *>(ws + b.rows);
  int32_t *off = reinterpret_cast<int32_t *>(ws + b.off);
  hipError_t e = hipSuccess;
  if (T > 0) {
    // without dx nothing sums the parts of v: one split
    const int64_t S = q.dx ? shrink_splits(T, N) : 1;
    float *part = S > 1 ? reinterpret_cast<float *>(ws + b.part) : v;
    e = shrink(q.dy, q.lddy, q.ids, q.b, part, T, N, r, L, S, s);
    if (e != hipSuccess) return e;
    if (q.dx) {
      e = expand_as(q.dtype, part, S, q.ids, q.a, q.scale, q.base, q.ldb, q.dx, q.lddx,
                    S > 1 ? v : nullptr, T, K, r, L, s);
      if (e != hipSuccess) return e;
    }
  }
  if (!q.sums) return hipSuccess;
  e = launch_group_rows(q.ids, rows, off, ws + b.group, T, L, s);
  if (e != hipSuccess) return e;
  const Side sa = {v, q.x, q.xs, q.ldx, K, q.da, reinterpret_cast<float *>(ws + b.slot_a)};
  const Side sb = {q.u, q.dy, nullptr, q.lddy, N, q.db, reinterpret_cast<float *>(ws + b.slot_b)};
  const int split = (int)((K + 511) / 512), cols = split + (int)((N + 511) / 512);
  const int64_t most = (T < L ? T : L) + T / b.chunk;
  if (most > 0) {
    const unsigned ty = (unsigned)(most < 65535 ? most : 65535);
#define BNN_OUTER(RT)                                                                            \
  if (q.xs)                                                                                      \
    adapter_outer_kernel<RT, true><<<dim3(cols, ty, (r + RT * 16 - 1) / (RT * 16)), 256, 0, s>>>( \
        sa, sb, split, rows, off, q.scale, r, L, (int)b.chunk);                                  \
  else                                                                                           \
    adapter_outer_kernel<RT, false><<<dim3(cols, ty, (r + RT * 16 - 1) / (RT * 16)), 256, 0, s>>>( \
        sa, sb, split, rows, off, q.scale, r, L, (int)b.chunk);
    if (r <= 16) {
      BNN_OUTER(1)
    } else {
      BNN_OUTER(2)
    }
#undef BNN_OUTER
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t na = ((int64_t)r * K + 255) / 256, nb = ((int64_t)r * N + 255) / 256;
  const int ja = (int)(na < 1024 ? na : 1024), jb = (int)(nb < 1024 ? nb : 1024);
  adapter_join_kernel<<<dim3(ja + jb, L < 16 ? L : 16), 256, 0, s>>>(sa, sb, ja, off, r, L,
                                                                     (int)b.chunk);
  return hipGetLastError();
}

}  // namespace bnn
