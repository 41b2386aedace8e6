// Low-rank adapters of many groups at once, beside a projection:
//   h[s][:]      = x[row(s)][:] A_g^T                      (shrink, K -> R)
//   out[o(s)][:] = base[o(s)][:] + scale_g h[s][:] B_g^T   (expand, R -> N)
// and their gradients
//   dh[s][:] = scale_g dy[o(s)][:] B_g                     (shrink, N -> R)
//   dx[s][:] = dh[s][:] A_g                                (expand, R -> K)
//   dA_g = sum_s dh[s]^T x[row(s)]       dB_g = scale_g sum_s dy[o(s)]^T h[s]   (outer)
// over the rows s of each group g.
//
// At ranks of 8 to 256 the products are thin: every kernel is bound by its
// pass over the wide operand (x, base and out, dy, dx), so each reads it once,
// in 16-byte pieces straight into MFMA registers.  All use the 16x16x32 MFMA,
// whose contraction order is free as long as both operands share it; that
// freedom is used twice:
//   * shrink: lane slice q takes k = 32 q .. 32 q + 31 of a 128-wide step, so
//     a wave reads 256 contiguous bytes of each row;
//   * expand, outer: MFMA j's column c stands for column 8 c + j of a 128-wide
//     block, so a lane's eight results (or operands) are 8 consecutive columns,
//     one 16-byte access, 256 contiguous bytes per row and wave.
//
// The low-rank operand (h, dh) is fp32.  It enters the MFMAs as a sum of
// 16-bit parts that carries all its 24 bits: three of bf16 (8 bits each), or
// two of binary16 (11 each and the sign between) after scaling by a power of
// two to the middle of binary16's range (per row in expand; per wave, raised
// when a step outgrows it, in outer).  A single 16-bit rounding would have put
// its 2^-9 (2^-12) error into every product; the extra MFMAs are free here.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

struct Dev {
  const int* offsets;
  const int* sorted_ids;
  int P, E, R;
  const float* scale;
};

// Which row of a wide operand belongs to sorted row s: s itself (ROW_SORTED),
// its pair (1), or pair / div (div > 1).
struct RowMap {
  int sorted;
  int div;
};

// Pair id of sorted row s, -1 where the table holds none.
__device__ __forceinline__ int pair_of(const Dev& g, int s) {
  if (!g.sorted_ids) return s;
  const int p = g.sorted_ids[s];
  return p >= 0 && p < g.P ? p : -1;
}
__device__ __forceinline__ int map_row(const RowMap& m, int s, int pair) { return m.sorted ? s : pair / m.div; }
__device__ __forceinline__ float scale_of(const Dev& g, int e) { return g.scale ? g.scale[e] : 1.f; }

// Schedule table and scan scratch for up to 1024 groups.
constexpr int kTableInts = 1025 + 2 * kMaxWaves;
constexpr int cmax(int a, int b) { return a > b ? a : b; }

template <int KIND>
__device__ __forceinline__ v4f mfma16(u32x4 a, u32x4 b, v4f c) {
  if (KIND == OUT_BF16)
    return mfma_bf16_16x16x32(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c);
  return mfma_f16_16x16x32(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c);
}

// 16-bit parts of an fp32 value, largest first.
template <int KIND>
constexpr int kParts = KIND == OUT_BF16 ? 3 : 2;

// The parts of v (F16: |v| <= 2^15 where finite).  Infinities and NaN go to
// the first part alone: their remainders would be NaN.
template <int KIND>
__device__ __forceinline__ void split(float v, uint16_t p[kParts<KIND>]) {
#pragma unroll
  for (int i = 0; i < kParts<KIND>; ++i) {
    p[i] = OutT<KIND>::from(v);
    const float got = KIND == OUT_BF16 ? bf16_bits_to_f32(p[i]) : f16_bits_to_f32(p[i]);
    v = __builtin_fabsf(got) < __builtin_inff() ? v - got : 0.f;
  }
}

// 8 rows of 8 elements to 8 columns of 8, in registers: column j's word t
// holds rows 2t and 2t + 1.
__device__ __forceinline__ u32x4 column_of(const u32x4 rows[8], int j) {
  const u32 sel = j & 1 ? 0x07060302u : 0x05040100u;
  u32x4 v;
#pragma unroll
  for (int t = 0; t < 4; ++t) v[t] = __builtin_amdgcn_perm(rows[2 * t + 1][j >> 1], rows[2 * t][j >> 1], sel);
  return v;
}

// Two transposing LDS reads: lane i of each 16 gets column i of the 4 x 16
// block whose row j/4, columns 4 (j % 4) .. +3 its lane j points at.
__device__ __forceinline__ u32x4 transposed8(const uint16_t* a, const uint16_t* b) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds4;
  typedef u32 u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)a));
  const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)b));
  return u32x4{x[0], x[1], y[0], y[1]};
}

// Exponent of the power of two that brings m (finite, >= 0) to [2^8, 2^9):
// far from both ends of binary16, with 2^6 of room before 2^15.
__device__ __forceinline__ int half_exp(float m) { return 135 - max(1, __float_as_int(m) >> 23); }
__device__ __forceinline__ float ldexp2(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }

// ------------------------------------------------------------------ shrink
constexpr int kShrinkWaves = 8;
constexpr int kShrinkThreads = 64 * kShrinkWaves;

// part[split][s][r] = sum over the split's columns of X[row(s)][k] W[e][r][k]
// (W [E][R][C]; C_MAJOR: W [E][C][R], as B is stored for dh).  One workgroup: 16 RT rows of one group, 16 NR ranks, one split of the
// columns, dealt to its 8 waves in steps of 128.  Rows past the tile and ranks
// past R repeat valid ones: they only reach results that are not stored.
// C_MAJOR weights pass through the wave's own piece of LDS, 32 columns at a
// time, and come back through the transposing read (lane i of 16 gets column
// i of a 4 x 16 block), so that B needs no transposed copy in memory.
template <int KIND, int RT, int NR, bool C_MAJOR>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(Dev g, const uint16_t* __restrict__ X, RowMap xm,
                                                                int C, const uint16_t* __restrict__ W,
                                                                float* __restrict__ part, int splits, int rchunks) {
  constexpr int BM = 16 * RT, RW = 16 * NR + 4;
  __shared__ __align__(16) int sm[cmax(kTableInts, kShrinkWaves * BM * RW)];
  __shared__ __align__(16) uint16_t turn[C_MAJOR ? kShrinkWaves : 1][32 * 16 * NR];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, c = lane & 15, q = lane >> 4;
  const int rc = blockIdx.x % rchunks, sp = blockIdx.x / rchunks % splits, w = blockIdx.x / rchunks / splits;
  sched_build(sm, sm + g.E + 1, g.offsets, g.E, g.P, BM, 1);
  if (w >= sm[g.E]) return;
  const Tile t = sched_tile<1>(sm, g.offsets, g.E, g.P, BM, 1, w);

  const uint16_t* xp[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int s = t.row0 + min(rt * 16 + c, t.rows - 1), pair = pair_of(g, s);
    xp[rt] = X + (int64_t)(pair < 0 ? 0 : map_row(xm, s, pair)) * C;
  }
  const uint16_t* wp[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    if (C_MAJOR) {  // piece p of 32 columns: row p / 2NR, 8 ranks
      const int p = lane + 64 * n, row = p / (2 * NR), o = min(rc * 8 + p % (2 * NR), g.R / 8 - 1);
      wp[n] = W + ((int64_t)t.e * C + (row / 8) * 32 + row % 8) * g.R + o * 8;
    } else {
      wp[n] = W + ((int64_t)t.e * g.R + min(rc * 64 + n * 16 + c, g.R - 1)) * C;
    }
  }

  v4f acc[RT][NR];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[rt][n] = v4f{0.f, 0.f, 0.f, 0.f};

  const int steps = (C + 127) / 128, slot = sp * kShrinkWaves + wid, slots = splits * kShrinkWaves;
  const int st0 = (int)((int64_t)steps * slot / slots), st1 = (int)((int64_t)steps * (slot + 1) / slots);
  u32x4 xb[RT][4], wb[NR][4];
  auto load = [&](int st, u32x4 (&xv)[RT][4], u32x4 (&wv)[NR][4]) {
    const int k = st * 128 + q * 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = st * 128 + 128 <= C || k + i * 8 < C;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) xv[rt][i] = in ? ld16(xp[rt] + k + i * 8) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (C_MAJOR) {
          const int row = (lane + 64 * n) / (2 * NR), col = st * 128 + (row / 8) * 32 + i * 8 + row % 8;
          wv[n][i] = col < C ? ld16(wp[n] + (int64_t)(st * 128 + i * 8) * g.R) : u32x4{0, 0, 0, 0};
        } else {
          wv[n][i] = in ? ld16(wp[n] + k + i * 8) : u32x4{0, 0, 0, 0};
        }
      }
    }
  };
  if (st0 < st1) load(st0, xb, wb);
#pragma unroll 2
  for (int st = st0; st < st1; ++st) {
    u32x4 xn[RT][4], wn[NR][4];
    if (st + 1 < st1) load(st + 1, xn, wn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 wf[NR];
      if (C_MAJOR) {
        uint16_t* tw = turn[wid];
#pragma unroll
        for (int n = 0; n < NR; ++n) *reinterpret_cast<u32x4*>(tw + (lane + 64 * n) * 8) = wb[n][i];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint16_t* p = tw + (q * 8 + c / 4) * (16 * NR) + n * 16 + (c & 3) * 4;
          wf[n] = transposed8(p, p + 4 * 16 * NR);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NR; ++n) wf[n] = wb[n][i];
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[rt][n] = mfma16<KIND>(wf[n], xb[rt][i], acc[rt][n]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) xb[rt][i] = xn[rt][i];
#pragma unroll
      for (int n = 0; n < NR; ++n) wb[n][i] = wn[n][i];
    }
  }

  // The waves' sums meet in LDS (over the schedule, which is done with).
  __syncthreads();
  float* red = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < NR; ++n)
      *reinterpret_cast<v4f*>(red + (wid * BM + rt * 16 + c) * RW + n * 16 + 4 * q) = acc[rt][n];
  __syncthreads();
  for (int i = tid; i < BM * NR * 4; i += kShrinkThreads) {
    const int row = i / (NR * 4), r = (i - row * (NR * 4)) * 4;
    if (row >= t.rows || rc * 64 + r >= g.R || pair_of(g, t.row0 + row) < 0) continue;
    v4f sum = *reinterpret_cast<v4f*>(red + row * RW + r);
#pragma unroll
    for (int v = 1; v < kShrinkWaves; ++v) {
      const v4f o = *reinterpret_cast<v4f*>(red + (v * BM + row) * RW + r);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += o[j];
    }
    *reinterpret_cast<v4f*>(part + ((int64_t)sp * g.P + t.row0 + row) * g.R + rc * 64 + r) = sum;
  }
}

// ------------------------------------------------------------------ expand
constexpr int kExpandThreads = 256;
constexpr int kExpandWaves = kExpandThreads / 64;

struct ExpandArgs {
  const float* part;     // [splits][P][R], summed here
  int splits;
  float* h;              // [P][R] or null: receives the sums
  const uint16_t* W;     // [E][C][R], or TR: [E][R][C]
  int C;
  const uint16_t* base;  // or null
  uint16_t* out;
  int out_pair;          // row of out: the pair (else s)
  int iters;             // 512-column blocks a workgroup walks
  int cblocks;           // workgroups across the columns
  int main_blocks;       // workgroups of the rows with a group; the others copy
  const int* p2s;        // the rows without one
};

__host__ __device__ constexpr int padded_rank(int R) { return (R + 31) / 32 * 32 + 8; }

// out[o(s)][n] = base + sum_r (scale h[s][r]) W[e][n][r] for 16 RT rows of one
// group.  The rows' low-rank operand is split once into LDS; each wave then
// walks blocks of 128 columns.  Ranks are taken 32 at a time (zero past R).
template <int KIND, int RT, bool TR>
__global__ __launch_bounds__(kExpandThreads, 2) void expand_kernel(Dev g, ExpandArgs a) {
  constexpr int BM = 16 * RT, NP = kParts<KIND>;
  extern __shared__ int sm[];
  __shared__ int orow[BM];
  __shared__ u32 rmax[BM];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, c = lane & 15, q = lane >> 4;
  if ((int)blockIdx.x >= a.main_blocks) {
    const int nw = (gridDim.x - a.main_blocks) * kExpandWaves;
    for (int p = (blockIdx.x - a.main_blocks) * kExpandWaves + wid; p < g.P; p += nw) {
      const int s = a.p2s[p];
      if (s >= 0 && s < g.P) continue;
      for (int n = lane * 8; n < a.C; n += 512)
        st16(a.out + (int64_t)p * a.C + n, a.base ? ld16(a.base + (int64_t)p * a.C + n) : u32x4{0, 0, 0, 0});
    }
    return;
  }
  const int w = blockIdx.x / a.cblocks, cb = blockIdx.x - w * a.cblocks;
  sched_build(sm, sm + g.E + 1, g.offsets, g.E, g.P, BM, 1);
  if (w >= sm[g.E]) return;
  const Tile t = sched_tile<1>(sm, g.offsets, g.E, g.P, BM, 1, w);
  __syncthreads();

  // The split operand: parts[p][row][r], rows of RP.
  const int octs = g.R / 8, RP = padded_rank(g.R), ochunks = (octs + 3) / 4;
  uint16_t* parts = reinterpret_cast<uint16_t*>(sm);
  const float sc = scale_of(g, t.e);
  if (tid < BM) {
    const int pair = tid < t.rows ? pair_of(g, t.row0 + tid) : -1;
    orow[tid] = pair < 0 ? -1 : (a.out_pair ? pair : t.row0 + tid);
    rmax[tid] = 0;
  }
  __syncthreads();
  auto value = [&](int row, int o, float v[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (o >= octs || orow[row] < 0) return;
    for (int sp = 0; sp < a.splits; ++sp) {
      float u[8];
      load8<OUT_F32, false>(a.part, ((int64_t)sp * g.P + t.row0 + row) * g.R + o * 8, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    if (a.h && cb == 0 && KIND == OUT_BF16) store8<OUT_F32, false>(a.h, (int64_t)(t.row0 + row) * g.R + o * 8, v);
  };
  if (KIND == OUT_F16) {
    // each row's largest finite magnitude, for its scale
    for (int i = tid; i < BM * octs; i += kExpandThreads) {
      const int row = i / octs, o = i - row * octs;
      float v[8], m = 0.f;
      value(row, o, v);
      if (a.h && cb == 0 && orow[row] >= 0) store8<OUT_F32, false>(a.h, (int64_t)(t.row0 + row) * g.R + o * 8, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = __builtin_fabsf(sc * v[j]);
        m = u < __builtin_inff() ? fmaxf(m, u) : m;
      }
      atomicMax(&rmax[row], __float_as_uint(m));
    }
    __syncthreads();
  }
  for (int i = tid; i < BM * ochunks * 4; i += kExpandThreads) {
    const int row = i / (ochunks * 4), o = i - row * (ochunks * 4);
    float v[8];
    value(row, o, v);
    const int f = KIND == OUT_F16 ? half_exp(__uint_as_float(rmax[row])) : 0;
    u32x4 pk[NP];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint16_t lo[NP], hi[NP];
      split<KIND>(KIND == OUT_F16 ? ldexp2(sc * v[j], f) : sc * v[j], lo);
      split<KIND>(KIND == OUT_F16 ? ldexp2(sc * v[j + 1], f) : sc * v[j + 1], hi);
#pragma unroll
      for (int p = 0; p < NP; ++p) pk[p][j / 2] = (u32)lo[p] | ((u32)hi[p] << 16);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<u32x4*>(parts + (p * BM + row) * RP + o * 8) = pk[p];
  }
  __syncthreads();

  for (int it = 0; it < a.iters; ++it) {
    const int n0 = ((cb * a.iters + it) * kExpandWaves + wid) * 128;
    if (n0 >= a.C) break;
    const int col = n0 + c * 8;
    const bool in = col < a.C;
    u32x4 bv[RT][4];
    if (a.base) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = orow[rt * 16 + 4 * q + i];
          bv[rt][i] = in && o >= 0 ? ld16(a.base + (int64_t)o * a.C + col) : u32x4{0, 0, 0, 0};
        }
    }
    v4f acc[RT][8];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[rt][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int oc = 0; oc < ochunks; ++oc) {
      const int o = min(oc * 4 + q, octs - 1);  // past R: times the operand's zeros
      u32x4 raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (TR) raw[i] = ld16(a.W + ((int64_t)t.e * g.R + o * 8 + i) * a.C + (in ? col : a.C - 8));
        else raw[i] = ld16(a.W + ((int64_t)t.e * a.C + min(col + i, a.C - 1)) * g.R + o * 8);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        u32x4 l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          l[rt] = *reinterpret_cast<u32x4*>(parts + (p * BM + rt * 16 + c) * RP + (oc * 4 + q) * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32x4 b = TR ? column_of(raw, j) : raw[j];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt][j] = mfma16<KIND>(l[rt], b, acc[rt][j]);
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = rt * 16 + 4 * q + i, o = orow[row];
        if (!in || o < 0) continue;
        const int f = KIND == OUT_F16 ? -half_exp(__uint_as_float(rmax[row])) : 0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = KIND == OUT_F16 ? ldexp2(acc[rt][j][i], f) : acc[rt][j][i];
          if (a.base) {
            const u32 b = bv[rt][i][j >> 1] >> (16 * (j & 1)) & 0xffffu;
            v[j] += KIND == OUT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32((uint16_t)b);
          }
        }
        store8<KIND, false>(a.out, (int64_t)o * a.C + col, v);
      }
  }
}

// ------------------------------------------------------------------- outer
constexpr int kOuterWaves = 4;
constexpr int kOuterThreads = 64 * kOuterWaves;

// What outer's waves read of a tile of 32 rows of one group, made once by
// split_kernel: the low-rank operands of both weight gradients as MFMA
// fragments, fr[side][tile][part][16 ranks][lane][8 rows], the exponents of
// their scales (F16), and the rows of the wide operands (-1: none).
struct Tiles {
  uint16_t* fr;
  int* exps;       // [side][tile]
  int* rows;       // [side][tile][32]
  int64_t tiles;   // allocated
  int rank_tiles;
};

struct Side {
  const float* L;      // [splits][P][R], summed here; times the group's scale
  int splits;
  const uint16_t* X;   // the wide operand
  RowMap xm;
  int C;
  uint16_t* out;       // [E][R][C], or col_major: [E][C][R]
  int col_major;
  float* part;         // [slots][R][C] of the cut groups
  int slabs;           // 128 columns each
};

// Exponent of a 32-row tile's scale, a multiple of 16 so that neighbours
// rarely differ: brings m to [2^-2, 2^14).
__device__ __forceinline__ int tile_exp(float m) {
  return ((13 + 127 - max(1, __float_as_int(m) >> 23) + 128) & ~15) - 128;
}

template <int KIND>
__global__ __launch_bounds__(256) void split_kernel(Dev g, Side sa, Side sb, Tiles tl) {
  constexpr int NP = kParts<KIND>;
  __shared__ int sm[kTableInts];
  __shared__ u32 tmax[2];
  const int tid = threadIdx.x;
  sched_build(sm, sm + g.E + 1, g.offsets, g.E, g.P, 32, 1);
  const int w = blockIdx.x;
  if (w >= sm[g.E]) return;
  const Tile t = sched_tile<1>(sm, g.offsets, g.E, g.P, 32, 1, w);
  const float sc = scale_of(g, t.e);
  if (tid < 64) {
    const int side = tid >> 5, i = tid & 31;
    const int pair = i < t.rows ? pair_of(g, t.row0 + i) : -1;
    tl.rows[(side * tl.tiles + w) * 32 + i] = pair < 0 ? -1 : map_row(side ? sb.xm : sa.xm, t.row0 + i, pair);
  }
  if (tid < 2) tmax[tid] = 0;
  __syncthreads();
  // task: 8 rows (slice q) of one rank of one side
  const int per = 64 * tl.rank_tiles;
  const auto low = [&](int i, float (&v)[8]) {
    const int side = i >= per, k = i - side * per, rank = (k >> 6) * 16 + (k & 15), q = k >> 4 & 3;
    const Side& d = side ? sb : sa;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.f;
      const int s = t.row0 + q * 8 + j;
      if (rank < g.R && q * 8 + j < t.rows && pair_of(g, s) >= 0)
        for (int sp = 0; sp < d.splits; ++sp) v[j] += d.L[((int64_t)sp * g.P + s) * g.R + rank];
      v[j] *= sc;
    }
  };
  if (KIND == OUT_F16) {
    for (int i = tid; i < 2 * per; i += 256) {
      float v[8], big = 0.f;
      low(i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = __builtin_fabsf(v[j]);
        big = u < __builtin_inff() ? fmaxf(big, u) : big;
      }
      atomicMax(&tmax[i >= per], __float_as_uint(big));
    }
    __syncthreads();
    if (tid < 2) tl.exps[tid * tl.tiles + w] = tile_exp(__uint_as_float(tmax[tid]));
  }
  for (int i = tid; i < 2 * per; i += 256) {
    const int side = i >= per, k = i - side * per;
    float v[8];
    low(i, v);
    const int f = KIND == OUT_F16 ? tile_exp(__uint_as_float(tmax[side])) : 0;
    u32x4 pk[NP];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint16_t u0[NP], u1[NP];
      split<KIND>(KIND == OUT_F16 ? ldexp2(v[j], f) : v[j], u0);
      split<KIND>(KIND == OUT_F16 ? ldexp2(v[j + 1], f) : v[j + 1], u1);
#pragma unroll
      for (int p = 0; p < NP; ++p) pk[p][j / 2] = (u32)u0[p] | ((u32)u1[p] << 16);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) st16(tl.fr + (((side * tl.tiles + w) * NP + p) * per + k) * 8, pk[p]);
  }
}

// Slot of the partial sums of the chunk that starts at sorted row s: at most
// one first and one later chunk of the groups longer than a chunk start in
// the same `chunk` rows.
__host__ __device__ constexpr int outer_slot(int s, bool first, int chunk) { return 2 * (s / chunk) + (first ? 1 : 0); }
__host__ __device__ constexpr int64_t outer_slots(int64_t P, int chunk) { return P > chunk ? 2 * ((P - 1) / chunk + 1) : 0; }

// Chunks of a group of m rows; a group without rows has one that writes zeros.
__device__ __forceinline__ int chunks_of(int m, int chunk) { return max(1, (m + chunk - 1) / chunk); }

// dW[r][n] = sum_s (scale L[s][r]) X[row(s)][n]: each wave by itself takes one
// chunk of a group's rows, 128 columns and 16 NR ranks, and walks the chunk's
// tiles of 32 rows (the MFMA's contraction) with the next tile's 8 KB in
// flight.  Waves of the same columns and other ranks sit side by side, where
// the second finds the wide operand in the L1.
template <int KIND, int NR>
__global__ __launch_bounds__(kOuterThreads, 2) void outer_kernel(Dev g, Side sa, Side sb, Tiles tl, int rchunks,
                                                                 int chunk) {
  constexpr int NP = kParts<KIND>;
  __shared__ int tab[1025], tiles[1025], scratch[2 * kOuterWaves];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, c = lane & 15, q = lane >> 4;

  // Tables of the groups' chunks and 32-row tiles: one scan of both counts.
  {
    const int per = (g.E + kOuterThreads - 1) / kOuterThreads;
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int nc = 0, nt = 0, lo, hi;
    for (int e = e0; e < e1; ++e) {
      expert_range(g.offsets, e, g.P, lo, hi);
      nc += chunks_of(hi - lo, chunk);
      nt += (hi - lo + 31) / 32;
    }
    int ic = nc, it = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int vc = __shfl_up(ic, o, 64), vt = __shfl_up(it, o, 64);
      if (lane >= o) {
        ic += vc;
        it += vt;
      }
    }
    if (lane == 63) {
      scratch[wid] = ic;
      scratch[kOuterWaves + wid] = it;
    }
    __syncthreads();
    int rc = ic - nc, rt = it - nt;
    for (int v = 0; v < wid; ++v) {
      rc += scratch[v];
      rt += scratch[kOuterWaves + v];
    }
    for (int e = e0; e < e1; ++e) {
      tab[e] = rc;
      tiles[e] = rt;
      expert_range(g.offsets, e, g.P, lo, hi);
      rc += chunks_of(hi - lo, chunk);
      rt += (hi - lo + 31) / 32;
    }
    if (tid == kOuterThreads - 1) tab[g.E] = rc;
    __syncthreads();
  }
  const int slabs = sa.slabs + sb.slabs;
  const int task = blockIdx.x * kOuterWaves + wid;
  const int rc = task % rchunks, w = task / rchunks / slabs;
  int slab = task / rchunks % slabs;
  if (w >= tab[g.E]) return;
  const int side = slab >= sa.slabs;
  const Side& d = side ? sb : sa;
  if (side) slab -= sa.slabs;
  int bl = 0, bh = g.E - 1;
  while (bl < bh) {
    const int mid = (bl + bh + 1) >> 1;
    if (tab[mid] <= w) bl = mid; else bh = mid - 1;
  }
  const int e = bl, ch = w - tab[e];
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  const int s0 = lo + ch * chunk, first = tiles[e] + ch * (chunk / 32);
  // (a malformed offsets table may count more tiles than there can be)
  const int nt = min((min(chunk, hi - s0) + 31) / 32, (int)max<int64_t>(0, tl.tiles - first));
  const int64_t t0 = side * tl.tiles + first;

  const int col = min(slab * 128 + c * 8, d.C - 8);
  const uint16_t* X = d.X + col;
  const int* rowp = tl.rows + t0 * 32 + q * 8;
  // ranks past R: results that are not stored
  const uint16_t* fp[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n)
    fp[n] = tl.fr + t0 * NP * tl.rank_tiles * 512 + min(rc * NR + n, tl.rank_tiles - 1) * 512 + lane * 8;

  v4f acc[NR][8];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[n][j] = v4f{0.f, 0.f, 0.f, 0.f};
  u32x4 raw[8], fr[NR][NP];
  int row[8];
  const auto load_rows = [&](int k) {
    const v4i r0 = *reinterpret_cast<const v4i*>(rowp + k * 32), r1 = *reinterpret_cast<const v4i*>(rowp + k * 32 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row[i] = r0[i];
      row[4 + i] = r1[i];
    }
  };
  const auto load_x = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = row[i] >= 0 ? ld16(X + (int64_t)row[i] * d.C) : u32x4{0, 0, 0, 0};
  };
  const auto load_fr = [&](int k) {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int p = 0; p < NP; ++p) fr[n][p] = ld16(fp[n] + ((int64_t)k * NP + p) * tl.rank_tiles * 512);
  };
  int f = 0;
  if (nt > 0) {
    load_rows(0);
    load_x();
    load_fr(0);
    if (nt > 1) load_rows(1);
    f = KIND == OUT_F16 ? tl.exps[t0] : 0;
  }
  for (int k = 0; k < nt; ++k) {
    if (KIND == OUT_F16) {
      // The sums keep the smallest scale so far; a tile with a larger one is
      // brought down to it (what that drops is below 2^-22 of the largest).
      const int ft = tl.exps[t0 + k];
      if (ft < f) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][j][i] = ldexp2(acc[n][j][i], ft - f);
        f = ft;
      } else if (ft > f) {
        const _Float16 down = (_Float16)ldexp2(1.f, f - ft);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int p = 0; p < NP; ++p) fr[n][p] = __builtin_bit_cast(u32x4, __builtin_bit_cast(v8h, fr[n][p]) * down);
      }
    }
#pragma unroll
    for (int jh = 0; jh < 8; jh += 4) {  // half of the columns at a time: fewer live registers
      u32x4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = column_of(raw, jh + j);
      if (jh == 4 && k + 1 < nt) {
        load_x();
        if (k + 2 < nt) load_rows(k + 2);
      }
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][jh + j] = mfma16<KIND>(fr[n][p], x[j], acc[n][jh + j]);
    }
    if (k + 1 < nt) load_fr(k + 1);
  }

  // Lane: ranks 4q .. 4q+3 of each tile, columns col .. col+7.
  if (slab * 128 + c * 8 >= d.C) return;
  const bool cut = hi - lo > chunk;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r0 = (rc * NR + n) * 16 + 4 * q;
    if (r0 >= g.R) continue;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = KIND == OUT_F16 ? ldexp2(acc[n][j][i], -f) : acc[n][j][i];
    if (cut) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store8<OUT_F32, false>(d.part, ((int64_t)outer_slot(s0, ch == 0, chunk) * g.R + r0 + i) * d.C + col, v[i]);
    } else if (d.col_major) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u32 o0 = (u32)OutT<KIND>::from(v[0][j]) | ((u32)OutT<KIND>::from(v[1][j]) << 16);
        const u32 o1 = (u32)OutT<KIND>::from(v[2][j]) | ((u32)OutT<KIND>::from(v[3][j]) << 16);
        *reinterpret_cast<uint2*>(d.out + ((int64_t)e * d.C + col + j) * g.R + r0) = make_uint2(o0, o1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) store8<KIND, false>(d.out, ((int64_t)e * g.R + r0 + i) * d.C + col, v[i]);
    }
  }
}

// Joins the chunks of the groups longer than one: a thread takes 4 ranks of
// one column, so that both output orders store 4 values at once or in runs.
template <int KIND>
__global__ __launch_bounds__(256) void join_kernel(Dev g, Side sa, Side sb, int blocks_a, int blocks_b,
                                                  int chunk) {
  const int per = blocks_a + blocks_b, e = blockIdx.x / per;
  int b = blockIdx.x - e * per;
  const Side& d = b < blocks_a ? sa : sb;
  if (b >= blocks_a) b -= blocks_a;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  if (hi - lo <= chunk) return;
  const int64_t i = (int64_t)b * 256 + threadIdx.x;
  const int r = (int)(i / d.C) * 4, n = (int)(i % d.C);
  if (r >= g.R) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = lo; s < hi; s += chunk) {
    const float* p = d.part + ((int64_t)outer_slot(s, s == lo, chunk) * g.R + r) * d.C + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += p[(int64_t)j * d.C];
  }
  if (d.col_major) {
    const u32 o0 = (u32)OutT<KIND>::from(sum[0]) | ((u32)OutT<KIND>::from(sum[1]) << 16);
    const u32 o1 = (u32)OutT<KIND>::from(sum[2]) | ((u32)OutT<KIND>::from(sum[3]) << 16);
    *reinterpret_cast<uint2*>(d.out + ((int64_t)e * d.C + n) * g.R + r) = make_uint2(o0, o1);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) d.out[((int64_t)e * g.R + r + j) * d.C + n] = OutT<KIND>::from(sum[j]);
  }
}

// ---------------------------------------------------------------- launches
Dev dev_args(const LoraArgs& g) { return Dev{g.offsets, g.sorted_ids, (int)g.P, g.E, g.R, g.scale}; }
RowMap x_map(const LoraArgs& g) { return RowMap{g.x_div == 0, std::max(1, g.x_div)}; }
RowMap o_map(const LoraArgs& g) { return RowMap{!g.out_pair, 1}; }

// Upper bound of the row tiles of bm rows: every group may end in a part tile.
int64_t max_tiles(int64_t P, int E, int bm) { return P / bm + std::min<int64_t>(P, E); }

// Row tiles (of 16) a workgroup takes: as many as the average group fills.
int shrink_rt(int64_t P, int E, int nr) {
  if (P >= 64 * (int64_t)E && nr == 1) return 4;
  return P >= 24 * (int64_t)E ? 2 : 1;
}
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }  // per workgroup; 64 ranks at most

// Row tiles (of 16) of an expand workgroup; the split operand has to fit LDS.
int expand_rt(int64_t P, int E, int R) {
  if (P >= 64 * (int64_t)E && R <= 128) return 4;
  return P >= 24 * (int64_t)E ? 2 : 1;
}

// 512-column blocks an expand workgroup walks: up to 8 while 2048 workgroups
// remain, more where one grid could not hold the workgroups.
int expand_iters(int64_t tiles, int blocks) {
  int iters = (int)std::max<int64_t>(1, std::min<int64_t>(8, tiles * blocks / 2048));
  while (iters < blocks && tiles * ((blocks + iters - 1) / iters) > kMaxBlocks) iters *= 2;
  return iters;
}

// Column splits of a shrink: enough workgroups for two on each of 256 compute
// units, at least one 128-column step per wave.
int shrink_splits(int64_t P, int E, int C, int R) {
  const int nr = rank_tiles(R), steps = (C + 127) / 128;
  const int64_t wgs = max_tiles(P, E, 16 * shrink_rt(P, E, nr)) * ((R + 63) / 64);
  const int64_t want = (512 + wgs - 1) / std::max<int64_t>(1, wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, (steps + kShrinkWaves - 1) / kShrinkWaves, 8}));
}

template <int KIND, int RT, int NR, bool CM>
hipError_t shrink_launch(const Dev& d, const uint16_t* X, RowMap xm, int C, const uint16_t* W, float* part, int splits,
                         hipStream_t stream) {
  const int rchunks = (d.R + 63) / 64;
  const int64_t grid = max_tiles(d.P, d.E, 16 * RT) * splits * rchunks;
  hipLaunchKernelGGL((shrink_kernel<KIND, RT, NR, CM>), dim3((unsigned)grid), dim3(kShrinkThreads), 0, stream, d, X, xm, C,
                     W, part, splits, rchunks);
  return hipGetLastError();
}

template <int KIND, bool CM>
hipError_t shrink(const Dev& d, const uint16_t* X, RowMap xm, int C, const uint16_t* W, float* part, int splits,
                  hipStream_t stream) {
  const int nr = rank_tiles(d.R), rt = shrink_rt(d.P, d.E, nr);
  if (nr == 1 && rt == 4) return shrink_launch<KIND, 4, 1, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 1 && rt == 2) return shrink_launch<KIND, 2, 1, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 1) return shrink_launch<KIND, 1, 1, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2 && rt == 2) return shrink_launch<KIND, 2, 2, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2) return shrink_launch<KIND, 1, 2, CM>(d, X, xm, C, W, part, splits, stream);
  if (rt == 2) return shrink_launch<KIND, 2, 4, CM>(d, X, xm, C, W, part, splits, stream);
  return shrink_launch<KIND, 1, 4, CM>(d, X, xm, C, W, part, splits, stream);
}

template <int KIND, int RT, bool TR>
hipError_t expand_launch(const Dev& d, ExpandArgs a, bool copy, hipStream_t stream) {
  const int64_t tiles = max_tiles(d.P, d.E, 16 * RT);
  const int blocks = (a.C + 511) / 512;
  a.iters = expand_iters(tiles, blocks);
  a.cblocks = (blocks + a.iters - 1) / a.iters;
  a.main_blocks = (int)(tiles * a.cblocks);
  const int copies = copy ? std::min((d.P + kExpandWaves - 1) / kExpandWaves, 1024) : 0;
  const size_t lds = std::max(sizeof(int) * (d.E + 1 + 2 * kMaxWaves),
                              sizeof(uint16_t) * kParts<KIND> * 16 * RT * padded_rank(d.R));
  hipLaunchKernelGGL((expand_kernel<KIND, RT, TR>), dim3(a.main_blocks + copies), dim3(kExpandThreads), lds, stream, d,
                     a);
  return hipGetLastError();
}

template <int KIND, bool TR>
hipError_t expand(const Dev& d, const ExpandArgs& a, bool copy, hipStream_t stream) {
  switch (expand_rt(d.P, d.E, d.R)) {
    case 4: return expand_launch<KIND, 4, TR>(d, a, copy, stream);
    case 2: return expand_launch<KIND, 2, TR>(d, a, copy, stream);
    default: return expand_launch<KIND, 1, TR>(d, a, copy, stream);
  }
}

int outer_nr(int R) { return R <= 16 ? 1 : 2; }
int64_t outer_tasks(int E, int N, int K, int R) {  // waves per chunk of rows
  const int nr = outer_nr(R);
  return (int64_t)((N + 127) / 128 + (K + 127) / 128) * ((R + 16 * nr - 1) / (16 * nr));
}

// Rows a wave sums before a longer group is cut: short enough for eight waves
// on each of 256 compute units, where the rows allow it.
int outer_chunk(int64_t P, int E, int N, int K, int R) {
  for (int chunk = 1024; chunk > 128; chunk /= 2)
    if (std::max<int64_t>(P / chunk, std::min<int64_t>(P, E)) * outer_tasks(E, N, K, R) >= 2048) return chunk;
  return 128;
}

template <int KIND>
hipError_t outer(const Dev& d, const Side& sa, const Side& sb, const Tiles& tl, int N, int K, hipStream_t stream) {
  const int chunk = outer_chunk(d.P, d.E, N, K, d.R), nr = outer_nr(d.R);
  const int64_t tasks = (d.P / chunk + d.E) * outer_tasks(d.E, N, K, d.R);
  const dim3 grid((unsigned)((tasks + kOuterWaves - 1) / kOuterWaves));
  const int rchunks = (d.R + 16 * nr - 1) / (16 * nr);
  if (nr == 1)
    hipLaunchKernelGGL((outer_kernel<KIND, 1>), grid, dim3(kOuterThreads), 0, stream, d, sa, sb, tl, rchunks, chunk);
  else
    hipLaunchKernelGGL((outer_kernel<KIND, 2>), grid, dim3(kOuterThreads), 0, stream, d, sa, sb, tl, rchunks, chunk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || d.P <= chunk) return e;
  const int ba = (int)(((int64_t)K * (d.R / 4) + 255) / 256), bb = (int)(((int64_t)N * (d.R / 4) + 255) / 256);
  hipLaunchKernelGGL(join_kernel<KIND>, dim3((unsigned)(d.E * (ba + bb))), dim3(256), 0, stream, d, sa, sb, ba, bb,
                     chunk);
  return hipGetLastError();
}

template <int KIND>
hipError_t forward(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b, const uint16_t* base,
                   uint16_t* out, float* h, float* ws, hipStream_t stream) {
  const Dev d = dev_args(g);
  const int splits = shrink_splits(g.P, g.E, g.K, g.R);
  float* part = splits == 1 && h ? h : ws;
  hipError_t e = shrink<KIND, false>(d, x, x_map(g), g.K, a, part, splits, stream);
  if (e != hipSuccess) return e;
  ExpandArgs ea = {part, splits, part == h ? nullptr : h, b, g.N, base, out, g.out_pair, 0, 0, 0, g.p2s};
  return expand<KIND, false>(d, ea, g.out_pair && base != out, stream);
}

// Workspace of the gradients: dh's partial sums, the tiles of both low-rank
// operands (exponents, rows, fragments), and the cut groups' partial weight
// gradients, each at a multiple of 256 bytes.
struct BwdLayout {
  int64_t tiles;
  size_t exps, rows, fr, pa, pb, bytes;
};
BwdLayout bwd_layout(int64_t P, int E, int N, int K, int R) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  BwdLayout l = {};
  if (P == 0) return l;
  l.tiles = max_tiles(P, E, 32);
  l.exps = up((size_t)P * R * sizeof(float) * shrink_splits(P, E, N, R));
  l.rows = l.exps + up((size_t)l.tiles * 2 * sizeof(int));
  l.fr = l.rows + up((size_t)l.tiles * 2 * 32 * sizeof(int));
  l.pa = l.fr + up((size_t)l.tiles * 2 * kParts<OUT_BF16> * ((R + 15) / 16) * 1024);
  const size_t slots = outer_slots(P, outer_chunk(P, E, N, K, R));
  l.pb = l.pa + up(slots * R * K * sizeof(float));
  l.bytes = l.pb + up(slots * R * N * sizeof(float));
  return l;
}

template <int KIND>
hipError_t backward(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                    const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, char* ws, hipStream_t stream) {
  const Dev d = dev_args(g);
  const BwdLayout l = bwd_layout(g.P, g.E, g.N, g.K, g.R);
  float* dh = reinterpret_cast<float*>(ws);
  const int splits = shrink_splits(g.P, g.E, g.N, g.R);
  const Side sa = {dh, splits, x, x_map(g), g.K, da, 0, reinterpret_cast<float*>(ws + l.pa), (g.K + 127) / 128};
  const Side sb = {h, 1, dy, o_map(g), g.N, db, 1, reinterpret_cast<float*>(ws + l.pb), (g.N + 127) / 128};
  const Tiles tl = {reinterpret_cast<uint16_t*>(ws + l.fr), reinterpret_cast<int*>(ws + l.exps),
                    reinterpret_cast<int*>(ws + l.rows), l.tiles, (g.R + 15) / 16};
  if (g.P > 0) {
    hipError_t e = shrink<KIND, true>(d, dy, o_map(g), g.N, b, dh, splits, stream);
    if (e != hipSuccess) return e;
    if (dx) {
      ExpandArgs ea = {dh, splits, nullptr, a, g.K, nullptr, dx, 0, 0, 0, 0, nullptr};
      if ((e = expand<KIND, true>(d, ea, false, stream)) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(split_kernel<KIND>, dim3((unsigned)l.tiles), dim3(256), 0, stream, d, sa, sb, tl);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return outer<KIND>(d, sa, sb, tl, g.N, g.K, stream);
}

}  // namespace

bool lora_fits(int64_t P, int E, int N, int K, int R) {
  constexpr int64_t kThreadsMax = int64_t(1) << 31;  // per launch, half the packet's limit
  const int64_t rchunks = (R + 63) / 64;
  for (const int C : {N, K}) {
    if (max_tiles(P, E, 16 * shrink_rt(P, E, rank_tiles(R))) * shrink_splits(P, E, C, R) * rchunks *
            kShrinkThreads > kThreadsMax)
      return false;
    const int64_t tiles = max_tiles(P, E, 16 * expand_rt(P, E, R));
    const int blocks = (C + 511) / 512, iters = expand_iters(tiles, blocks);
    if (tiles * ((blocks + iters - 1) / iters) > kMaxBlocks) return false;
  }
  return max_tiles(P, E, 32) * 256 <= kThreadsMax &&
         (P / outer_chunk(P, E, N, K, R) + E) * outer_tasks(E, N, K, R) * 64 <= kThreadsMax &&
         E * (((int64_t)N + K) * (R / 4) / 256 + 2) * 256 <= kThreadsMax;
}

size_t lora_workspace_bytes(int64_t P, int E, int N, int K, int R) {
  return P ? (size_t)P * R * sizeof(float) * shrink_splits(P, E, K, R) : 0;
}
size_t lora_bwd_workspace_bytes(int64_t P, int E, int N, int K, int R) { return bwd_layout(P, E, N, K, R).bytes; }

hipError_t launch_lora(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                       const uint16_t* base, uint16_t* out, float* h, void* ws, hipStream_t stream) {
  if (g.P == 0) return hipSuccess;
  float* w = static_cast<float*>(ws);
  return g.f16 ? forward<OUT_F16>(g, x, a, b, base, out, h, w, stream)
               : forward<OUT_BF16>(g, x, a, b, base, out, h, w, stream);
}

hipError_t launch_lora_bwd(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a,
                           const uint16_t* b, const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                           hipStream_t stream) {
  char* w = static_cast<char*>(ws);
  return g.f16 ? backward<OUT_F16>(g, dy, x, a, b, h, dx, da, db, w, stream)
               : backward<OUT_BF16>(g, dy, x, a, b, h, dx, da, db, w, stream);
}

}  // namespace moeq
