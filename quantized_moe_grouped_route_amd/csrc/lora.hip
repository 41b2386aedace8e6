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
// freedom is used in expand and outer: MFMA j's column c stands for column
// 8 c + j of a 128-wide block, so a lane's eight results (or operands) are 8
// consecutive columns, one 16-byte access, 256 contiguous bytes per row and
// wave.  shrink keeps the plain order, 64 contiguous bytes of each of 16 rows
// in an access: with a lane's 64 bytes in a row (and so 16-byte pieces 64
// bytes apart in an access) the L1 saw 45 lookups per access and not 16, and
// dh of 256 experts under Zipf routing took 167 us, not 145.
//
// The low-rank operand (h, dh) is fp32.  It enters the MFMAs as a sum of
// 16-bit parts: three of bf16 (8 bits each), exactly, or two of binary16 (11
// bits each and the sign between), to 2^-23 of itself, after scaling by a power
// of two to the middle of binary16's range: per row in expand, where values far
// below the row's largest keep 2^-33 of that; per tile of 32 rows in outer,
// 2^-35 of the tile's largest, with sums that move to the scale of the tile at
// work.  A single 16-bit rounding would have put its 2^-9 (2^-12) error into
// every product; the extra MFMAs are free here.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "pipeline.h"
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

// Inclusive sum over the wave.
__device__ __forceinline__ int wave_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

struct Item {
  int e, lo, hi;  // group and its rows
  int local;      // the item's number within the group
  int before;     // sum of count2 over the groups before
};

// Item w of the groups' items in order, count(rows) of each group: every wave
// finds it by itself from the offsets, with two sums over the lanes and no
// barrier, which takes about one trip to the L2 where E <= 256 (a table in LDS
// took three barriers and a search more; a small call is little else).
// False past the last item.  All results are wave-uniform.
template <class F, class F2>
__device__ __forceinline__ bool find_item(const int* __restrict__ offsets, int E, int P, int w, F count, F2 count2,
                                          Item& it) {
  const int lane = threadIdx.x & 63, per = (E + 63) >> 6, e0 = lane * per;
  int n = 0, n2 = 0, lo = 0, hi = 0;
  for (int i = 0; i < per; i += 4) {
    int o[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) o[j] = offsets[min(e0 + i + j, E)];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < per && e0 + i + j < E) {
        lo = min(max(o[j], 0), P);
        hi = min(max(o[j + 1], lo), P);
        n += count(hi - lo);
        n2 += count2(hi - lo);
      }
  }
  int sum = wave_sum(n, lane), sum2 = wave_sum(n2, lane);
  if (w >= __builtin_amdgcn_readlane(sum, 63)) return false;
  const int owner = __ffsll(__ballot(sum > w)) - 1;
  it.e = owner;
  it.local = w - __builtin_amdgcn_readlane(sum - n, owner);
  it.before = __builtin_amdgcn_readlane(sum2 - n2, owner);
  int at = owner;
  if (per > 1) {  // among the owner's groups
    const int e = owner * per + lane;
    const bool mine = lane < per && e < E;
    const int a = offsets[min(e, E)], b = offsets[min(e + 1, E)];
    lo = min(max(a, 0), P);
    hi = min(max(b, lo), P);
    n = mine ? count(hi - lo) : 0;
    n2 = mine ? count2(hi - lo) : 0;
    sum = wave_sum(n, lane);
    sum2 = wave_sum(n2, lane);
    at = __ffsll(__ballot(sum > it.local)) - 1;
    it.e = owner * per + at;
    it.local -= __builtin_amdgcn_readlane(sum - n, at);
    it.before += __builtin_amdgcn_readlane(sum2 - n2, at);
  }
  it.lo = __builtin_amdgcn_readlane(lo, at);
  it.hi = __builtin_amdgcn_readlane(hi, at);
  return true;
}

// Tile w of bm rows of the groups' rows; false past the last.
__device__ __forceinline__ bool find_tile(const Dev& g, int bm, int w, Tile& t) {
  Item it;
  if (!find_item(g.offsets, g.E, g.P, w, [=](int m) { return (m + bm - 1) / bm; }, [](int) { return 0; }, it)) return false;
  t.e = it.e;
  t.row0 = it.lo + it.local * bm;
  t.rows = min(bm, it.hi - t.row0);
  t.nt = 0;
  return true;
}

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

// Column j of 8 rows of elements held in registers: word t has rows 2t, 2t + 1.
template <class V>
__device__ __forceinline__ u32x4 column_of(const V (&rows)[8], int j) {
  const u32 sel = j & 1 ? 0x07060302u : 0x05040100u;
  u32x4 v;
#pragma unroll
  for (int t = 0; t < 4; ++t) v[t] = __builtin_amdgcn_perm(rows[2 * t + 1][j >> 1], rows[2 * t][j >> 1], sel);
  return v;
}

typedef u32 u32x2 __attribute__((ext_vector_type(2)));
template <int KIND>
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<u32x2*>(p) = u32x2{(u32)OutT<KIND>::from(a) | ((u32)OutT<KIND>::from(b) << 16),
                                       (u32)OutT<KIND>::from(c) | ((u32)OutT<KIND>::from(d) << 16)};
}

// Two transposing LDS reads: lane i of each 16 gets column i of the 4 x 16
// block whose row j/4, columns 4 (j % 4) .. +3 its lane j points at.
__device__ __forceinline__ u32x4 transposed8(const uint16_t* a, const uint16_t* b) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds4;
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

// red[wave][row][rank] = the wave's share of sum_k X[row(s)][k] W[e][r][k] for
// 16 RT rows of one group and 16 NR ranks (W [E][R][C]; C_MAJOR: W [E][C][R],
// as B is stored for dh), complete behind the barrier at the end.  The columns
// are dealt in steps of 128: this wave takes share `slot` of `slots`.  Rows
// past the tile and ranks past R repeat valid ones: they only reach results
// that are not used.  C_MAJOR weights pass through the wave's own piece of LDS,
// 32 columns at a time, and come back through the transposing read (lane i of
// 16 gets column i of a 4 x 16 block), so that B needs no transposed copy in
// memory.
template <int RT, int NR, bool C_MAJOR>
struct ShrinkLds {
  static constexpr int BM = 16 * RT, RW = 16 * NR + 4;
  float red[kShrinkWaves * BM * RW] __attribute__((aligned(16)));
  uint16_t turn[C_MAJOR ? kShrinkWaves : 1][32 * 16 * NR] __attribute__((aligned(16)));
  // Four ranks from r of a row, over the waves.
  __device__ __forceinline__ v4f sum4(int row, int r) const {
    v4f sum = *reinterpret_cast<const v4f*>(red + row * RW + r);
#pragma unroll
    for (int v = 1; v < kShrinkWaves; ++v) {
      const v4f o = *reinterpret_cast<const v4f*>(red + (v * BM + row) * RW + r);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += o[j];
    }
    return sum;
  }
};

template <int KIND, int RT, int NR, bool C_MAJOR>
__device__ __forceinline__ void shrink_tile(const Dev& g, const uint16_t* __restrict__ X, const RowMap& xm, int C,
                                            const uint16_t* __restrict__ W, const Tile& t, int rc, int slot, int slots,
                                            ShrinkLds<RT, NR, C_MAJOR>& lds) {
  constexpr int BM = 16 * RT, RW = 16 * NR + 4;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
      wp[n] = W + (int64_t)t.e * C * g.R + min(rc * 8 + (lane + 64 * n) % (2 * NR), g.R / 8 - 1) * 8;
    } else {
      wp[n] = W + ((int64_t)t.e * g.R + min(rc * 64 + n * 16 + c, g.R - 1)) * C;
    }
  }

  v4f acc[RT][NR];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[rt][n] = v4f{0.f, 0.f, 0.f, 0.f};

  const int steps = (C + 127) / 128;
  const int st0 = (int)((int64_t)steps * slot / slots), st1 = (int)((int64_t)steps * (slot + 1) / slots);
  u32x4 xb[RT][4], wb[NR][4];
  // Columns past C repeat the last 8 of each operand, W's as zeros.
  auto load = [&](int st, u32x4 (&xv)[RT][4], u32x4 (&wv)[NR][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = st * 128 + i * 32 + q * 8, kc = min(k, C - 8);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) xv[rt][i] = ld16(xp[rt] + kc);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (C_MAJOR) {
          const int col = st * 128 + i * 32 + (lane + 64 * n) / (2 * NR);
          wv[n][i] = ld16(wp[n] + (int64_t)min(col, C - 1) * g.R);
          if (col >= C) wv[n][i] = u32x4{0, 0, 0, 0};
        } else {
          wv[n][i] = ld16(wp[n] + kc);
          if (k >= C) wv[n][i] = u32x4{0, 0, 0, 0};
        }
      }
    }
  };
  const auto multiply = [&](const u32x4 (&xv)[RT][4], const u32x4 (&wv)[NR][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 wf[NR];
      if (C_MAJOR) {
        uint16_t* tw = lds.turn[wid];
#pragma unroll
        for (int n = 0; n < NR; ++n) *reinterpret_cast<u32x4*>(tw + (lane + 64 * n) * 8) = wv[n][i];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint16_t* p = tw + (q * 8 + c / 4) * (16 * NR) + n * 16 + (c & 3) * 4;
          wf[n] = transposed8(p, p + 4 * 16 * NR);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NR; ++n) wf[n] = wv[n][i];
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[rt][n] = mfma16<KIND>(wf[n], xv[rt][i], acc[rt][n]);
    }
  };
  // Two register sets; inside the loop no load is conditional, which would
  // make the compiler wait for all of them.
  int st = st0;
  if (st < st1) load(st, xb, wb);
  u32x4 xn[RT][4], wn[NR][4];
  for (; st + 2 < st1; st += 2) {
    load(st + 1, xn, wn);
    multiply(xb, wb);
    load(st + 2, xb, wb);
    multiply(xn, wn);
  }
  if (st + 1 < st1) {
    load(st + 1, xn, wn);
    multiply(xb, wb);
    multiply(xn, wn);
  } else if (st < st1) {
    multiply(xb, wb);
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < NR; ++n)
      *reinterpret_cast<v4f*>(lds.red + (wid * BM + rt * 16 + c) * RW + n * 16 + 4 * q) = acc[rt][n];
  __syncthreads();
}

// part[split][s][r]: one workgroup takes 16 RT rows of one group, 64 ranks at
// most, and one split of the columns.
// Up to rank 32 bound by its one read of X with what it has in flight, below
// what reads alone reach (7.0 TB/s).  dh of 32768 bf16 rows of 7168, 256 experts
// under Zipf routing, rank 16: 124 - 129 us, 0.53 GB, 4.3 TB/s; h of 16384 f16
// rows of 4096 from 8192 tokens, 8 experts: 36 - 46 us.  4 waves or 8, 1, 2 or 4
// row tiles, 1 split or 2 are within 2 % there.
// At rank 64 W bounds it: every workgroup reads the group's whole W through the
// L2, 512 KB for 256 KB of X in 32 rows (1 MB in 16), and the two-row-tile form
// spills 8 to 12 registers in its loop, with 74 - 102 KB of LDS one workgroup on
// a compute unit.  dh of 16384 f16 rows of 4096, 8 experts: 68 - 80 us, 0.15 GB.
// Above rank 64, X is read again for every 64 ranks.
template <int KIND, int RT, int NR, bool C_MAJOR>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(Dev g, const uint16_t* __restrict__ X, RowMap xm,
                                                                int C, const uint16_t* __restrict__ W,
                                                                float* __restrict__ part, int splits, int rchunks) {
  constexpr int BM = 16 * RT;
  __shared__ ShrinkLds<RT, NR, C_MAJOR> lds;
  const int tid = threadIdx.x, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rc = blockIdx.x % rchunks, sp = blockIdx.x / rchunks % splits, w = blockIdx.x / rchunks / splits;
  Tile t;
  if (!find_tile(g, BM, w, t)) return;
  shrink_tile<KIND>(g, X, xm, C, W, t, rc, sp * kShrinkWaves + wid, splits * kShrinkWaves, lds);
  for (int i = tid; i < BM * NR * 4; i += kShrinkThreads) {
    const int row = i / (NR * 4), r = (i - row * (NR * 4)) * 4;
    if (row >= t.rows || rc * 64 + r >= g.R || pair_of(g, t.row0 + row) < 0) continue;
    *reinterpret_cast<v4f*>(part + ((int64_t)sp * g.P + t.row0 + row) * g.R + rc * 64 + r) = lds.sum4(row, r);
  }
}

// ------------------------------------------------------------------- split
// What outer's waves read of a tile of 32 rows of one group, made once by
// split_tile: the low-rank operands of both weight gradients as MFMA
// fragments, fr[side][tile][part][16 ranks][lane][8 rows], the exponents of
// their scales (F16), and the rows of the wide operands.  A row that is not
// there stands as a row of the tile that is: its low-rank operand is zero, and
// what the row holds enters its group's sums anyway.  A tile without any row
// has the exponent kNoRows.
constexpr int kNoRows = 1 << 20;
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
  int blocks;          // kOuterWaves * kOuterCols columns each
};

// Exponent of a 32-row tile's scale, a multiple of 4 so that neighbours often
// agree: brings m (finite, >= 0) to [2^10, 2^14), so that the parts resolve
// 2^-35 of the tile's largest value.  (Multiples of 16 left 2^-23 where m came
// out lowest: ranks 2^-20 below the others came out wrong.)
constexpr int kMaxTileExp = 136;
constexpr int kMaxSpread = 80;  // of the exponents among which outer's sums move
__device__ __forceinline__ int tile_exp(float m) {
  return ((13 + 127 - max(1, __float_as_int(m) >> 23) + 128) & ~3) - 128;
}

// One workgroup of 256 threads: one side of one tile.
template <int KIND>
__device__ void split_tile(const Dev& g, const Side& sa, const Side& sb, const Tiles& tl, int unit) {
  constexpr int NP = kParts<KIND>;
  __shared__ u32 tmax;
  __shared__ int some;
  const int tid = threadIdx.x;
  const int side = unit & 1, w = unit >> 1;
  Tile t;
  if (!find_tile(g, 32, w, t)) return;
  const float sc = scale_of(g, t.e);
  const float* L = side ? sb.L : sa.L;
  const int splits = side ? sb.splits : sa.splits;
  const int64_t at = side * tl.tiles + w;
  if (tid < 64) {
    const int i = tid & 31;
    const int pair = i < t.rows ? pair_of(g, t.row0 + i) : -1;
    const int row = pair < 0 ? -1 : map_row(side ? sb.xm : sa.xm, t.row0 + i, pair);
    const unsigned long long there = __ballot(row >= 0);
    const int stand_in = __shfl(row, max(0, __ffsll(there) - 1), 64);
    if (tid < 32) tl.rows[at * 32 + i] = row >= 0 ? row : max(0, stand_in);
    if (tid == 0) {
      tmax = 0;
      some = there != 0;
    }
  }
  __syncthreads();
  // task: 8 rows (slice q) of one rank
  const int per = 64 * tl.rank_tiles;
  const auto low = [&](int k, float (&v)[8]) {
    const int rank = (k >> 6) * 16 + (k & 15), q = k >> 4 & 3;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.f;
      const int s = t.row0 + q * 8 + j;
      if (rank < g.R && q * 8 + j < t.rows && pair_of(g, s) >= 0)
        for (int sp = 0; sp < splits; ++sp) v[j] += L[((int64_t)sp * g.P + s) * g.R + rank];
      v[j] *= sc;
    }
  };
  float v[8];
  if (tid < per) low(tid, v);
  if (KIND == OUT_F16) {
    float big = 0.f;
    const auto raise = [&](const float (&u)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = __builtin_fabsf(u[j]);
        big = m < __builtin_inff() ? fmaxf(big, m) : big;
      }
    };
    if (tid < per) raise(v);
    for (int k = tid + 256; k < per; k += 256) {
      float u[8];
      low(k, u);
      raise(u);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
    if ((tid & 63) == 0) atomicMax(&tmax, __float_as_uint(big));
    __syncthreads();
  }
  const int f = KIND == OUT_F16 ? tile_exp(__uint_as_float(tmax)) : 0;
  if (tid == 0) tl.exps[at] = some ? f : kNoRows;
  for (int k = tid; k < per; k += 256) {
    if (k >= 256) low(k, v);
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
    for (int p = 0; p < NP; ++p) st16(tl.fr + ((at * NP + p) * per + k) * 8, pk[p]);
  }
}

// ------------------------------------------------------------------ expand
constexpr int kExpandThreads = 256;
constexpr int kExpandWaves = kExpandThreads / 64;
constexpr int kExpandRows = 64;

struct ExpandArgs {
  const float* part;     // [splits][P][R], summed here
  int splits;
  float* h;              // [P][R] or null: receives the sums
  const uint16_t* W;     // [E][C][R], or TR: [E][R][C]
  int C;
  const uint16_t* base;  // or null
  uint16_t* out;
  int out_pair;          // row of out: the pair (else s)
  int bm;                // rows a workgroup takes, a multiple of 16 up to kExpandRows
  int iters;             // 512-column blocks a workgroup walks
  int cblocks;           // workgroups across the columns
  int main_blocks;       // workgroups of the rows with a group; the others
  const int* p2s;        // copy the rows without one (by pair_to_sorted), or, in
  Side sa, sb;           // the gradient, make the outer kernel's tiles
  Tiles tl;
};

__host__ __device__ constexpr int padded_rank(int R) { return (R + 31) / 32 * 32 + 8; }

// Weights of columns n0 + 8c + j, ranks 32 oc + 8q .. +7 (TR: their rows, to be
// turned by column_of); columns past C and ranks past R repeat the last ones
// (for results not stored, times zeros).
template <bool TR>
__device__ __forceinline__ void load_weights(const ExpandArgs& a, int R, int e, int n0, int oc, u32x4 (&v)[8]) {
  const int lane = threadIdx.x & 63, o = min(oc * 4 + (lane >> 4), R / 8 - 1), col = n0 + (lane & 15) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (TR) v[i] = ld16(a.W + ((int64_t)e * R + o * 8 + i) * a.C + min(col, a.C - 8));
    else v[i] = ld16(a.W + ((int64_t)e * a.C + min(col + i, a.C - 1)) * R + o * 8);
  }
}

// The 16-bit parts of 8 ranks of one row, times 2^f (F16), to parts[p * stride].
template <int KIND>
__device__ __forceinline__ void put_parts(uint16_t* parts, int stride, const float v[8], int f) {
  constexpr int NP = kParts<KIND>;
  u32x4 pk[NP];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint16_t lo[NP], hi[NP];
    split<KIND>(KIND == OUT_F16 ? ldexp2(v[j], f) : v[j], lo);
    split<KIND>(KIND == OUT_F16 ? ldexp2(v[j + 1], f) : v[j + 1], hi);
#pragma unroll
    for (int p = 0; p < NP; ++p) pk[p][j / 2] = (u32)lo[p] | ((u32)hi[p] << 16);
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) *reinterpret_cast<u32x4*>(parts + p * stride) = pk[p];
}

// Row i of the lane's four: 8 columns, times 2^-f (F16), with the base.
template <int KIND, bool NT>
__device__ __forceinline__ void store_row(const v4f (&acc)[8], int i, int f, bool has_base, u32x4 base, uint16_t* out) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = KIND == OUT_F16 ? ldexp2(acc[j][i], -f) : acc[j][i];
    if (has_base) {
      const u32 b = base[j >> 1] >> (16 * (j & 1)) & 0xffffu;
      v[j] += KIND == OUT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32((uint16_t)b);
    }
  }
  store8<KIND, NT>(out, 0, v);
}

// Pair-ordered rows without a group: base, or zeros.
__device__ __forceinline__ void copy_rows_without(const Dev& g, const ExpandArgs& a, int wave, int waves) {
  for (int p = wave; p < g.P; p += waves) {
    const int s = a.p2s[p];
    if (s >= 0 && s < g.P) continue;
    for (int n = (threadIdx.x & 63) * 8; n < a.C; n += 512)
      st16(a.out + (int64_t)p * a.C + n, a.base ? ld16(a.base + (int64_t)p * a.C + n) : u32x4{0, 0, 0, 0});
  }
}

// out[o(s)][n] = base + sum_r (scale h[s][r]) W[e][n][r] for bm rows of one
// group.  The rows' low-rank operand is split once into LDS (zero past R).
// Each wave then takes 128 columns at a time, keeps their weights of OC x 32
// ranks in registers and walks the rows 16 at a time, the next rows' base in
// flight; OC = 0 takes any rank, reloading the weights for every 32 rows.
// Bound by base and out: 16384 f16 rows of 28672 at rank 16, 1.88 GB, 341 us,
// 5.5 TB/s.  dx with the outer kernel's tiles: 16384 f16 rows of 14336 at rank
// 64 96 - 116 us (0.47 GB written), 32768 bf16 rows of 2048 47 - 51 us.  Above
// rank 64 (OC = 0) bound by the weights, read again for every 32 rows.
template <int KIND, int OC, bool TR, bool NT>
__global__ __launch_bounds__(kExpandThreads, OC ? 3 : 2) void expand_kernel(Dev g, ExpandArgs a) {
  constexpr int NP = kParts<KIND>, RTI = OC ? 1 : 2;
  extern __shared__ __align__(16) int sm[];
  __shared__ int orow[kExpandRows];
  __shared__ u32 rmax[kExpandRows];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);  // what a wave shares stays in scalar registers
  if ((int)blockIdx.x >= a.main_blocks) {
    if (TR) {
      split_tile<KIND>(g, a.sa, a.sb, a.tl, blockIdx.x - a.main_blocks);
      return;
    }
    copy_rows_without(g, a, (blockIdx.x - a.main_blocks) * kExpandWaves + wid,
                      (gridDim.x - a.main_blocks) * kExpandWaves);
    return;
  }
  const int w = blockIdx.x / a.cblocks, cb = blockIdx.x - w * a.cblocks;
  Tile t;
  if (!find_tile(g, a.bm, w, t)) return;

  const bool has_base = !TR && a.base;  // dx has none
  const int octs = g.R / 8, RP = padded_rank(g.R), ochunks = (octs + 3) / 4;
  const auto load_w = [&](int n0, int oc, u32x4 (&v)[8]) { load_weights<TR>(a, g.R, t.e, n0, oc, v); };
  const auto turn_w = [&](u32x4 (&v)[8]) {
    if (TR) {
      u32x4 r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = column_of(r, j);
    }
  };
  const int first = (cb * a.iters * kExpandWaves + wid) * 128;
  u32x4 wr[OC ? OC : 1][8];
  if (OC) {
#pragma unroll
    for (int oc = 0; oc < OC; ++oc) load_w(first, oc, wr[oc]);
  }

  // The split operand: parts[p][row][r], rows of RP.
  uint16_t* parts = reinterpret_cast<uint16_t*>(sm);
  const int nrt = (t.rows + 15) / 16, rows16 = nrt * 16;
  const float sc = scale_of(g, t.e);
  if (tid < rows16) {
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
  };
  if (KIND == OUT_F16) {
    // each row's largest finite magnitude, for its scale
    for (int i = tid; i < rows16 * octs; i += kExpandThreads) {
      const int row = i / octs, o = i - row * octs;
      float v[8], m = 0.f;
      value(row, o, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = __builtin_fabsf(sc * v[j]);
        m = u < __builtin_inff() ? fmaxf(m, u) : m;
      }
      atomicMax(&rmax[row], __float_as_uint(m));
    }
    __syncthreads();
  }
  for (int i = tid; i < rows16 * ochunks * 4; i += kExpandThreads) {
    const int row = i / (ochunks * 4), o = i - row * (ochunks * 4);
    float v[8];
    value(row, o, v);
    if (a.h && cb == 0 && o < octs && orow[row] >= 0)
      store8<OUT_F32, false>(a.h, (int64_t)(t.row0 + row) * g.R + o * 8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= sc;
    put_parts<KIND>(parts + row * RP + o * 8, a.bm * RP, v, KIND == OUT_F16 ? half_exp(__uint_as_float(rmax[row])) : 0);
  }
  __syncthreads();

  for (int it = 0; it < a.iters; ++it) {
    const int n0 = first + it * kExpandWaves * 128;
    if (n0 >= a.C) break;
    const int col = n0 + c * 8, colc = min(col, a.C - 8);
    if (OC) {
#pragma unroll
      for (int oc = 0; oc < OC; ++oc) {
        if (it > 0) load_w(n0, oc, wr[oc]);
        turn_w(wr[oc]);
      }
    }
    u32x4 bv[RTI][4], bn[RTI][4];
    const auto load_base = [&](int rt, u32x4 (&v)[RTI][4]) {
#pragma unroll
      for (int x = 0; x < RTI; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[x][i] = ld16_nt<NT>(a.base + (int64_t)max(orow[min(rt + x, nrt - 1) * 16 + 4 * q + i], 0) * a.C + colc);
    };
    if (has_base) load_base(0, bv);
    for (int rt = 0; rt < nrt; rt += RTI) {
      if (has_base && rt + RTI < nrt) load_base(rt + RTI, bn);
      v4f acc[RTI][8];
#pragma unroll
      for (int x = 0; x < RTI; ++x)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[x][j] = v4f{0.f, 0.f, 0.f, 0.f};
      const auto multiply = [&](int oc, const u32x4 (&v)[8]) {
#pragma unroll
        for (int x = 0; x < RTI; ++x)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const u32x4 l = *reinterpret_cast<u32x4*>(
                parts + (p * a.bm + min(rt + x, nrt - 1) * 16 + c) * RP + (oc * 4 + q) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[x][j] = mfma16<KIND>(l, v[j], acc[x][j]);
          }
      };
      if (OC) {
#pragma unroll
        for (int oc = 0; oc < OC; ++oc) multiply(oc, wr[oc]);
      } else {
        for (int oc = 0; oc < ochunks; ++oc) {
          load_w(n0, oc, wr[0]);
          turn_w(wr[0]);
          multiply(oc, wr[0]);
        }
      }
#pragma unroll
      for (int x = 0; x < RTI; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (rt + x) * 16 + 4 * q + i;
          const int o = rt + x < nrt ? orow[row] : -1;
          if (col >= a.C || o < 0) continue;
          store_row<KIND, NT>(acc[x], i, KIND == OUT_F16 ? half_exp(__uint_as_float(rmax[row])) : 0, has_base, bv[x][i],
                              a.out + (int64_t)o * a.C + col);
        }
#pragma unroll
      for (int x = 0; x < RTI; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) bv[x][i] = bn[x][i];
    }
  }
}

// ------------------------------------------------------------------- small
constexpr int kSmallCols = 128 * kShrinkWaves;

// Shrink and expand in one launch, for few rows: one workgroup takes 16 rows of
// one group and 1024 columns of the output, and computes the rows' low-rank
// values for itself.  The column blocks of a tile repeat that, which costs
// less than a second launch and its trip through memory while A is short.
// Bound by its chain of trips to memory and one compute unit's loads of A.  In
// series: the offsets; the row's pair, whose wait holds for B's loads too; the
// pair again for x's row; x and A, two steps of 128 columns a wave at a time; the
// scale, after the reduction; base, after the barrier behind it.  One row, K = N
// = 4096, rank 16, 10.0 us (two launches 4.6 + 6.8 us); K = N = 1024, rank 8, 6.1
// us in a graph for 8.8.
template <int KIND, int NR>
__global__ __launch_bounds__(kShrinkThreads) void small_kernel(Dev g, const uint16_t* __restrict__ X, RowMap xm, int K,
                                                               const uint16_t* __restrict__ A, ExpandArgs a) {
  constexpr int NP = kParts<KIND>, OC = (NR + 1) / 2, LANES = 4 * OC, RP = 32 * OC + 8;
  __shared__ ShrinkLds<1, NR, false> lds;
  __shared__ __align__(16) uint16_t parts[NP * 16 * RP];
  __shared__ int orow[16], rexp[16];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  if ((int)blockIdx.x >= a.main_blocks) {
    copy_rows_without(g, a, (blockIdx.x - a.main_blocks) * kShrinkWaves + wid,
                      (gridDim.x - a.main_blocks) * kShrinkWaves);
    return;
  }
  const int w = blockIdx.x / a.cblocks, cb = blockIdx.x - w * a.cblocks;
  Tile t;
  if (!find_tile(g, 16, w, t)) return;
  const int n0 = (cb * kShrinkWaves + wid) * 128, col = n0 + c * 8;
  u32x4 wr[OC][8];
#pragma unroll
  for (int oc = 0; oc < OC; ++oc) load_weights<false>(a, g.R, t.e, n0, oc, wr[oc]);
  if (tid < 16) {
    const int pair = tid < t.rows ? pair_of(g, t.row0 + tid) : -1;
    orow[tid] = pair < 0 ? -1 : (a.out_pair ? pair : t.row0 + tid);
  }
  shrink_tile<KIND>(g, X, xm, K, A, t, 0, wid, kShrinkWaves, lds);
  if (tid < 16 * LANES) {  // 8 ranks of one row; a row's lanes are neighbours
    const int row = tid / LANES, o = tid % LANES;
    float v[8], m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (o * 8 < g.R && orow[row] >= 0) {
      const v4f x = lds.sum4(row, o * 8), y = lds.sum4(row, o * 8 + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = x[j];
        v[4 + j] = y[j];
      }
      if (a.h && cb == 0) store8<OUT_F32, false>(a.h, (int64_t)(t.row0 + row) * g.R + o * 8, v);
    }
    const float sc = scale_of(g, t.e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] *= sc;
      const float u = __builtin_fabsf(v[j]);
      m = u < __builtin_inff() ? fmaxf(m, u) : m;
    }
#pragma unroll
    for (int x = 1; x < LANES; x <<= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    const int f = KIND == OUT_F16 ? half_exp(m) : 0;
    if (o == 0) rexp[row] = f;
    put_parts<KIND>(parts + row * RP + o * 8, 16 * RP, v, f);
  }
  __syncthreads();
  if (n0 >= a.C) return;
  u32x4 bv[4];  // (loaded before the shrink, 0.6 us slower: its pairs hold up x)
  if (a.base) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bv[i] = ld16(a.base + (int64_t)max(orow[4 * q + i], 0) * a.C + min(col, a.C - 8));
  }
  v4f acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int oc = 0; oc < OC; ++oc)
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const u32x4 l = *reinterpret_cast<u32x4*>(parts + (p * 16 + c) * RP + (oc * 4 + q) * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = mfma16<KIND>(l, wr[oc][j], acc[j]);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int o = orow[4 * q + i];
    if (col < a.C && o >= 0)
      store_row<KIND, false>(acc, i, KIND == OUT_F16 ? rexp[4 * q + i] : 0, a.base != nullptr, bv[i],
                             a.out + (int64_t)o * a.C + col);
  }
}

// ------------------------------------------------------------------- outer
constexpr int kOuterWaves = 4;
constexpr int kOuterThreads = 64 * kOuterWaves;
constexpr int kOuterCols = 64;   // columns of a wave
constexpr int kOuterDepth = 3;   // tiles of the wide operand in flight
constexpr int kOuterChunk = 4096;              // most rows of a chunk, but for the half more of one not cut
constexpr int kOuterTiles = kOuterChunk / 32 * 2;

// A group of m rows is cut into chunks_of(m) runs of its tiles, equal to a
// tile, of 3/4 to 3/2 of `chunk` rows (at least 256); without rows it has one
// that writes zeros.
__host__ __device__ constexpr int chunks_of(int m, int chunk) { return m < chunk ? 1 : (m + chunk / 2) / chunk; }
__device__ __forceinline__ int chunk_tile(int nt, int i, int n) { return (int)((int64_t)nt * i / n); }

// Slot of the partial sums of the chunk of a cut group that starts at sorted
// row s: starts of one group are more than chunk / 2 rows apart, so in the same
// chunk / 2 rows lie at most one group's first and another's later start.
__host__ __device__ constexpr int outer_slot(int s, bool first, int chunk) { return 2 * (s / (chunk / 2)) + (first ? 1 : 0); }
__host__ __device__ constexpr int64_t outer_slots(int64_t P, int chunk) {
  return chunks_of((int)P, chunk) > 1 ? 2 * ((P - 1) / (chunk / 2) + 1) : 0;
}

// dW[r][n] = sum_s (scale L[s][r]) X[row(s)][n] for one chunk of a group's
// rows, 256 columns and 16 NR ranks.  Each of the 4 waves owns 64 columns and
// walks the chunk's tiles of 32 rows (the MFMA's contraction), three tiles of
// 4 KB in flight to registers.  The low-rank fragments, which all columns
// share, and the rows come through LDS by direct-to-LDS copies, pairs of tiles
// ahead: a row or an exponent that came through a register would be the newest
// load when it is needed, and waiting for it would be waiting for everything
// in flight.
// One read of both wide operands, 0.60 GB together: bf16 rows of 7168 and 2048,
// 256 experts under Zipf routing, rank 16, 136 - 148 us, 4.4 TB/s; f16 rows of
// 4096 and 14336, 8 experts, rank 64, 132 - 152 us.  What holds it below the 7.0
// TB/s of reads alone is not shown; it is not HBM, as the second takes dy from
// the Infinity Cache and is no faster.  Two tiles in flight, double buffers for
// the MFMA operands, or 128 columns a wave were no faster.  Above rank 64, both
// operands are read again for every 64 ranks.
template <int KIND, int NR>
__global__ __launch_bounds__(kOuterThreads, 3) void outer_kernel(Dev g, Side sa, Side sb, Tiles tl, int rchunks,
                                                                 int chunk) {
  constexpr int NP = kParts<KIND>, kPieces = NR * NP;  // 1 KB fragments of a tile
  __shared__ __align__(16) uint16_t ring[2][2][kPieces][512];
  __shared__ __align__(16) int rows[4][64], exps[kOuterTiles];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);  // what a wave shares stays in scalar registers

  const int rc = blockIdx.x % rchunks, w = blockIdx.x / rchunks / (sa.blocks + sb.blocks);
  int block = blockIdx.x / rchunks % (sa.blocks + sb.blocks);
  Item it;
  if (!find_item(g.offsets, g.E, g.P, w, [=](int m) { return chunks_of(m, chunk); },
                 [](int m) { return (m + 31) / 32; }, it))
    return;
  const int side = block >= sa.blocks;
  if (side) block -= sa.blocks;
  const Side& d = side ? sb : sa;
  const int e = it.e, ch = it.local, lo = it.lo, hi = it.hi;
  const int cuts = chunks_of(hi - lo, chunk), all = (hi - lo + 31) / 32;
  const int k0 = chunk_tile(all, ch, cuts), s0 = lo + k0 * 32;
  const int first = it.before + k0;
  // (a malformed offsets table may count more tiles than there can be)
  const int nt = min(chunk_tile(all, ch + 1, cuts) - k0, (int)max<int64_t>(0, tl.tiles - first));
  const int64_t t0 = side * tl.tiles + first;

  // Lane: columns col .. col+3 (past C the last ones again, not stored).
  const int n0 = (block * kOuterWaves + wid) * kOuterCols + c * 4, col = min(n0, d.C - 4);
  const uint16_t* X = d.X + col;
  v4f acc[NR][4];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = v4f{0.f, 0.f, 0.f, 0.f};
  u32x2 raw[kOuterDepth][8];
  const auto load_x = [&](int k, u32x2 (&v)[8]) {
    if (k >= nt) return;
    const int* p = &rows[(k >> 1) & 3][(k & 1) * 32 + q * 8];
    const v4i r0 = *reinterpret_cast<const v4i*>(p), r1 = *reinterpret_cast<const v4i*>(p + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x2*>(X + (int64_t)(i < 4 ? r0[i] : r1[i - 4]) * d.C));
  };
  // The rows of tiles k and k + 1.
  const auto copy_rows = [&](int k) {
    if (wid == 0 && k < nt)
      dma4(tl.rows + (t0 + min(k + (lane >> 5), nt - 1)) * 32 + (lane & 31), lds_addr(rows[(k >> 1) & 3]));
  };
  // The fragments of tiles k and k + 1, dealt to the waves; ranks past R
  // repeat the last ones.
  const auto copy_fr = [&](int k) {
    for (int i = wid; i < 2 * kPieces; i += kOuterWaves) {
      const int x = i / kPieces, p = (i - x * kPieces) / NR, n = i % NR;
      const int64_t piece = ((t0 + min(k + x, nt - 1)) * NP + p) * tl.rank_tiles + min(rc * NR + n, tl.rank_tiles - 1);
      dma16(tl.fr + piece * 512 + lane * 8, lds_addr(ring[(k >> 1) & 1][x][p * NR + n]));
    }
  };
  static_assert(kOuterDepth == 3, "rows are copied for tiles up to k + 4 while tile k is at work");
  int f = kMaxTileExp, low = f;  // F16: exponent of the scale of the sums, the smallest so far
  const auto step = [&](int k, u32x2 (&x8)[8]) {
    if ((k & 1) == 0) {
      // The pair's fragments, and the rows of pair k + 4, were copied before
      // the loads of wide tiles k + 1 and k + 2, 16 of them where both tiles
      // are there; all waves have them, and are done with the other half of
      // the ring, behind the barrier.
      if (k == 0 && nt >= kOuterDepth) wait_vmcnt<8 * kOuterDepth>();
      else if (k > 0 && k - 1 + kOuterDepth < nt) wait_vmcnt<16>();
      else wait_vmcnt<0>();
      raw_barrier();
      if (k + 2 < nt) copy_fr(k + 2);
      copy_rows(k + 6);
    }
    const int te = __builtin_amdgcn_readfirstlane(exps[k]);
    if (te == kNoRows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x8[i] = u32x2{0, 0};
    }
    bool lost = false;
    if (KIND == OUT_F16 && te != kNoRows) {
      // The sums move to the tile's scale, in fp32 and so without loss.  At the
      // smallest scale so far they are below 2^43 (2^14, times x's 2^16, times
      // 6144 rows), so 2^kMaxSpread above it they cannot overflow.  A tile past
      // that, all below 2^-80 of the largest value so far, is dropped but for
      // its infinities and NaN.  (Fragments brought down to the smaller scale
      // in binary16 stopped at its lowest step, 2^-34 of the largest value,
      // however small they were.)
      low = min(low, te);
      lost = te - low > kMaxSpread;
      if (!lost && te != f) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][j][i] = ldexp2(acc[n][j][i], te - f);
        f = te;
      }
    }
    u32x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = column_of(x8, j);
    load_x(k + kOuterDepth, x8);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        u32x4 a = ld16(&ring[(k >> 1) & 1][k & 1][p * NR + n][lane * 8]);
        if (KIND == OUT_F16 && lost) {  // times 2^-42: zero, but infinities stay
          const _Float16 tiny = (_Float16)0x1p-14f;
          a = __builtin_bit_cast(u32x4, __builtin_bit_cast(v8h, a) * tiny * tiny * tiny);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][j] = mfma16<KIND>(a, x[j], acc[n][j]);
      }
  };
  if (nt > 0) {
    copy_rows(0);
    copy_rows(2);
    copy_rows(4);
    for (int i = wid * 64; i < nt; i += kOuterThreads) dma4(tl.exps + t0 + min(i + lane, nt - 1), lds_addr(exps + i));
    wait_vmcnt<0>();
    raw_barrier();
    copy_fr(0);
#pragma unroll
    for (int i = 0; i < kOuterDepth; ++i) load_x(i, raw[i]);
  }
  for (int k = 0; k < nt; k += kOuterDepth) {
#pragma unroll
    for (int i = 0; i < kOuterDepth; ++i)
      if (k + i < nt) step(k + i, raw[i]);
  }

  // Lane: ranks 4q .. 4q+3 of each 16, columns col .. col+3.
  if (n0 >= d.C) return;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r0 = (rc * NR + n) * 16 + 4 * q;
    if (r0 >= g.R) continue;
    v4f v[4];  // [rank][column]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = KIND == OUT_F16 ? ldexp2(acc[n][j][i], -f) : acc[n][j][i];
    if (cuts > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(d.part + ((int64_t)outer_slot(s0, ch == 0, chunk) * g.R + r0 + i) * d.C + col) = v[i];
    } else if (d.col_major) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store4<KIND>(d.out + ((int64_t)e * d.C + col + j) * g.R + r0, v[0][j], v[1][j], v[2][j], v[3][j]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store4<KIND>(d.out + ((int64_t)e * g.R + r0 + i) * d.C + col, v[i][0], v[i][1], v[i][2], v[i][3]);
    }
  }
}

// Joins the chunks of the groups longer than one: a thread takes 4 ranks of
// one column, so that both output orders store 4 values at once or in runs.
// 14 - 16 us (256 experts, most of them whole) and 4 - 6 us (8 experts, none cut:
// the launch covers every group whose rows could fill one that is) after the above.
template <int KIND>
__global__ __launch_bounds__(256) void join_kernel(Dev g, Side sa, Side sb, int blocks_a, int blocks_b,
                                                  int chunk) {
  const int per = blocks_a + blocks_b, e = blockIdx.x / per;
  int b = blockIdx.x - e * per;
  const Side& d = b < blocks_a ? sa : sb;
  if (b >= blocks_a) b -= blocks_a;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  const int cuts = chunks_of(hi - lo, chunk), all = (hi - lo + 31) / 32;
  if (cuts == 1) return;
  const int64_t i = (int64_t)b * 256 + threadIdx.x;
  const int r = (int)(i / d.C) * 4, n = (int)(i % d.C);
  if (r >= g.R) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < cuts; ++c) {
    const float* p = d.part + ((int64_t)outer_slot(lo + 32 * chunk_tile(all, c, cuts), c == 0, chunk) * g.R + r) * d.C + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += p[(int64_t)j * d.C];
  }
  if (d.col_major) {
    store4<KIND>(d.out + ((int64_t)e * d.C + n) * g.R + r, sum[0], sum[1], sum[2], sum[3]);
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

// Row tiles (of 16) a workgroup takes.  Two halve the reads of the weights;
// four took more registers than that gave back (Zipf over 256 experts, dh: 120
// us at two, 145 at four).  At rank 64 two spill, and one, which reads the
// weights twice as often, was no faster.
int shrink_rt(int64_t P, int E) { return P >= 24 * (int64_t)E ? 2 : 1; }
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }  // per workgroup; 64 ranks at most

// Rows of an expand workgroup: about the average group's, up to 64 (beside the
// Mixtral-sized gate+up projection 128 rows took 405 us for 387); their split
// operand has to leave LDS for three workgroups on a compute unit.
int expand_rows(int64_t P, int E, int R, int f16) {
  int bm = kExpandRows;
  while (bm > 16 && ((f16 ? 2 : 3) * bm * padded_rank(R) * 2 > 52 * 1024 || P < bm * (int64_t)E)) bm /= 2;
  return bm;
}

// 512-column blocks an expand workgroup walks: up to 2 while 2048 workgroups
// remain (there 4 blocks took 414 us for 387), more where one grid could not
// hold the workgroups.
int expand_iters(int64_t tiles, int blocks) {
  int iters = (int)std::max<int64_t>(1, std::min<int64_t>(2, tiles * blocks / 2048));
  while (iters < blocks && tiles * ((blocks + iters - 1) / iters) > kMaxBlocks) iters *= 2;
  return iters;
}

// Column splits of a shrink: enough workgroups for two on each of 256 compute
// units, at least one 128-column step per wave.
int shrink_splits(int64_t P, int E, int C, int R) {
  const int steps = (C + 127) / 128;
  const int64_t wgs = max_tiles(P, E, 16 * shrink_rt(P, E)) * ((R + 63) / 64);
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
  const int nr = rank_tiles(d.R), rt = shrink_rt(d.P, d.E);
  if (nr == 1 && rt == 2) return shrink_launch<KIND, 2, 1, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 1) return shrink_launch<KIND, 1, 1, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2 && rt == 2) return shrink_launch<KIND, 2, 2, CM>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2) return shrink_launch<KIND, 1, 2, CM>(d, X, xm, C, W, part, splits, stream);
  if (rt == 2) return shrink_launch<KIND, 2, 4, CM>(d, X, xm, C, W, part, splits, stream);
  return shrink_launch<KIND, 1, 4, CM>(d, X, xm, C, W, part, splits, stream);
}

template <int KIND, int OC, bool TR, bool NT>
hipError_t expand_launch(const Dev& d, ExpandArgs a, int others, hipStream_t stream) {
  a.bm = expand_rows(d.P, d.E, d.R, KIND == OUT_F16);
  const int64_t tiles = max_tiles(d.P, d.E, a.bm);
  const int blocks = (a.C + 511) / 512;
  a.iters = expand_iters(tiles, blocks);
  a.cblocks = (blocks + a.iters - 1) / a.iters;
  a.main_blocks = (int)(tiles * a.cblocks);
  if (!a.out) a.main_blocks = 0;
  const size_t lds = sizeof(uint16_t) * kParts<KIND> * a.bm * padded_rank(d.R);
  hipLaunchKernelGGL((expand_kernel<KIND, OC, TR, NT>), dim3(a.main_blocks + others), dim3(kExpandThreads), lds, stream, d,
                     a);
  return hipGetLastError();
}

template <int KIND, bool TR, bool NT>
hipError_t expand_nt(const Dev& d, const ExpandArgs& a, int others, hipStream_t stream) {
  if (d.R <= 32) return expand_launch<KIND, 1, TR, NT>(d, a, others, stream);
  if (d.R <= 64) return expand_launch<KIND, 2, TR, NT>(d, a, others, stream);
  return expand_launch<KIND, 0, TR, NT>(d, a, others, stream);
}

// `bytes`: what the launch streams, with what the launches after it read
// again.  Where that is more than the Infinity Cache holds, base and out go
// past it: beside the Mixtral-sized gate+up projection 386 -> 369 us, and the
// gradients, whose next launch reads dy again, 387 -> 346 us (rank 64,
// Mixtral-sized) and 345 -> 335 us (Zipf over 256 experts).
template <int KIND, bool TR>
hipError_t expand(const Dev& d, const ExpandArgs& a, int others, int64_t bytes, hipStream_t stream) {
  return bytes >= (int64_t(256) << 20) ? expand_nt<KIND, TR, true>(d, a, others, stream)
                                       : expand_nt<KIND, TR, false>(d, a, others, stream);
}

int outer_nr(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }
int outer_blocks(int C) { return (C + kOuterWaves * kOuterCols - 1) / (kOuterWaves * kOuterCols); }
int outer_rchunks(int R) { return (R + 16 * outer_nr(R) - 1) / (16 * outer_nr(R)); }
int64_t outer_tasks(int N, int K, int R) {  // workgroups per chunk of rows
  return (int64_t)(outer_blocks(N) + outer_blocks(K)) * outer_rchunks(R);
}

// About the rows a workgroup sums before a longer group is cut: four times the
// average group's, so that the longest of skewed groups do not outlast the
// others (256 experts of 128 rows on average under Zipf routing: 355 us at 512
// rows, 364 at 256, 382 at 2048; cutting equal groups costs the join: 8 of 2048
// rows, 418 us whole, 438 in halves), and less where the rows then make no two
// workgroups for each of 256 compute units.
int outer_chunk(int64_t P, int E, int N, int K, int R) {
  int chunk = 256;
  while (chunk < kOuterChunk && chunk < 4 * P / E) chunk *= 2;
  while (chunk > 256 && std::max<int64_t>(P / chunk, std::min<int64_t>(P, E)) * outer_tasks(N, K, R) < 512) chunk /= 2;
  return chunk;
}
// Upper bound of all groups' chunks.
int64_t max_chunks(int64_t P, int E, int chunk) { return P / chunk + E; }

template <int KIND>
hipError_t outer(const Dev& d, const Side& sa, const Side& sb, const Tiles& tl, int N, int K, hipStream_t stream) {
  const int chunk = outer_chunk(d.P, d.E, N, K, d.R), nr = outer_nr(d.R);
  const int64_t tasks = max_chunks(d.P, d.E, chunk) * outer_tasks(N, K, d.R);
  const dim3 grid((unsigned)tasks);
  const int rchunks = outer_rchunks(d.R);
  if (nr == 1)
    hipLaunchKernelGGL((outer_kernel<KIND, 1>), grid, dim3(kOuterThreads), 0, stream, d, sa, sb, tl, rchunks, chunk);
  else if (nr == 2)
    hipLaunchKernelGGL((outer_kernel<KIND, 2>), grid, dim3(kOuterThreads), 0, stream, d, sa, sb, tl, rchunks, chunk);
  else
    hipLaunchKernelGGL((outer_kernel<KIND, 4>), grid, dim3(kOuterThreads), 0, stream, d, sa, sb, tl, rchunks, chunk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || outer_slots(d.P, chunk) == 0) return e;
  const int ba = (int)(((int64_t)K * (d.R / 4) + 255) / 256), bb = (int)(((int64_t)N * (d.R / 4) + 255) / 256);
  hipLaunchKernelGGL(join_kernel<KIND>, dim3((unsigned)(d.E * (ba + bb))), dim3(256), 0, stream, d, sa, sb, ba, bb,
                     chunk);
  return hipGetLastError();
}

// Whether a call takes one launch (small_kernel).  Against the two kernels, in
// graphs, one row to 200: A of 16 KB a group 6.1 - 7.7 us for 8.8 - 10.9, of
// 64 KB 8.2 - 8.4 for 10.5 - 10.9, of 128 KB 9.8 - 11.2 for 9.9 - 11.0 (and a
// launch less for the host), of 224 KB 13.0 - 19.1 for 10.8 - 13.7; with more
// workgroups than CUs 16.8 for 14.4.  (256 is an MI355X's number, written out: the
// workspace's size may not depend on the device that is current when it is asked.)
bool one_launch(int64_t P, int E, int N, int K, int R) {
  return R <= 64 && max_tiles(P, E, 16) * ((N + kSmallCols - 1) / kSmallCols) <= 256 &&
         (int64_t)rank_tiles(R) * 16 * K <= 65536;
}

template <int KIND>
hipError_t small(const Dev& d, const uint16_t* x, RowMap xm, int K, const uint16_t* A, ExpandArgs a, bool copy,
                 hipStream_t stream) {
  a.cblocks = (a.C + kSmallCols - 1) / kSmallCols;
  a.main_blocks = (int)(max_tiles(d.P, d.E, 16) * a.cblocks);
  const dim3 grid(a.main_blocks + (copy ? (d.P + kShrinkWaves - 1) / kShrinkWaves : 0)), block(kShrinkThreads);
  switch (rank_tiles(d.R)) {
    case 1: hipLaunchKernelGGL((small_kernel<KIND, 1>), grid, block, 0, stream, d, x, xm, K, A, a); break;
    case 2: hipLaunchKernelGGL((small_kernel<KIND, 2>), grid, block, 0, stream, d, x, xm, K, A, a); break;
    default: hipLaunchKernelGGL((small_kernel<KIND, 4>), grid, block, 0, stream, d, x, xm, K, A, a); break;
  }
  return hipGetLastError();
}

template <int KIND>
hipError_t forward(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b, const uint16_t* base,
                   uint16_t* out, float* h, float* ws, hipStream_t stream) {
  const Dev d = dev_args(g);
  const bool copy = g.out_pair && base != out;
  if (one_launch(g.P, g.E, g.N, g.K, g.R)) {
    const ExpandArgs ea = {nullptr, 0, h, b, g.N, base, out, g.out_pair, 0, 0, 0, 0, g.p2s};
    return small<KIND>(d, x, x_map(g), g.K, a, ea, copy, stream);
  }
  const int splits = shrink_splits(g.P, g.E, g.K, g.R);
  float* part = splits == 1 && h ? h : ws;
  hipError_t e = shrink<KIND, false>(d, x, x_map(g), g.K, a, part, splits, stream);
  if (e != hipSuccess) return e;
  const int copies = copy ? std::min((d.P + kExpandWaves - 1) / kExpandWaves, 1024) : 0;
  ExpandArgs ea = {part, splits, part == h ? nullptr : h, b, g.N, base, out, g.out_pair, 0, 0, 0, 0, g.p2s};
  return expand<KIND, false>(d, ea, copies, g.P * g.N * (base ? 4 : 2), stream);
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
  const Side sa = {dh, splits, x, x_map(g), g.K, da, 0, reinterpret_cast<float*>(ws + l.pa), outer_blocks(g.K)};
  const Side sb = {h, 1, dy, o_map(g), g.N, db, 1, reinterpret_cast<float*>(ws + l.pb), outer_blocks(g.N)};
  const Tiles tl = {reinterpret_cast<uint16_t*>(ws + l.fr), reinterpret_cast<int*>(ws + l.exps),
                    reinterpret_cast<int*>(ws + l.rows), l.tiles, (g.R + 15) / 16};
  if (g.P > 0) {
    hipError_t e = shrink<KIND, true>(d, dy, o_map(g), g.N, b, dh, splits, stream);
    if (e != hipSuccess) return e;
    ExpandArgs ea = {dh, splits, nullptr, a, g.K, nullptr, dx, 0, 0, 0, 0, 0, nullptr, sa, sb, tl};
    if ((e = expand<KIND, true>(d, ea, (int)(2 * l.tiles), g.P * (g.N + 2 * (int64_t)g.K) * 2, stream)) != hipSuccess)
      return e;
  }
  return outer<KIND>(d, sa, sb, tl, g.N, g.K, stream);
}

}  // namespace

namespace {
constexpr int64_t kThreadsMax = int64_t(1) << 31;  // per launch, half the packet's limit

// Whether a shrink of C columns and an expand to C2 fit one grid each.
bool products_fit(int64_t P, int E, int C, int C2, int R) {
  if (max_tiles(P, E, 16 * shrink_rt(P, E)) * shrink_splits(P, E, C, R) * ((R + 63) / 64) *
          kShrinkThreads > kThreadsMax)
    return false;
  const int64_t tiles = max_tiles(P, E, expand_rows(P, E, R, 0));
  const int blocks = (C2 + 511) / 512, iters = expand_iters(tiles, blocks);
  return tiles * ((blocks + iters - 1) / iters) <= kMaxBlocks;
}
}  // namespace

bool lora_fits(int64_t P, int E, int N, int K, int R) { return products_fit(P, E, K, N, R); }

bool lora_bwd_fits(int64_t P, int E, int N, int K, int R) {
  return products_fit(P, E, N, K, R) && max_tiles(P, E, 32) * 512 <= kThreadsMax / 2 &&
         max_chunks(P, E, outer_chunk(P, E, N, K, R)) * outer_tasks(N, K, R) * kOuterThreads <= kThreadsMax &&
         E * (((int64_t)N + K) * (R / 4) / 256 + 2) * 256 <= kThreadsMax;
}

size_t lora_workspace_bytes(int64_t P, int E, int N, int K, int R) {
  return P && !one_launch(P, E, N, K, R) ? (size_t)P * R * sizeof(float) * shrink_splits(P, E, K, R) : 0;
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
