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

// Exponent of the power of two that brings m (finite, >= 0) to [2^8, 2^9):
// far from both ends of binary16, with 2^6 of room before 2^15.
__device__ __forceinline__ int half_exp(float m) { return 135 - max(1, __float_as_int(m) >> 23); }
__device__ __forceinline__ float ldexp2(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }

// ------------------------------------------------------------------ shrink
constexpr int kShrinkWaves = 8;
constexpr int kShrinkThreads = 64 * kShrinkWaves;

// part[split][s][r] = sum over the split's columns of X[row(s)][k] W[e][r][k].
// One workgroup: 16 RT rows of one group, 16 NR ranks, one split of the
// columns, dealt to its 8 waves in steps of 128.  Rows past the tile and ranks
// past R repeat valid ones: they only reach results that are not stored.
template <int KIND, int RT, int NR>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(Dev g, const uint16_t* __restrict__ X, RowMap xm,
                                                                int C, const uint16_t* __restrict__ W,
                                                                float* __restrict__ part, int splits, int rchunks) {
  constexpr int BM = 16 * RT, RW = 16 * NR + 4;
  __shared__ __align__(16) int sm[cmax(kTableInts, kShrinkWaves * BM * RW)];
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
  for (int n = 0; n < NR; ++n)
    wp[n] = W + ((int64_t)t.e * g.R + min(rc * 64 + n * 16 + c, g.R - 1)) * C;

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
      for (int n = 0; n < NR; ++n) wv[n][i] = in ? ld16(wp[n] + k + i * 8) : u32x4{0, 0, 0, 0};
    }
  };
  if (st0 < st1) load(st0, xb, wb);
#pragma unroll 2
  for (int st = st0; st < st1; ++st) {
    u32x4 xn[RT][4], wn[NR][4];
    if (st + 1 < st1) load(st + 1, xn, wn);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[rt][n] = mfma16<KIND>(wb[n][i], xb[rt][i], acc[rt][n]);
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
constexpr int kOuterWaves = 8;
constexpr int kOuterThreads = 64 * kOuterWaves;
constexpr int kOuterRows = 1024;  // rows a workgroup sums; longer groups are cut and joined

struct Side {
  const float* L;      // [splits][P][R], summed here; times the group's scale
  int splits;
  const uint16_t* X;   // the wide operand
  RowMap xm;
  int C;
  uint16_t* out;       // [E][R][C], or col_major: [E][C][R]
  int col_major;
  float* part;         // [slots][R][C] of the cut groups
  int slabs;           // 128-column slabs
};

// Slot of the partial sums of the chunk that starts at sorted row s: at most
// one first and one later chunk of the groups longer than a chunk start in
// the same kOuterRows rows.
__host__ __device__ constexpr int outer_slot(int s, bool first) { return 2 * (s / kOuterRows) + (first ? 1 : 0); }
__host__ __device__ constexpr int64_t outer_slots(int64_t P) { return P > kOuterRows ? 2 * ((P - 1) / kOuterRows + 1) : 0; }

// Chunks of a group of m rows; a group without rows has one that writes zeros.
__device__ __forceinline__ int chunks_of(int m) { return max(1, (m + kOuterRows - 1) / kOuterRows); }

// dW[r][n] = sum_s (scale L[s][r]) X[row(s)][n] for one chunk of a group's
// rows, 128 columns and 16 NR ranks.  The 8 waves deal the rows in steps of
// 32 (the MFMA's contraction) and meet in LDS.
template <int KIND, int NR>
__global__ __launch_bounds__(kOuterThreads) void outer_kernel(Dev g, Side sa, Side sb, int rchunks) {
  constexpr int NP = kParts<KIND>, CW = 132;
  __shared__ __align__(16) int sm[kOuterWaves * 16 * CW];
  static_assert(kOuterWaves * 16 * CW >= kTableInts, "the schedule fits under the sums");
  __shared__ int rows[kOuterRows];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, c = lane & 15, q = lane >> 4;
  const int slabs = sa.slabs + sb.slabs;
  const int rc = blockIdx.x % rchunks;
  int slab = blockIdx.x / rchunks % slabs, w = blockIdx.x / rchunks / slabs;
  const Side& d = slab < sa.slabs ? sa : sb;
  if (slab >= sa.slabs) slab -= sa.slabs;

  // Work item w: chunk `ch` of group e, the groups' chunks in order.
  int* tab = sm;
  {
    int* scratch = tab + g.E + 1;
    const int per = (g.E + kOuterThreads - 1) / kOuterThreads;
    const int e0 = min(g.E, tid * per), e1 = min(g.E, e0 + per);
    int local = 0, lo, hi;
    for (int e = e0; e < e1; ++e) {
      expert_range(g.offsets, e, g.P, lo, hi);
      local += chunks_of(hi - lo);
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (lane == 63) scratch[wid] = incl;
    __syncthreads();
    int run = incl - local;
    for (int v = 0; v < wid; ++v) run += scratch[v];
    for (int e = e0; e < e1; ++e) {
      tab[e] = run;
      expert_range(g.offsets, e, g.P, lo, hi);
      run += chunks_of(hi - lo);
    }
    if (tid == kOuterThreads - 1) tab[g.E] = run;
    __syncthreads();
  }
  if (w >= tab[g.E]) return;
  int bl = 0, bh = g.E - 1;
  while (bl < bh) {
    const int mid = (bl + bh + 1) >> 1;
    if (tab[mid] <= w) bl = mid; else bh = mid - 1;
  }
  const int e = bl, ch = w - tab[e];
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  const int s0 = lo + ch * kOuterRows, m = min(kOuterRows, hi - s0);
  for (int i = tid; i < (m + 31) / 32 * 32; i += kOuterThreads) {
    const int pair = i < m ? pair_of(g, s0 + i) : -1;
    rows[i] = pair < 0 ? -1 : map_row(d.xm, s0 + i, pair);
  }
  __syncthreads();

  const float sc = scale_of(g, e);
  const int col = min(slab * 128 + c * 8, d.C - 8);
  int rank[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) rank[n] = min(rc * 64 + n * 16 + c, g.R - 1);
  v4f acc[NR][8];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[n][j] = v4f{0.f, 0.f, 0.f, 0.f};
  int f = 0;  // F16: exponent of the wave's scale of L
  bool first = true;
  for (int st = wid * 32; st < m; st += kOuterWaves * 32) {
    u32x4 raw[8];
    float l[NR][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = st + q * 8 + i, row = rows[k];
      raw[i] = row >= 0 ? ld16(d.X + (int64_t)row * d.C + col) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float v = 0.f;
        if (row >= 0)
          for (int sp = 0; sp < d.splits; ++sp) v += d.L[((int64_t)sp * g.P + s0 + k) * g.R + rank[n]];
        l[n][i] = sc * v;
      }
    }
    if (KIND == OUT_F16) {
      float big = 0.f;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = __builtin_fabsf(l[n][i]);
          big = u < __builtin_inff() ? fmaxf(big, u) : big;
        }
      if (first || __any(ldexp2(big, f) > 32768.f)) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
        const int nf = half_exp(big);
        if (!first) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[n][j][i] = ldexp2(acc[n][j][i], nf - f);
        }
        f = nf;
        first = false;
      }
    }
    u32x4 lp[NR][NP];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        uint16_t u0[NP], u1[NP];
        split<KIND>(KIND == OUT_F16 ? ldexp2(l[n][i], f) : l[n][i], u0);
        split<KIND>(KIND == OUT_F16 ? ldexp2(l[n][i + 1], f) : l[n][i + 1], u1);
#pragma unroll
        for (int p = 0; p < NP; ++p) lp[n][p][i / 2] = (u32)u0[p] | ((u32)u1[p] << 16);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u32x4 x = column_of(raw, j);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int p = 0; p < NP; ++p) acc[n][j] = mfma16<KIND>(lp[n][p], x, acc[n][j]);
    }
  }

  // Join the waves 16 ranks at a time: red[wave][rank][column].
  const bool cut = hi - lo > kOuterRows;
  float* red = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* p = red + (wid * 16 + 4 * q + i) * CW + c * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = KIND == OUT_F16 ? ldexp2(acc[n][j][i], -f) : acc[n][j][i];
    }
    __syncthreads();
    // thread: 4 columns of one rank
    const int r = tid >> 5, x = (tid & 31) * 4;
    v4f sum = *reinterpret_cast<v4f*>(red + r * CW + x);
#pragma unroll
    for (int v = 1; v < kOuterWaves; ++v) {
      const v4f o = *reinterpret_cast<v4f*>(red + (v * 16 + r) * CW + x);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += o[j];
    }
    const int rr = rc * 64 + n * 16 + r, cc = slab * 128 + x;
    if (!cut && d.col_major) {  // transposed through wave 0's part of red
      __syncthreads();
      *reinterpret_cast<v4f*>(red + r * CW + x) = sum;
      __syncthreads();
      const int n4 = (tid & 3) * 4, y = tid >> 2, rb = rc * 64 + n * 16 + n4, yc = slab * 128 + y;
      if (rb < g.R && yc < d.C) {
        u32 o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o[j] = (u32)OutT<KIND>::from(red[(n4 + 2 * j) * CW + y]) |
                 ((u32)OutT<KIND>::from(red[(n4 + 2 * j + 1) * CW + y]) << 16);
        *reinterpret_cast<uint2*>(d.out + ((int64_t)e * d.C + yc) * g.R + rb) = make_uint2(o[0], o[1]);
      }
    } else if (rr < g.R && cc < d.C) {
      if (cut) {
        *reinterpret_cast<v4f*>(d.part + ((int64_t)outer_slot(s0, ch == 0) * g.R + rr) * d.C + cc) = sum;
      } else {
        const u32 o0 = (u32)OutT<KIND>::from(sum[0]) | ((u32)OutT<KIND>::from(sum[1]) << 16);
        const u32 o1 = (u32)OutT<KIND>::from(sum[2]) | ((u32)OutT<KIND>::from(sum[3]) << 16);
        *reinterpret_cast<uint2*>(d.out + ((int64_t)e * g.R + rr) * d.C + cc) = make_uint2(o0, o1);
      }
    }
  }
}

// Joins the chunks of the groups longer than one: a thread takes 4 ranks of
// one column, so that both output orders store 4 values at once or in runs.
template <int KIND>
__global__ __launch_bounds__(256) void join_kernel(Dev g, Side sa, Side sb, int blocks_a, int blocks_b) {
  const int per = blocks_a + blocks_b, e = blockIdx.x / per;
  int b = blockIdx.x - e * per;
  const Side& d = b < blocks_a ? sa : sb;
  if (b >= blocks_a) b -= blocks_a;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  if (hi - lo <= kOuterRows) return;
  const int64_t i = (int64_t)b * 256 + threadIdx.x;
  const int r = (int)(i / d.C) * 4, n = (int)(i % d.C);
  if (r >= g.R) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = lo; s < hi; s += kOuterRows) {
    const float* p = d.part + ((int64_t)outer_slot(s, s == lo) * g.R + r) * d.C + n;
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

// --------------------------------------------------------------- transpose
// bt[e][r][n] = b[e][n][r] of the groups with rows: 64 rows of b at a time.
__global__ __launch_bounds__(256) void transpose_kernel(Dev g, const uint16_t* __restrict__ b, int N,
                                                        uint16_t* __restrict__ bt) {
  __shared__ uint16_t tile[64][66];
  const int nblocks = (N + 63) / 64, rblocks = (g.R + 63) / 64;
  const int e = blockIdx.x / (nblocks * rblocks), i = blockIdx.x - e * nblocks * rblocks;
  const int n0 = i / rblocks * 64, r0 = i % rblocks * 64;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  if (lo == hi) return;
  const int rn = min(64, g.R - r0), nn = min(64, N - n0);
  for (int k = threadIdx.x; k < nn * rn; k += 256) {
    const int n = k / rn, r = k - n * rn;
    tile[r][n] = b[((int64_t)e * N + n0 + n) * g.R + r0 + r];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 64 * rn; k += 256) {
    const int r = k >> 6, n = k & 63;
    if (n < nn) bt[((int64_t)e * g.R + r0 + r) * N + n0 + n] = tile[r][n];
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

template <int KIND, int RT, int NR>
hipError_t shrink_launch(const Dev& d, const uint16_t* X, RowMap xm, int C, const uint16_t* W, float* part, int splits,
                         hipStream_t stream) {
  const int rchunks = (d.R + 63) / 64;
  const int64_t grid = max_tiles(d.P, d.E, 16 * RT) * splits * rchunks;
  hipLaunchKernelGGL((shrink_kernel<KIND, RT, NR>), dim3((unsigned)grid), dim3(kShrinkThreads), 0, stream, d, X, xm, C,
                     W, part, splits, rchunks);
  return hipGetLastError();
}

template <int KIND>
hipError_t shrink(const Dev& d, const uint16_t* X, RowMap xm, int C, const uint16_t* W, float* part, int splits,
                  hipStream_t stream) {
  const int nr = rank_tiles(d.R), rt = shrink_rt(d.P, d.E, nr);
  if (nr == 1 && rt == 4) return shrink_launch<KIND, 4, 1>(d, X, xm, C, W, part, splits, stream);
  if (nr == 1 && rt == 2) return shrink_launch<KIND, 2, 1>(d, X, xm, C, W, part, splits, stream);
  if (nr == 1) return shrink_launch<KIND, 1, 1>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2 && rt == 2) return shrink_launch<KIND, 2, 2>(d, X, xm, C, W, part, splits, stream);
  if (nr == 2) return shrink_launch<KIND, 1, 2>(d, X, xm, C, W, part, splits, stream);
  if (rt == 2) return shrink_launch<KIND, 2, 4>(d, X, xm, C, W, part, splits, stream);
  return shrink_launch<KIND, 1, 4>(d, X, xm, C, W, part, splits, stream);
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

template <int KIND, int NR>
hipError_t outer_launch(const Dev& d, const Side& sa, const Side& sb, hipStream_t stream) {
  const int rchunks = (d.R + 63) / 64;
  const int64_t grid = (d.P / kOuterRows + d.E) * (int64_t)(sa.slabs + sb.slabs) * rchunks;
  hipLaunchKernelGGL((outer_kernel<KIND, NR>), dim3((unsigned)grid), dim3(kOuterThreads), 0, stream, d, sa, sb,
                     rchunks);
  return hipGetLastError();
}

template <int KIND>
hipError_t forward(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b, const uint16_t* base,
                   uint16_t* out, float* h, float* ws, hipStream_t stream) {
  const Dev d = dev_args(g);
  const int splits = shrink_splits(g.P, g.E, g.K, g.R);
  float* part = splits == 1 && h ? h : ws;
  hipError_t e = shrink<KIND>(d, x, x_map(g), g.K, a, part, splits, stream);
  if (e != hipSuccess) return e;
  ExpandArgs ea = {part, splits, part == h ? nullptr : h, b, g.N, base, out, g.out_pair, 0, 0, 0, g.p2s};
  return expand<KIND, false>(d, ea, g.out_pair && base != out, stream);
}

// Workspace of the gradients: dh's partial sums, B transposed, and the cut
// groups' partial weight gradients, each at a multiple of 256 bytes.
struct BwdLayout {
  size_t bt, pa, pb, bytes;
};
BwdLayout bwd_layout(int64_t P, int E, int N, int K, int R) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  BwdLayout l;
  l.bt = up((size_t)P * R * sizeof(float) * (P ? shrink_splits(P, E, N, R) : 0));
  l.pa = l.bt + (P ? up((size_t)E * N * R * 2) : 0);
  l.pb = l.pa + up((size_t)outer_slots(P) * R * K * sizeof(float));
  l.bytes = l.pb + up((size_t)outer_slots(P) * R * N * sizeof(float));
  return l;
}

template <int KIND>
hipError_t backward(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                    const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, char* ws, hipStream_t stream) {
  const Dev d = dev_args(g);
  Dev d1 = d;  // without the scale
  d1.scale = nullptr;
  const BwdLayout l = bwd_layout(g.P, g.E, g.N, g.K, g.R);
  float* dh = reinterpret_cast<float*>(ws);
  const int splits = g.P ? shrink_splits(g.P, g.E, g.N, g.R) : 1;
  hipError_t e;
  if (g.P > 0) {
    uint16_t* bt = reinterpret_cast<uint16_t*>(ws + l.bt);
    hipLaunchKernelGGL(transpose_kernel, dim3(g.E * ((g.N + 63) / 64) * ((g.R + 63) / 64)), dim3(256), 0, stream, d, b,
                       g.N, bt);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = shrink<KIND>(d1, dy, o_map(g), g.N, bt, dh, splits, stream)) != hipSuccess) return e;
    if (dx) {
      ExpandArgs ea = {dh, splits, nullptr, a, g.K, nullptr, dx, 0, 0, 0, 0, nullptr};
      if ((e = expand<KIND, true>(d, ea, false, stream)) != hipSuccess) return e;
    }
  }
  const Side sa = {dh, splits, x, x_map(g), g.K, da, 0, reinterpret_cast<float*>(ws + l.pa), (g.K + 127) / 128};
  const Side sb = {h, 1, dy, o_map(g), g.N, db, 1, reinterpret_cast<float*>(ws + l.pb), (g.N + 127) / 128};
  switch (rank_tiles(g.R)) {
    case 1: e = outer_launch<KIND, 1>(d, sa, sb, stream); break;
    case 2: e = outer_launch<KIND, 2>(d, sa, sb, stream); break;
    default: e = outer_launch<KIND, 4>(d, sa, sb, stream); break;
  }
  if (e != hipSuccess || g.P <= kOuterRows) return e;
  const int ba = (int)(((int64_t)g.K * (g.R / 4) + 255) / 256), bb = (int)(((int64_t)g.N * (g.R / 4) + 255) / 256);
  hipLaunchKernelGGL(join_kernel<KIND>, dim3((unsigned)(g.E * (ba + bb))), dim3(256), 0, stream, d, sa, sb, ba, bb);
  return hipGetLastError();
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
  const int64_t slabs = (N + 127) / 128 + (K + 127) / 128;
  return (P / kOuterRows + E) * slabs * rchunks * kOuterThreads <= kThreadsMax &&
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
