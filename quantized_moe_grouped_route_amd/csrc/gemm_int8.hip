// W8A8 INT8 grouped GEMM with per-token x per-channel scales, and its
// gradient towards the activations.
//
// Forward:  acc[s][n] = sum_k a[row(s)][k] w[e][n][k]   (int32, exact)
//           y = a_scale * w_scale * acc, optionally silu(gate) * up.
// Gradient: dx[s][k] = sum_n dy[s][n] w_scale[e][n] w[e][n][k]  (+ base)
// The int8 MFMA takes w as it is stored in both.  For the gradient a first
// kernel writes d = dy * w_scale, an fp32 value, as 24-bit fixed point of its
// row's largest value, d = step (65536 hi + 256 mid + lo) with a code of at most
// 8355711, in three int8 planes; the planes' products with w are exact int32
// sums, joined in fp32.  So the sums lose no more than fp32 products and sums
// would: d is off by 2^-24 of its row's largest, its own fp32 rounding there.
// Two planes (16 bits) would be half again as fast, but where one column is 100
// times the others they lose more than f16's own rounding.  Three int8 MFMAs
// take as long as one and a half bf16 MFMAs and need no conversion of w in the
// loop; d's 24 bits would take three bf16 operands.
//
// Measured, 8 experts, 16384 rows, f16: gate+up 4096 -> 28672 with SiLU 1.58-1.71
// ms (2.26-2.44 POP/s; the MFMAs alone take 1.15 ms at the clock that they are
// left), its gradient 5.51-5.58 ms with the planes' 0.49 (two planes: 3.67-3.77).
// 256 experts, 32768 rows under Zipf, gradient 7168 -> 2048, bf16: 1.90-1.92 ms
// with the planes' 0.25 (two planes: 1.54-1.59), 7.6 GB read past the L2s at 4.5
// TB/s.  8 tokens to 8 of 256 experts, 7168 -> 4096: 241-253 us, the weights at 6.7
// to 7.0 TB/s.
#include <algorithm>
#include <type_traits>

#include "int8.h"
#include "kernels.h"
#include "pipeline.h"
#include "tile.h"
#include "vec8.h"

namespace moeq {
namespace {

enum Mode { NONE = 0, SILU = 1, GRAD = 2 };

constexpr int kRowBytes = 128;  // K (GRAD: N) values of a row per stage: one cache line
constexpr int kGroupM = 4;      // m-tiles per n-tile sweep

constexpr int kPlanes = 3;      // int8 digits of a gradient's value: hi, mid, lo

// WM x WN waves; a wave owns XO 16-row operands of the A tile and WO 16-wide
// operands of the weight tile.  GRAD: A operands 3i, 3i + 1, 3i + 2 of a wave
// hold the hi, mid and lo plane of its i-th 16 rows.
template <int WM_, int WN_, int XO_, int WO_, int STAGES_>
struct Cfg {
  static constexpr int WM = WM_, WN = WN_, XO = XO_, WO = WO_, kStages = STAGES_;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kBM = 16 * XO * WM;                   // A tile rows
  static constexpr int kBN = 16 * WO * WN;                   // weight rows of a tile (GRAD: weight columns)
  // 1 KB copies (8 rows) per wave, the same for every wave: a tile of 96 rows
  // and 8 waves has 32 rows more that nobody reads
  static constexpr int kCopiesA = (kBM / 8 + kWaves - 1) / kWaves;
  static constexpr int kATile = kCopiesA * 8 * kWaves * kRowBytes;
  static constexpr int kStageBytes = kATile + kBN * kRowBytes;
  static constexpr int kCopiesB = kBN / 8 / kWaves;
  static constexpr int kCopies = kCopiesA + kCopiesB;
  static constexpr int kRW = 8 * kCopiesA;                   // A rows per wave
  static constexpr int kCW = kBN / kWaves;                   // weight-scale columns per wave
  static constexpr int kScaleBytes = kWaves * 256;           // [waves][32 row | 32 column scales]
  // Tile t's scales are read at its epilogue, after its last stage; by then
  // at most kStages later tiles have been issued.
  static constexpr int kScaleBufs = kStages + 1;
  static constexpr int kWaveCols = 16 * WO;
  // Whether both substeps' operands fit in registers beside the accumulators.
  static constexpr bool kDouble = XO * WO <= 16;
  static_assert((kBN == 256 || kBN == 128) && kCW <= 32 && kRW <= 32, "scale and weight layouts");
  static_assert(kBM % 8 == 0 && kCopiesB * 8 * kWaves == kBN, "copies cover the tile");
};

typedef __attribute__((address_space(4))) const int cint_t;
typedef int i32x8_a4 __attribute__((ext_vector_type(8), aligned(4)));
typedef __attribute__((address_space(4))) const i32x8_a4 ci32x8_t;
// Wave-uniform reads through the constant address space (scalar loads).
__device__ __forceinline__ int ld_uniform(const int* p, int64_t i) { return ((cint_t*)(p))[i]; }
__device__ __forceinline__ i32x8_a4 ld_uniform8(const int* p) { return *(ci32x8_t*)(p); }

__device__ __forceinline__ v4i mfma_i8_16x16x64(v4i a, v4i b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

struct TileAt {
  int e, row0, rows, nt;
};

// Work item -> tile, wave-uniform: expert-major, and inside an expert
// kGroupM m-tiles are visited for each n-tile before the next n-tile (1, 2, 4, 8
// of them: 1.73, 1.65, 1.62, 1.66 ms for the Mixtral-sized product above, when
// it took 1.62; 1.59, 1.56, 1.56, 1.54 for the gradient under Zipf, when it had
// two planes).
__device__ __forceinline__ TileAt tile_at(const int* tile_start, const int* __restrict__ offsets, int E, int P,
                                          int first, int bm, int n_tiles, int item) {
  int bl = 0, bh = E - 1;
  while (bl < bh) {
    const int mid = (bl + bh + 1) >> 1;
    if (__builtin_amdgcn_readfirstlane(tile_start[mid]) <= item) bl = mid; else bh = mid - 1;
  }
  const int e = __builtin_amdgcn_readfirstlane(bl);
  const int local = item - __builtin_amdgcn_readfirstlane(tile_start[e]);
  const int lo = min(max(ld_uniform(offsets, e), first) - first, P);
  const int hi = max(min(max(ld_uniform(offsets, e + 1), first) - first, P), lo);
  const int m = hi - lo;
  const int mtiles = tiles_of(m, bm);
  const int group = local / (kGroupM * n_tiles);
  const int in_group = local - group * kGroupM * n_tiles;
  const int gm = min(kGroupM, mtiles - group * kGroupM);
  const int mt = group * kGroupM + in_group % gm;
  return TileAt{e, lo + mt * bm, min(bm, m - mt * bm), in_group / gm};
}

// Expert-local weight row of tile row rb.  SILU: a wave's first half are gate
// rows, its second half the up rows of the same columns.  Rows past N are
// clamped (their outputs are not stored).
template <class C, int MODE>
__device__ __forceinline__ int weight_row(int nt, int rb, int N) {
  if (MODE == SILU) {
    constexpr int W = C::kWaveCols, H = W / 2;
    const int I = N / 2;
    int col = nt * (C::kBN / 2) + H * (rb / W) + rb % H;
    if (col >= I) col = nt * (C::kBN / 2);
    return (rb / H % 2) * I + col;
  }
  const int r = nt * C::kBN + rb;
  return r < N ? r : nt * C::kBN;
}

typedef __attribute__((address_space(3))) v2i_t lds_v2i;

// Operands of one 64-value substep j (two per stage): lane l holds row l % 16
// and the 16 values of chunk 4j + l / 16 of its row.  LDS rows are 128 bytes,
// chunk c of row r at c ^ ((r >> 1) & 7): 16 consecutive rows reading one chunk
// land on 16 bank groups.
template <class C>
__device__ __forceinline__ v4i read_x(const uint8_t* As, int wm, int lane, int j, int o) {
  const int r = 16 * (C::XO * wm + o) + (lane & 15);
  return __builtin_bit_cast(v4i, ld16(As + r * kRowBytes + (((4 * j + (lane >> 4)) ^ ((lane >> 1) & 7)) << 4)));
}
// GRAD: the weight tile is [128 n][kBN k] and a transposing read gives lane i
// of each 16 column i of the 8 x 16 block whose row i/2, half i%2 it points at.
// Chunk c of row n stands at c ^ key(n): the 8 rows of a block, and the blocks
// 16 rows further down that the next 16 lanes read, on different banks.
template <class C>
__device__ __forceinline__ int grad_key(int n) {
  return C::kBN == 256 ? (2 * (n & 7)) ^ ((n >> 4) & 1) : ((n >> 1) & 3) ^ (((n >> 4) & 1) << 2);
}
template <class C, int MODE>
__device__ __forceinline__ v4i read_w(const uint8_t* As, int wn, int lane, int j, int o) {
  const uint8_t* Bs = As + C::kATile;
  if constexpr (MODE == GRAD) {
    const int i = lane & 15, g = lane >> 4;
    const int n = 16 * g + (i >> 1);
    const uint8_t* row = Bs + (64 * j + n) * C::kBN + 8 * (i & 1) + (((C::WO * wn + o) ^ grad_key<C>(n)) << 4);
    const v2i_t a = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)row);
    const v2i_t b = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(row + 8 * C::kBN));
    return v4i{a[0], a[1], b[0], b[1]};
  } else {
    const int r = C::kWaveCols * wn + 16 * o + (lane & 15);
    return __builtin_bit_cast(v4i, ld16(Bs + r * kRowBytes + (((4 * j + (lane >> 4)) ^ ((lane >> 1) & 7)) << 4)));
  }
}

// The WO x NX products of one substep, its reads of another substep's operands
// (read(0 .. WO + NX - 1)) and copies (copy(0 .. kCopies - 1)) spread over them
// in a pinned order: the reads over the first half, so that they are there in
// time.
template <class C, int NX, class Read, class Copy>
__device__ __forceinline__ void mma_reading(v4i (&acc)[C::WO][NX ? NX : 1], const v4i (&w)[C::WO],
                                            const v4i (&x)[NX ? NX : 1], Read read, Copy copy) {
  constexpr int kM = C::WO * NX, kR = C::WO + NX;
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    acc[m / NX][m % NX] = mfma_i8_16x16x64(w[m / NX], x[m % NX], acc[m / NX][m % NX]);
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if (r * (kM / 2) / kR == m) read(r);
#pragma unroll
    for (int i = 0; i < C::kCopies; ++i)
      if (i * kM / C::kCopies == m) copy(i);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int OUT>
__device__ __forceinline__ void put4(void* out, int64_t idx, const float (&o)[4]) {
  typedef typename OutT<OUT>::T T;
  T* dst = static_cast<T*>(out) + idx;
  if constexpr (sizeof(T) == 2) {
    u32 w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (u32)OutT<OUT>::from(rounded(o[2 * i])) | ((u32)OutT<OUT>::from(rounded(o[2 * i + 1])) << 16);
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<v4f*>(dst) = v4f{o[0], o[1], o[2], o[3]};
  }
}

struct Int8Args {
  const uint8_t* a;        // activations, or the planes of d
  const float* a_scale;    // per activation row, or step per sorted row
  const uint8_t* w;
  const float* w_scale;    // not read by GRAD
  const int* offsets;
  const int* sorted_ids;   // or null
  const void* base;        // GRAD: added to dx, or null
  void* out;
  int64_t rows_a;
  int a_sorted, topk, E, P, N, K;
  int first;               // sorted row that a, base and out begin at (GRAD: of a round of rows)
};

// An accumulator with its scales.  The weight's goes first: an accumulator is zero
// or at least 1 and below 2^31, so that only a w_scale past 2^96 can leave fp32's
// range before the result does, whatever a_scale is.  (a_scale * w_scale first
// made NaN of accumulators of zero, and lost the bits of small products.)
__device__ __forceinline__ float scaled(int acc, float w_scale, float a_scale) {
  return a_scale * (w_scale * (float)acc);
}

// Epilogue of one tile: value i of accumulator [wo][xo] in lane l is weight
// row kWaveCols wn + 16wo + 4(l/16) + i of the tile and A row 16(XO wm + xo) +
// l%16.
template <class C, int OUT, int MODE, int NX>
__device__ __forceinline__ void epilogue(const TileAt& t, const float* sb, int wm, int wn, int lane, const Int8Args& g,
                                         const v4i (&acc)[C::WO][NX]) {
  constexpr int kP = MODE == GRAD ? kPlanes : 1;  // A operands per 16 routed rows
  const int l16 = lane & 15, m0 = 4 * (lane >> 4);
  // every scale first: read one by one they cost a trip to LDS per operand
  v4f sw[C::WO];
  float sa[NX];
#pragma unroll
  for (int wo = 0; wo < C::WO; ++wo) {
    const int c = C::kWaveCols * wn + 16 * wo + m0;
    if (MODE != GRAD) sw[wo] = *reinterpret_cast<const v4f*>(sb + 32 + (c / C::kCW) * 64 + c % C::kCW);
  }
#pragma unroll
  for (int xo = 0; xo < NX; xo += kP) {
    const int ar = 16 * (C::XO * wm + xo) + l16;  // row of the A tile
    sa[xo] = sb[(ar / C::kRW) * 64 + ar % C::kRW];
  }
#pragma unroll
  for (int xo = 0; xo < NX; xo += kP) {
    const int r = 16 * ((C::XO * wm + xo) / kP) + l16;  // row of the tile's routed rows
    if (r >= t.rows) continue;
    const int64_t orow = t.row0 + r;
    if constexpr (MODE == SILU) {
      constexpr int H = C::WO / 2;
      const int I = g.N / 2;
#pragma unroll
      for (int wo = 0; wo < H; ++wo) {
        const int col0 = t.nt * (C::kBN / 2) + C::kWaveCols / 2 * wn + 16 * wo + m0;
        if (col0 >= I) continue;
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = silu<OUT>(scaled(acc[wo][xo][i], sw[wo][i], sa[xo])) * scaled(acc[wo + H][xo][i], sw[wo + H][i], sa[xo]);
        put4<OUT>(g.out, orow * I + col0, o);
      }
    } else {
#pragma unroll
      for (int wo = 0; wo < C::WO; ++wo) {
        const int col0 = t.nt * C::kBN + C::kWaveCols * wn + 16 * wo + m0;
        if (col0 >= (MODE == GRAD ? g.K : g.N)) continue;
        if constexpr (MODE == GRAD) {
          float b[4] = {0.f, 0.f, 0.f, 0.f}, o[4];
          const int64_t idx = orow * g.K + col0;
          if (g.base) {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g.base) + idx);
            const u32 v[2] = {q.x, q.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const u32 bits = i & 1 ? v[i >> 1] >> 16 : v[i >> 1] & 0xffffu;
              b[i] = OUT == OUT_BF16 ? bf16_bits_to_f32(bits) : f16_bits_to_f32((uint16_t)bits);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float hm = __builtin_fmaf((float)acc[wo][xo][i], 256.0f, (float)acc[wo][xo + 1][i]);
            o[i] = __builtin_fmaf(__builtin_fmaf(hm, 256.0f, (float)acc[wo][xo + 2][i]), sa[xo], b[i]);
          }
          put4<OUT>(g.out, idx, o);
        } else if constexpr (OUT == OUT_I32) {
          *reinterpret_cast<v4i*>(static_cast<int*>(g.out) + orow * g.N + col0) = acc[wo][xo];
        } else {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = scaled(acc[wo][xo][i], sw[wo][i], sa[xo]);
          put4<OUT>(g.out, orow * g.N + col0, o);
        }
      }
    }
  }
}

template <class C, int OUT, int MODE>
__global__ __launch_bounds__(C::kThreads, 1) void int8_tiles(Int8Args g) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[C::kStages * C::kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t sbuf[C::kScaleBufs * C::kScaleBytes];
  __shared__ int tile_start[kMaxExperts + 1];
  __shared__ int sched_scratch[2 * kMaxWaves];

  constexpr int kBMt = MODE == GRAD ? C::kBM / kPlanes : C::kBM;  // routed rows per tile
  // The dies start their sums an eighth of K apart (exact sums: any order gives
  // the same bits).  Starting together they all read the same columns of rows K
  // apart, on the same few memory channels where K is a power of two: 32 experts
  // of 4096 x 4096 with 64 rows each take 131 us, staggered 111; 8 of 8192 x
  // 8192 126, 99; K = 1536, 7168 and 14336 the same within 2 %.  Large's calls
  // are not held by the channels (no gain), the gradient's go down the rows
  // (1 to 2 % slower).
  constexpr bool kStagger = MODE != GRAD && C::kDouble;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / C::WN, wn = wid % C::WN;
  const int N = g.N, K = g.K, P = g.P, E = g.E;
  const int cols = MODE == SILU ? N / 2 : MODE == GRAD ? K : N;
  const int n_tiles = MODE == SILU ? (cols + C::kBN / 2 - 1) / (C::kBN / 2) : (cols + C::kBN - 1) / C::kBN;
  const int a_pitch = MODE == GRAD ? plane_pitch(N) : K;
  const int steps = a_pitch / kRowBytes;
  const bool ragged = N % kRowBytes != 0;  // GRAD: the last stage ends inside
  const int row_base = MODE == GRAD ? g.first : 0;
  sched_build(tile_start, sched_scratch, g.offsets, E, P, kBMt, n_tiles, row_base);
  const int total = __builtin_amdgcn_readfirstlane(tile_start[E]);
  const int G = gridDim.x;
  const int first = xcd_logical_id(blockIdx.x, G);
  if (first >= total) return;

  // ---- issue cursor: sources of the next stage to copy.  Wave w copies A
  // rows [kRW w, +kRW) and weight rows (GRAD: n rows) of its own.
  const uint8_t* pa[C::kCopiesA];
  const uint8_t* pb[C::kCopiesB];
  const float* psc = g.a_scale;
  int is_item = first, is_step = 0, is_sbuf = 0;
  // kStagger: where the tiles' sums start, and the sources' move to their next
  // stage (at the last one back to stage 0)
  const int phase = kStagger ? (int)((blockIdx.x & 7) * steps) >> 3 : 0;
  int is_pos = phase;
  int64_t move = kStagger && phase == steps - 1 ? kRowBytes - K : kRowBytes;
  auto set_tile = [&](int item) __attribute__((always_inline)) {
    const TileAt t = tile_at(tile_start, g.offsets, E, P, row_base, kBMt, n_tiles, item);
    int arow[C::kCopiesA];
#pragma unroll
    for (int i = 0; i < C::kCopiesA; ++i) {
      const int r0 = C::kRW * wid + 8 * i;  // A tile row of the copy's first row
      const int chunk = dma_chunk(lane, r0 / 8);
      if constexpr (MODE == GRAD) {
        // a copy's 8 rows lie in one 16-row operand, hence in one plane
        static_assert(C::XO == 2 * kPlanes, "a wave owns two groups of 16 rows");
        const int op = r0 / 16;
        arow[i] = t.row0 + min(16 * (op / kPlanes) + r0 % 16 + (lane >> 3), t.rows - 1);
        pa[i] = g.a + ((int64_t)(op % kPlanes) * P + arow[i]) * a_pitch + chunk;
      } else {
        int r;
        if (g.a_sorted || g.sorted_ids == nullptr) {
          r = t.row0 + min(r0 + (lane >> 3), t.rows - 1);
        } else {
          // the copy's 8 sorted ids (one 32-byte scalar load when all 8 rows
          // are in the tile); each lane picks its own
          i32x8_a4 ids;
          if (r0 + 8 <= t.rows) {
            ids = ld_uniform8(g.sorted_ids + t.row0 + r0);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) ids[k] = ld_uniform(g.sorted_ids, t.row0 + min(r0 + k, t.rows - 1));
          }
          int v = ids[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) v = (lane >> 3) == k ? ids[k] : v;
          r = v / g.topk;
        }
        arow[i] = (r < 0 || r >= g.rows_a) ? 0 : r;
        pa[i] = g.a + (int64_t)arow[i] * a_pitch + chunk + phase * kRowBytes;
      }
    }
#pragma unroll
    for (int i = 0; i < C::kCopiesB; ++i) {
      const int q = C::kCopiesB * wid + i;
      if constexpr (MODE == GRAD) {
        // kN rows n of the stage, kBN / 16 chunks of 16 columns each
        constexpr int kChunks = C::kBN / 16, kN = 64 / kChunks;
        const int n = kN * q + lane / kChunks;
        int col = t.nt * C::kBN + 16 * ((lane % kChunks) ^ grad_key<C>(n));
        if (col >= K) col -= 128;  // K is a multiple of 128: only the upper half of 256 may be past it
        pb[i] = g.w + ((int64_t)t.e * N + n) * K + col;
      } else {
        pb[i] = g.w + ((int64_t)t.e * N + weight_row<C, MODE>(t.nt, 8 * q + (lane >> 3), N)) * K + dma_chunk(lane, q) +
                phase * kRowBytes;
      }
    }
    // scales: lanes 0..31 the wave's A rows (row l of them was gathered by
    // copy l / 8, whose lanes 8 (l % 8) .. +7 hold it), 32..63 its columns
    const int lr = lane % C::kRW, src = 8 * (lr & 7);
    int s = __shfl(arow[0], src, 64);
#pragma unroll
    for (int i = 1; i < C::kCopiesA; ++i) {
      const int v = __shfl(arow[i], src, 64);
      s = (lr >> 3) == i ? v : s;
    }
    psc = MODE != GRAD && lane >= 32
              ? g.w_scale + (int64_t)t.e * N + weight_row<C, MODE>(t.nt, C::kCW * wid + lane % C::kCW, N)
              : g.a_scale + s;
  };
  const uint32_t ring_lds = lds_addr(ring), sbuf_lds = lds_addr(sbuf);
  // Copy i of this wave's share of the cursor's stage, into the slot at `base`;
  // its source moves on to the next stage.
  const int64_t b_step = MODE == GRAD ? (int64_t)kRowBytes * K : kRowBytes;
  auto copy = [&](uint32_t base, int i) __attribute__((always_inline)) {
    if (i < C::kCopiesA) {
      dma16(pa[i], __builtin_amdgcn_readfirstlane(base + (C::kCopiesA * wid + i) * 1024));
      pa[i] += kStagger ? move : kRowBytes;
    } else {
      const int q = C::kCopiesB * wid + i - C::kCopiesA;
      const uint8_t* src = pb[i - C::kCopiesA];
      if (MODE == GRAD && ragged && is_step == steps - 1) {
        // rows past N meet zeros of the planes, so any row's bytes do: the
        // stage's rows n % 32 are there, N being a multiple of 32
        const int n = 1024 / C::kBN * q;
        if (is_step * kRowBytes + n >= N) src -= (int64_t)(n & ~31) * K;
      }
      dma16(src, __builtin_amdgcn_readfirstlane(base + C::kATile + q * 1024));
      pb[i - C::kCopiesA] += kStagger ? move : b_step;
    }
  };
  // After a stage's copies: a tile's scales ride with its first stage, and the
  // cursor moves on.  Past the last tile it goes over that tile again, into
  // slots that nobody reads: every wave then waits for constant counts.
  const int last_item = first + (total - 1 - first) / G * G;
  auto advance = [&]() __attribute__((always_inline)) {
    if (is_step == 0) {
      dma4(psc, __builtin_amdgcn_readfirstlane(sbuf_lds + is_sbuf * C::kScaleBytes + wid * 256));
      is_sbuf = is_sbuf == C::kScaleBufs - 1 ? 0 : is_sbuf + 1;
    }
    if constexpr (kStagger) {
      is_pos = is_pos == steps - 1 ? 0 : is_pos + 1;
      move = is_pos == steps - 1 ? kRowBytes - K : kRowBytes;
    }
    if (++is_step == steps) {
      is_step = 0;
      if (C::kBN == 128 && is_item >= last_item) {
        // the same sources without a look-up, in the tile of short calls: 7.4 us
        // for 8.5 with 128 rows and 4 experts of 256 x 256 (the branch costs
        // long calls 4 % in Large, 0.5 % in Medium)
        if constexpr (!kStagger) {  // (kStagger: they are back by themselves)
#pragma unroll
          for (int i = 0; i < C::kCopiesA; ++i) pa[i] -= a_pitch;
#pragma unroll
          for (int i = 0; i < C::kCopiesB; ++i) pb[i] -= steps * b_step;
        }
      } else {
        is_item += G;
        set_tile(min(is_item, last_item));
      }
    }
  };
  // Stage q is there once at most `newer` later stages of this wave's copies
  // are in flight (a scale copy among them only lengthens the wait) and every
  // wave has said so; the stage before it has then been read by all.
  auto arrive = [&](auto newer) __attribute__((always_inline)) {
    wait_vmcnt<decltype(newer)::value * C::kCopies>();
    raw_barrier();
  };

  set_tile(first);
#pragma nounroll
  for (int s = 0; s < C::kStages; ++s) {
#pragma unroll
    for (int i = 0; i < C::kCopies; ++i) copy(ring_lds + s * C::kStageBytes, i);
    advance();
  }
  arrive(std::integral_constant<int, C::kStages - 1>());

  // One tile of a wave with NX A operands in use (those of rows past a partial
  // tile's last are left out: the tile then costs its copies, not its MFMAs).
  //
  // Per stage: the 64-value substeps 0 and 1, each WO passes over the A
  // operands with one weight operand.  An operand's registers take its next
  // substep's values right after its last use (weights after their pass, A
  // operands in the last pass), so 48 registers hold the fragments.  The
  // barrier comes after substep 1's first pass, when all of the stage has been
  // read: the next stage's reads and the copies into this stage's slot are
  // spread over the passes that remain.  (kDouble: both substeps' operands have
  // registers, and the barrier stands between them.)  The order is pinned: left
  // to itself the compiler gathers the reads, and the matrix cores wait for them
  // (2.07 ms for 1.85, before the wider stages and the other MFMA).
  int slot = 0, ep_sbuf = 0;
  auto run_tile = [&](const TileAt& t, auto operands) __attribute__((always_inline)) {
    constexpr int NX = decltype(operands)::value, NA = NX ? NX : 1;
    const uint8_t* As = ring + slot * C::kStageBytes;
    v4i x[NA], w[C::WO], acc[C::WO][NA];
#pragma unroll
    for (int wo = 0; wo < C::WO; ++wo) {
#pragma unroll
      for (int xo = 0; xo < NX; ++xo) acc[wo][xo] = v4i{};
      if (NX) w[wo] = read_w<C, MODE>(As, wn, lane, 0, wo);
    }
#pragma unroll
    for (int xo = 0; xo < NX; ++xo) x[xo] = read_x<C>(As, wm, lane, 0, xo);
    v4i x1[NA], w1[C::WO];  // kDouble
    int st = 0;
    do {
      if constexpr (C::kDouble) {
        mma_reading<C, NX>(acc, w, x, [&](int r) __attribute__((always_inline)) {
          if (r < C::WO) w1[r] = read_w<C, MODE>(As, wn, lane, 1, r);
          else x1[r - C::WO] = read_x<C>(As, wm, lane, 1, r - C::WO);
        }, [](int) {});
      } else {
#pragma unroll
        for (int wo = 0; wo < (NX ? C::WO : 0); ++wo) {
#pragma unroll
          for (int xo = 0; xo < NX; ++xo) {
            acc[wo][xo] = mfma_i8_16x16x64(w[wo], x[xo], acc[wo][xo]);
            if (wo == C::WO - 1) x[xo] = read_x<C>(As, wm, lane, 1, xo);
            __builtin_amdgcn_sched_barrier(0);
          }
          w[wo] = read_w<C, MODE>(As, wn, lane, 1, wo);
        }
#pragma unroll
        for (int xo = 0; xo < NX; ++xo) {
          acc[0][xo] = mfma_i8_16x16x64(w[0], x[xo], acc[0][xo]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      arrive(std::integral_constant<int, C::kStages - 2>());
      const uint32_t refill = __builtin_amdgcn_readfirstlane(ring_lds + slot * C::kStageBytes);
      slot = slot == C::kStages - 1 ? 0 : slot + 1;
      As = ring + slot * C::kStageBytes;
      if constexpr (NX == 0) {
#pragma unroll
        for (int i = 0; i < C::kCopies; ++i) copy(refill, i);
      } else if constexpr (C::kDouble) {
        mma_reading<C, NX>(acc, w1, x1, [&](int r) __attribute__((always_inline)) {
          if (r < C::WO) w[r] = read_w<C, MODE>(As, wn, lane, 0, r);
          else x[r - C::WO] = read_x<C>(As, wm, lane, 0, r - C::WO);
        }, [&](int i) __attribute__((always_inline)) { copy(refill, i); });
      } else {
        w[0] = read_w<C, MODE>(As, wn, lane, 0, 0);
        constexpr int kRest = (C::WO - 1) * NX;
#pragma unroll
        for (int wo = 1; wo < C::WO; ++wo) {
#pragma unroll
          for (int xo = 0; xo < NX; ++xo) {
            acc[wo][xo] = mfma_i8_16x16x64(w[wo], x[xo], acc[wo][xo]);
            if (wo == C::WO - 1) x[xo] = read_x<C>(As, wm, lane, 0, xo);
#pragma unroll
            for (int i = 0; i < C::kCopies; ++i)
              if (i * kRest / C::kCopies == (wo - 1) * NX + xo) copy(refill, i);
            __builtin_amdgcn_sched_barrier(0);
          }
          w[wo] = read_w<C, MODE>(As, wn, lane, 0, wo);
        }
      }
      advance();
    } while (++st < steps);
    if constexpr (NX > 0)
      epilogue<C, OUT, MODE, NX>(t, reinterpret_cast<const float*>(sbuf + ep_sbuf * C::kScaleBytes), wm, wn, lane, g,
                                 acc);
    wait_vmcnt<0>();  // the stores leave before the next stages are counted
    ep_sbuf = ep_sbuf == C::kScaleBufs - 1 ? 0 : ep_sbuf + 1;
  };
  for (int item = first; item < total; item += G) {
    const TileAt t = tile_at(tile_start, g.offsets, E, P, row_base, kBMt, n_tiles, item);
    const int left = t.rows - kBMt / C::WM * wm;  // routed rows of this wave
    constexpr int kRows = kBMt / C::WM;
    if constexpr (MODE == GRAD) {
      if (left > kRows / 2) run_tile(t, std::integral_constant<int, C::XO>());
      else if (left > 0) run_tile(t, std::integral_constant<int, kPlanes>());
      else run_tile(t, std::integral_constant<int, 0>());
    } else if (left > kRows / 2) run_tile(t, std::integral_constant<int, C::XO>());
    else if (C::XO > 4 && left > kRows / 4) run_tile(t, std::integral_constant<int, C::XO / 2>());
    else if (C::XO > 4 && left > 0) run_tile(t, std::integral_constant<int, C::XO / 4>());
    else if (C::XO <= 4 && left > 0) run_tile(t, std::integral_constant<int, C::XO / 2>());
    else run_tile(t, std::integral_constant<int, 0>());
  }
}

// ------------------------------------------------------------------ decode
// Few routed rows per expert: the weight stream is the whole cost.  The wave
// is the unit of work: item = (at most 16 routed rows of one expert) x (16
// weight rows; SILU: 8 gate rows and the 8 up rows of the same columns).  Per
// K group of 128 values (one cache line of a row) a ring slot of the wave
// holds the 16 weight rows (two whole-line copies of 8 rows) and the activation
// rows (a copy for each 8 that the item has), 16-byte piece p of row r at p ^
// ((r >> 1) & 7).  The item's scales ride in group 0's slot (one
// 4-byte-per-lane copy: lanes 0..15 the rows', 16..31 the weights').  Two
// v_mfma_i32_16x16x64_i8 per group take the weights as the 16-row operand and
// the routed rows as the columns: lane l supplies pieces 2(l/16) and 2(l/16) +
// 1 of row l % 16, value i of lane l is weight row 4(l/16) + i and routed row
// l % 16.  64 rows over 57-60 experts of 4096 x 7168, with SiLU: 247-254 us, 7.0
// TB/s; rings of 5 and 6 groups take 255 and 262.
namespace dd {
constexpr int kM = 16;
constexpr int kRowsW = 16;
constexpr int kWaves = 4;                              // waves per workgroup, independent
constexpr int kDepth = 4;                              // K groups in flight per wave
constexpr int kW = 0, kX = 2048, kS = 4096;            // slot regions
constexpr int kSlot = 4352;
constexpr int kGroupK = 128;
}  // namespace dd

template <int COPIES>
__device__ __forceinline__ void wait_decode(int n) {  // vmcnt(n * COPIES)
  static_assert(dd::kDepth == 4, "wait table");
  if (n <= 0) wait_vmcnt<0>();
  else if (n == 1) wait_vmcnt<COPIES>();
  else if (n == 2) wait_vmcnt<2 * COPIES>();
  else wait_vmcnt<3 * COPIES>();
  asm volatile("" ::: "memory");
}

// Activation row of sorted position `pos`, one of the 8 from `first` on
// (wave-uniform): one scalar load of their ids, moved down where it would pass
// the table's end, and one division.  (Eight loads in turn cost 8 us at the start
// of every item.)
__device__ __forceinline__ int act_row(const int* __restrict__ ids, int topk, int64_t rows_a, int P, int first,
                                       int pos) {
  int r = pos;
  if (ids != nullptr) {
    if (P >= 8) {
      const int at = min(first, P - 8), k = pos - at;
      const i32x8_a4 v = ld_uniform8(ids + at);
      r = v[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) r = k == j ? v[j] : r;
    } else {
      r = ids[pos];
    }
    r /= topk;
  }
  return (r < 0 || r >= rows_a) ? 0 : r;
}

template <int OUT, int MODE>
__global__ __launch_bounds__(64 * dd::kWaves) void int8_decode(Int8Args g) {
  __shared__ int tile_start[kMaxExperts + 1];
  __shared__ int sched_scratch[2 * kMaxWaves];
  __shared__ __attribute__((aligned(1024))) uint8_t ring[dd::kWaves][dd::kDepth][dd::kSlot];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = g.N, K = g.K, P = g.P, E = g.E, I = N / 2;
  const int n_blocks = N / dd::kRowsW;
  sched_build(tile_start, sched_scratch, g.offsets, E, P, dd::kM, n_blocks);
  const int total = __builtin_amdgcn_readfirstlane(tile_start[E]);
  const int active = gridDim.x * dd::kWaves;
  const int wid = blockIdx.x * dd::kWaves + wv;
  const int G = K / dd::kGroupK;
  uint8_t* myring = &ring[wv][0][0];
  const uint32_t lb = lds_addr(myring);
  const int l16 = lane & 15, quarter = lane >> 4;
  const int crow = lane >> 3;  // row of a weight copy, + 8 for the second
  const int cp0 = ((lane & 7) ^ ((crow >> 1) & 7)) << 4;
  const int cp1 = ((lane & 7) ^ (((crow + 8) >> 1) & 7)) << 4;
  const int wkey = (l16 >> 1) & 7;
  const int wf0 = dd::kW + l16 * 128 + (((2 * quarter) ^ wkey) << 4);
  const int wf1 = dd::kW + l16 * 128 + (((2 * quarter + 1) ^ wkey) << 4);
  const int* ids = g.a_sorted ? nullptr : g.sorted_ids;
  // Where K is a power of two, 64 neighbouring waves start their (exact) sums at
  // different groups of it: together they would read the same columns of rows K
  // apart, on the same few memory channels.  8 rows an expert: 32 experts of 4096
  // x 4096 94 us and 85 staggered, 8 of 8192 x 8192 94 and 85; other K lose by
  // it, 64 of 4096 x 7168 284 and 288, 16 of 4096 x 14336 142 and 146.
  const int phase = (K & (K - 1)) == 0 ? (wid & 63) * G >> 6 : 0;

  for (int item = wid; item < total; item += active) {
    // m-tile major, then blocks; every field wave-uniform
    int bl = 0, bh = E - 1;
    while (bl < bh) {
      const int mid = (bl + bh + 1) >> 1;
      if (__builtin_amdgcn_readfirstlane(tile_start[mid]) <= item) bl = mid; else bh = mid - 1;
    }
    const int e = __builtin_amdgcn_readfirstlane(bl);
    const int local = item - __builtin_amdgcn_readfirstlane(tile_start[e]);
    const int lo = min(max(ld_uniform(g.offsets, e), 0), P);
    const int hi = min(max(ld_uniform(g.offsets, e + 1), lo), P);
    const int mt = local / n_blocks;
    const int nb = local - mt * n_blocks;
    const int row0 = lo + mt * dd::kM;
    const int rows = min(dd::kM, hi - row0);
    auto wrow = [&](int rb) __attribute__((always_inline)) {
      return MODE == SILU ? (rb < 8 ? 0 : I) + nb * 8 + (rb & 7) : nb * dd::kRowsW + rb;
    };
    const uint8_t* wbase = g.w + (int64_t)e * N * K;
    const uint8_t* sw0 = wbase + (int64_t)wrow(crow) * K + cp0;
    const uint8_t* sw1 = wbase + (int64_t)wrow(8 + crow) * K + cp1;
    // XC: copies of activation rows, 8 rows each and 8 lanes a row
    auto run_item = [&](auto copies) __attribute__((always_inline)) {
      constexpr int XC = decltype(copies)::value;
      int xrow[XC];
      const uint8_t* sx[XC];
#pragma unroll
      for (int c = 0; c < XC; ++c) {
        xrow[c] = act_row(ids, g.topk, g.rows_a, P, row0 + 8 * c, row0 + min(8 * c + (lane >> 3), rows - 1));
        sx[c] = g.a + (int64_t)xrow[c] * K + (((lane & 7) ^ ((4 * c + (lane >> 4)) & 7)) << 4);
      }
      // row i's number is in lanes 8 (i % 8) .. +7 of xrow[i / 8]; read by
      // every lane, as lanes on both sides of the select below hold it
      const int s0 = __shfl(xrow[0], 8 * (lane & 7), 64), s1 = __shfl(xrow[XC - 1], 8 * (lane & 7), 64);
      const float* ss = lane >= dd::kM && lane < dd::kM + dd::kRowsW
                            ? g.w_scale + (int64_t)e * N + wrow(lane - dd::kM)
                            : g.a_scale + (XC > 1 && lane >= 8 ? s1 : s0);
      auto issue = [&](int k) __attribute__((always_inline)) {
        const uint32_t sl = lb + (uint32_t)((k % dd::kDepth) * dd::kSlot);
        const int kk = k + phase;
        const int64_t ko = (int64_t)(kk < G ? kk : kk - G) * dd::kGroupK;
        dma16_nt(sw0 + ko, sl + dd::kW);
        dma16_nt(sw1 + ko, sl + dd::kW + 1024);
#pragma unroll
        for (int c = 0; c < XC; ++c) dma16(sx[c] + ko, sl + dd::kX + 1024 * c);
        if (k == 0) dma4(ss, sl + dd::kS);
      };
      const int npre = G < dd::kDepth ? G : dd::kDepth;
      for (int k = 0; k < npre; ++k) issue(k);
      const int xslot = l16 < 8 * XC ? l16 : 0;
      const int xkey = (xslot >> 1) & 7;
      const int xf0 = dd::kX + xslot * 128 + (((2 * quarter) ^ xkey) << 4);
      const int xf1 = dd::kX + xslot * 128 + (((2 * quarter + 1) ^ xkey) << 4);
      v4i acc = v4i{};
      float sa = 0.f;
      v4f sw = v4f{};
      for (int k = 0; k < G; ++k) {
        const int after = G - 1 - k;
        wait_decode<2 + XC>(after < dd::kDepth - 1 ? after : dd::kDepth - 1);
        const uint8_t* sp = myring + (k % dd::kDepth) * dd::kSlot;
        const v4i w0 = __builtin_bit_cast(v4i, ld16(sp + wf0)), w1 = __builtin_bit_cast(v4i, ld16(sp + wf1));
        const v4i x0 = __builtin_bit_cast(v4i, ld16(sp + xf0)), x1 = __builtin_bit_cast(v4i, ld16(sp + xf1));
        if (k == 0) {
          const float* s = reinterpret_cast<const float*>(sp + dd::kS);
          sa = s[xslot];
          sw = *reinterpret_cast<const v4f*>(s + dd::kM + 4 * quarter);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read; it may be refilled
        if (k + dd::kDepth < G) issue(k + dd::kDepth);
        acc = mfma_i8_16x16x64(w0, x0, acc);
        acc = mfma_i8_16x16x64(w1, x1, acc);
      }
      const int64_t orow = row0 + l16;
      if constexpr (MODE == SILU) {
        float v[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = scaled(acc[i], sw[i], sa);
          u[i] = __shfl_xor(v[i], 32, 64);  // quarters 0, 1 hold gates, 2, 3 the ups
        }
        if (l16 < rows && quarter < 2) {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = silu<OUT>(v[i]) * u[i];
          put4<OUT>(g.out, orow * I + nb * 8 + 4 * quarter, o);
        }
      } else if (l16 < rows) {
        const int64_t idx = orow * N + nb * dd::kRowsW + 4 * quarter;
        if constexpr (OUT == OUT_I32) {
          *reinterpret_cast<v4i*>(static_cast<int*>(g.out) + idx) = acc;
        } else {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = scaled(acc[i], sw[i], sa);
          put4<OUT>(g.out, idx, o);
        }
      }
    };
    if (rows > 8) run_item(std::integral_constant<int, 2>());
    else run_item(std::integral_constant<int, 1>());
  }
}

// ------------------------------------------------------- gradient's planes
// d[s][n] = dy[s][n] * w_scale[e][n] as step * (65536 hi + 256 mid + lo): step =
// max |d| / 8355711, the code rne(d * (8355711 / max)), its digits from -128 to
// 127.  WAVES waves work on a row, whose d stays in their registers (LOADS times
// 8 values a lane; 0: the row is read twice).  A row whose largest value is below
// 2^-100 counts as zero; one that holds an infinity or NaN gets step NaN, so all
// of its dx is NaN.  The rows are those from `first` on, at most P of them; dy,
// the planes and step begin at the first.
//
// HBM-bound: dy is read once, past the caches, and the three planes are written,
// 16384 rows of 28672 (2.35 GB) in 489-494 us, 4.8 TB/s, 32768 rows of 7168 (1.17
// GB) in 248-254.  Waves a row, timed with two planes (394-422 and 213-225 us): 8
// for rows of 28672 (16: 437, 4: 480), 2 for rows of 7168 (1: 311, 4: 251).

// Expert of sorted row s, by the whole wave: the number of experts that end
// (ends[e], in LDS) at or before it.
__device__ __forceinline__ int expert_of(const int* ends, int E, int s, int lane) {
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    n += __popcll(__ballot(e < E && ends[e] <= s));
  }
  return min(n, E - 1);
}

// The largest code: digits 127, 127, 127.
constexpr float kTopCode = 127 * 65536 + 127 * 256 + 127;

template <int YK, int WAVES, int LOADS>
__global__ __launch_bounds__(64 * (WAVES == 1 ? 4 : WAVES)) void grad_planes(
    const void* __restrict__ dy, const float* __restrict__ w_scale, const int* __restrict__ offsets, int E, int first, int P,
    int N, uint8_t* __restrict__ planes, float* __restrict__ step) {
  constexpr int kRows = WAVES == 1 ? 4 : 1;  // rows of a workgroup at a time
  constexpr int kT = 64 * WAVES;
  __shared__ u32 wmax[WAVES];
  __shared__ int ends[kMaxExperts];
  // in LDS, so that the search for a row's expert does not wait for dy's loads
  for (int e = threadIdx.x; e < E; e += blockDim.x) ends[e] = offsets[e + 1];
  __syncthreads();
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, sub = wid / WAVES, tid = threadIdx.x % kT;
  const int n = min(max(offsets[E], first) - first, P), Np = plane_pitch(N);
  for (int64_t s = (int64_t)blockIdx.x * kRows + sub; s < n; s += (int64_t)gridDim.x * kRows) {
    const int64_t base = s * N;
    float d[LOADS ? LOADS : 1][8];
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        if ((i * kT + tid) * 8 < N) load8<YK, true>(dy, base + (i * kT + tid) * 8, d[i]);
    }
    const float* ws = w_scale + (int64_t)expert_of(ends, E, first + (int)s, lane) * N;
    auto scale8 = [&](int k, float (&v)[8]) __attribute__((always_inline)) {
      float c[8];
      load8<OUT_F32, false>(ws, k, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= c[j];
    };
    u32 m = 0;
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (i * kT + tid) * 8;
        if (k < N) {
          scale8(k, d[i]);
          m = max(m, amax_bits(d[i]));
        }
      }
    } else {
      for (int k = tid * 8; k < N; k += kT * 8) {
        load8<YK, false>(dy, base + k, d[0]);
        scale8(k, d[0]);
        m = max(m, amax_bits(d[0]));
      }
    }
    m = wave_max(m);
    if constexpr (WAVES > 1) {
      static_assert(kRows == 1, "the rows of a workgroup may end in different rounds: no barrier then");
      if (lane == 0) wmax[wid] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) m = max(m, wmax[w]);
      __syncthreads();  // wmax is reused by the next row
    }
    const Scale c = scale_of(m, kTopCode, 0x1p-100f);
    uint8_t* row = planes + s * Np;
    const int64_t plane = (int64_t)P * Np;
    auto put = [&](int k, const float (&v)[8]) __attribute__((always_inline)) {
      u32 w[kPlanes][2] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = code_of(v[j], c.recip, kTopCode);
        w[0][j >> 2] |= ((u32)((q + 0x8080) >> 16) & 255u) << (8 * (j & 3));
        w[1][j >> 2] |= ((u32)((q + 0x80) >> 8) & 255u) << (8 * (j & 3));
        w[2][j >> 2] |= ((u32)q & 255u) << (8 * (j & 3));
      }
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) *reinterpret_cast<uint2*>(row + p * plane + k) = make_uint2(w[p][0], w[p][1]);
    };
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (i * kT + tid) * 8;
        if (k < N) put(k, d[i]);
      }
    } else {
      for (int k = tid * 8; k < N; k += kT * 8) {
        load8<YK, false>(dy, base + k, d[0]);
        scale8(k, d[0]);
        put(k, d[0]);
      }
    }
    if (tid < (Np - N) / 8) {  // the planes' zeros up to a whole stage
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) *reinterpret_cast<uint2*>(row + p * plane + N + 8 * tid) = make_uint2(0, 0);
    }
    if (tid == 0) step[s] = c.scale;
  }
}

// ------------------------------------------------------------------ launch
struct Forward {
  typedef Cfg<2, 4, 8, 4, 2> Large;   // 256 rows x 256 columns
  typedef Cfg<2, 4, 4, 4, 3> Medium;  // 128 x 256
  typedef Cfg<1, 8, 4, 2, 3> Small;   // 64 x 256
  typedef Cfg<1, 4, 4, 2, 5> Narrow;  // 64 x 128
};
struct Gradient {                     // three A rows for a routed row
  typedef Cfg<2, 4, 6, 4, 2> Large;   // 64 routed rows x 256 columns
  typedef Cfg<1, 8, 6, 2, 3> Small;   // 32 x 256
  typedef Cfg<1, 4, 6, 2, 5> Narrow;  // 32 x 128
};

int out_cols(const Int8Args& g, int mode) { return mode == SILU ? g.N / 2 : mode == GRAD ? g.K : g.N; }

template <class C, int MODE>
int64_t n_tiles(const Int8Args& g) {
  const int w = MODE == SILU ? C::kBN / 2 : C::kBN;
  return (out_cols(g, MODE) + w - 1) / w;
}

template <class C, int OUT, int MODE>
hipError_t go_tiles(const Int8Args& g, int num_cus, hipStream_t stream) {
  const int bm = MODE == GRAD ? C::kBM / kPlanes : C::kBM;
  // upper bound on tiles: every expert adds at most one partial m-tile
  const int64_t tiles = (((int64_t)g.P + bm - 1) / bm + std::min(g.E, g.P)) * n_tiles<C, MODE>(g);
  const int grid = (int)std::min<int64_t>(tiles, num_cus);
  hipLaunchKernelGGL((int8_tiles<C, OUT, MODE>), dim3(grid), dim3(C::kThreads), 0, stream, g);
  return hipGetLastError();
}

// Tiles that a compute unit works through, at the least one, with half a
// partial m-tile for every expert, times the time of one relative to Large's.
template <class C, int MODE>
double cost(const Int8Args& g, int num_cus, double one) {
  const double mt = (double)g.P * (MODE == GRAD ? kPlanes : 1) / C::kBM + 0.5 * std::min(g.E, g.P);
  return one * std::max(1.0, mt * (double)n_tiles<C, MODE>(g) / num_cus);
}

// The tile of the least cost.  Relative times of a tile: 1, 0.54, 0.36, 0.22, from
// 32 experts of 4096 x 4096, bf16, each tile forced, 256, 128 and 64 rows x 256 and
// 64 x 128, us: 512 rows each 315, 319, 430 and 520, 128 rows 155, 139, 153 and
// 171, 64 rows 143, 112, 120 and 125, 16 rows 134, 104, 103 and 103 (by the rule
// 512 rows take 128-row tiles, 64 rows 64-row ones).  4 of 256 x 256 with 256 rows:
// 18.6, 12.8, 10.3 and 9.2.
template <int OUT, int MODE>
hipError_t go_prefill(const Int8Args& g, int num_cus, hipStream_t stream) {
  typedef Forward F;
  const double l = cost<F::Large, MODE>(g, num_cus, 1.0), m = cost<F::Medium, MODE>(g, num_cus, 0.54),
               s = cost<F::Small, MODE>(g, num_cus, 0.36), n = cost<F::Narrow, MODE>(g, num_cus, 0.22);
  if (n <= s && n <= m && n <= l) return go_tiles<F::Narrow, OUT, MODE>(g, num_cus, stream);
  if (s <= m && s <= l) return go_tiles<F::Small, OUT, MODE>(g, num_cus, stream);
  if (m <= l) return go_tiles<F::Medium, OUT, MODE>(g, num_cus, stream);
  return go_tiles<F::Large, OUT, MODE>(g, num_cus, stream);
}

// The gradient's tile, as above.  32 experts of 4096 x 4096, bf16, each tile
// forced, 64 x 256, 32 x 256 and 32 x 128, us with the planes: 512 rows each 848,
// 1025 and 1243, 128 rows 267, 304 and 372, 64 rows 202, 191 and 215, 16 rows 124,
// 115 and 131; so 1, 0.62 and 0.37.  4 of 256 x 256 with 256 rows: 14.3, 13.6 and
// 12.1.
template <int OUT>
hipError_t go_gradient(const Int8Args& g, int num_cus, hipStream_t stream) {
  typedef Gradient B;
  const double l = cost<B::Large, GRAD>(g, num_cus, 1.0), s = cost<B::Small, GRAD>(g, num_cus, 0.62),
               n = cost<B::Narrow, GRAD>(g, num_cus, 0.37);
  if (n <= s && n <= l) return go_tiles<B::Narrow, OUT, GRAD>(g, num_cus, stream);
  if (s <= l) return go_tiles<B::Small, OUT, GRAD>(g, num_cus, stream);
  return go_tiles<B::Large, OUT, GRAD>(g, num_cus, stream);
}

// AUTO streams below 10 rows an expert on average: with 32 experts of 4096 x 4096,
// 4 rows each take 83 us streamed and 102 in tiles, 8 rows 84 and 102, 10 rows 87
// and 100, 12 rows 107 and 101, 16 rows 125 and 100 (experts past 16 rows stream
// their weights again); with 256 experts of 2048 x 2048 8 rows take 180 and 185, 10
// rows 191 and 187.  The counts are on the device, so the rule cannot see skewed
// routing, where the large experts' weights stream more than once: under Zipf 4
// rows an expert take 67 and 88 us with the 32 experts, 8 rows 97 and 97; with the
// 256, 129 and 134, 187 and 163.  A caller that knows of stronger skew asks for
// PREFILL.
// And where no wave gets a second item, so that a call is as long as one item:
// one expert of 4096 x 4096 with 64 rows 11 us streamed and 22 in tiles, with 256
// rows 26 and 22.
template <int OUT, int MODE>
hipError_t go(const Int8Args& g, int sched, int num_cus, hipStream_t stream) {
  if (g.P == 0) return hipSuccess;
  const int64_t items = (((int64_t)g.P + dd::kM - 1) / dd::kM + std::min(g.E, g.P)) * (g.N / dd::kRowsW);
  if (sched == 1 || (sched == 0 && (g.P < (int64_t)10 * g.E || items <= (int64_t)num_cus * 2 * dd::kWaves))) {
    hipLaunchKernelGGL((int8_decode<OUT, MODE>), dim3(num_cus * 2), dim3(64 * dd::kWaves), 0, stream, g);
    return hipGetLastError();
  }
  return go_prefill<OUT, MODE>(g, num_cus, stream);
}

Int8Args int8_args(const GroupedArgs& g, const void* a, const float* a_scale, const int8_t* w, const float* w_scale) {
  return Int8Args{static_cast<const uint8_t*>(a), a_scale, reinterpret_cast<const uint8_t*>(w), w_scale, g.offsets,
                  g.sorted_ids, nullptr, g.out, g.rows_a, g.a_sorted, g.topk, g.E, (int)g.P, g.N, g.K, 0};
}

}  // namespace

hipError_t launch_gemm_int8(const GroupedArgs& g, const int8_t* a, const float* a_scale, const int8_t* w,
                            const float* w_scale, hipStream_t stream) {
  const Int8Args k = int8_args(g, a, a_scale, w, w_scale);
  if (g.silu_mul) {
    switch (g.out_kind) {
      case OUT_F16: return go<OUT_F16, SILU>(k, g.sched, g.num_cus, stream);
      case OUT_BF16: return go<OUT_BF16, SILU>(k, g.sched, g.num_cus, stream);
      default: return go<OUT_F32, SILU>(k, g.sched, g.num_cus, stream);
    }
  }
  switch (g.out_kind) {
    case OUT_F16: return go<OUT_F16, NONE>(k, g.sched, g.num_cus, stream);
    case OUT_BF16: return go<OUT_BF16, NONE>(k, g.sched, g.num_cus, stream);
    case OUT_I32: return go<OUT_I32, NONE>(k, g.sched, g.num_cus, stream);
    default: return go<OUT_F32, NONE>(k, g.sched, g.num_cus, stream);
  }
}

// Work items are counted in 32 bits.  Every expert adds at most one partial item,
// and the tiles are fewer than the streamed items (GRAD: than the narrow tiles).
bool int8_fits(int64_t P, int E, int64_t N) {
  return (P / dd::kM + E) * (N / dd::kRowsW) < (1 << 30);
}
bool int8_bwd_fits(int64_t P, int E, int64_t K) {
  typedef Gradient::Narrow C;
  return (P / (C::kBM / kPlanes) + E) * (K / C::kBN) < (1 << 30);
}

// Bytes of the workspace that one row takes: its planes and its step.
static int64_t row_bytes(int N) { return kPlanes * plane_pitch(N) + 4; }

size_t int8_bwd_workspace_bytes(int64_t P, int N) {
  return P == 0 ? 0 : (size_t)std::max(P * (2 * plane_pitch(N) + 4), row_bytes(N));
}
size_t int8_bwd_workspace_most(int64_t P, int N) { return (size_t)(P * row_bytes(N)); }

// One plane and one tile launch for as many rows as the workspace holds: all of
// them, or, with the least workspace, two thirds of them and then the rest.
hipError_t launch_gemm_int8_bwd(const GroupedArgs& g, const void* dy, const int8_t* w, const float* w_scale,
                                const void* base, void* ws, size_t ws_bytes, hipStream_t stream) {
  const bool bf = g.out_kind == OUT_BF16;
  const int64_t room = std::min<int64_t>(ws_bytes / row_bytes(g.N), g.P);
  uint8_t* planes = static_cast<uint8_t*>(ws);
  float* step = reinterpret_cast<float*>(planes + kPlanes * room * plane_pitch(g.N));
  for (int64_t first = 0; first < g.P; first += room) {
    const int P = (int)std::min(room, g.P - first);
    const uint16_t* y = static_cast<const uint16_t*>(dy) + first * g.N;
#define MOEQ_PLANES(WAVES, LOADS)                                                                                  \
  do {                                                                                                             \
    const int64_t rows = WAVES == 1 ? 4 : 1;                                                                       \
    const dim3 grid((int)std::min<int64_t>((P + rows - 1) / rows, g.num_cus * 8)), block(64 * WAVES * rows);       \
    if (bf)                                                                                                        \
      hipLaunchKernelGGL((grad_planes<OUT_BF16, WAVES, LOADS>), grid, block, 0, stream, y, w_scale, g.offsets,     \
                         g.E, (int)first, P, g.N, planes, step);                                                   \
    else                                                                                                           \
      hipLaunchKernelGGL((grad_planes<OUT_F16, WAVES, LOADS>), grid, block, 0, stream, y, w_scale, g.offsets,      \
                         g.E, (int)first, P, g.N, planes, step);                                                   \
  } while (0)
    if (g.N <= 64 * 8 * 4) MOEQ_PLANES(1, 4);
    else if (g.N <= 128 * 8 * 8) MOEQ_PLANES(2, 8);
    else if (g.N <= 512 * 8 * 8) MOEQ_PLANES(8, 8);
    else MOEQ_PLANES(8, 0);
#undef MOEQ_PLANES
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    Int8Args k = int8_args(g, planes, step, w, w_scale);
    k.P = P;
    k.first = (int)first;
    k.base = base ? static_cast<const uint16_t*>(base) + first * g.K : nullptr;
    k.out = static_cast<uint16_t*>(g.out) + first * g.K;
    e = bf ? go_gradient<OUT_BF16>(k, g.num_cus, stream) : go_gradient<OUT_F16>(k, g.num_cus, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moeq
