// The gated activation as a call of its own, for projections whose columns
// change between the GEMM and the activation (adapters), with an 8-bit
// checkpoint of its input, and its gradient:
//   h  = g sig(g) u            sig(g) = 1 / (1 + exp(-g)), rows [g | u]
//   dg = dh u sig (1 + g (1 - sig)),  du = dh g sig
// The checkpoint keeps g and u as int8 codes with an fp32 scale for every 128
// columns of a row (amax / 127): 1.03 bytes a value where 16-bit columns take
// 2.  The gradient reads the columns or the checkpoint, and can give h again,
// with the gradient or alone, before dh exists (what the gradients of the next
// projection's adapters read), so h need not be kept either.
//
// HBM-bound.  16 lanes own a block of 128 columns, 8 columns each, of gate and
// up alike; a workgroup covers 16 blocks of one row, or of several rows where
// a row has fewer.  Rows past the last expert's are left as they are.  16384
// rows of 28672 f16 columns: with the checkpoint 353 us (1.89 GB), the gradient
// and h from it 447 us (2.36 GB), 5.3 TB/s both, above a copy's 5.1.
#include <algorithm>

#include "int8.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kThreadsS = 256;
constexpr int kUnits = kThreadsS / 16;  // blocks of 128 columns per workgroup

// Where this thread works: column `col` (8 of them; none where col >= I) of
// block `block` in row `row`, for work group `item` of 2^lu blocks per row.
struct Place {
  int64_t row;
  int block, col;
};
__device__ __forceinline__ Place place(int64_t item, int chunks, int lu) {
  const int64_t rg = item / chunks;
  const int chunk = (int)(item - rg * chunks), unit = threadIdx.x >> 4;
  const int block = (chunk << lu) + (unit & ((1 << lu) - 1));
  return Place{rg * (kUnits >> lu) + (unit >> lu), block, block * 128 + 8 * (int)(threadIdx.x & 15)};
}

__device__ __forceinline__ u32 max16(u32 m) {  // over the block's 16 lanes
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = max(m, (u32)__shfl_xor((int)m, o, 16));
  return m;
}

template <bool NT>
__device__ __forceinline__ void st8(uint8_t* p, uint2 v) {
  const v2i_t w = {(int)v.x, (int)v.y};
  if (NT) __builtin_nontemporal_store(w, reinterpret_cast<v2i_t*>(p));
  else *reinterpret_cast<v2i_t*>(p) = w;
}

__device__ __forceinline__ int64_t valid_rows(const int* __restrict__ offsets, int E, int64_t P) {
  if (offsets == nullptr) return P;
  return min((int64_t)max(offsets[E], 0), P);
}

template <int XK, bool SAVE, bool NT>
__global__ __launch_bounds__(kThreadsS) void silu_mul_rows(const void* __restrict__ gu,
                                                           const int* __restrict__ offsets, int E, int64_t P, int I,
                                                           int lu, void* __restrict__ h, uint8_t* __restrict__ ck,
                                                           float* __restrict__ cs) {
  const int64_t n = valid_rows(offsets, E, P);
  const int nb = (I + 127) / 128, chunks = (nb + (1 << lu) - 1) >> lu, rpw = kUnits >> lu;
  const int64_t items = (n + rpw - 1) / rpw * chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const Place p = place(item, chunks, lu);
    const bool live = p.row < n && p.col < I;
    float g[8] = {}, u[8] = {};
    const int64_t at = p.row * 2 * I + p.col;
    if (live) {
      load8<XK, NT>(gu, at, g);
      load8<XK, NT>(gu, at + I, u);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rounded(silu<XK>(g[j]) * u[j]);
      store8<XK, NT>(h, p.row * I + p.col, o);
    }
    if constexpr (SAVE) {
      const Scale a = scale_of(max16(amax_bits(g)), 127.0f, 0x1p-120f);
      const Scale b = scale_of(max16(amax_bits(u)), 127.0f, 0x1p-120f);
      if (live) {
        st8<NT>(ck + at, codes8(g, a.recip));
        st8<NT>(ck + at + I, codes8(u, b.recip));
        if ((threadIdx.x & 15) == 0) {
          cs[p.row * 2 * nb + p.block] = a.scale;
          cs[p.row * 2 * nb + nb + p.block] = b.scale;
        }
      }
    }
  }
}

__device__ __forceinline__ void decode8(const uint8_t* p, float scale, float (&v)[8]) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  const u32 w[2] = {q.x, q.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = scale * (float)(int8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// SAVED: g and u from the checkpoint (else from gu).  dh null: h alone.
template <int XK, bool SAVED, bool NT>
__global__ __launch_bounds__(kThreadsS) void silu_mul_grad(const void* __restrict__ dh, const void* gu,
                                                           const uint8_t* __restrict__ ck,
                                                           const float* __restrict__ cs,
                                                           const int* __restrict__ offsets, int E, int64_t P, int I,
                                                           int lu, void* dgu, void* __restrict__ h) {
  const int64_t n = valid_rows(offsets, E, P);
  const int nb = (I + 127) / 128, chunks = (nb + (1 << lu) - 1) >> lu, rpw = kUnits >> lu;
  const int64_t items = (n + rpw - 1) / rpw * chunks;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const Place p = place(item, chunks, lu);
    if (p.row >= n || p.col >= I) continue;
    const int64_t at = p.row * 2 * I + p.col;
    float g[8], u[8], d[8] = {};
    if (dh) load8<XK, NT>(dh, p.row * I + p.col, d);
    if constexpr (SAVED) {
      decode8(ck + at, cs[p.row * 2 * nb + p.block], g);
      decode8(ck + at + I, cs[p.row * 2 * nb + nb + p.block], u);
    } else {
      load8<XK, NT>(gu, at, g);
      load8<XK, NT>(gu, at + I, u);
    }
    float a[8], b[8], o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Sigmoid q = sigmoid<XK>(g[j]);
      const float t = g[j] * q.s;
      a[j] = rounded(d[j] * u[j] * __builtin_fmaf(t, q.c, q.s));
      b[j] = rounded(d[j] * t);
      o[j] = rounded(t * u[j]);
    }
    if (dh) {
      store8<XK, NT>(dgu, at, a);
      store8<XK, NT>(dgu, at + I, b);
    }
    if (h) store8<XK, NT>(h, p.row * I + p.col, o);
  }
}

// log2 of the blocks of one row that a workgroup takes
int log_units(int I) {
  const int nb = (I + 127) / 128;
  int lu = 0;
  while ((1 << lu) < nb && (1 << lu) < kUnits) ++lu;
  return lu;
}
int grid_of(int64_t P, int I, int lu, int num_cus) {
  const int nb = (I + 127) / 128, rpw = kUnits >> lu;
  const int64_t items = (P + rpw - 1) / rpw * ((nb + (1 << lu) - 1) >> lu);
  return (int)std::min<int64_t>(items, (int64_t)num_cus * 16);
}

}  // namespace

hipError_t launch_silu_mul(const void* gu, int kind, const int* offsets, int E, int64_t P, int I, void* h, int8_t* ck,
                           float* cs, int num_cus, hipStream_t stream) {
  if (P == 0) return hipSuccess;
  const int lu = log_units(I), grid = grid_of(P, I, lu, num_cus);
  // streams past the 256 MB Infinity Cache go past it
  const bool nt = P * I * (kind == OUT_F32 ? 4 : 2) * 3 >= (int64_t(256) << 20);
  uint8_t* c = reinterpret_cast<uint8_t*>(ck);
#define MOEQ_SM(XK, SAVE, NT)                                                                                      \
  hipLaunchKernelGGL((silu_mul_rows<XK, SAVE, NT>), dim3(grid), dim3(kThreadsS), 0, stream, gu, offsets, E, P, I, \
                     lu, h, c, cs)
#define MOEQ_SM2(XK)                                                     \
  do {                                                                   \
    if (ck && nt) MOEQ_SM(XK, true, true);                               \
    else if (ck) MOEQ_SM(XK, true, false);                               \
    else if (nt) MOEQ_SM(XK, false, true);                               \
    else MOEQ_SM(XK, false, false);                                      \
  } while (0)
  switch (kind) {
    case OUT_F16: MOEQ_SM2(OUT_F16); break;
    case OUT_BF16: MOEQ_SM2(OUT_BF16); break;
    default: MOEQ_SM2(OUT_F32); break;
  }
#undef MOEQ_SM2
#undef MOEQ_SM
  return hipGetLastError();
}

hipError_t launch_silu_mul_bwd(const void* dh, int kind, const void* gu, const int8_t* ck, const float* cs,
                               const int* offsets, int E, int64_t P, int I, void* dgu, void* h, int num_cus,
                               hipStream_t stream) {
  if (P == 0) return hipSuccess;
  const int lu = log_units(I), grid = grid_of(P, I, lu, num_cus);
  const bool nt = P * I * (kind == OUT_F32 ? 4 : 2) * 3 >= (int64_t(256) << 20);
  const uint8_t* c = reinterpret_cast<const uint8_t*>(ck);
#define MOEQ_SB(XK, SAVED, NT)                                                                                     \
  hipLaunchKernelGGL((silu_mul_grad<XK, SAVED, NT>), dim3(grid), dim3(kThreadsS), 0, stream, dh, gu, c, cs,       \
                     offsets, E, P, I, lu, dgu, h)
#define MOEQ_SB2(XK)                                                     \
  do {                                                                   \
    if (ck && nt) MOEQ_SB(XK, true, true);                               \
    else if (ck) MOEQ_SB(XK, true, false);                               \
    else if (nt) MOEQ_SB(XK, false, true);                               \
    else MOEQ_SB(XK, false, false);                                      \
  } while (0)
  switch (kind) {
    case OUT_F16: MOEQ_SB2(OUT_F16); break;
    case OUT_BF16: MOEQ_SB2(OUT_BF16); break;
    default: MOEQ_SB2(OUT_F32); break;
  }
#undef MOEQ_SB2
#undef MOEQ_SB
  return hipGetLastError();
}

}  // namespace moeq
