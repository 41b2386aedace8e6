// Low-rank adapters of many groups at once, beside a projection:
//   h[s][:]      = x[row(s)][:] A_g^T                  (shrink, K -> R)
//   out[o(s)][:] = base[o(s)][:] + scale_g h[s][:] B_g^T   (expand, R -> N)
// and their gradients
//   dh[s][:] = scale_g dy[o(s)][:] B_g      dx[s][:] = dh[s][:] A_g
//   dA_g = sum_s dh[s]^T x[row(s)]          dB_g = scale_g sum_s dy[o(s)]^T h[s]
// over the rows s of each group g.
//
// First form: one workgroup per row (or per weight tile), plain fp32
// arithmetic, nothing shared between rows.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kThreads = 256;

struct Dev {
  const int* offsets;
  const int* sorted_ids;
  int P, E, x_div, out_pair, N, K, R;
  const float* scale;
};

// Group of sorted row s (the last e with offsets[e] <= s), -1 past the last.
__device__ __forceinline__ int group_of(const Dev& g, int s) {
  if (s >= min(max(g.offsets[g.E], 0), g.P)) return -1;
  int lo = 0, hi = g.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.offsets[mid] <= s) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Pair id of sorted row s, -1 where the table holds none.
__device__ __forceinline__ int pair_of(const Dev& g, int s) {
  if (!g.sorted_ids) return s;
  const int p = g.sorted_ids[s];
  return p >= 0 && p < g.P ? p : -1;
}
__device__ __forceinline__ int64_t x_row(const Dev& g, int s, int pair) { return g.x_div ? pair / g.x_div : s; }
__device__ __forceinline__ int64_t o_row(const Dev& g, int s, int pair) { return g.out_pair ? pair : s; }
__device__ __forceinline__ float scale_of(const Dev& g, int e) { return g.scale ? g.scale[e] : 1.f; }

// h[s][r] = sum_k x[row][k] a[e][r][k]
template <int KIND>
__global__ __launch_bounds__(kThreads) void shrink_rows(Dev g, const uint16_t* x, const uint16_t* a, float* h) {
  const int s = blockIdx.x, lane = threadIdx.x & 63;
  const int e = group_of(g, s), pair = e < 0 ? -1 : pair_of(g, s);
  if (pair < 0) return;
  const int64_t row = x_row(g, s, pair);
  for (int r = threadIdx.x >> 6; r < g.R; r += kThreads / 64) {
    float sum = 0.f;
    for (int c = lane * 8; c < g.K; c += 512) {
      float u[8], v[8];
      load8<KIND, false>(x, row * g.K + c, u);
      load8<KIND, false>(a, ((int64_t)e * g.R + r) * g.K + c, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum = __builtin_fmaf(u[q], v[q], sum);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) h[(int64_t)s * g.R + r] = sum;
  }
}

// out[o][n] = base[o][n] + scale sum_r h[s][r] b[e][n][r]
template <int KIND>
__global__ __launch_bounds__(kThreads) void expand_rows(Dev g, const float* h, const uint16_t* b, const uint16_t* base,
                                                        uint16_t* out) {
  const int s = blockIdx.x;
  const int e = group_of(g, s), pair = e < 0 ? -1 : pair_of(g, s);
  if (pair < 0) return;
  const int64_t o = o_row(g, s, pair) * g.N;
  const float sc = scale_of(g, e);
  for (int c = threadIdx.x * 8; c < g.N; c += kThreads * 8) {
    float acc[8], v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      acc[q] = 0.f;
      for (int r = 0; r < g.R; r += 8) {
        load8<KIND, false>(b, ((int64_t)e * g.N + c + q) * g.R + r, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[q] = __builtin_fmaf(h[(int64_t)s * g.R + r + i], v[i], acc[q]);
      }
    }
    if (base) load8<KIND, false>(base, o + c, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = base ? __builtin_fmaf(sc, acc[q], v[q]) : sc * acc[q];
    store8<KIND, false>(out, o + c, acc);
  }
}

// Pair-ordered rows without a group: base, or zero.
__global__ __launch_bounds__(kThreads) void copy_skipped(const int* p2s, int64_t P, int units, const u32x4* base,
                                                         u32x4* out) {
  const int64_t p = blockIdx.x;
  if (p2s[p] >= 0 && p2s[p] < P) return;
  for (int u = threadIdx.x; u < units; u += kThreads) out[p * units + u] = base ? base[p * units + u] : u32x4{0, 0, 0, 0};
}

// dh[s][r] = scale sum_n dy[o][n] b[e][n][r]
template <int KIND>
__global__ __launch_bounds__(kThreads) void shrink_dy(Dev g, const uint16_t* dy, const uint16_t* b, float* dh) {
  const int s = blockIdx.x, lane = threadIdx.x & 63;
  const int e = group_of(g, s), pair = e < 0 ? -1 : pair_of(g, s);
  if (pair < 0) return;
  const int64_t row = o_row(g, s, pair);
  for (int r = threadIdx.x >> 6; r < g.R; r += kThreads / 64) {
    float sum = 0.f;
    for (int n = lane; n < g.N; n += 64)
      sum = __builtin_fmaf(load_as_f32<KIND>(dy, row * g.N + n), load_as_f32<KIND>(b, ((int64_t)e * g.N + n) * g.R + r),
                           sum);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) dh[(int64_t)s * g.R + r] = scale_of(g, e) * sum;
  }
}

// dx[s][k] = sum_r dh[s][r] a[e][r][k]
template <int KIND>
__global__ __launch_bounds__(kThreads) void expand_dx(Dev g, const float* dh, const uint16_t* a, uint16_t* dx) {
  const int s = blockIdx.x;
  const int e = group_of(g, s), pair = e < 0 ? -1 : pair_of(g, s);
  if (pair < 0) return;
  for (int c = threadIdx.x * 8; c < g.K; c += kThreads * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
    for (int r = 0; r < g.R; ++r) {
      load8<KIND, false>(a, ((int64_t)e * g.R + r) * g.K + c, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(dh[(int64_t)s * g.R + r], v[q], acc[q]);
    }
    store8<KIND, false>(dx, (int64_t)s * g.K + c, acc);
  }
}

// da[e][r][c] = sum_s dh[s][r] x[row][c], one thread per (r, 8 columns)
template <int KIND>
__global__ __launch_bounds__(kThreads) void outer_a(Dev g, const float* dh, const uint16_t* x, uint16_t* da) {
  const int e = blockIdx.x / g.R, r = blockIdx.x - e * g.R;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  for (int c = threadIdx.x * 8; c < g.K; c += kThreads * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
    for (int s = lo; s < hi; ++s) {
      const int pair = pair_of(g, s);
      if (pair < 0) continue;
      load8<KIND, false>(x, x_row(g, s, pair) * g.K + c, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(dh[(int64_t)s * g.R + r], v[q], acc[q]);
    }
    store8<KIND, false>(da, ((int64_t)e * g.R + r) * g.K + c, acc);
  }
}

// db[e][n][r] = scale sum_s dy[o][n] h[s][r], one thread per (n, 8 ranks)
template <int KIND>
__global__ __launch_bounds__(kThreads) void outer_b(Dev g, const float* h, const uint16_t* dy, uint16_t* db) {
  const int per = (g.N * (g.R / 8) + kThreads - 1) / kThreads;
  const int e = blockIdx.x / per;
  const int i = (blockIdx.x - e * per) * kThreads + threadIdx.x;
  const int n = i / (g.R / 8), r = (i - n * (g.R / 8)) * 8;
  if (n >= g.N) return;
  int lo, hi;
  expert_range(g.offsets, e, g.P, lo, hi);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
  for (int s = lo; s < hi; ++s) {
    const int pair = pair_of(g, s);
    if (pair < 0) continue;
    const float d = load_as_f32<KIND>(dy, o_row(g, s, pair) * g.N + n);
    load8<OUT_F32, false>(h, (int64_t)s * g.R + r, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(d, v[q], acc[q]);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] *= scale_of(g, e);
  store8<KIND, false>(db, ((int64_t)e * g.N + n) * g.R + r, acc);
}

Dev dev_args(const LoraArgs& g) {
  return Dev{g.offsets, g.sorted_ids, (int)g.P, g.E, g.x_div, g.out_pair, g.N, g.K, g.R, g.scale};
}

template <int KIND>
hipError_t forward(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b, const uint16_t* base,
                   uint16_t* out, float* h, hipStream_t stream) {
  const Dev d = dev_args(g);
  hipLaunchKernelGGL(shrink_rows<KIND>, dim3((unsigned)g.P), dim3(kThreads), 0, stream, d, x, a, h);
  hipLaunchKernelGGL(expand_rows<KIND>, dim3((unsigned)g.P), dim3(kThreads), 0, stream, d, h, b, base, out);
  if (g.out_pair && base != out)
    hipLaunchKernelGGL(copy_skipped, dim3((unsigned)g.P), dim3(kThreads), 0, stream, g.p2s, g.P, g.N / 8,
                       reinterpret_cast<const u32x4*>(base), reinterpret_cast<u32x4*>(out));
  return hipGetLastError();
}

template <int KIND>
hipError_t backward(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                    const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, float* dh, hipStream_t stream) {
  const Dev d = dev_args(g);
  if (g.P > 0) {
    hipLaunchKernelGGL(shrink_dy<KIND>, dim3((unsigned)g.P), dim3(kThreads), 0, stream, d, dy, b, dh);
    if (dx) hipLaunchKernelGGL(expand_dx<KIND>, dim3((unsigned)g.P), dim3(kThreads), 0, stream, d, dh, a, dx);
  }
  hipLaunchKernelGGL(outer_a<KIND>, dim3(g.E * g.R), dim3(kThreads), 0, stream, d, dh, x, da);
  const int per = (g.N * (g.R / 8) + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(outer_b<KIND>, dim3(g.E * per), dim3(kThreads), 0, stream, d, h, dy, db);
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t P, int E, int N, int K, int R) { return (size_t)P * R * sizeof(float); }
size_t lora_bwd_workspace_bytes(int64_t P, int E, int N, int K, int R) { return (size_t)P * R * sizeof(float); }

hipError_t launch_lora(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                       const uint16_t* base, uint16_t* out, float* h, void* ws, hipStream_t stream) {
  if (g.P == 0) return hipSuccess;
  if (!h) h = static_cast<float*>(ws);
  return g.f16 ? forward<OUT_F16>(g, x, a, b, base, out, h, stream)
               : forward<OUT_BF16>(g, x, a, b, base, out, h, stream);
}

hipError_t launch_lora_bwd(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a,
                           const uint16_t* b, const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                           hipStream_t stream) {
  float* dh = static_cast<float*>(ws);
  return g.f16 ? backward<OUT_F16>(g, dy, x, a, b, h, dx, da, db, dh, stream)
               : backward<OUT_BF16>(g, dy, x, a, b, h, dx, da, db, dh, stream);
}

}  // namespace moeq
