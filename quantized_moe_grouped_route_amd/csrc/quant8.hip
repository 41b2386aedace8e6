// Per-row symmetric INT8 quantization of activations, the operand rows of
// grouped_gemm_qint8: amax = max |x|, scale = amax / 127, code =
// clamp(rne(x * (127 / amax)), -127, 127), each step one fp32 operation.  A row
// with amax < 2^-120 becomes zeros with scale 1; a row that holds an infinity
// or NaN gets scale NaN, so its products show it.
//
// HBM-bound: 8 elements per lane and step, 16 input bytes (32 for f32) and 8
// output bytes.  Rows of up to kThreadsQ8 * 8 * kLoadsQ8 = 16384 elements are
// held in one workgroup's registers and read once; longer ones are read twice.
#include <algorithm>

#include "int8.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kThreadsQ8 = 256;
constexpr int kLoadsQ8 = 8;

// LOADS: register loads per thread (0: the row is read twice).
template <int XK, int LOADS, bool NT>
__global__ __launch_bounds__(kThreadsQ8) void quant_int8_rows(const void* __restrict__ x, int64_t rows, int K,
                                                             uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ u32 wmax[kThreadsQ8 / 64];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * K;
    float v[LOADS ? LOADS : 1][8];
    u32 m = 0;
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (i * kThreadsQ8 + tid) * 8;
        if (k < K) load8<XK, NT>(x, base + k, v[i]);
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        if ((i * kThreadsQ8 + tid) * 8 < K) m = max(m, amax_bits(v[i]));
    } else {
      for (int k = tid * 8; k < K; k += kThreadsQ8 * 8) {
        load8<XK, false>(x, base + k, v[0]);
        m = max(m, amax_bits(v[0]));
      }
    }
    m = wave_max(m);
    if (lane == 0) wmax[wid] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreadsQ8 / 64; ++w) m = max(m, wmax[w]);
    __syncthreads();  // wmax is reused by the next row
    const Scale c = scale_of(m, 127.0f, 0x1p-120f);
    auto put = [&](int k, const float (&t)[8]) __attribute__((always_inline)) {
      const uint2 p = codes8(t, c.recip);
      v2i_t* dst = reinterpret_cast<v2i_t*>(q + base + k);
      const v2i_t w = {(int)p.x, (int)p.y};
      if (NT) __builtin_nontemporal_store(w, dst);
      else *dst = w;
    };
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (i * kThreadsQ8 + tid) * 8;
        if (k < K) put(k, v[i]);
      }
    } else {
      for (int k = tid * 8; k < K; k += kThreadsQ8 * 8) {
        load8<XK, false>(x, base + k, v[0]);
        put(k, v[0]);
      }
    }
    if (tid == 0) scale[row] = c.scale;
  }
}

template <int XK>
hipError_t go(const void* x, int64_t rows, int K, uint8_t* q, float* scale, int num_cus, hipStream_t stream) {
  const int grid = (int)std::min<int64_t>(rows, (int64_t)num_cus * 8);
  // inputs past the 256 MB Infinity Cache are read, and their codes written, past it
  const bool nt = rows * K * (XK == OUT_F32 ? 4 : 2) >= (int64_t(256) << 20);
#define MOEQ_Q8(LOADS, NT) \
  hipLaunchKernelGGL((quant_int8_rows<XK, LOADS, NT>), dim3(grid), dim3(kThreadsQ8), 0, stream, x, rows, K, q, scale)
  if (K > kThreadsQ8 * 8 * kLoadsQ8) MOEQ_Q8(0, false);
  else if (nt) MOEQ_Q8(kLoadsQ8, true);
  else MOEQ_Q8(kLoadsQ8, false);
#undef MOEQ_Q8
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_int8(const void* x, int x_kind, int64_t rows, int K, int8_t* q, float* scale, int num_cus,
                             hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  uint8_t* out = reinterpret_cast<uint8_t*>(q);
  switch (x_kind) {
    case OUT_F16: return go<OUT_F16>(x, rows, K, out, scale, num_cus, stream);
    case OUT_BF16: return go<OUT_BF16>(x, rows, K, out, scale, num_cus, stream);
    default: return go<OUT_F32>(x, rows, K, out, scale, num_cus, stream);
  }
}

}  // namespace moeq
