// Per-row symmetric INT8 quantization of activations, the operand rows of
// grouped_gemm_qint8: amax = max |x|, scale = amax / 127, code =
// clamp(rne(x * (127 / amax)), -127, 127), each step one fp32 operation.  A row
// with amax < 2^-120 becomes zeros with scale 1; a row that holds an infinity
// or NaN gets scale NaN, so its products show it.
//
// HBM-bound: 8 elements per lane and step, 16 input bytes (32 for f32) and 8
// output bytes.  Rows of up to 16384 elements are held in registers and read
// once: by one wave each up to 2048, four rows of a workgroup at a time (16384
// rows of 256 bf16: 7 us, against 19 with a workgroup each), by a workgroup
// above (16384 rows of 14336 f16, 705 MB: 125 us, 5.6 TB/s).  Longer rows are
// read twice.
#include <algorithm>

#include "int8.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kWavesQ8 = 4;

// WAVES waves work on a row (1 or the whole workgroup's).  LOADS: register
// loads per thread (0: the row is read twice).
template <int XK, int WAVES, int LOADS, bool NT>
__global__ __launch_bounds__(64 * kWavesQ8) void quant_int8_rows(const void* __restrict__ x, int64_t rows, int K,
                                                                uint8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int kRows = kWavesQ8 / WAVES, kT = 64 * WAVES;
  static_assert(WAVES == 1 || kRows == 1, "the rows of a workgroup may end in different rounds: no barrier then");
  __shared__ u32 wmax[WAVES];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, tid = threadIdx.x % kT;
  for (int64_t row = (int64_t)blockIdx.x * kRows + wid / WAVES; row < rows; row += (int64_t)gridDim.x * kRows) {
    const int64_t base = row * K;
    float v[LOADS ? LOADS : 1][8];
    u32 m = 0;
    if constexpr (LOADS > 0) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int k = (i * kT + tid) * 8;
        if (k < K) load8<XK, NT>(x, base + k, v[i]);
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        if ((i * kT + tid) * 8 < K) m = max(m, amax_bits(v[i]));
    } else {
      for (int k = tid * 8; k < K; k += kT * 8) {
        load8<XK, false>(x, base + k, v[0]);
        m = max(m, amax_bits(v[0]));
      }
    }
    m = wave_max(m);
    if constexpr (WAVES > 1) {
      if (lane == 0) wmax[wid] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) m = max(m, wmax[w]);
      __syncthreads();  // wmax is reused by the next row
    }
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
        const int k = (i * kT + tid) * 8;
        if (k < K) put(k, v[i]);
      }
    } else {
      for (int k = tid * 8; k < K; k += kT * 8) {
        load8<XK, false>(x, base + k, v[0]);
        put(k, v[0]);
      }
    }
    if (tid == 0) scale[row] = c.scale;
  }
}

template <int XK>
hipError_t go(const void* x, int64_t rows, int K, uint8_t* q, float* scale, int num_cus, hipStream_t stream) {
  // inputs past the 256 MB Infinity Cache are read, and their codes written, past it
  const bool nt = rows * K * (XK == OUT_F32 ? 4 : 2) >= (int64_t(256) << 20);
#define MOEQ_Q8(WAVES, LOADS, NT)                                                                              \
  hipLaunchKernelGGL((quant_int8_rows<XK, WAVES, LOADS, NT>),                                                  \
                     dim3((int)std::min<int64_t>((rows + kWavesQ8 / WAVES - 1) / (kWavesQ8 / WAVES), (int64_t)num_cus * 8)), \
                     dim3(64 * kWavesQ8), 0, stream, x, rows, K, q, scale)
  if (K > kWavesQ8 * 64 * 8 * 8) MOEQ_Q8(4, 0, false);
  else if (K <= 64 * 8 * 4 && nt) MOEQ_Q8(1, 4, true);
  else if (K <= 64 * 8 * 4) MOEQ_Q8(1, 4, false);
  else if (nt) MOEQ_Q8(4, 8, true);
  else MOEQ_Q8(4, 8, false);
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
