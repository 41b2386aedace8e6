// Token rows to rows sorted by expert, and the gradients of the way back
// (the gradient of the way there is combine.hip's unweighted sum):
//   permute           xs[s][:] = x[t][:]                 s = pair_to_sorted[t*topk + j]
//   combine backward  dy[s][:] = w[t][j] * dout[t][:]
//                     dw[t][j] = sum_n dout[t][n] * y[s][n]
// Both are bound by HBM: they walk the tokens and not the sorted rows, so a
// token's row is read once into registers and used for its topk slots.  One
// workgroup takes one token and `per` of its slots; few tokens give each
// slot its own workgroup, so that a decode batch still fills the chip.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesPB = kThreads / 64;
// Sorted rows of more bytes than the Infinity Cache holds: the combine's
// gradient reads and writes them past it (nontemporal; bf16, 32768 x 7168 rows:
// 212 -> 196 us at topk 8, 236 -> 191 at topk 2).  The permutation, which only
// writes them, gained nothing (107 us either way) and keeps ordinary accesses.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

// xs rows of 16-byte units; unit counts fit int (N <= 2^24 elements).
// Bound by its stores: 8192 f16 rows of 4096 to 16384, 201 MB, 30 us, 6.7 TB/s
// (the rows come from the Infinity Cache); 8 rows to 64 slots 3.2 us, a launch.
__global__ __launch_bounds__(kThreads) void permute_kernel(const u32x4* __restrict__ x,
                                                           const int* __restrict__ p2s, int topk, int per,
                                                           int64_t P, int units, u32x4* __restrict__ xs) {
  const int groups = (topk + per - 1) / per;
  const int t = blockIdx.x / groups, j0 = (blockIdx.x - t * groups) * per, j1 = min(topk, j0 + per);
  const u32x4* src = x + (int64_t)t * units;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    const u32x4 v = src[u];
    for (int j = j0; j < j1; ++j) {
      const int s = p2s[(int64_t)t * topk + j];
      if (s < 0 || s >= P) continue;
      xs[(int64_t)s * units + u] = v;
    }
  }
}

// Bound by the three streams: 4096 bf16 rows of 7168 with 8 slots each, 1.0 GB,
// 194 us, 5.2 TB/s, above a plain copy's 4.9.  w * dout is rounded once, to dy's
// type; dw's sums are fp32, over a thread's columns, its wave, its workgroup.
template <int DK, int YK, bool NT>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(const void* __restrict__ dout,
                                                               const void* __restrict__ y,
                                                               const int* __restrict__ p2s,
                                                               const float* __restrict__ tw, int topk, int per,
                                                               int64_t P, int N, void* __restrict__ dy,
                                                               float* __restrict__ dw) {
  __shared__ float part[64][kWavesPB];  // topk <= 64
  const int groups = (topk + per - 1) / per;
  const int t = blockIdx.x / groups, j0 = (blockIdx.x - t * groups) * per, j1 = min(topk, j0 + per);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  for (int j = j0; j < j1; ++j) {
    const int64_t p = (int64_t)t * topk + j;
    const int s = p2s[p];
    float sum = 0.f;
    if (s >= 0 && s < P) {
      const float w = tw[p];
      for (int c = threadIdx.x * 8; c < N; c += kThreads * 8) {
        float d[8], v[8];
        load8<DK, false>(dout, (int64_t)t * N + c, d);
        load8<YK, NT>(y, (int64_t)s * N + c, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sum = __builtin_fmaf(d[q], v[q], sum);
          d[q] *= w;
        }
        store8<YK, NT>(dy, (int64_t)s * N + c, d);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane == 0) part[j - j0][wid] = sum;
  }
  __syncthreads();
  for (int j = j0 + threadIdx.x; j < j1; j += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWavesPB; ++w) sum += part[j - j0][w];
    dw[(int64_t)t * topk + j] = sum;
  }
}

// Slots a workgroup walks: all of a token's (its row is read once) from `full`
// tokens on, one otherwise.  One slot and all of 8, bf16 rows of 7168:
//   tokens              64          256         512          2048
//   permute             3.7  5.3    9.6  7.2   18.1 11.7    67.6 39.1 us
//   combine's gradient  4.5 12.7   14.6 17.8   26.9 21.4   102.8 106.1 us
// so a workgroup for each compute unit is enough to copy, two where every slot
// ends in a reduction (at 2048 tokens the gradient would still be 3 % faster the
// other way).  Only rows of 4096 and 7168 were compared; 8 slots of 64 to 1024
// columns, the gradient, take 10.4 - 11.5 us a call at 512 and 2048 tokens (14.4 at
// 2048 x 1024), near the 9 us of any small call.
int slots_per_group(int T, int topk, int full) { return T >= full ? topk : 1; }

template <int DK, bool NT>
hipError_t launch_bwd_nt(const void* dout, const void* y, int y_kind, const int* p2s, const float* tw, int T, int topk,
                      int per, int64_t P, int N, void* dy, float* dw, hipStream_t stream) {
  const dim3 grid(T * ((topk + per - 1) / per));
  switch (y_kind) {
    case OUT_F16:
      hipLaunchKernelGGL((combine_bwd_kernel<DK, OUT_F16, NT>), grid, dim3(kThreads), 0, stream, dout, y, p2s, tw, topk,
                         per, P, N, dy, dw);
      break;
    case OUT_BF16:
      hipLaunchKernelGGL((combine_bwd_kernel<DK, OUT_BF16, NT>), grid, dim3(kThreads), 0, stream, dout, y, p2s, tw, topk,
                         per, P, N, dy, dw);
      break;
    default:
      hipLaunchKernelGGL((combine_bwd_kernel<DK, OUT_F32, NT>), grid, dim3(kThreads), 0, stream, dout, y, p2s, tw, topk,
                         per, P, N, dy, dw);
      break;
  }
  return hipGetLastError();
}

template <int DK>
hipError_t launch_bwd(const void* dout, const void* y, int y_kind, const int* p2s, const float* tw, int T, int topk,
                      int per, int64_t P, int N, void* dy, float* dw, hipStream_t stream) {
  if (P * N * (y_kind == OUT_F32 ? 4 : 2) >= kStreamBytes)
    return launch_bwd_nt<DK, true>(dout, y, y_kind, p2s, tw, T, topk, per, P, N, dy, dw, stream);
  return launch_bwd_nt<DK, false>(dout, y, y_kind, p2s, tw, T, topk, per, P, N, dy, dw, stream);
}

// Calls launch(t0, tn) for runs of tokens small enough for one grid.
template <class F>
hipError_t for_token_runs(int T, int groups, F launch) {
  const int run = kMaxBlocks / groups;
  for (int t0 = 0; t0 < T;) {
    const int tn = std::min(run, T - t0);
    hipError_t e = launch(t0, tn);
    if (e != hipSuccess) return e;
    t0 += tn;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_permute(const void* x, const int* p2s, int T, int topk, int64_t row_bytes, void* xs, int num_cus,
                          hipStream_t stream) {
  const int per = slots_per_group(T, topk, num_cus), groups = (topk + per - 1) / per;
  return for_token_runs(T, groups, [&](int t0, int tn) {
    hipLaunchKernelGGL(permute_kernel, dim3(tn * groups), dim3(kThreads), 0, stream,
                       reinterpret_cast<const u32x4*>(static_cast<const char*>(x) + t0 * row_bytes),
                       p2s + (int64_t)t0 * topk, topk, per, (int64_t)T * topk, (int)(row_bytes / 16),
                       static_cast<u32x4*>(xs));
    return hipGetLastError();
  });
}

hipError_t launch_combine_bwd(const void* dout, int dout_kind, const void* y, int y_kind, const int* p2s,
                              const float* tw, int T, int topk, int N, void* dy, float* dw, int num_cus,
                              hipStream_t stream) {
  const int per = slots_per_group(T, topk, 2 * num_cus), groups = (topk + per - 1) / per;
  const int64_t P = (int64_t)T * topk, row_bytes = (int64_t)N * (dout_kind == OUT_F32 ? 4 : 2);
  return for_token_runs(T, groups, [&](int t0, int tn) {
    const int64_t p0 = (int64_t)t0 * topk;
    const void* d = static_cast<const char*>(dout) + t0 * row_bytes;
    switch (dout_kind) {
      case OUT_F16:
        return launch_bwd<OUT_F16>(d, y, y_kind, p2s + p0, tw + p0, tn, topk, per, P, N, dy, dw + p0, stream);
      case OUT_BF16:
        return launch_bwd<OUT_BF16>(d, y, y_kind, p2s + p0, tw + p0, tn, topk, per, P, N, dy, dw + p0, stream);
      default:
        return launch_bwd<OUT_F32>(d, y, y_kind, p2s + p0, tw + p0, tn, topk, per, P, N, dy, dw + p0, stream);
    }
  });
}

}  // namespace moeq
