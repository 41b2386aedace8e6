// Top-k weighted scatter back to token rows (megamoe_rm.cu's combine: a
// token's pairs that have an expert, summed in slot order in fp32 and
// rounded once; tilelang_kernels.py: zero output plus weighted rows).
// ROWS_PAIRS: the rows are already weighted and in pair order (the output of
// fc2_rm's epilogue), so token t's rows are t*topk .. t*topk+topk-1.
// ROWS_PLAIN: rows in sorted order summed without weights, the gradient of
// the permutation (each token's row was copied to its slots' rows): 32768 bf16
// rows of 7168 to 4096, 0.53 GB, 88 us, 6.0 TB/s.
//
// One thread owns 8 consecutive columns of one token row: it reads the
// pair table entries of its token, then 8 elements (16 or 32 bytes) of each
// routed expert row, so every wave reads and writes contiguous runs.
// When y is larger than the 256 MB Infinity Cache it streams from HBM, and
// nontemporal loads and stores measured 17 % faster (bf16 y of 32768 x
// 7168: 107 -> 89 us); a y that fits may still sit in the cache from the
// GEMM that wrote it, and there ordinary accesses measured 9 % faster
// (f16 y of 16384 x 4096: 29.8 against 32.4 us).
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "vec8.h"

namespace moeq {
namespace {

constexpr int kThreads = 256;

constexpr int64_t kStreamBytes = int64_t(256) << 20;

enum Rows { ROWS_WEIGHTED, ROWS_PAIRS, ROWS_PLAIN };

template <int YK, int OK, int ROWS, bool NT>
__global__ __launch_bounds__(kThreads) void combine_kernel(const void* __restrict__ y,
                                                           const int* __restrict__ p2s,
                                                           const float* __restrict__ tw, int T,
                                                           int topk, int N, int64_t P,
                                                           void* __restrict__ out) {
  const int cblocks = (N / 8 + kThreads - 1) / kThreads;
  const int t = blockIdx.x / cblocks;
  const int c = ((blockIdx.x - t * cblocks) * kThreads + threadIdx.x) * 8;
  if (c >= N) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < topk; ++j) {
    const int64_t p = (int64_t)t * topk + j;
    const int s = p2s[p];
    if (s < 0 || s >= P) continue;
    float v[8];
    load8<YK, NT>(y, (ROWS == ROWS_PAIRS ? p : (int64_t)s) * N + c, v);
    if (ROWS != ROWS_WEIGHTED) {
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += v[q];
    } else {
      const float w = tw[p];
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(w, v[q], acc[q]);
    }
  }
  store8<OK, NT>(out, (int64_t)t * N + c, acc);
}

template <int YK, int ROWS, bool NT>
hipError_t launch_nt(const void* y, const int* p2s, const float* tw, int T, int topk, int N,
                     int64_t P, int out_kind, void* out, hipStream_t stream) {
  const dim3 grid(((N / 8 + kThreads - 1) / kThreads) * T);
  switch (out_kind) {
    case OUT_F16:
      hipLaunchKernelGGL((combine_kernel<YK, OUT_F16, ROWS, NT>), grid, dim3(kThreads), 0, stream, y, p2s, tw,
                         T, topk, N, P, out);
      break;
    case OUT_BF16:
      hipLaunchKernelGGL((combine_kernel<YK, OUT_BF16, ROWS, NT>), grid, dim3(kThreads), 0, stream, y, p2s,
                         tw, T, topk, N, P, out);
      break;
    default:
      hipLaunchKernelGGL((combine_kernel<YK, OUT_F32, ROWS, NT>), grid, dim3(kThreads), 0, stream, y, p2s, tw,
                         T, topk, N, P, out);
      break;
  }
  return hipGetLastError();
}

template <int YK, int ROWS>
hipError_t launch_y(const void* y, const int* p2s, const float* tw, int T, int topk, int N,
                    int64_t P, int out_kind, void* out, hipStream_t stream) {
  // the rows actually read: T * topk of them at most
  const int64_t y_bytes = std::min<int64_t>(P, (int64_t)T * topk) * N * (YK == OUT_F32 ? 4 : 2);
  if (y_bytes >= kStreamBytes)
    return launch_nt<YK, ROWS, true>(y, p2s, tw, T, topk, N, P, out_kind, out, stream);
  return launch_nt<YK, ROWS, false>(y, p2s, tw, T, topk, N, P, out_kind, out, stream);
}

template <int ROWS>
hipError_t launch_kind(const void* y, int y_kind, const int* p2s, const float* tw, int T, int topk, int N,
                       int64_t P, int out_kind, void* out, hipStream_t stream) {
  switch (y_kind) {
    case OUT_F16: return launch_y<OUT_F16, ROWS>(y, p2s, tw, T, topk, N, P, out_kind, out, stream);
    case OUT_BF16: return launch_y<OUT_BF16, ROWS>(y, p2s, tw, T, topk, N, P, out_kind, out, stream);
    default: return launch_y<OUT_F32, ROWS>(y, p2s, tw, T, topk, N, P, out_kind, out, stream);
  }
}

// Launches in runs of tokens small enough for one grid (the packet's grid
// size in threads is 32 bits wide).
template <int ROWS>
hipError_t launch_tokens(const void* y, int y_kind, const int* p2s, const float* tw, int T, int topk, int N,
                         int out_kind, void* out, hipStream_t stream) {
  const int64_t P = (int64_t)T * topk;
  const int run = std::max(1, kMaxBlocks / ((N / 8 + kThreads - 1) / kThreads));
  for (int t0 = 0; t0 < T;) {
    const int tn = std::min(run, T - t0);
    const int64_t p0 = (int64_t)t0 * topk;
    // pair-ordered rows move with the tokens, sorted rows are addressed whole
    const char* yt = static_cast<const char*>(y) + (ROWS == ROWS_PAIRS ? p0 * N * (y_kind == OUT_F32 ? 4 : 2) : 0);
    hipError_t e = launch_kind<ROWS>(yt, y_kind, p2s + p0, tw ? tw + p0 : nullptr, tn, topk, N, P, out_kind,
                                     static_cast<char*>(out) + (int64_t)t0 * N * (out_kind == OUT_F32 ? 4 : 2), stream);
    if (e != hipSuccess) return e;
    t0 += tn;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_combine(const void* y, int y_kind, const int* p2s, const float* tw, int T, int topk, int N,
                          int out_kind, void* out, hipStream_t stream) {
  if (tw == nullptr)
    return launch_tokens<ROWS_PAIRS>(y, y_kind, p2s, tw, T, topk, N, out_kind, out, stream);
  return launch_tokens<ROWS_WEIGHTED>(y, y_kind, p2s, tw, T, topk, N, out_kind, out, stream);
}

hipError_t launch_permute_bwd(const void* dxs, int dxs_kind, const int* p2s, int T, int topk, int N, int out_kind,
                              void* dx, hipStream_t stream) {
  return launch_tokens<ROWS_PLAIN>(dxs, dxs_kind, p2s, nullptr, T, topk, N, out_kind, dx, stream);
}

}  // namespace moeq
