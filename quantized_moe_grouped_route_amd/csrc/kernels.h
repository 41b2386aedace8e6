// Internal launchers (host side of each kernel file).  Arguments are
// validated by the C-ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moeq {

// Route prep.
size_t route_workspace_bytes(int64_t P, int E);
hipError_t launch_route(const int* ids, int P, int E, int* offsets, int* sorted_ids,
                        int* pair_to_sorted, int* n_invalid, void* ws, hipStream_t stream);
// Route prep with its per-chunk counts in the library's fixed device array
// (kRouteNoallocScratchBytes per device) instead of a caller's workspace.
constexpr size_t kRouteNoallocScratchBytes = size_t(1) << 20;
// Counters of the NVFP4 tiled schedule's work queue: one claim counter per
// XCD (8) and one count of finished workgroups.
constexpr int kWorkQueueInts = 16;
hipError_t launch_route_noalloc(const int* ids, int P, int E, int* offsets, int* sorted_ids,
                                int* pair_to_sorted, int* n_invalid, hipStream_t stream);

// Combine.  y_kind / out_kind are OutKind values.  tw == null: y holds
// pre-weighted rows in pair order (row t*topk + j), summed unweighted.
hipError_t launch_combine(const void* y, int y_kind, const int* p2s, const float* tw, int T,
                          int topk, int N, int out_kind, void* out, hipStream_t stream);

// Workgroups of 256 threads one launch may have: a grid's size in threads is
// a 32-bit field of the dispatch packet.
constexpr int kMaxBlocks = 1 << 23;

// Token rows to sorted rows (row_bytes % 16 == 0), and its gradient: the
// unweighted sum of each token's sorted rows.
hipError_t launch_permute(const void* x, const int* p2s, int T, int topk, int64_t row_bytes, void* xs, int num_cus,
                          hipStream_t stream);
hipError_t launch_permute_bwd(const void* dxs, int dxs_kind, const int* p2s, int T, int topk, int N, int out_kind,
                              void* dx, hipStream_t stream);
// Gradients of the weighted combine.
hipError_t launch_combine_bwd(const void* dout, int dout_kind, const void* y, int y_kind, const int* p2s,
                              const float* tw, int T, int topk, int N, void* dy, float* dw, int num_cus,
                              hipStream_t stream);

// Per-row symmetric INT4 quantization (x_kind: OutKind of the input).
hipError_t launch_quant_int4(const void* x, int x_kind, int64_t rows, int K, uint8_t* q, float* scale,
                             int num_cus, hipStream_t stream);

// Arguments common to the grouped GEMMs.
struct GroupedArgs {
  const int* offsets;       // [E+1]
  const int* sorted_ids;    // [P] or null (identity rows)
  int64_t rows_a;           // rows of the activation operand
  int a_sorted;             // 1: row = s, 0: row = sorted_ids[s] / topk
  int topk;
  int E;
  int64_t P;
  int N;                    // GEMM columns (2I for SILU_MUL)
  int K;
  int silu_mul;             // 1: write I = N/2 columns silu(gate) * up
  float act_limit;          // SwiGLU clamp (NVFP4 only); +inf: none
  const float* pair_weights;  // [P] or null: write w[p] * y to row p = sorted_ids[s] (NVFP4 only)
  int x_f16;                // NVFP4: activations are binary16 (else bf16)
  int sf_quads;             // NVFP4: scales [E][K/64][N][4] (else [E][N][K/16])
  int w_tiled;              // NVFP4: codes in 16-row x 64-K blocks (else [E][N][K/2])
  int out_kind;             // OutKind
  void* out;
  int sched;                // 0 auto, 1 decode, 2 prefill
  int* queue;               // NVFP4 tiled schedule: [kWorkQueueInts] zeroed counters, or null
  int num_cus;              // compute units of the current device
};

hipError_t launch_gemm_int4(const GroupedArgs& g, const uint8_t* a, const float* a_scale,
                            const uint8_t* w, const float* w_scale, hipStream_t stream);
hipError_t launch_gemm_fp8(const GroupedArgs& g, const uint8_t* a, const float* a_scale,
                           const uint8_t* w, const float* w_scale, hipStream_t stream);
hipError_t launch_gemm_nvfp4(const GroupedArgs& g, const uint16_t* x, const uint8_t* w,
                             const uint8_t* w_sf, const float* w_gscale, hipStream_t stream);

// W8A8: whether every launch of these sizes fits, the GEMM, and its gradient
// towards the activations (GroupedArgs: offsets, E, P, N, K, out = dx and its
// kind, which is dy's; the other fields are not read).
bool int8_fits(int64_t P, int E, int64_t N);
bool int8_bwd_fits(int64_t P, int E, int64_t K);
hipError_t launch_gemm_int8(const GroupedArgs& g, const int8_t* a, const float* a_scale, const int8_t* w,
                            const float* w_scale, hipStream_t stream);
// The least workspace, and the one beyond which more is not used.
size_t int8_bwd_workspace_bytes(int64_t P, int N);
size_t int8_bwd_workspace_most(int64_t P, int N);
hipError_t launch_gemm_int8_bwd(const GroupedArgs& g, const void* dy, const int8_t* w, const float* w_scale,
                                const void* base, void* ws, size_t ws_bytes, hipStream_t stream);

// Per-row symmetric INT8 quantization (x_kind: OutKind of the input).
hipError_t launch_quant_int8(const void* x, int x_kind, int64_t rows, int K, int8_t* q, float* scale, int num_cus,
                             hipStream_t stream);

// h = silu(gate) * up of rows [gate | up]; ck, cs: null, or the 8-bit
// checkpoint.  offsets null: all P rows, else the first offsets[E].  Its
// gradient reads gu, or the checkpoint where ck is given; h null: not written;
// dh and dgu null: h alone.
hipError_t launch_silu_mul(const void* gu, int kind, const int* offsets, int E, int64_t P, int I, void* h, int8_t* ck,
                           float* cs, int num_cus, hipStream_t stream);
hipError_t launch_silu_mul_bwd(const void* dh, int kind, const void* gu, const int8_t* ck, const float* cs,
                               const int* offsets, int E, int64_t P, int I, void* dgu, void* h, int num_cus,
                               hipStream_t stream);

// Low-rank adapters beside a projection, rows grouped by adapter.
struct LoraArgs {
  const int* offsets;       // [E+1]
  const int* sorted_ids;    // [P] or null (identity rows)
  const int* p2s;           // [P] or null (pair-ordered output only)
  int64_t P;                // rows
  int E;                    // adapters
  int x_div;                // row of x: sorted_ids[s] / x_div, or s where 0
  int out_pair;             // 1: row of out / base / dy is sorted_ids[s], 0: s
  int N;
  int K;
  int R;
  int f16;                  // element type: binary16 (else bf16)
  const float* scale;       // [E] or null (1)
};
// Whether every launch of these sizes fits one grid, forward and gradients.
bool lora_fits(int64_t P, int E, int N, int K, int R);
bool lora_bwd_fits(int64_t P, int E, int N, int K, int R);
size_t lora_workspace_bytes(int64_t P, int E, int N, int K, int R);
size_t lora_bwd_workspace_bytes(int64_t P, int E, int N, int K, int R);
// h: null, or [P][R] that receives the shrunk rows.
hipError_t launch_lora(const LoraArgs& g, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                       const uint16_t* base, uint16_t* out, float* h, void* ws, hipStream_t stream);
// dx: null where it is not wanted.
hipError_t launch_lora_bwd(const LoraArgs& g, const uint16_t* dy, const uint16_t* x, const uint16_t* a,
                           const uint16_t* b, const float* h, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                           hipStream_t stream);

// bf16 -> binary16 (round to nearest even), n values, n % 8 == 0.
hipError_t launch_cast_bf16_f16(const uint16_t* x, int64_t n, uint16_t* y, int num_cus, hipStream_t stream);

// NVFP4 weight repack: megamoe_rm.cu layout (swizzled scales, optionally up
// rows first) -> grouped_gemm_qnvfp4's, E experts of N rows and K columns.
hipError_t launch_repack_nvfp4(const uint8_t* w_in, const uint8_t* sf_in, int64_t E, int64_t N, int64_t K,
                               int swap_halves, int w_tiled, int out_quads, uint8_t* w_out, uint8_t* sf_out,
                               hipStream_t stream);

}  // namespace moeq
