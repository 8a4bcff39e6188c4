// Internal launchers behind the C ABI.  Every launcher enqueues on `stream`,
// trusts that api.hip has validated its arguments, and returns
// hipGetLastError() of its last launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

hipError_t launch_gate(const float* logits, int T, int E, int k, int renormalize, int* topk_ids,
                       float* topk_w, hipStream_t stream);
hipError_t launch_gate_record(const float* logits, int T, int E, int k, int renormalize, int* topk_ids,
                              float* topk_w, int block_tokens, int layer, int L, int* block_counts,
                              hipStream_t stream);

// ---- routing with scores -----------------------------------------------------
struct RouteArgs {
  int T, E, k;
  int bf16;      // logits: 1 bf16, 0 fp32
  int sigmoid;   // 0: softmax
  int n_groups, top_groups;
  int group_lanes = 0;   // set by the launcher: lanes that hold a group's experts (0: no whole, power-of-two run)
  int top2;      // group value: sum of the two best, 0: the best
  int renormalize;
  float scale;
  int* topk_ids;
  float* topk_w;
};
hipError_t launch_route(const void* logits, const float* bias, const RouteArgs& a, hipStream_t stream);

// ---- router projection -------------------------------------------------------
hipError_t launch_router(const void* x, const void* w_router, int T, int d, int E, int bf16, float* logits,
                         hipStream_t stream);

// ---- permutation -----------------------------------------------------------
struct PermuteArgs {
  const int* topk_ids;
  int T, E, k, n_shared, n_priority;
  const void* x;
  int elem_bytes;  // 2 (bf16) or 4 (f32)
  int d;
  int* group_offsets;
  int* sorted_to_flat;
  int* flat_to_sorted;
  int* sorted_token;  // may be nullptr
  void* x_sorted;
};
size_t permute_workspace_bytes(int T, int E, int k, int n_shared, int n_priority);
hipError_t launch_permute(const PermuteArgs& a, void* workspace, hipStream_t stream);

// ---- grouped FFN -----------------------------------------------------------
struct FfnArgs {
  const void* x_sorted;
  const int* x_rows;  // nullptr: x_sorted is already in sorted order
  int n_x;            // rows of x_sorted when x_rows is given
  const int* group_offsets;
  int n_rows, E, n_shared, nseg, d, I;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  int bf16;  // 1: bf16 operands, 0: fp32
  void* h_sorted;
  // FP8-weight call only: one fp32 scale per weight row ([E+S][I], [E+S][I], [E+S][d])
  const float* s_gate = nullptr;
  const float* s_up = nullptr;
  const float* s_down = nullptr;
  // weights pre-packed in 1 KiB blocks of 16 rows: 32 K values for bf16
  // (moe_grouped_ffn_packed), 64 for FP8 codes (moe_grouped_ffn_fp8w_packed)
  bool packed = false;
  // per-tile timeline of the persistent queue (moe_grouped_ffn_traced): records
  // of 4 uint64, nullptr for none
  unsigned long long* trace = nullptr;
  int trace_capacity = 0;
  // combine folded into the down projection (moe_grouped_ffn_combine): y32 is
  // the [T][d] fp32 sums in the workspace, y the [T][d] bf16 result; nullptr
  // for the plain call
  float* y32 = nullptr;
  void* y = nullptr;
  const int* s2f = nullptr;
  const float* topk_w = nullptr;
  int T = 0, k = 0;
};
size_t ffn_workspace_bytes(int n_rows, int E, int n_shared, int nseg, int d, int I, int bf16);
// moe_grouped_ffn_combine: batches on the decode-shaped kernels only
bool ffn_fused_combine_supported(int n_rows, int E, int n_shared, int nseg, int d, int I);
hipError_t launch_ffn(const FfnArgs& a, void* workspace, hipStream_t stream);
size_t ffn_fp8w_workspace_bytes(int n_rows, int E, int n_shared, int nseg, int d, int I, bool packed);
// FP8 batches that run on the GEMM kernel (packed codes, groups averaging more
// than 48 rows, d and I multiples of 64 and at least 128, 16-byte aligned scales)
bool fp8w_uses_gemm(int n_rows, int G, int d, int I, bool packed, const void* s_gate, const void* s_up,
                    const void* s_down);
hipError_t launch_ffn_fp8w(const FfnArgs& a, void* workspace, hipStream_t stream);

// ---- int8 rows and products ----------------------------------------------------
hipError_t launch_quantize_rows(const void* x, int bf16, int T, int d, int8_t* q, float* s, hipStream_t stream);

struct GroupedI8 {
  const int* x_rows;   // nullptr: sorted row n reads row n
  int n_x;
  const int* group_offsets;
  int n_rows, E, n_shared, nseg;
};
// y[n][o], packed int8 weights [E+S][O][K]; bf16: output type
hipError_t launch_grouped_linear_i8(const GroupedI8& g, const int8_t* xq, const float* xs, int K, int O,
                                    const int8_t* w, const float* ws, int bf16, void* y, hipStream_t stream);
struct FfnI8Args {
  GroupedI8 g;
  const void* x;       // bf16 tokens
  int d, I;
  const int8_t *w_gate, *w_up, *w_down;
  const float *s_gate, *s_up, *s_down;
  void* h_sorted;
};
size_t ffn_i8_workspace_bytes(int n_rows, int n_tokens, int d, int I);
hipError_t launch_ffn_i8(const FfnI8Args& a, void* workspace, hipStream_t stream);

// ---- norm and FP8 block codes -----------------------------------------------------
enum CodeKind { kCodeNone, kCodeI8, kCodeFp8 };
struct NormArgs {
  int T, d;
  int x_bf16, residual_bf16, weight_bf16, y_bf16;   // 1 bf16, 0 fp32
  const void *x, *residual, *weight;                // residual: nullptr for none
  void *residual_out, *y;                           // y: nullptr for none
  int code;                                         // CodeKind of q and s
  uint8_t* q;
  float* s;
  float eps;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream);
hipError_t launch_quantize_blocks(const void* x, int bf16, int T, int d, uint8_t* q, float* s, hipStream_t stream);

// ---- FP8 products -----------------------------------------------------------------
struct GroupedFp8 {
  const int* x_rows;   // nullptr: sorted row n reads row n
  int n_x;
  const int* group_offsets;
  int n_rows, E, n_shared, nseg;
};
// y[n][o], packed E4M3 weights [E+S][O][K]; bf16: output type
hipError_t launch_grouped_linear_fp8(const GroupedFp8& g, const uint8_t* xq, const float* xs, int K, int O,
                                     const uint8_t* w, const float* ws, int bf16, void* y, hipStream_t stream);
struct FfnFp8Args {
  GroupedFp8 g;
  const uint8_t* xq;
  const float* xs;
  int d, I;
  const uint8_t *w_gate, *w_up, *w_down;
  const float *s_gate, *s_up, *s_down;
  void* h_sorted;
};
size_t ffn_fp8_workspace_bytes(int n_rows, int I);
hipError_t launch_ffn_fp8(const FfnFp8Args& a, void* workspace, hipStream_t stream);

// ---- combine ---------------------------------------------------------------
hipError_t launch_combine(const void* h_sorted, const int* flat_to_sorted, const float* topk_w, int T,
                          int k, int n_shared, int d, int bf16, void* y, hipStream_t stream);

// ---- statistics ------------------------------------------------------------
struct StatsArgs {
  const int* topk_ids;
  int L, T, k, E;
  const int* req_offsets;
  int R;
  const float* idf;
  int* counts;
  int* union_size;
  uint8_t* union_mask;
  int* affinity;
  int* req_counts;
  float* signature;
};
size_t stats_workspace_bytes(int L, int T, int k, int E, int R);
hipError_t launch_stats(const StatsArgs& a, void* workspace, hipStream_t stream);

// ---- continuous (softmax-probability) request signature ---------------------
hipError_t launch_prob_signature(const float* logits, int L, int T, int E, const int* req_offsets, int R,
                                 float* signature, hipStream_t stream);

}  // namespace moe
