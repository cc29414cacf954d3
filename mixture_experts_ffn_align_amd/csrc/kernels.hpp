// Internal launch interface between the C ABI (api.hip) and the kernels.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_ffn.h"

namespace moe {

// Per-kernel timing of moe_ffn_forward_profiled: while a LaunchTiming is
// installed (one per host thread), every launch records the kernel's own
// start and end timestamps into these events (hipExtLaunchKernel); the start
// event is consumed by the first launch of a stage, the end event is
// re-recorded by each launch, so a stage of several launches spans them all.
struct LaunchTiming {
  hipEvent_t start;
  hipEvent_t stop;
};
LaunchTiming*& launch_timing();

template <typename... KArgs, typename... Args>
void launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, uint32_t lds_bytes, hipStream_t stream,
            Args... args) {
  LaunchTiming* t = launch_timing();
  if (t == nullptr) {
    hipLaunchKernelGGL(kernel, grid, block, lds_bytes, stream, args...);
  } else {
    hipExtLaunchKernelGGL(kernel, grid, block, lds_bytes, stream, t->start, t->stop, 0, args...);
    t->start = nullptr;
  }
}

// Every kernel strides over its tasks, so its grid may be smaller than its
// task count; launches are capped at kMaxGrid workgroups (and at a caller's
// max_workgroups > 0), which keeps the work-item count of a dispatch within
// 32 bits. Task counts themselves are int32 in the layer and the ragged products
// (the C ABI rejects larger ones) and 64 bits wide in routing, the sums of routes
// and the 4-bit products, whose limits on sizes admit more.
constexpr int64_t kMaxGrid = int64_t(1) << 20;
inline int grid_for(int64_t work_groups, int max_workgroups) {
  if (work_groups < 1) work_groups = 1;
  if (work_groups > kMaxGrid) work_groups = kMaxGrid;
  return (max_workgroups > 0 && max_workgroups < work_groups) ? max_workgroups : static_cast<int>(work_groups);
}

// Route alignment (align.hip). Up to kAlignSingleMaxRoutes routes run as one
// workgroup; more (with a workspace of align_ws_bytes) as three launches over
// workgroups of kAlignRoutesPerGroup routes. Experts [ebase, ebase + E) are
// held here.
constexpr int kAlignSingleMaxRoutes = 8192;
constexpr int kAlignRoutesPerGroup = 4096;
size_t align_lds_bytes(int E);
size_t align_ws_bytes(int mk, int E);
hipError_t launch_align(const int32_t* ids, int mk, int E, int ebase, int b, int32_t* sorted, int32_t* blocks,
                        int32_t* num_padded, int cap, void* ws, size_t ws_bytes, hipStream_t stream);

// Decode path (decode.hip).
struct DecodeArgs {
  const uint16_t* x;
  const int32_t* ids;
  const float* topk_w;
  moe_weights w13, w2;
  uint16_t* a_hi;  // bf16 [M*k][I] intermediate, high part
  uint16_t* a_lo;  // bf16 [M*k][I] intermediate, low part
  float* w13_out;  // fp32 [M*k][2I] W13 outputs (gate, up) or null: capture surface
  float* y;        // fp32 [M][H]
  int M, H, I, E, k;
  int ebase;       // experts [ebase, ebase + E) are held here
  int max_workgroups;
};
bool decode_shape_ok(int fmt, int H, int I, int k, int g13, int g2);
hipError_t launch_decode_gate_up(const DecodeArgs& p, hipStream_t stream);
hipError_t launch_decode_down(const DecodeArgs& p, hipStream_t stream);

// Grouped path (grouped.hip).
struct GroupedArgs {
  const uint16_t* x;
  const int32_t* ids;
  const float* topk_w;
  const int32_t* sorted;
  const int32_t* blocks;
  const int32_t* num_padded;
  moe_weights w13, w2;
  uint16_t* a16;   // fp16 [M*k][I] intermediate, each 64-neuron chunk of a route scaled by a power of two
  float* a_scale;  // fp32 [M*k][ceil(I/128)][4]: entries 0 and 1 undo the scaling of the slab's two chunks
  float* yhat;     // fp32 [M*k][H]
  float* w13_out;  // fp32 [M*k][2I] W13 outputs (gate, up) or null: capture surface
  float* y;        // fp32 [M][H]
  int M, H, I, E, k, b;
  int ebase;       // experts [ebase, ebase + E) are held here
  int nblk;        // blocks in the alignment buffers (capacity / b)
  int max_workgroups;
};
bool grouped_shape_ok(int fmt, int H, int I, int b, int g13, int g2);
hipError_t launch_grouped_gate_up(const GroupedArgs& p, hipStream_t stream);
hipError_t launch_grouped_down(const GroupedArgs& p, hipStream_t stream);
hipError_t launch_combine(const GroupedArgs& p, hipStream_t stream);

// The two grouped GEMMs on the fixed-capacity batched layout: expert e's rows
// are e * cap .. e * cap + counts[e] - 1 of x / the intermediate (a16 and
// a_scale) / yhat (counts on the device, clamped to [0, cap]); rows past the
// count are not read or written. Uses x, w13, w2, a16, a_scale, yhat, H, I,
// E, b and max_workgroups of p.
hipError_t launch_grouped_gate_up_batched(const GroupedArgs& p, const int32_t* counts, int cap, hipStream_t stream);
hipError_t launch_grouped_down_batched(const GroupedArgs& p, const int32_t* counts, int cap, hipStream_t stream);

// Products on rows grouped by expert with ragged counts (ragged.hip). `a` is
// the operand whose index runs along the output's contiguous dimension.
struct RaggedArgs {
  const void* a;            // forward, input gradient: w [E][N][K]; weight gradient: x
  const void* b;            // forward: x; input and weight gradient: dy
  const uint8_t* a_scale;   // MXFP4 forward: exponents of w [E][N][K/32] and x [rows][K/32]
  const uint8_t* b_scale;
  const int32_t* offsets;   // [E + 1]
  void* out;                // y, dx or dW
  int64_t lda, ldb, ldo;    // row strides in elements (weights, codes and dW are contiguous)
  int rows, E, N, K;
  int out_dtype;            // moe_dtype
};
hipError_t launch_ragged_forward(const RaggedArgs& p, int dtype, hipStream_t stream);
hipError_t launch_ragged_input_grad(const RaggedArgs& p, int dtype, hipStream_t stream);
hipError_t launch_ragged_weight_grad(const RaggedArgs& p, int dtype, hipStream_t stream);

// MXFP4 (mxfp4.hip). K a multiple of 32; ldx, ldy in elements.
hipError_t launch_mxfp4_quantize(int dtype, const void* x, int64_t ldx, int64_t rows, int K, void* q, uint8_t* scale,
                                 hipStream_t stream);
hipError_t launch_mxfp4_dequantize(int dtype, const void* q, const uint8_t* scale, int64_t rows, int K, void* y,
                                   int64_t ldy, hipStream_t stream);

// Routing (route.hip). ld, ldd in elements.
struct RouteLayout {         // how a row's experts are dealt to lanes
  int per_group, per_lane;
};
struct RouteArgs {
  const void* logits;
  const float* bias;        // or null
  int32_t* topk_ids;
  float* topk_w;
  int64_t ld, M;
  int E, k, dtype, score;
  bool renormalize;
  float scale;
  int groups, topk_groups, group_top;
  // Set by launch_route:
  int group_size;
  RouteLayout wide, narrow;  // over 64 and over 16 lanes
  bool exact_scores;         // the choice takes scores, not logits alone
  bool vector;               // rows are read in 16-byte pieces
};
hipError_t launch_route(const RouteArgs& p, hipStream_t stream);

struct RouteGradArgs {
  const void* logits;
  const int32_t* topk_ids;
  const float* dtopk_w;
  void* dlogits;
  int64_t ld, ldd, M;
  int E, k, dtype, out_dtype, score;
  bool renormalize;
  float scale;
  bool vector, vector_out;   // set by launch_route_grad: rows in pieces of four elements
};
hipError_t launch_route_grad(const RouteGradArgs& p, hipStream_t stream);

// The weighted sum of routes (combine.hip); strides in elements.
struct CombineArgs {
  const void* rows;          // [rows_n][H]
  const int32_t* positions;  // [M * k], or null: route r in row r
  const float* topk_w;       // [M * k], or null: ones
  void* y;                   // [M][H]
  const void* dy;            // gradient of y
  void* drows;
  float* dtopk_w;            // or null
  int64_t ldr, ldy, lddr;    // ldy: of y or dy
  int64_t M, rows_n;
  int k, H;
};
hipError_t launch_combine_rows(const CombineArgs& p, int dtype, int y_dtype, hipStream_t stream);
hipError_t launch_combine_grad(const CombineArgs& p, int dtype, int y_dtype, hipStream_t stream);
hipError_t launch_positions(const int32_t* sorted, const int32_t* num_padded, int capacity, int routes,
                            int32_t* positions, hipStream_t stream);

// Products with packed 4-bit weights (matvec.hip).
struct MatvecArgs {
  const void* x;             // row r of y reads row r / per
  const int32_t* ids;        // [rows], or null: one matrix
  void* y;
  moe_weights w;
  int64_t ldx, ldy, rows;
  int64_t tasks;             // set by launch_matvec, as the next
  uint32_t group_inverse;    // 2^31 / (group / 32), rounded up
  int per, E, N, K, group, out_dtype;
};
hipError_t launch_matvec(const MatvecArgs& p, int dtype, hipStream_t stream);

// Row offsets of an alignment (align.hip).
hipError_t launch_align_offsets(const int32_t* blocks, const int32_t* num_padded, int nblk, int E, int b,
                                int32_t* offsets, hipStream_t stream);

}  // namespace moe
