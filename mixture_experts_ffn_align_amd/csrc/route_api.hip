// C ABI of routing, the weighted sum of routes and the products with packed
// 4-bit weights: argument checks and launches. Nothing here allocates device
// memory or synchronises the host.
#include <cstdint>

#include "kernels.hpp"
#include "moe_ffn.h"

namespace {

constexpr int32_t kMaxExperts = 2048;
constexpr int32_t kMaxSlots = 64;                    // routes per token: one lane each
constexpr int32_t kMaxGroups = 64;
constexpr int32_t kMaxDim = 1 << 20;                 // H, N, K
constexpr int32_t kMaxRows = INT32_MAX - 255;
constexpr int64_t kMaxStride = 1 << 22;
constexpr int64_t kMaxTasks = int64_t(1) << 40;

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool is_dtype(int32_t t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32; }

uintptr_t size_of(int32_t t) { return t == MOE_DTYPE_F32 ? 4 : 2; }

moe_status check_route(const moe_route_desc* d) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->M < 0 || d->E < 1 || d->k < 1 || d->k > d->E || !is_dtype(d->dtype)) return MOE_ERR_INVALID_ARG;
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (d->groups < 1 || d->E % d->groups != 0 || d->topk_groups < 1 || d->topk_groups > d->groups)
    return MOE_ERR_INVALID_ARG;
  if (d->group_top != 1 && d->group_top != 2) return MOE_ERR_INVALID_ARG;
  if (int64_t(d->topk_groups) * (d->E / d->groups) < d->k) return MOE_ERR_INVALID_ARG;
  if (d->E > kMaxExperts || d->k > kMaxSlots || d->groups > kMaxGroups || d->M > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows of logits: any stride from E on; elements at their own alignment.
moe_status check_logits(const void* p, int64_t ld, int32_t E, int32_t dtype) {
  if (p == nullptr || ld < E || !aligned(p, size_of(dtype))) return MOE_ERR_INVALID_ARG;
  return ld > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows of values: 16-byte aligned, a stride of a multiple of 8 elements.
moe_status check_rows(const void* p, int64_t ld, int32_t cols) {
  if (p == nullptr || !aligned(p, 16) || ld < cols || ld % 8 != 0) return MOE_ERR_INVALID_ARG;
  return ld > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_combine(const moe_combine_desc* d) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->M < 0 || d->k < 1 || d->H < 1 || d->rows < 0 || d->H % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(d->dtype) || !is_dtype(d->y_dtype)) return MOE_ERR_INVALID_ARG;
  if (d->H > kMaxDim || d->rows > kMaxRows || int64_t(d->M) * d->k > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::CombineArgs args_of(const moe_combine_desc* d, const int32_t* positions, const float* topk_w) {
  moe::CombineArgs p{};
  p.positions = positions;
  p.topk_w = topk_w;
  p.M = d->M; p.k = d->k; p.H = d->H; p.rows_n = d->rows;
  return p;
}

}  // namespace

extern "C" {

moe_status moe_route(const moe_route_desc* d, const void* logits, int64_t ld, const float* bias, int32_t* topk_ids,
                     float* topk_w, hipStream_t stream) {
  moe_status st = check_route(d);
  if (st != MOE_OK) return st;
  if (d->M == 0) return MOE_OK;
  if ((st = check_logits(logits, ld, d->E, d->dtype)) != MOE_OK) return st;
  if (topk_ids == nullptr || topk_w == nullptr || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  moe::RouteArgs p{};
  p.logits = logits;
  p.ld = ld;
  p.bias = bias;
  p.topk_ids = topk_ids;
  p.topk_w = topk_w;
  p.M = d->M; p.E = d->E; p.k = d->k;
  p.dtype = d->dtype; p.score = d->score;
  p.renormalize = d->renormalize != 0;
  p.scale = d->scale;
  p.groups = d->groups; p.topk_groups = d->topk_groups; p.group_top = d->group_top;
  return hip_status(moe::launch_route(p, stream));
}

moe_status moe_route_grad(const moe_route_desc* d, const void* logits, int64_t ld, const int32_t* topk_ids,
                          const float* dtopk_w, int32_t out_dtype, void* dlogits, int64_t ldd, hipStream_t stream) {
  moe_status st = check_route(d);
  if (st != MOE_OK) return st;
  if (out_dtype != d->dtype && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (d->M == 0) return MOE_OK;
  if ((st = check_logits(logits, ld, d->E, d->dtype)) != MOE_OK ||
      (st = check_logits(dlogits, ldd, d->E, out_dtype)) != MOE_OK)
    return st;
  if (topk_ids == nullptr || dtopk_w == nullptr || !aligned(topk_ids, 4) || !aligned(dtopk_w, 4))
    return MOE_ERR_INVALID_ARG;
  moe::RouteGradArgs p{};
  p.logits = logits;
  p.ld = ld;
  p.topk_ids = topk_ids;
  p.dtopk_w = dtopk_w;
  p.dlogits = dlogits;
  p.ldd = ldd;
  p.M = d->M; p.E = d->E; p.k = d->k;
  p.dtype = d->dtype; p.out_dtype = out_dtype; p.score = d->score;
  p.renormalize = d->renormalize != 0;
  p.scale = d->scale;
  return hip_status(moe::launch_route_grad(p, stream));
}

moe_status moe_align_positions(const int32_t* sorted_route_ids, const int32_t* num_padded, size_t capacity,
                               int32_t routes, int32_t* positions, hipStream_t stream) {
  if (routes < 0) return MOE_ERR_INVALID_ARG;
  if (capacity > size_t(kMaxRows) || routes > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (routes == 0) return MOE_OK;
  if (num_padded == nullptr || positions == nullptr || (capacity > 0 && sorted_route_ids == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(num_padded, 4) || !aligned(positions, 4) || !aligned(sorted_route_ids, 4)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_positions(sorted_route_ids, num_padded, static_cast<int>(capacity), routes, positions,
                                          stream));
}

moe_status moe_combine(const moe_combine_desc* d, const void* rows, int64_t ldr, const int32_t* positions,
                       const float* topk_w, void* y, int64_t ldy, hipStream_t stream) {
  moe_status st = check_combine(d);
  if (st != MOE_OK) return st;
  if (d->M == 0) return MOE_OK;
  if (!aligned(positions, 4) || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(y, ldy, d->H)) != MOE_OK) return st;
  // Without rows there is nothing to read, but every sum is zero.
  if (d->rows > 0 && (st = check_rows(rows, ldr, d->H)) != MOE_OK) return st;
  moe::CombineArgs p = args_of(d, positions, topk_w);
  p.rows = rows;
  p.ldr = ldr;
  p.y = y;
  p.ldy = ldy;
  return hip_status(moe::launch_combine_rows(p, d->dtype, d->y_dtype, stream));
}

moe_status moe_combine_grad(const moe_combine_desc* d, const void* dy, int64_t lddy, const void* rows, int64_t ldr,
                            const int32_t* positions, const float* topk_w, void* drows, int64_t lddr, float* dtopk_w,
                            hipStream_t stream) {
  moe_status st = check_combine(d);
  if (st != MOE_OK) return st;
  if (d->M == 0) return MOE_OK;
  if (!aligned(positions, 4) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4)) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(dy, lddy, d->H)) != MOE_OK) return st;
  if (d->rows > 0) {
    if ((st = check_rows(drows, lddr, d->H)) != MOE_OK) return st;
    if (dtopk_w != nullptr && (st = check_rows(rows, ldr, d->H)) != MOE_OK) return st;
  }
  moe::CombineArgs p = args_of(d, positions, topk_w);
  p.rows = rows;
  p.ldr = ldr;
  p.dy = dy;
  p.ldy = lddy;
  p.drows = drows;
  p.lddr = lddr;
  p.dtopk_w = dtopk_w;
  return hip_status(moe::launch_combine_grad(p, d->dtype, d->y_dtype, stream));
}

moe_status moe_matvec_int4(const moe_matvec_desc* d, const void* x, int64_t ldx, const int32_t* topk_ids, void* y,
                           int64_t ldy, hipStream_t stream) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->M < 0 || d->k < 1 || d->E < 1 || d->N < 1 || d->K < 1) return MOE_ERR_INVALID_ARG;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (d->out_dtype != d->dtype && d->out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (d->w.fmt != MOE_W_INT4_AWQ) return d->w.fmt == MOE_W_MXFP8 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (d->w.group < 32 || d->w.group % 32 != 0 || d->K % d->w.group != 0) return MOE_ERR_INVALID_ARG;
  if (d->E > kMaxExperts || d->N > kMaxDim || d->K > kMaxDim || int64_t(d->M) * d->k > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  if (int64_t(d->M) * d->k * d->N > kMaxTasks) return MOE_ERR_UNSUPPORTED;
  if (d->M == 0) return MOE_OK;
  if ((topk_ids == nullptr && (d->E != 1 || d->k != 1)) || !aligned(topk_ids, 4)) return MOE_ERR_INVALID_ARG;
  moe_status st = check_rows(x, ldx, d->K);
  if (st != MOE_OK) return st;
  // The output is written by single elements.
  if (y == nullptr || ldy < d->N || !aligned(y, size_of(d->out_dtype))) return MOE_ERR_INVALID_ARG;
  if (ldy > kMaxStride) return MOE_ERR_UNSUPPORTED;
  if (d->w.q == nullptr || d->w.scale == nullptr || !aligned(d->w.q, 16) || !aligned(d->w.scale, 2))
    return MOE_ERR_INVALID_ARG;
  moe::MatvecArgs p{};
  p.x = x;
  p.ldx = ldx;
  p.ids = topk_ids;
  p.y = y;
  p.ldy = ldy;
  p.w = d->w;
  p.rows = int64_t(d->M) * d->k;
  p.per = d->k;
  p.E = d->E; p.N = d->N; p.K = d->K;
  p.group = d->w.group;
  p.out_dtype = d->out_dtype;
  return hip_status(moe::launch_matvec(p, d->dtype, stream));
}

}  // extern "C"
