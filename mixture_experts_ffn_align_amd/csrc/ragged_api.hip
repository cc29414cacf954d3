// C ABI of the ragged expert products, MXFP4 and the alignment's row offsets:
// argument checks and launches. Nothing here allocates device memory or
// synchronises the host.
#include <cstdint>

#include "kernels.hpp"
#include "moe_ffn.h"

namespace {

constexpr int32_t kMaxExperts = 2048;
constexpr int32_t kMaxDim = 1 << 20;          // N, K
constexpr int32_t kMaxRows = INT32_MAX - 255; // a tile's last row, and the rounding up of a row count to tiles, stay int32
constexpr int64_t kMaxStride = 1 << 22;       // row strides: a tile's 256 rows stay within 32-bit byte offsets
constexpr int64_t kMaxTasks = int64_t(1) << 30;
constexpr int64_t kMaxElements = int64_t(1) << 40;   // MXFP4 calls

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool is_dtype(int32_t t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32; }

// Shape checks shared by the products; `unit` is what N and K are multiples of.
moe_status check_shape(const moe_grouped_matmul_desc* d, int32_t unit) {
  if (d == nullptr) return MOE_ERR_INVALID_ARG;
  if (d->rows < 0 || d->E < 1 || d->N < 1 || d->K < 1) return MOE_ERR_INVALID_ARG;
  if (d->N % 8 != 0 || d->K % unit != 0) return MOE_ERR_INVALID_ARG;
  if (!is_dtype(d->out_dtype)) return MOE_ERR_INVALID_ARG;
  if (d->rows > kMaxRows || d->E > kMaxExperts || d->N > kMaxDim || d->K > kMaxDim) return MOE_ERR_UNSUPPORTED;
  // Tasks of the smallest tiles (16 x 16) in every direction.
  const int64_t nt = (d->N + 15) / 16, kt = (d->K + 15) / 16;
  const int64_t mt = d->rows / 16 + int64_t(d->E);
  if (mt * nt > kMaxTasks || mt * kt > kMaxTasks) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The 16-bit products: operand type, and an output of that type or fp32.
moe_status check_desc(const moe_grouped_matmul_desc* d) {
  const moe_status st = check_shape(d, 8);
  if (st != MOE_OK) return st;
  if (d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (d->out_dtype != d->dtype && d->out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// A row operand: 16-byte aligned rows of `cols` elements every `ld`.
moe_status check_rows(const void* p, int64_t ld, int32_t cols) {
  if (p == nullptr || !aligned16(p) || ld < cols || ld % 8 != 0) return MOE_ERR_INVALID_ARG;
  return ld > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe::RaggedArgs args_of(const moe_grouped_matmul_desc* d, const int32_t* offsets, void* out) {
  moe::RaggedArgs p{};
  p.offsets = offsets;
  p.out = out;
  p.rows = d->rows; p.E = d->E; p.N = d->N; p.K = d->K;
  p.out_dtype = d->out_dtype;
  return p;
}

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(const moe_grouped_matmul_desc* d, const void* x, int64_t ldx, const void* w,
                              const int32_t* offsets, void* y, int64_t ldy, hipStream_t stream) {
  moe_status st = check_desc(d);
  if (st != MOE_OK) return st;
  if (d->rows == 0) return MOE_OK;
  if ((st = check_rows(x, ldx, d->K)) != MOE_OK || (st = check_rows(y, ldy, d->N)) != MOE_OK) return st;
  if (w == nullptr || offsets == nullptr || !aligned16(w)) return MOE_ERR_INVALID_ARG;
  moe::RaggedArgs p = args_of(d, offsets, y);
  p.a = w;
  p.b = x;
  p.ldb = ldx; p.ldo = ldy;
  return hip_status(moe::launch_ragged_forward(p, d->dtype, stream));
}

moe_status moe_grouped_matmul_dx(const moe_grouped_matmul_desc* d, const void* dy, int64_t lddy, const void* w,
                                 const int32_t* offsets, void* dx, int64_t lddx, hipStream_t stream) {
  moe_status st = check_desc(d);
  if (st != MOE_OK) return st;
  if (d->rows == 0) return MOE_OK;
  if ((st = check_rows(dy, lddy, d->N)) != MOE_OK || (st = check_rows(dx, lddx, d->K)) != MOE_OK) return st;
  if (w == nullptr || offsets == nullptr || !aligned16(w)) return MOE_ERR_INVALID_ARG;
  moe::RaggedArgs p = args_of(d, offsets, dx);
  p.a = w;
  p.b = dy;
  p.ldb = lddy; p.ldo = lddx;
  return hip_status(moe::launch_ragged_input_grad(p, d->dtype, stream));
}

moe_status moe_grouped_matmul_dw(const moe_grouped_matmul_desc* d, const void* dy, int64_t lddy, const void* x,
                                 int64_t ldx, const int32_t* offsets, void* dw, hipStream_t stream) {
  moe_status st = check_desc(d);
  if (st != MOE_OK) return st;
  if (int64_t(d->E) * ((d->N + 15) / 16) * ((d->K + 15) / 16) > kMaxTasks) return MOE_ERR_UNSUPPORTED;
  if (offsets == nullptr || dw == nullptr || !aligned16(dw)) return MOE_ERR_INVALID_ARG;
  // Without rows there is nothing to read, but every gradient is zero.
  if (d->rows > 0 &&
      ((st = check_rows(dy, lddy, d->N)) != MOE_OK || (st = check_rows(x, ldx, d->K)) != MOE_OK))
    return st;
  moe::RaggedArgs p = args_of(d, offsets, dw);
  p.a = x;
  p.b = dy;
  p.lda = ldx; p.ldb = lddy;
  return hip_status(moe::launch_ragged_weight_grad(p, d->dtype, stream));
}

moe_status moe_grouped_matmul_mxfp4(const moe_grouped_matmul_desc* d, const void* xq, const uint8_t* x_scale,
                                    const void* wq, const uint8_t* w_scale, const int32_t* offsets, void* y,
                                    int64_t ldy, hipStream_t stream) {
  moe_status st = check_shape(d, 32);
  if (st != MOE_OK) return st;
  if (d->dtype != MOE_DTYPE_MXFP4) return MOE_ERR_INVALID_ARG;
  if (d->rows == 0) return MOE_OK;
  if ((st = check_rows(y, ldy, d->N)) != MOE_OK) return st;
  if (xq == nullptr || x_scale == nullptr || wq == nullptr || w_scale == nullptr || offsets == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(wq)) return MOE_ERR_INVALID_ARG;
  moe::RaggedArgs p = args_of(d, offsets, y);
  p.a = wq;
  p.b = xq;
  p.a_scale = w_scale;
  p.b_scale = x_scale;
  p.ldo = ldy;
  return hip_status(moe::launch_ragged_forward(p, MOE_DTYPE_MXFP4, stream));
}

moe_status moe_mxfp4_quantize(int32_t dtype, const void* x, int64_t ldx, int64_t rows, int32_t K, void* q,
                              uint8_t* scale, hipStream_t stream) {
  if (!is_dtype(dtype) || rows < 0 || K < 1 || K % 32 != 0) return MOE_ERR_INVALID_ARG;
  if (K > kMaxDim || rows > kMaxElements / K) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const moe_status st = check_rows(x, ldx, K);
  if (st != MOE_OK) return st;
  if (q == nullptr || scale == nullptr || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_mxfp4_quantize(dtype, x, ldx, rows, K, q, scale, stream));
}

moe_status moe_mxfp4_dequantize(int32_t dtype, const void* q, const uint8_t* scale, int64_t rows, int32_t K, void* y,
                                int64_t ldy, hipStream_t stream) {
  if (!is_dtype(dtype) || rows < 0 || K < 1 || K % 32 != 0) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
  if (K > kMaxDim || rows > kMaxElements / K) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const moe_status st = check_rows(y, ldy, K);
  if (st != MOE_OK) return st;
  if (q == nullptr || scale == nullptr || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_mxfp4_dequantize(dtype, q, scale, rows, K, y, ldy, stream));
}

moe_status moe_align_offsets(const int32_t* expert_block_ids, const int32_t* num_padded, size_t blocks, int32_t E,
                             int32_t b, int32_t* offsets, hipStream_t stream) {
  if (E < 1 || b < 1 || num_padded == nullptr || offsets == nullptr || (blocks > 0 && expert_block_ids == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || blocks > size_t(INT32_MAX / b)) return MOE_ERR_UNSUPPORTED;
  return hip_status(moe::launch_align_offsets(expert_block_ids, num_padded, static_cast<int>(blocks), E, b, offsets,
                                              stream));
}

}  // extern "C"
