// MXFP4 quantisation and dequantisation (gfx950).
//
// A row of K elements becomes K / 2 bytes of E2M1 codes (even element in the
// low nibble) and K / 32 E8M0 bytes. For a block of 32 elements with largest
// magnitude m, the exponent is s = clamp(floor(log2 m) - 2, -127, 127) (E2M1's
// largest value is 1.5 * 2^2) and the code of x is x / 2^s rounded to the
// nearest E2M1 value, ties to the even code, saturating at 6. A block of zeros
// gets s = -127. A block holding an infinity or a NaN gets the NaN exponent
// byte 255 and codes 0: it decodes to NaN, so a bad value is not lost.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));

// Eight consecutive elements as fp32.
template <int kDtype>
__device__ __forceinline__ floatx8 load8(const void* x, int64_t i) {
  floatx8 v;
  if constexpr (kDtype == MOE_DTYPE_F32) {
    const floatx4* p = reinterpret_cast<const floatx4*>(static_cast<const float*>(x) + i);
    const floatx4 a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[j + 4] = b[j];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = w[j];
      if constexpr (kDtype == MOE_DTYPE_BF16) {
        v[2 * j] = bf16_lo(u);
        v[2 * j + 1] = bf16_hi(u);
      } else {
        const halfx2 h = __builtin_bit_cast(halfx2, u);
        v[2 * j] = static_cast<float>(h[0]);
        v[2 * j + 1] = static_cast<float>(h[1]);
      }
    }
  }
  return v;
}

// A lane takes eight consecutive elements; four lanes share a block. `pieces`
// is K / 8: loads and stores are contiguous over the wave, and the block's
// largest magnitude needs two exchanges within four lanes. Bound: HBM (each
// element is read once, 17 bytes per 32 written): 196608 x 2048 fp32 347 us,
// 5.3 TB/s; 21 x 2048 bf16 2.6 us.
template <int kDtype>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize(const void* __restrict__ x, int64_t ldx, int64_t rows,
                                                           int pieces, uint32_t* __restrict__ q,
                                                           uint8_t* __restrict__ scale) {
  const int64_t n = rows * pieces;
  for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = i / pieces;
    const int c = static_cast<int>(i - row * pieces);
    const floatx8 v = load8<kDtype>(x, row * ldx + c * 8);
    // Magnitudes compare as their bit patterns; an infinity or a NaN is above every finite value.
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    // The four lanes of a block are neighbours and all active: K is a multiple of 32.
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xF, 0xF, true)));
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xF, 0xF, true)));
    const bool bad = m >= 0x7F800000u;
    // Biased exponent of m less 2; below 2^-125 (subnormals among them) it is 0.
    const int e = bad ? 255 : max(0, static_cast<int>(m >> 23) - 2);
    const float unit = e8m0_to_float(bad ? 127 : e);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], unit, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], unit, 3);
    q[i] = bad ? 0 : w;
    if ((c & 3) == 0) scale[i >> 2] = static_cast<uint8_t>(e);
  }
}

// A lane decodes eight codes; 196608 x 2048 to bf16 191 us, 5.3 TB/s. Every value is exact in bf16 and fp32 (but
// those from 2^128 on, which are infinite; the quantiser above does not make them).
template <int kDtype>
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize(const uint32_t* __restrict__ q,
                                                             const uint8_t* __restrict__ scale, int64_t rows,
                                                             int pieces, void* __restrict__ y, int64_t ldy) {
  const int64_t n = rows * pieces;
  for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = i / pieces;
    const int c = static_cast<int>(i - row * pieces);
    const uint32_t w = q[i];
    const float unit = e8m0_to_float(scale[i >> 2]);
    const floatx2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 0);
    const floatx2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 1);
    const floatx2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 2);
    const floatx2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 3);
    const int64_t at = row * ldy + c * 8;
    if constexpr (kDtype == MOE_DTYPE_F32) {
      floatx4* o = reinterpret_cast<floatx4*>(static_cast<float*>(y) + at);
      o[0] = floatx4{v0[0], v0[1], v1[0], v1[1]};
      o[1] = floatx4{v2[0], v2[1], v3[0], v3[1]};
    } else {
      bf16x8 o;
      o[0] = static_cast<__bf16>(v0[0]);
      o[1] = static_cast<__bf16>(v0[1]);
      o[2] = static_cast<__bf16>(v1[0]);
      o[3] = static_cast<__bf16>(v1[1]);
      o[4] = static_cast<__bf16>(v2[0]);
      o[5] = static_cast<__bf16>(v2[1]);
      o[6] = static_cast<__bf16>(v3[0]);
      o[7] = static_cast<__bf16>(v3[1]);
      *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(y) + at) = o;
    }
  }
}

int grid_of(int64_t n) { return grid_for((n + kThreads - 1) / kThreads, 0); }

}  // namespace

hipError_t launch_mxfp4_quantize(int dtype, const void* x, int64_t ldx, int64_t rows, int K, void* q, uint8_t* scale,
                                 hipStream_t stream) {
  const int pieces = K / 8;
  const dim3 grid(grid_of(rows * pieces)), block(kThreads);
  uint32_t* qw = static_cast<uint32_t*>(q);
  if (dtype == MOE_DTYPE_F32)
    launch(mxfp4_quantize<MOE_DTYPE_F32>, grid, block, 0, stream, x, ldx, rows, pieces, qw, scale);
  else if (dtype == MOE_DTYPE_BF16)
    launch(mxfp4_quantize<MOE_DTYPE_BF16>, grid, block, 0, stream, x, ldx, rows, pieces, qw, scale);
  else
    launch(mxfp4_quantize<MOE_DTYPE_F16>, grid, block, 0, stream, x, ldx, rows, pieces, qw, scale);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(int dtype, const void* q, const uint8_t* scale, int64_t rows, int K, void* y,
                                   int64_t ldy, hipStream_t stream) {
  const int pieces = K / 8;
  const dim3 grid(grid_of(rows * pieces)), block(kThreads);
  const uint32_t* qw = static_cast<const uint32_t*>(q);
  if (dtype == MOE_DTYPE_F32)
    launch(mxfp4_dequantize<MOE_DTYPE_F32>, grid, block, 0, stream, qw, scale, rows, pieces, y, ldy);
  else
    launch(mxfp4_dequantize<MOE_DTYPE_BF16>, grid, block, 0, stream, qw, scale, rows, pieces, y, ldy);
  return hipGetLastError();
}

}  // namespace moe
