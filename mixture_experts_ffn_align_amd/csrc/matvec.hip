// Products of a few rows with packed 4-bit weights (gfx950):
//   y[r][n] = sum_k (q[e][n][k] - z[e][n][k / g]) s[e][n][k / g] x[r / per][k]
// with one matrix for every row, or the matrix of the row's expert.
//
// The weights are the left operand of 16x16x32 matrix instructions, so up to
// sixteen rows cost the same unpacking. A nibble is OR-ed into the top of a
// 16-bit mantissa, which gives 16 + q exactly; a group's sum is then
//   s (sum (16 + q) x - (16 + z) sum x)
// in fp32, where sum x comes from a second matrix instruction with ones. (An
// offset of 128, from the mantissa's low bits, would cancel eight times as much.)
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kSplit = kThreads / kWave;   // waves that share a tile's summed index
constexpr int kTile = 16;                  // weight rows of a tile
constexpr int kChunk = 128;                // summed elements per 16-byte load of a lane

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8v __attribute__((ext_vector_type(8)));

template <bool kHalf>
__device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) {
  if constexpr (kHalf)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8v, a), __builtin_bit_cast(halfx8v, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0,
                                                   0, 0);
}

// Eight 4-bit values of a word as 16 + q, in element order.
template <bool kHalf>
__device__ __forceinline__ u32x4 unpack8(uint32_t w) {
  u32x4 v;
  if constexpr (kHalf) {
    const uint32_t m = 0x03C003C0u, c = 0x4C004C00u;
    v[0] = ((w << 6) & m) | c;
    v[1] = ((w << 2) & m) | c;
    v[2] = ((w >> 2) & m) | c;
    v[3] = ((w >> 6) & m) | c;
  } else {
    const uint32_t m = 0x00780078u, c = 0x41804180u;
    v[0] = ((w << 3) & m) | c;
    v[1] = ((w >> 1) & m) | c;
    v[2] = ((w >> 5) & m) | c;
    v[3] = ((w >> 9) & m) | c;
  }
  return v;
}

// Four registers of four groups of sixteen lanes, transposed: afterwards
// register j of lane group g holds what register g of lane group j held.
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{static_cast<uint32_t>(c[0]), static_cast<uint32_t>(c[1]), static_cast<uint32_t>(d[0]),
               static_cast<uint32_t>(d[1])};
}

// A workgroup takes sixteen weight rows and up to 16 kCols rows of x; its waves
// take quarters of the summed index, whose sums meet in LDS.
template <bool kHalf, int kCols>
__global__ __launch_bounds__(kThreads) void matvec(MatvecArgs p) {
  __shared__ floatx4 part[kSplit - 1][kCols][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int r = lane & 15, q = lane >> 4;
  const int tiles = (p.N + kTile - 1) / kTile;
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int c0 = static_cast<int>(int64_t(chunks) * wave / kSplit);
  const int c1 = static_cast<int>(int64_t(chunks) * (wave + 1) / kSplit);
  const int words = p.K / 8, groups = p.K / p.group;
  const uint32_t one = kHalf ? 0x3C003C00u : 0x3F803F80u;
  const u32x4 ones = {one, one, one, one};
  for (int64_t task = blockIdx.x; task < p.tasks; task += gridDim.x) {
    const int64_t block = task / tiles;
    const int n0 = static_cast<int>(task - block * tiles) * kTile;
    const int64_t row0 = p.ids != nullptr ? block : block * (kTile * kCols);
    const int rows = p.ids != nullptr ? 1 : static_cast<int>(min(int64_t(kTile * kCols), p.rows - row0));
    const int e = p.ids != nullptr ? p.ids[row0] : 0;
    floatx4 acc[kCols] = {};
    if (e >= 0 && e < p.E) {
      const int64_t wrow = int64_t(e) * p.N + min(n0 + r, p.N - 1);
      const uint32_t* w = static_cast<const uint32_t*>(p.w.q) + wrow * words;
      const uint16_t* x[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        x[c] = static_cast<const uint16_t*>(p.x) + (row0 + min(c * kTile + r, rows - 1)) / p.per * p.ldx + q * 8;
      int64_t srow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) srow[i] = (int64_t(e) * p.N + min(n0 + q * 4 + i, p.N - 1)) * groups;
      for (int c = c0; c < c1; ++c) {
        const int word = c * (kChunk / 8) + q * 4;
        u32x4 v = {0, 0, 0, 0};
        if (word < words) v = *reinterpret_cast<const u32x4*>(w + word);
        v = transpose4(v);
        const int steps = min(4, (p.K - c * kChunk) / 32);
        floatx4 sum[kCols] = {}, xs[kCols] = {};
        for (int j = 0; j < steps; ++j) {
          const int k = c * kChunk + j * 32;
          const u32x4 a = unpack8<kHalf>(j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3]);
#pragma unroll
          for (int m = 0; m < kCols; ++m) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(x[m] + k);
            sum[m] = mfma<kHalf>(a, b, sum[m]);
            xs[m] = mfma<kHalf>(ones, b, xs[m]);
          }
          if (j == steps - 1 || (k + 32) % p.group == 0) {
            const int g = k / p.group;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float s = half_bits_to_float(static_cast<const uint16_t*>(p.w.scale)[srow[i] + g]);
              const float z = 16.0f + (p.w.zero != nullptr ? static_cast<float>(p.w.zero[srow[i] + g]) : 8.0f);
#pragma unroll
              for (int m = 0; m < kCols; ++m) acc[m][i] += s * (sum[m][i] - z * xs[m][i]);
            }
#pragma unroll
            for (int m = 0; m < kCols; ++m) sum[m] = xs[m] = floatx4{0, 0, 0, 0};
          }
        }
      }
    }
    if (wave > 0) {
#pragma unroll
      for (int m = 0; m < kCols; ++m) part[wave - 1][m][lane] = acc[m];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
#pragma unroll
        for (int s = 0; s < kSplit - 1; ++s) acc[m] += part[s][m][lane];
        const int col = m * kTile + r;
        if (col >= rows) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + q * 4 + i;
          if (n >= p.N) continue;
          const int64_t at = (row0 + col) * p.ldy + n;
          if (p.out_dtype == MOE_DTYPE_F32)
            static_cast<float*>(p.y)[at] = acc[m][i];
          else if constexpr (kHalf)
            static_cast<_Float16*>(p.y)[at] = static_cast<_Float16>(acc[m][i]);
          else
            static_cast<__bf16*>(p.y)[at] = static_cast<__bf16>(acc[m][i]);
        }
      }
    }
    __syncthreads();
  }
}

template <int kCols>
void start(MatvecArgs p, int dtype, hipStream_t stream) {
  const int64_t tiles = (p.N + kTile - 1) / kTile;
  const int64_t blocks = p.ids != nullptr ? p.rows : (p.rows + kTile * kCols - 1) / (kTile * kCols);
  p.tasks = tiles * blocks;
  const dim3 grid(grid_for(p.tasks, 0)), block(kThreads);
  if (dtype == MOE_DTYPE_F16)
    launch(matvec<true, kCols>, grid, block, 0, stream, p);
  else
    launch(matvec<false, kCols>, grid, block, 0, stream, p);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& p, int dtype, hipStream_t stream) {
  if (p.ids != nullptr || p.rows <= kTile)
    start<1>(p, dtype, stream);
  else if (p.rows <= 2 * kTile)
    start<2>(p, dtype, stream);
  else
    start<4>(p, dtype, stream);
  return hipGetLastError();
}

}  // namespace moe
