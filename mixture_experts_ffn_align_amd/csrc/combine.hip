// The weighted sum of a token's routes and its gradient (gfx950):
//   y[t] = sum_j w[t][j] rows[p(t, j)]
//   drows[p(t, j)] = w[t][j] dy[t],  dw[t][j] = rows[p(t, j)] . dy[t]
// where p(t, j) is the row of route t * k + j, or none. Sums are fp32, in slot
// order; each output is rounded once. Both kernels go by tokens, so nothing is
// atomic and a token's dy is read once for all its routes.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;              // routes whose loads are in flight together
constexpr int kPositionThreads = 1024;    // in one workgroup
constexpr int kScatterThreads = 256;      // in several
// Routes and rows up to which one workgroup inverts the alignment: 1.8 us for 168, 3.4 for 4096, 5.9 for 8192;
// two launches 3.3, 3.7, 3.7 (32768: 3.8, one workgroup 21).
constexpr int kPositionsSingle = 4096;

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

// What a route without a row reads.
__device__ const floatx8 kZeros = {0, 0, 0, 0, 0, 0, 0, 0};

template <int kDtype>
struct Elem;
template <>
struct Elem<MOE_DTYPE_F32> {
  typedef floatx8 Vec;
  static constexpr int kBytes = 4;
};
template <>
struct Elem<MOE_DTYPE_BF16> {
  typedef bf16x8 Vec;
  static constexpr int kBytes = 2;
};
template <>
struct Elem<MOE_DTYPE_F16> {
  typedef halfx8 Vec;
  static constexpr int kBytes = 2;
};

// Elements 8 c .. 8 c + 7 of a row, as stored and as fp32.
template <int kDtype>
__device__ __forceinline__ typename Elem<kDtype>::Vec load8(const void* base, int64_t elem) {
  return *reinterpret_cast<const typename Elem<kDtype>::Vec*>(static_cast<const char*>(base) +
                                                              elem * Elem<kDtype>::kBytes);
}
template <typename V>
__device__ __forceinline__ floatx8 to_f32(V v) {
  return __builtin_convertvector(v, floatx8);
}
template <int kDtype>
__device__ __forceinline__ void store8(void* base, int64_t elem, floatx8 v) {
  typedef typename Elem<kDtype>::Vec V;
  *reinterpret_cast<V*>(static_cast<char*>(base) + elem * Elem<kDtype>::kBytes) = __builtin_convertvector(v, V);
}

// Row of slot j of token t, or -1.
__device__ __forceinline__ int row_of(const CombineArgs& p, int64_t t, int j) {
  if (j >= p.k) return -1;
  const int64_t r = t * p.k + j;
  const int at = p.positions != nullptr ? p.positions[r] : static_cast<int>(r);
  return (at >= 0 && at < p.rows_n) ? at : -1;
}

// A lane takes eight columns of a token, with the loads of eight routes in flight. Bound: HBM; 4096 tokens of
// 2048 columns, top-8, bf16: 32 us, 4.7 TB/s.
template <int kIn, int kOut>
__global__ __launch_bounds__(kThreads) void combine(CombineArgs p) {
  const int pieces = p.H / 8;
  const int64_t n = p.M * int64_t(pieces);
  for (int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    const int64_t t = i / pieces;
    const int c = static_cast<int>(i - t * pieces);
    floatx8 y = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      typename Elem<kIn>::Vec v[kSlots];
      float w[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const int at = row_of(p, t, j0 + j);
        w[j] = at < 0 ? 0.0f : p.topk_w != nullptr ? p.topk_w[t * p.k + j0 + j] : 1.0f;
        const void* src = at < 0 ? static_cast<const void*>(&kZeros)
                                 : static_cast<const char*>(p.rows) + (at * p.ldr + c * 8) * Elem<kIn>::kBytes;
        v[j] = *reinterpret_cast<const typename Elem<kIn>::Vec*>(src);
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) y += w[j] * to_f32(v[j]);
    }
    store8<kOut>(p.y, t * p.ldy + c * 8, y);
  }
}

// The sum over kLanes lanes, a wave's at most.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = min(kLanes, kWave) / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// kLanes lanes take a token, eight columns to a lane and step. Bound: HBM. Rows
// are read and written once, past the caches that others use: 4096 tokens of 2048
// columns, top-8, bf16: 56 us, 5.1 TB/s.
template <int kIn, int kOut, int kLanes>
__global__ __launch_bounds__(kThreads) void combine_grad(CombineArgs p) {
  typedef typename Elem<kIn>::Vec V;
  constexpr int kTokens = kThreads / kLanes;
  constexpr int kParts = kLanes / kWave;               // waves of a token, where they are several
  __shared__ float part[kThreads / kWave][kSlots];
  const int pieces = p.H / 8;
  const int lane = threadIdx.x % kLanes;
  for (int64_t t0 = blockIdx.x * int64_t(kTokens); t0 < p.M; t0 += int64_t(gridDim.x) * kTokens) {
    const int64_t t = t0 + threadIdx.x / kLanes;
    const bool here = t < p.M;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      float w[kSlots], dot[kSlots];
      int at[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        at[j] = here ? row_of(p, t, j0 + j) : -1;
        w[j] = at[j] < 0 ? 0.0f : p.topk_w != nullptr ? p.topk_w[t * p.k + j0 + j] : 1.0f;
        dot[j] = 0.0f;
      }
      for (int c = lane; here && c < pieces; c += kLanes) {
        const floatx8 dy = to_f32(load8<kOut>(p.dy, t * p.ldy + c * 8));
        if (p.dtopk_w != nullptr) {
          V v[kSlots];
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            const void* src = at[j] < 0 ? static_cast<const void*>(&kZeros)
                                        : static_cast<const char*>(p.rows) +
                                              (at[j] * p.ldr + c * 8) * Elem<kIn>::kBytes;
            v[j] = __builtin_nontemporal_load(static_cast<const V*>(src));
          }
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            const floatx8 r = to_f32(v[j]);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[j] += r[q] * dy[q];
          }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          if (at[j] < 0) continue;
          void* dst = static_cast<char*>(p.drows) + (at[j] * p.lddr + c * 8) * Elem<kIn>::kBytes;
          __builtin_nontemporal_store(__builtin_convertvector(w[j] * dy, V), static_cast<V*>(dst));
        }
      }
      if (p.dtopk_w == nullptr) continue;
#pragma unroll
      for (int j = 0; j < kSlots; ++j) dot[j] = lanes_sum<kLanes>(dot[j]);
      if constexpr (kParts > 1) {
        if (threadIdx.x % kWave == 0) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j) part[threadIdx.x / kWave][j] = dot[j];
        }
        lds_barrier();                        // (__syncthreads would wait for the stores, too)
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j) {
            dot[j] = part[threadIdx.x / kWave][j];
            for (int v = 1; v < kParts; ++v) dot[j] += part[threadIdx.x / kWave + v][j];
          }
        }
        lds_barrier();
      }
      if (here && lane == 0) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)       // a slot without a row: 0, whatever dy holds
          if (j0 + j < p.k) p.dtopk_w[t * p.k + j0 + j] = at[j] < 0 ? 0.0f : dot[j];
      }
    }
  }
}

// positions[r] = the row of route r, -1 without one. The fill comes before the
// scatter: by a barrier in one workgroup, by a second launch in several. Routes
// have one row each, so the stores meet no others (a maximum by atomics, which
// would order them, takes 6.5 us for 4096 routes in place of 3.4, 43 for 2^20 in
// place of 16).
__device__ __forceinline__ void scatter_positions(const int32_t* sorted, int live, int routes, int32_t* positions,
                                                  int first, int step) {
  constexpr int kBatch = 4;                 // loads in flight
  for (int64_t i = first; i < live; i += int64_t(kBatch) * step) {
    int r[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) r[q] = i + int64_t(q) * step < live ? sorted[i + int64_t(q) * step] : -1;
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
      if (r[q] >= 0 && r[q] < routes) positions[r[q]] = static_cast<int>(i + int64_t(q) * step);
  }
}

__global__ __launch_bounds__(kPositionThreads) void positions_single(const int32_t* __restrict__ sorted,
                                                                     const int32_t* __restrict__ num_padded,
                                                                     int capacity, int routes, int32_t* positions) {
  for (int r = threadIdx.x; r < routes; r += kPositionThreads) positions[r] = -1;
  __syncthreads();
  scatter_positions(sorted, min(capacity, num_padded[0]), routes, positions, threadIdx.x, kPositionThreads);
}

__global__ __launch_bounds__(kScatterThreads) void positions_fill(int routes, int32_t* positions) {
  for (int64_t r = blockIdx.x * kScatterThreads + threadIdx.x; r < routes; r += gridDim.x * kScatterThreads)
    positions[r] = -1;
}

__global__ __launch_bounds__(kScatterThreads) void positions_scatter(const int32_t* __restrict__ sorted,
                                                                     const int32_t* __restrict__ num_padded,
                                                                     int capacity, int routes, int32_t* positions) {
  scatter_positions(sorted, min(capacity, num_padded[0]), routes, positions,
                    blockIdx.x * kScatterThreads + threadIdx.x, gridDim.x * kScatterThreads);
}

template <int kIn, int kOut>
void start_combine(const CombineArgs& p, hipStream_t stream) {
  const int64_t n = p.M * int64_t(p.H / 8);
  launch(combine<kIn, kOut>, dim3(grid_for((n + kThreads - 1) / kThreads, 0)), dim3(kThreads), 0, stream, p);
}

template <int kIn, int kOut>
void start_combine_grad(const CombineArgs& p, hipStream_t stream) {
  // As many lanes as a row has pieces, up to a workgroup: 4096 tokens of 2048 columns, top-8, bf16: 256 lanes 56 us,
  // 64 lanes 74 (through the caches: 67 and 77); 16384 of 256: 32 lanes 31, 64 lanes 46, 256 lanes 136. Two routes
  // of 1024 columns in fp32 alone would do better with fewer (128 lanes 50, 64 lanes 42).
  const int pieces = p.H / 8;
  const auto grid = [&](int lanes) { return dim3(grid_for((p.M * lanes + kThreads - 1) / kThreads, 0)); };
  if (pieces <= 32)
    launch(combine_grad<kIn, kOut, 32>, grid(32), dim3(kThreads), 0, stream, p);
  else if (pieces <= 64)
    launch(combine_grad<kIn, kOut, 64>, grid(64), dim3(kThreads), 0, stream, p);
  else if (pieces <= 128)
    launch(combine_grad<kIn, kOut, 128>, grid(128), dim3(kThreads), 0, stream, p);
  else
    launch(combine_grad<kIn, kOut, 256>, grid(256), dim3(kThreads), 0, stream, p);
}

template <int kIn>
void by_output(const CombineArgs& p, int out, bool grad, hipStream_t stream) {
  if (out == MOE_DTYPE_F32)
    grad ? start_combine_grad<kIn, MOE_DTYPE_F32>(p, stream) : start_combine<kIn, MOE_DTYPE_F32>(p, stream);
  else if (out == MOE_DTYPE_BF16)
    grad ? start_combine_grad<kIn, MOE_DTYPE_BF16>(p, stream) : start_combine<kIn, MOE_DTYPE_BF16>(p, stream);
  else
    grad ? start_combine_grad<kIn, MOE_DTYPE_F16>(p, stream) : start_combine<kIn, MOE_DTYPE_F16>(p, stream);
}

hipError_t by_input(const CombineArgs& p, int dtype, int y_dtype, bool grad, hipStream_t stream) {
  if (dtype == MOE_DTYPE_F32)
    by_output<MOE_DTYPE_F32>(p, y_dtype, grad, stream);
  else if (dtype == MOE_DTYPE_BF16)
    by_output<MOE_DTYPE_BF16>(p, y_dtype, grad, stream);
  else
    by_output<MOE_DTYPE_F16>(p, y_dtype, grad, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& p, int dtype, int y_dtype, hipStream_t stream) {
  return by_input(p, dtype, y_dtype, false, stream);
}

hipError_t launch_combine_grad(const CombineArgs& p, int dtype, int y_dtype, hipStream_t stream) {
  return by_input(p, dtype, y_dtype, true, stream);
}

hipError_t launch_positions(const int32_t* sorted, const int32_t* num_padded, int capacity, int routes,
                            int32_t* positions, hipStream_t stream) {
  if (routes <= kPositionsSingle && capacity <= kPositionsSingle) {
    launch(positions_single, dim3(1), dim3(kPositionThreads), 0, stream, sorted, num_padded, capacity, routes,
           positions);
  } else {
    const int fill = (routes + kScatterThreads - 1) / kScatterThreads;
    const int scatter = (capacity + kScatterThreads - 1) / kScatterThreads;
    launch(positions_fill, dim3(min(fill, 4096)), dim3(kScatterThreads), 0, stream, routes, positions);
    launch(positions_scatter, dim3(min(max(scatter, 1), 4096)), dim3(kScatterThreads), 0, stream, sorted, num_padded,
           capacity, routes, positions);
  }
  return hipGetLastError();
}

}  // namespace moe
