// Routing to experts (gfx950): scores, choice in groups, top-k, weights, and
// the gradient of the weights with respect to the logits.
//
// Score s_e = softmax(l)_e or sigmoid(l_e); choice value c_e = s_e + b_e, or
// without a bias the logit itself, whose order is the score's. Groups are
// ranked by the sum of their group_top largest choice values, the k largest of
// the kept groups win, ties go to the lowest index.
//
// The choice is made on 64-bit values: an fp32 evaluation would order close
// experts by its own rounding, and the same token would take other routes in
// another kernel, batch or framework. The weights are fp32.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// An element of a row of logits as fp32 (exact for the 16-bit types).
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype) {
  if (dtype == MOE_DTYPE_F32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == MOE_DTYPE_BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : half_bits_to_float(h);
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int dtype, float v) {
  if (dtype == MOE_DTYPE_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_DTYPE_BF16)
    static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
  else
    static_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
}

// Ordered 64-bit keys of choice values: larger key, larger value; -0 equals 0,
// a NaN is above every number, kNoKey (below every number) is no candidate.
constexpr int64_t kNoKey = INT64_MIN;
constexpr int64_t kNanKey = INT64_MAX;

__device__ __forceinline__ int64_t key_of(double v) {
  if (v != v) return kNanKey;
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & INT64_MAX);
}

__device__ __forceinline__ double value_of(int64_t key) {   // of a key that is neither kNoKey nor kNanKey
  return __longlong_as_double(key ^ ((key >> 63) & INT64_MAX));
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

// A wave takes a row. Lanes are dealt to groups (`per_group` of them each, a
// power of two), a lane owns C consecutive experts of its group at most, so
// that experts ascend with (lane, place).
template <int C>
__global__ __launch_bounds__(kThreads) void route(RouteArgs p) {
  const int lane = threadIdx.x & (kWave - 1);
  const int group = lane / p.per_group;
  const int first = group * p.group_size + (lane % p.per_group) * p.per_lane;
  const int end = group < p.groups ? min(first + p.per_lane, (group + 1) * p.group_size) : first;
  for (int64_t row = blockIdx.x * int64_t(kWaves) + threadIdx.x / kWave; row < p.M; row += int64_t(gridDim.x) * kWaves) {
    const int64_t at = row * p.ld;
    float l[C];
    bool live[C];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const bool here = first + i < end;
      l[i] = here ? load_elem(p.logits, at + first + i, p.dtype) : -INFINITY;
      live[i] = here && !(l[i] == -INFINITY);
      top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    float total = 0.0f;       // of the softmax, relative to `top`
    if (p.score == MOE_SCORE_SOFTMAX && !p.renormalize) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (live[i]) total += expf(l[i] - top);
      total = wave_sum(total);
    }
    // Choice values as keys; `by_score` holds the scores' where groups are summed and no bias is given.
    int64_t key[C], by_score[C];
    double total64 = 0.0;
    if (p.exact_scores && p.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (live[i]) total64 += exp(static_cast<double>(l[i]) - top);
      total64 = wave_sum64(total64);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      key[i] = by_score[i] = kNoKey;
      if (!live[i]) continue;
      double s = l[i];
      if (p.exact_scores)
        s = p.score == MOE_SCORE_SOFTMAX ? exp(s - top) / total64 : 1.0 / (1.0 + exp(-s));
      if (p.bias != nullptr) {
        const float b = p.bias[first + i];
        if (b == -INFINITY) continue;
        key[i] = by_score[i] = key_of(s + b);
      } else {
        key[i] = key_of(static_cast<double>(l[i]));
        by_score[i] = key_of(s);
      }
    }
    if (p.topk_groups < p.groups) {
      int64_t a = kNoKey, b = kNoKey;       // the two largest of the group
#pragma unroll
      for (int i = 0; i < C; ++i) {
        b = max(b, min(a, by_score[i]));
        a = max(a, by_score[i]);
      }
      for (int off = 1; off < p.per_group; off <<= 1) {
        const int64_t oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
        b = max(min(a, oa), max(b, ob));
        a = max(a, oa);
      }
      int64_t g = a;
      if (p.group_top == 2 && a != kNanKey && b != kNoKey) g = key_of(value_of(a) + value_of(b));
      int rank = 0;
      for (int o = 0; o < p.groups; ++o) {
        const int64_t og = __shfl(g, o * p.per_group, kWave);
        rank += (og > g || (og == g && o < group)) ? 1 : 0;
      }
      if (rank >= p.topk_groups) {
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = kNoKey;
      }
    }
    int mine = -1;                          // expert of slot `lane`
    for (int j = 0; j < p.k; ++j) {
      int64_t best = kNoKey;
      int e = INT32_MAX;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (key[i] > best) {
          best = key[i];
          e = first + i;
        }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        const int64_t ob = __shfl_xor(best, off, kWave);
        const int oe = __shfl_xor(e, off, kWave);
        if (ob > best || (ob == best && oe < e)) {
          best = ob;
          e = oe;
        }
      }
      if (best == kNoKey) break;
      if (lane == j) mine = e;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (first + i == e) key[i] = kNoKey;
    }
    float s = 0.0f;
    const float chosen = mine >= 0 ? load_elem(p.logits, at + mine, p.dtype) : -INFINITY;
    if (p.renormalize) {
      // Relative to the largest chosen score, so that small scores do not vanish.
      float m = wave_max(chosen);
      if (p.score == MOE_SCORE_SOFTMAX) {
        s = mine >= 0 ? expf(chosen - m) : 0.0f;
      } else {
        m = fminf(m, 0.0f);
        s = mine >= 0 ? expf(fminf(chosen, 0.0f) - m) / (1.0f + expf(-fabsf(chosen))) : 0.0f;
      }
      s /= wave_sum(s);
    } else if (p.score == MOE_SCORE_SOFTMAX) {
      s = expf(chosen - top) / total;
    } else {
      s = 1.0f / (1.0f + expf(-chosen));
    }
    if (lane < p.k) {
      p.topk_ids[row * p.k + lane] = mine;
      p.topk_w[row * p.k + lane] = mine >= 0 ? p.scale * s : 0.0f;
    }
  }
}

// A wave takes a row: lane j holds slot j. With c = scale, p the scores and
// u = p / sum of the chosen p:
//   softmax               dl_e = c p_e ([e chosen] g_e - sum_j g_j p_j)
//   softmax, renormalised dl_j = c u_j (g_j - sum_i g_i u_i), 0 elsewhere
//   sigmoid               dl_j = c g_j p_j (1 - p_j)
//   sigmoid, renormalised dl_j = c u_j (1 - p_j) (g_j - sum_i g_i u_i)
// Slots are separate arguments: an expert named twice gets both slots' shares.
__global__ __launch_bounds__(kThreads) void route_grad(RouteGradArgs p) {
  extern __shared__ float rows_lds[];
  const int lane = threadIdx.x & (kWave - 1);
  float* buf = rows_lds + (threadIdx.x / kWave) * p.E;
  for (int64_t row = blockIdx.x * int64_t(kWaves) + threadIdx.x / kWave; row < p.M; row += int64_t(gridDim.x) * kWaves) {
    const int64_t at = row * p.ld;
    int id = lane < p.k ? p.topk_ids[row * p.k + lane] : -1;
    if (id >= p.E) id = -1;
    const bool valid = id >= 0;
    const float g = valid ? p.scale * p.dtopk_w[row * p.k + lane] : 0.0f;
    const float l = valid ? load_elem(p.logits, at + id, p.dtype) : -INFINITY;
    float d = 0.0f, back = 0.0f, top = 0.0f, total = 1.0f;
    const bool dense = p.score == MOE_SCORE_SOFTMAX && !p.renormalize;
    const bool any = __ballot(valid) != 0;
    if (dense && any) {
      top = -INFINITY;
      for (int e = lane; e < p.E; e += kWave) top = fmaxf(top, load_elem(p.logits, at + e, p.dtype));
      top = wave_max(top);
      total = 0.0f;
      for (int e = lane; e < p.E; e += kWave) {
        const float v = load_elem(p.logits, at + e, p.dtype);
        total += v == -INFINITY ? 0.0f : expf(v - top);
      }
      total = wave_sum(total);
      const float s = valid ? expf(l - top) / total : 0.0f;
      d = valid ? g * s : 0.0f;
      back = wave_sum(d);
    } else if (p.score == MOE_SCORE_SOFTMAX) {
      const float m = wave_max(l);
      const float e = valid ? expf(l - m) : 0.0f;
      const float u = e / wave_sum(e);
      const float dot = wave_sum(valid ? g * u : 0.0f);
      d = valid ? u * (g - dot) : 0.0f;
    } else {
      const float q = 1.0f / (1.0f + expf(l));       // 1 - p
      if (p.renormalize) {
        const float m = fminf(wave_max(l), 0.0f);
        const float e = valid ? expf(fminf(l, 0.0f) - m) / (1.0f + expf(-fabsf(l))) : 0.0f;
        const float u = e / wave_sum(e);
        const float dot = wave_sum(valid ? g * u : 0.0f);
        d = valid ? u * q * (g - dot) : 0.0f;
      } else {
        d = valid ? g * q / (1.0f + expf(-l)) : 0.0f;
      }
    }
    // Slots that name the same expert: each takes their sum, in slot order.
    float sum = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int oid = __shfl(id, j, kWave);
      const float od = __shfl(d, j, kWave);
      if (oid == id) sum += od;
    }
    for (int e = lane; e < p.E; e += kWave) {
      float v = 0.0f;
      if (dense && any) {
        const float x = load_elem(p.logits, at + e, p.dtype);
        v = x == -INFINITY ? 0.0f : -expf(x - top) / total * back;
      }
      buf[e] = v;
    }
    // The lanes of a wave exchange through LDS without a barrier: its accesses stay in order.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float before = valid ? buf[id] : 0.0f;
    __builtin_amdgcn_wave_barrier();
    if (valid) buf[id] = before + sum;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int e = lane; e < p.E; e += kWave) store_elem(p.dlogits, row * p.ldd + e, p.out_dtype, buf[e]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  RouteArgs p = a;
  p.group_size = p.E / p.groups;
  p.per_group = 1;
  while (p.per_group * 2 * p.groups <= kWave) p.per_group *= 2;
  p.per_lane = (p.group_size + p.per_group - 1) / p.per_group;
  // Scores are needed for the choice with a bias, and where they are summed over a group.
  p.exact_scores = p.bias != nullptr || (p.topk_groups < p.groups && p.group_top == 2);
  const dim3 grid(grid_for((p.M + kWaves - 1) / kWaves, 0)), block(kThreads);
  if (p.per_lane <= 2)
    launch(route<2>, grid, block, 0, stream, p);
  else if (p.per_lane <= 8)
    launch(route<8>, grid, block, 0, stream, p);
  else if (p.per_lane <= 32)
    launch(route<32>, grid, block, 0, stream, p);
  else
    launch(route<64>, grid, block, 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& p, hipStream_t stream) {
  const dim3 grid(grid_for((p.M + kWaves - 1) / kWaves, 0)), block(kThreads);
  launch(route_grad, grid, block, sizeof(float) * kWaves * p.E, stream, p);
  return hipGetLastError();
}

}  // namespace moe
