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
#include <type_traits>

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

// How the experts of a row are dealt to `lanes` lanes: `per_group` of them (a
// power of two) to each group, each with `per_lane` consecutive experts of it at
// most, so that experts ascend with (lane, place).
struct Deal {
  int group, first, end;
};
__device__ __forceinline__ Deal deal(const RouteLayout& y, int lane, int groups, int group_size) {
  Deal d;
  d.group = lane / y.per_group;
  d.first = d.group * group_size + (lane % y.per_group) * y.per_lane;
  d.end = d.group < groups ? min(d.first + y.per_lane, (d.group + 1) * group_size) : d.first;
  return d;
}

// The weight of this lane's slot (expert `mine`, or -1), before p.scale; `top` and
// `total` are the largest logit and the softmax's sum relative to it. kMax and
// kSum reduce over the lanes that hold the row's slots.
template <typename Max, typename Sum>
__device__ __forceinline__ float weight_of(const RouteArgs& p, int mine, float chosen, float top, float total, Max kMax,
                                           Sum kSum) {
  if (p.renormalize) {
    // Relative to the largest chosen score, so that small scores do not vanish.
    float m = kMax(mine >= 0 ? chosen : -INFINITY);
    float s;
    if (p.score == MOE_SCORE_SOFTMAX) {
      s = mine >= 0 ? expf(chosen - m) : 0.0f;
    } else {
      m = fminf(m, 0.0f);
      s = mine >= 0 ? expf(fminf(chosen, 0.0f) - m) / (1.0f + expf(-fabsf(chosen))) : 0.0f;
    }
    return s / kSum(s);
  }
  return p.score == MOE_SCORE_SOFTMAX ? expf(chosen - top) / total : 1.0f / (1.0f + expf(-chosen));
}

// The lanes of a wave exchange through LDS without a barrier: its accesses stay in order.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A value of another of sixteen neighbouring lanes (rotated by kBy).
template <int kBy>
__device__ __forceinline__ float ror(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 | kBy, 0xF, 0xF, false));
}
template <int kBy>
__device__ __forceinline__ int ror(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 | kBy, 0xF, 0xF, false);
}

template <int kBy>
__device__ __forceinline__ int64_t ror(int64_t v) {
  const uint32_t lo = ror<kBy>(static_cast<int>(v)), hi = ror<kBy>(static_cast<int>(v >> 32));
  return static_cast<int64_t>(uint64_t(hi) << 32 | lo);
}
template <int kBy>
__device__ __forceinline__ double ror(double v) {
  return __longlong_as_double(ror<kBy>(static_cast<int64_t>(__double_as_longlong(v))));
}

// One row by a whole wave, every choice value in 64 bits and kept in LDS (E
// keys): any sizes, and the rows that `route_narrow` cannot decide.
__device__ __forceinline__ void route_exact(const RouteArgs& p, int64_t row, int64_t* key) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t at = row * p.ld;
  const auto logit = [&](int e) { return load_elem(p.logits, at + e, p.dtype); };
  float top = -INFINITY, total = 0.0f;      // of the softmax, relative to `top`
  double total64 = 0.0;
  if (p.score == MOE_SCORE_SOFTMAX) {
    for (int e = lane; e < p.E; e += kWave) top = fmaxf(top, logit(e));
    top = wave_max(top);
    for (int e = lane; e < p.E; e += kWave) {
      const float l = logit(e);
      if (l == -INFINITY) continue;
      if (!p.renormalize) total += expf(l - top);
      if (p.exact_scores) total64 += exp(static_cast<double>(l) - top);
    }
    total = wave_sum(total);
    total64 = wave_sum64(total64);
  }
  // Keys of the choice values; of the scores alone, where those are summed over groups without a bias.
  for (int e = lane; e < p.E; e += kWave) {
    const float l = logit(e), b = p.bias != nullptr ? p.bias[e] : 0.0f;
    double s = l;
    if (p.exact_scores) s = (p.score == MOE_SCORE_SOFTMAX ? exp(s - top) / total64 : 1.0 / (1.0 + exp(-s))) + b;
    key[e] = l == -INFINITY || b == -INFINITY ? kNoKey : key_of(s);
  }
  wave_lds_fence();
  if (p.topk_groups < p.groups) {
    const Deal d = deal(p.wide, lane, p.groups, p.group_size);
    int64_t a = kNoKey, b = kNoKey;         // the two largest of the group
    for (int e = d.first; e < d.end; ++e) {
      b = max(b, min(a, key[e]));
      a = max(a, key[e]);
    }
    for (int off = 1; off < p.wide.per_group; off <<= 1) {
      const int64_t oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    int64_t g = a;
    if (p.group_top == 2 && a != kNanKey && b != kNoKey) g = key_of(value_of(a) + value_of(b));
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const int64_t og = __shfl(g, o * p.wide.per_group, kWave);
      rank += (og > g || (og == g && o < d.group)) ? 1 : 0;
    }
    for (int e = d.first; e < d.end; ++e) {
      if (rank >= p.topk_groups)
        key[e] = kNoKey;
      else if (p.bias == nullptr && p.exact_scores && key[e] != kNoKey)
        key[e] = key_of(logit(e));
    }
    wave_lds_fence();
  }
  int mine = -1;                            // expert of slot `lane`
  for (int j = 0; j < p.k; ++j) {
    int64_t best = kNoKey;
    int e = INT32_MAX;
    for (int i = lane; i < p.E; i += kWave) {
      const int64_t t = key[i];
      if (t > best) {
        best = t;
        e = i;
      }
    }
    const auto take = [&](int64_t ob, int oe) {
      if (ob > best || (ob == best && oe < e)) {
        best = ob;
        e = oe;
      }
    };
    take(ror<8>(best), ror<8>(e));
    take(ror<4>(best), ror<4>(e));
    take(ror<2>(best), ror<2>(e));
    take(ror<1>(best), ror<1>(e));
    take(__shfl_xor(best, 16, kWave), __shfl_xor(e, 16, kWave));
    take(__shfl_xor(best, 32, kWave), __shfl_xor(e, 32, kWave));
    if (best == kNoKey) break;
    if (lane == j) mine = e;
    if (lane == 0) key[e] = kNoKey;
    wave_lds_fence();
  }
  const float chosen = mine >= 0 ? logit(mine) : -INFINITY;
  const float s = weight_of(p, mine, chosen, top, total, [](float v) { return wave_max(v); },
                            [](float v) { return wave_sum(v); });
  if (lane < p.k) {
    p.topk_ids[row * p.k + lane] = mine;
    p.topk_w[row * p.k + lane] = mine >= 0 ? p.scale * s : 0.0f;
  }
  wave_lds_fence();
}

__global__ __launch_bounds__(kThreads) void route_wide(RouteArgs p) {
  extern __shared__ int64_t keys[];
  for (int64_t row = blockIdx.x * int64_t(kWaves) + threadIdx.x / kWave; row < p.M; row += int64_t(gridDim.x) * kWaves)
    route_exact(p, row, keys + threadIdx.x / kWave * p.E);
}

constexpr int kLanes = 16;                 // of a row in route_narrow
constexpr int kRows = kThreads / kLanes;

// Reductions over a row's sixteen lanes; every lane ends with the same bits.
template <typename V>
__device__ __forceinline__ V row_max(V v) {
  v = max(v, ror<8>(v));
  v = max(v, ror<4>(v));
  v = max(v, ror<2>(v));
  return max(v, ror<1>(v));
}
template <typename V>
__device__ __forceinline__ V row_sum(V v) {
  v += ror<8>(v);
  v += ror<4>(v);
  v += ror<2>(v);
  return v + ror<1>(v);
}

// The value of a lane's partner in the merge of 2, 4, 8 and 16 lanes, when the
// halves that are merged hold the same values in all their lanes.
template <int kStep, typename V>
__device__ __forceinline__ V partner(V v) {
  constexpr int kCtrl = kStep == 1 ? 0xB1 : kStep == 2 ? 0x4E : kStep == 4 ? 0x141 : 0x140;
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, i, kCtrl, 0xF, 0xF, false));
}

template <typename V>
__device__ __forceinline__ V none();      // below every value
template <>
__device__ __forceinline__ float none<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ int none<int>() { return INT32_MIN; }

// Ordered 32-bit key of a logit, as key_of.
__device__ __forceinline__ int key32(float v) {
  if (v == -INFINITY) return INT32_MIN;
  if (v != v) return INT32_MAX;
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & INT32_MAX);
}

template <int kStep>
__device__ __forceinline__ double partner(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = partner<kStep>(static_cast<int>(b)), hi = partner<kStep>(static_cast<int>(b >> 32));
  return __longlong_as_double(static_cast<int64_t>(uint64_t(hi) << 32 | lo));
}

// The sum of the values of the row's lanes before this one.
__device__ __forceinline__ int row_before(int v) {
  int x = v;
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
  return x - v;
}

// The logit of a key32 that is none of its ends.
__device__ __forceinline__ float logit_of(int key) { return __int_as_float(key ^ ((key >> 31) & INT32_MAX)); }

// e^x from the hardware's 2^x: within |x| 2^-23 + 2^-22 of it, relatively. It serves the choice, whose bounds
// count it, and the sum and the gradient over a whole row, where it weighs p |x| 2^-23: below 2^-24 of the largest score.
// A chosen expert's weight takes expf.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Sixteen lanes take a row, so a wave chooses for four at once. Values to rank
// by: ordered keys of the logits, which are exact, or with a bias fp32 choice
// values c = s + b, off by err + |c| 2^-24 at most. err: a sigmoid moves by
// s (1 - s) |x| 2^-23 < 2^-25 through fast_exp's argument and by 2^-22 with its
// roundings, for which 2^-21 stands; a softmax by its own and its sum's share,
// (6.3 + 0.4) 2^-23 (the mean distance to the largest of 512 logits is below their
// entropy's bound, ln 512) and 36 additions of 2^-24, for which 2^-18 stands.
//   1. every lane finds the two largest of its C values;
//   2. groups are ranked by them; where two fp32 ranks are too close to decide, the
//      values that can be among the two largest are evaluated in 64 bits;
//   3. the k-th largest T of all lanes' two largest bounds the k-th largest of the
//      row from below: what is below T, less the errors, is out. That is near where k
//      is well below the number of those values (256 experts, 13 slots: 4 % of the rows
//      keep more than sixteen) and not where many slots or few groups make k of them
//      most (16 slots: 80 %; 6 slots of one of eight groups: all). Such a row bisects
//      its ordered keys for a T that at least k and at most sixteen values reach;
//   4. the rest, a few more than k, go one to a lane (through LDS, in index order),
//      are ranked by exact 64-bit values by counting, and those below k are chosen.
// A softmax's 64-bit sum is formed only for waves with values that its fp32 one does
// not tell apart. A row with a NaN, or with more than sixteen values left in step 4
// (with a bias: values equal to the k-th within the errors), goes to route_exact.
// Bound: VALU and its waits (1260 instructions a wave, three waves a SIMD): 32768
// rows of 256 experts in groups, with a bias, 8 slots 31 us, 12 slots 34, 16 slots 55
// (before the bisection 31, 100, 231; a wave a row 84, 107, 128); eight slots of one
// group 41 (157; 84); without bias and groups 8 slots 16, 16 slots 24 (16, 161; 120).
// Rows read in whole pieces stay in LDS, too, for step 4 (read again from memory they cost 4 us of 36).
template <int C, bool kBias>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(C > 16 ? 2 : kBias ? 3 : 4))) void route_narrow(
    RouteArgs p) {
  extern __shared__ int64_t keys[];         // for route_exact, then the rows' logits
  using V = std::conditional_t<kBias, float, int>;
  struct Row {
    union {
      V top[2 * kLanes];
      int64_t key[kLanes];
      double value[kLanes];
    };
    int id[kLanes];
    float logit[kLanes];
    uint32_t apart[4];                     // the four rows of a wave start in different banks
  };
  __shared__ __attribute__((aligned(16))) Row lds[kRows];
  const float err = p.score == MOE_SCORE_SIGMOID ? 0x1p-21f : 0x1p-18f;
  Row& mem = lds[threadIdx.x / kLanes];
  float* logits = reinterpret_cast<float*>(keys + kWaves * p.E) + threadIdx.x / kLanes * p.E;
  for (int64_t row0 = blockIdx.x * int64_t(kRows); row0 < p.M; row0 += int64_t(gridDim.x) * kRows) {
    // Opaque, or the compiler keeps what depends on it alone in (spilled) scalars across rows.
    const int lane = in_vgpr(threadIdx.x % kLanes);
    const Deal d = deal(p.narrow, lane, p.groups, p.group_size);
    const int64_t row = row0 + threadIdx.x / kLanes;
    const bool here = row < p.M;
    const int64_t at = row * p.ld;
    float l[C];
    if (p.vector && here) {
      const int64_t first = at + d.first;
      if (p.dtype == MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
          const floatx4 v = reinterpret_cast<const floatx4*>(static_cast<const float*>(p.logits) + first)[i];
#pragma unroll
          for (int q = 0; q < 4; ++q) l[4 * i + q] = v[q];
        }
      } else {
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
          const u32x4 v = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.logits) + first)[i];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            l[8 * i + 2 * q] = p.dtype == MOE_DTYPE_BF16 ? bf16_lo(v[q]) : half_bits_to_float(v[q] & 0xFFFF);
            l[8 * i + 2 * q + 1] = p.dtype == MOE_DTYPE_BF16 ? bf16_hi(v[q]) : half_bits_to_float(v[q] >> 16);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        l[i] = here && d.first + i < d.end ? load_elem(p.logits, at + d.first + i, p.dtype) : -INFINITY;
    }
    if (p.vector) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i)
        reinterpret_cast<floatx4*>(logits + d.first)[i] = floatx4{l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]};
    }
    // The softmax's largest logit and its sum, where something needs them.
    float top = 0.0f, total = 1.0f;
    if (p.score == MOE_SCORE_SOFTMAX && (kBias || !p.renormalize)) {
      top = l[0];
#pragma unroll
      for (int i = 1; i < C; ++i) top = fmaxf(top, l[i]);
      top = row_max(top);
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) total += l[i] == -INFINITY ? 0.0f : fast_exp(l[i] - top);
      total = row_sum(total);
    }
    V v[C];
    bool open = false;                       // the row goes to route_exact
    if constexpr (kBias) {
      const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float b = d.first + i < d.end ? p.bias[d.first + i] : -INFINITY;
        const float s = p.score == MOE_SCORE_SOFTMAX ? fast_exp(l[i] - top) * inv
                                                     : __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[i]));
        v[i] = l[i] == -INFINITY ? -INFINITY : s + b;
        open |= v[i] != v[i];                // a NaN has no place among fp32 maxima
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = key32(l[i]);
    }
    V a = v[0], b = none<V>();
#pragma unroll
    for (int i = 1; i < C; ++i) {
      b = max(min(a, b), min(max(a, b), v[i]));   // the median, one instruction
      a = max(a, v[i]);
    }
    double total64 = total;                  // the softmax's sum, fp32's until `sum_exactly`
    const auto logit_at = [&](int e) { return p.vector ? logits[e] : load_elem(p.logits, at + e, p.dtype); };
    const auto sum_exactly = [&] {
      double t = 0.0;
      for (int e = d.first; here && e < d.end; ++e) {
        const float x = logit_at(e);
        if (x != -INFINITY) t += exp(static_cast<double>(x) - top);
      }
      total64 = row_sum(t);
    };
    const auto exact_value = [&](int e, float x) {
      const double l64 = x;
      return (p.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l64)) : exp(l64 - top) / total64) + p.bias[e];
    };
    if (p.topk_groups < p.groups) {
      const auto merge = [&](auto& ga, auto& gb, auto oa, auto ob) {
        gb = max(min(ga, oa), max(gb, ob));
        ga = max(ga, oa);
      };
      const auto merge_group = [&](auto& ga, auto& gb) {
        if (p.narrow.per_group > 1) merge(ga, gb, partner<1>(ga), partner<1>(gb));
        if (p.narrow.per_group > 2) merge(ga, gb, partner<2>(ga), partner<2>(gb));
        if (p.narrow.per_group > 4) merge(ga, gb, partner<4>(ga), partner<4>(gb));
      };
      // The groups' ranks by the 64-bit values of their two largest.
      const auto rank_exactly = [&](double xa, double xb) {
        merge_group(xa, xb);
        const double x = p.group_top == 2 && xb != -INFINITY ? xa + xb : xa;
        wave_lds_fence();
        mem.key[lane] = x == -INFINITY ? kNoKey : key_of(x);
        wave_lds_fence();
        const int64_t key = mem.key[lane];
        int n = 0;
        for (int o = 0; o < p.groups; ++o) {
          const int64_t ok = mem.key[o * p.narrow.per_group];
          n += (ok > key || (ok == key && o < d.group)) ? 1 : 0;
        }
        return n;
      };
      V ga = a, gb = b;
      merge_group(ga, gb);
      V g = ga;
      float close = 0.0f;                    // ranks this near to each other decide nothing
      if constexpr (kBias) {
        const bool two = p.group_top == 2 && gb != -INFINITY;
        if (two) g = ga + gb;
        const float size = (ga == -INFINITY ? 0.0f : fabsf(ga)) + (two ? fabsf(gb) : 0.0f);
        close = 4.0f * err + row_max(size) * 0x1p-21f;
      }
      mem.top[lane] = g;
      wave_lds_fence();
      int rank = 0;
      bool unsure = false;
      for (int o = 0; o < p.groups; ++o) {
        const V og = mem.top[o * p.narrow.per_group];
        rank += (og > g || (og == g && o < d.group)) ? 1 : 0;
        if constexpr (kBias) unsure |= o != d.group && g != -INFINITY && fabsf(og - g) <= close;
      }
      if constexpr (kBias) {
        unsure |= g == INFINITY;
        if (__any(unsure)) {
          if (p.score == MOE_SCORE_SOFTMAX) sum_exactly();
          const float low = b - (2.0f * err + fabsf(b) * 0x1p-21f);
          uint32_t near = 0;
#pragma unroll
          for (int i = C - 1; i >= 0; --i) near = near + near + (v[i] != -INFINITY && !(v[i] < low) ? 1 : 0);
          double xa = -INFINITY, xb = -INFINITY;
          while (near != 0) {
            const int e = d.first + __ffs(near) - 1;
            near &= near - 1;
            const double x = exact_value(e, logit_at(e));
            xb = max(xb, min(xa, x));
            xa = max(xa, x);
          }
          rank = rank_exactly(xa, xb);
        }
      } else if (p.exact_scores) {
        // Sums of scores without a bias: the two largest logits have the two largest scores. The softmax's sum
        // is a factor of all.
        const float most = row_max(a == INT32_MIN ? -INFINITY : logit_of(a));
        const auto score = [&](int key) {
          const double x = logit_of(key);
          return key == INT32_MIN ? -INFINITY : p.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-x)) : exp(x - most);
        };
        // A NaN, or a softmax of an infinite logit, makes more of the row NaN.
        open = a == INT32_MAX || (p.score == MOE_SCORE_SOFTMAX && a != INT32_MIN && logit_of(a) == INFINITY);
        rank = rank_exactly(score(a), score(b));
      }
      if (rank >= p.topk_groups) {
        a = b = none<V>();
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = none<V>();
      }
      wave_lds_fence();
    }
    mem.top[lane] = a;
    mem.top[kLanes + lane] = b;
    wave_lds_fence();
    int from_a = 0, from_b = 0;              // values from a, from b on
#pragma unroll
    for (int o = 0; o < 2 * kLanes; ++o) {
      const V t = mem.top[o];
      from_a += t >= a ? 1 : 0;
      from_b += t >= b ? 1 : 0;
    }
    V bound = row_max(max(from_a >= p.k ? a : none<V>(), from_b >= p.k ? b : none<V>()));
    uint32_t left;                           // places that stay
    const auto keep = [&](int larger) {      // at least so many values above the bound
      left = 0;
      if constexpr (kBias) {
        const float low = bound == INFINITY ? bound : bound - (2.0f * err + fabsf(bound) * 0x1p-21f);
#pragma unroll
        for (int i = C - 1; i >= 0; --i) left = left + left + (v[i] >= low && v[i] != -INFINITY ? 1 : 0);
      } else {
        // Equal keys are equal values: the first of those at the bound are enough.
        uint32_t same = 0;
#pragma unroll
        for (int i = C - 1; i >= 0; --i) {
          left = left + left + (v[i] > bound ? 1 : 0);
          same = same + same + (v[i] == bound && v[i] != INT32_MIN ? 1 : 0);
        }
        int room = p.k - larger - row_before(__popc(same));
        for (; room > 0 && same != 0; --room) {
          left |= same & -same;
          same &= same - 1;
        }
      }
      return row_sum(static_cast<int>(__popc(left)));
    };
    int all = keep(0);
    if (__any(all > kLanes)) {
      // Many slots on few lanes. Where no value has at most sixteen at or above it, the k-th largest itself is found.
      const auto key = [](V t) { if constexpr (kBias) return key32(t); else return t; };
      const auto value = [](int t) { if constexpr (kBias) return logit_of(t); else return t; };
      // Opaque, or comparisons are kept from `keep` above, as scalars that others are spilled for.
#pragma unroll
      for (int i = 0; i < C; ++i) asm volatile("" : "+v"(v[i]));
      int lo = key(bound), hi = key(row_max(a));      // k values at least reach lo
      if (lo == INT32_MIN) {
        int least = INT32_MAX;
#pragma unroll
        for (int i = 0; i < C; ++i) least = min(least, v[i] == none<V>() ? INT32_MAX : key(v[i]));
        lo = -row_max(-least);
      }
      bool going = all > kLanes && lo < hi;
      while (__any(going)) {
        const int mid = lo + static_cast<int>((static_cast<uint32_t>(hi) - static_cast<uint32_t>(lo) + 1) / 2);
        const V t = value(mid);
        int n = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) n += v[i] >= t ? 1 : 0;
        n = row_sum(n);
        if (going && n >= p.k) lo = mid;
        if (going && n < p.k) hi = mid - 1;
        going = going && lo < hi && !(n >= p.k && n <= kLanes);
      }
      int larger = 0;
      if constexpr (!kBias) {
        if (all > kLanes) bound = lo;
#pragma unroll
        for (int i = 0; i < C; ++i) larger += v[i] > bound ? 1 : 0;
        larger = row_sum(larger);
      } else if (all > kLanes) {
        bound = value(lo);
      }
      all = keep(larger);
    }
    int slot = row_before(__popc(left));
    open = row_max(open || all > kLanes ? 1 : 0) != 0;
    if (!open) {
      while (left != 0) {
        mem.id[slot++] = d.first + __ffs(left) - 1;
        left &= left - 1;
      }
    }
    wave_lds_fence();
    int id = lane < all && !open ? mem.id[lane] : -1;
    float chosen = id < 0 ? -INFINITY : logit_at(id);
    int rank = 0;
    if constexpr (kBias) {
      for (bool exact = p.score == MOE_SCORE_SIGMOID;;) {
        const double c = id >= 0 ? exact_value(id, chosen) : -INFINITY;
        mem.value[lane] = c;
        wave_lds_fence();
        rank = 0;
        bool unsure = false;
#pragma unroll
        for (int o = 0; o < kLanes; ++o) {
          const double t = mem.value[o];
          rank += (t > c || (t == c && o < lane)) ? 1 : 0;
          unsure |= o != lane && fabs(t - c) <= 2.0 * err;
        }
        wave_lds_fence();
        if (exact || !__any(unsure && id >= 0)) break;
        sum_exactly();
        exact = true;
      }
    } else {
      const int key = id >= 0 ? key32(chosen) : INT32_MIN;
      mem.top[lane] = key;
      wave_lds_fence();
#pragma unroll
      for (int o = 0; o < kLanes; ++o) {
        const int t = mem.top[o];
        rank += (t > key || (t == key && o < lane)) ? 1 : 0;
      }
      wave_lds_fence();
    }
    if (id >= 0 && rank < p.k) {
      mem.id[rank] = id;
      mem.logit[rank] = chosen;
    }
    wave_lds_fence();
    id = lane < min(all, p.k) ? mem.id[lane] : -1;
    chosen = id >= 0 ? mem.logit[lane] : -INFINITY;
    const float s = weight_of(p, id, chosen, top, total, [](float x) { return row_max(x); },
                              [](float x) { return row_sum(x); });
    if (here && !open && lane < p.k) {
      p.topk_ids[row * p.k + lane] = id;
      p.topk_w[row * p.k + lane] = id >= 0 ? p.scale * s : 0.0f;
    }
    uint64_t rest = __ballot(here && open);
    while (rest != 0) {
      const int first = __ffsll(static_cast<unsigned long long>(rest)) - 1;
      route_exact(p, row0 + (threadIdx.x / kWave) * (kWave / kLanes) + first / kLanes,
                  keys + threadIdx.x / kWave * p.E);
      rest &= ~(uint64_t(0xFFFF) << (first / kLanes * kLanes));
    }
    wave_lds_fence();
  }
}

// Lane j of a row holds slot j. With c = scale, p the scores and
// u = p / sum of the chosen p:
//   softmax               dl_e = c p_e ([e chosen] g_e - sum_j g_j p_j)
//   softmax, renormalised dl_j = c u_j (g_j - sum_i g_i u_i), 0 elsewhere
//   sigmoid               dl_j = c g_j p_j (1 - p_j)
//   sigmoid, renormalised dl_j = c u_j (1 - p_j) (g_j - sum_i g_i u_i)
// Slots are separate arguments: an expert named twice gets both slots' shares.
//
// kLanes lanes take a row: a wave any row, sixteen lanes rows of up to 16 slots
// and 512 experts. Slots meet the row in LDS, and the row is written in pieces of
// four elements. Bound: HBM, by the writes where the row is not read: 32768 rows
// of 256 fp32, top-8, 11 us (12.4 alone).
template <int kRowLanes>
struct GradRow;

template <>
struct GradRow<kWave> {
  static __device__ __forceinline__ float max_of(float v) { return wave_max(v); }
  static __device__ __forceinline__ float sum_of(float v) { return wave_sum(v); }
};

template <>
struct GradRow<kLanes> {
  static __device__ __forceinline__ float max_of(float v) { return row_max(v); }
  static __device__ __forceinline__ float sum_of(float v) { return row_sum(v); }
};

// Four elements from element i on (i a multiple of four), or as many as the row has.
__device__ __forceinline__ floatx4 load_piece(const void* p, int64_t at, int i, int E, int dtype, bool vector) {
  floatx4 v;
  if (!vector) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = i + q < E ? load_elem(p, at + i + q, dtype) : -INFINITY;
  } else if (dtype == MOE_DTYPE_F32) {
    v = *reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + at + i);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + i);
    const bool bf = dtype == MOE_DTYPE_BF16;
    v[0] = bf ? bf16_lo(w.x) : half_bits_to_float(w.x & 0xFFFF);
    v[1] = bf ? bf16_hi(w.x) : half_bits_to_float(w.x >> 16);
    v[2] = bf ? bf16_lo(w.y) : half_bits_to_float(w.y & 0xFFFF);
    v[3] = bf ? bf16_hi(w.y) : half_bits_to_float(w.y >> 16);
  }
  return v;
}

__device__ __forceinline__ void store_piece(void* p, int64_t at, int i, int E, int dtype, bool vector, floatx4 v) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));
  if (!vector) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < E) store_elem(p, at + i + q, dtype, v[q]);
  } else if (dtype == MOE_DTYPE_F32) {
    *reinterpret_cast<floatx4*>(static_cast<float*>(p) + at + i) = v;
  } else if (dtype == MOE_DTYPE_BF16) {
    *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p) + at + i) = __builtin_convertvector(v, bf16x4);
  } else {
    *reinterpret_cast<halfx4*>(static_cast<_Float16*>(p) + at + i) = __builtin_convertvector(v, halfx4);
  }
}

template <int kRowLanes>
__global__ __launch_bounds__(kThreads) void route_grad(RouteGradArgs p) {
  extern __shared__ floatx4 rows_lds[];
  constexpr int kHere = kThreads / kRowLanes;          // rows of a workgroup
  using Row = GradRow<kRowLanes>;
  const int lane = threadIdx.x % kRowLanes;
  const int pieces = (p.E + 3) / 4;
  floatx4* buf = rows_lds + threadIdx.x / kRowLanes * pieces;
  float* one = reinterpret_cast<float*>(buf);
  const bool dense = p.score == MOE_SCORE_SOFTMAX && !p.renormalize;
  for (int64_t row0 = blockIdx.x * int64_t(kHere); row0 < p.M; row0 += int64_t(gridDim.x) * kHere) {
    const int64_t row = row0 + threadIdx.x / kRowLanes;
    const bool here = row < p.M;
    const int64_t at = row * p.ld;
    int id = here && lane < p.k ? p.topk_ids[row * p.k + lane] : -1;
    if (id >= p.E) id = -1;
    const bool valid = id >= 0;
    const float g = valid ? p.scale * p.dtopk_w[row * p.k + lane] : 0.0f;
    const float l = valid ? load_elem(p.logits, at + id, p.dtype) : -INFINITY;
    float d = 0.0f;
    if (dense) {
      // The row goes through LDS from here on: logits, then gradients.
      float top = -INFINITY;
      for (int i = lane; here && i < pieces; i += kRowLanes) {
        const floatx4 v = load_piece(p.logits, at, 4 * i, p.E, p.dtype, p.vector);
        buf[i] = v;
        top = fmaxf(fmaxf(fmaxf(top, v[0]), v[1]), fmaxf(v[2], v[3]));
      }
      top = Row::max_of(top);
      float total = 0.0f;
      for (int i = lane; here && i < pieces; i += kRowLanes) {
        floatx4 v = buf[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = v[q] == -INFINITY ? 0.0f : fast_exp(v[q] - top);
        buf[i] = v;
        total += (v[0] + v[1]) + (v[2] + v[3]);
      }
      total = Row::sum_of(total);
      const float s = valid ? fast_exp(l - top) / total : 0.0f;
      d = valid ? g * s : 0.0f;
      // A row without any route has no gradient, whatever its softmax.
      const bool any = Row::max_of(valid ? 1.0f : 0.0f) != 0.0f;
      const float back = any ? Row::sum_of(d) / total : 0.0f;
      for (int i = lane; here && i < pieces; i += kRowLanes) buf[i] = any ? -back * buf[i] : floatx4{0, 0, 0, 0};
    } else {
      for (int i = lane; here && i < pieces; i += kRowLanes) buf[i] = floatx4{0, 0, 0, 0};
      const float m = Row::max_of(l);
      if (p.score == MOE_SCORE_SOFTMAX) {
        const float e = valid ? expf(l - m) : 0.0f;
        const float u = e / Row::sum_of(e);
        const float dot = Row::sum_of(valid ? g * u : 0.0f);
        d = valid ? u * (g - dot) : 0.0f;
      } else {
        const float q = 1.0f / (1.0f + expf(l));       // 1 - p
        if (p.renormalize) {
          const float z = fminf(m, 0.0f);
          const float e = valid ? expf(fminf(l, 0.0f) - z) / (1.0f + expf(-fabsf(l))) : 0.0f;
          const float u = e / Row::sum_of(e);
          const float dot = Row::sum_of(valid ? g * u : 0.0f);
          d = valid ? u * q * (g - dot) : 0.0f;
        } else {
          d = valid ? g * q / (1.0f + expf(-l)) : 0.0f;
        }
      }
    }
    // Slots that name the same expert: the first of them brings their sum.
    float sum = 0.0f;
    bool first = valid;
    for (int j = 0; j < p.k; ++j) {
      const int oid = __shfl(id, j, kRowLanes);
      const float od = __shfl(d, j, kRowLanes);
      if (oid != id) continue;
      sum += od;
      first = first && j >= lane;
    }
    wave_lds_fence();
    if (first) one[id] += sum;
    wave_lds_fence();
    for (int i = lane; here && i < pieces; i += kRowLanes)
      store_piece(p.dlogits, row * p.ldd, 4 * i, p.E, p.out_dtype, p.vector_out, buf[i]);
    wave_lds_fence();
  }
}

}  // namespace

namespace {

RouteLayout layout(int lanes, int groups, int group_size) {
  RouteLayout y{1, 0};
  while (y.per_group * 2 * groups <= lanes) y.per_group *= 2;
  y.per_lane = (group_size + y.per_group - 1) / y.per_group;
  return y;
}

// LDS of route_exact's keys for every wave of a workgroup; of the rows' logits of route_narrow beside them.
uint32_t exact_bytes(const RouteArgs& p) { return sizeof(int64_t) * kWaves * p.E; }
uint32_t narrow_bytes(const RouteArgs& p) { return exact_bytes(p) + (p.vector ? sizeof(float) * kRows * p.E : 0); }

template <int C>
void start_narrow(RouteArgs p, hipStream_t stream) {
  // Whole 16-byte pieces for every lane of every row.
  const int64_t bytes = p.dtype == MOE_DTYPE_F32 ? 4 : 2;
  p.vector = p.groups * p.narrow.per_group == kLanes && p.narrow.per_lane == C &&
             p.group_size == p.narrow.per_group * C && C * bytes % 16 == 0 && p.ld * bytes % 16 == 0 &&
             reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
  const dim3 grid(grid_for((p.M + kRows - 1) / kRows, 0)), block(kThreads);
  if (p.bias != nullptr)
    launch(route_narrow<C, true>, grid, block, narrow_bytes(p), stream, p);
  else
    launch(route_narrow<C, false>, grid, block, narrow_bytes(p), stream, p);
}

}  // namespace

// Sixteen lanes a row where they hold it (32768 tokens, 256 experts, eight groups with a bias, four kept: 1, 8 and 16
// slots 30, 31 and 55 us, a wave a row 47, 84 and 128; one kept, 4, 8 and 16 slots: 30, 41, 59 and 63, 84, 125; 512
// experts, 8 slots: 52 and 102; 2048 tokens, 256 experts, 8 and 14 slots: 7.9, 9.6 and 12.1, 17.3, but 1 and 16, of which
// some row has a seventeenth within the errors: 7.8, 24.7 and 6.6, 18.9), a wave for more experts, slots or groups.
hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  RouteArgs p = a;
  p.group_size = p.E / p.groups;
  p.wide = layout(kWave, p.groups, p.group_size);
  // Scores are needed for the choice with a bias, and where they are summed over a group.
  const bool sums = p.topk_groups < p.groups && p.group_top == 2;
  p.exact_scores = p.bias != nullptr || sums;
  if (p.groups <= kLanes && p.k <= kLanes) {
    p.narrow = layout(kLanes, p.groups, p.group_size);
    if (p.narrow.per_lane <= 32) {
      if (p.narrow.per_lane <= 4)
        start_narrow<4>(p, stream);
      else if (p.narrow.per_lane <= 8)
        start_narrow<8>(p, stream);
      else if (p.narrow.per_lane <= 16)
        start_narrow<16>(p, stream);
      else
        start_narrow<32>(p, stream);
      return hipGetLastError();
    }
  }
  const dim3 grid(grid_for((p.M + kWaves - 1) / kWaves, 0)), block(kThreads);
  launch(route_wide, grid, block, exact_bytes(p), stream, p);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t stream) {
  RouteGradArgs p = a;
  // Pieces of four elements, aligned as such.
  const auto vector = [&](const void* v, int64_t ld, int dtype) {
    const uintptr_t bytes = dtype == MOE_DTYPE_F32 ? 16 : 8;
    return p.E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(v) % bytes == 0;
  };
  p.vector = vector(p.logits, p.ld, p.dtype);
  p.vector_out = vector(p.dlogits, p.ldd, p.out_dtype);
  const int lanes = p.k <= kLanes && p.E <= 512 ? kLanes : kWave;
  const int rows = kThreads / lanes;
  const dim3 grid(grid_for((p.M + rows - 1) / rows, 0)), block(kThreads);
  const uint32_t lds = sizeof(floatx4) * rows * ((p.E + 3) / 4);
  if (lanes == kLanes)
    launch(route_grad<kLanes>, grid, block, lds, stream, p);
  else
    launch(route_grad<kWave>, grid, block, lds, stream, p);
  return hipGetLastError();
}

}  // namespace moe
