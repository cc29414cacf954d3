// Expert products on rows grouped by expert with ragged counts (gfx950).
//
// Expert e owns rows offsets[e] .. offsets[e + 1] - 1 of the row operands; W is
// [E][N][K]. Three products, each a sum over one index, on 16-bit operands:
//   forward          y[r][n]     = sum_k x[r][k]  W[e][n][k]
//   input gradient   dx[r][k]    = sum_n dy[r][n] W[e][n][k]
//   weight gradient  dW[e][n][k] = sum_{r of e} dy[r][n] x[r][k]
// and the forward product on MXFP4 operands (E2M1 codes, one E8M0 exponent per
// 32 elements of k). Sums are fp32 in the matrix instructions' accumulators
// and rounded once to the output type. Every output has one writer and a
// fixed order of additions, so results do not depend on the grid.
//
// One kernel template computes a TA x TB tile of the output. The operand whose
// index runs along the output's contiguous dimension is the matrix
// instructions' A operand: a lane's four results are then consecutive in
// memory. Each operand is read in slabs of its summed index: one slab is 128
// bytes of a row (64 16-bit elements, or 256 codes) where the summed index is
// contiguous in memory ("direct"), or 64 rows where it is the row index
// ("transposed": W in the input gradient, both operands of the weight
// gradient). LDS-DMA brings a slab from global memory into a ring of S slots;
// direct tiles are read back 16 bytes a lane, transposed ones with gfx950's
// transposing LDS read, so neither operand needs a copy in another order.
//
// What is past the summed extent (the last slab's tail, rows after an expert's
// last one) is read from a zero page instead, in both operands, so that another
// expert's rows, whatever they hold, cannot reach a sum. What is past the
// output's extents re-reads the last valid row or chunk and is not stored.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

// Operand element types of the kernel template.
struct Bf16 {};
struct F16 {};
struct Fp4 {};

enum Kind { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

constexpr int kSlabBytes = 128;   // bytes of a direct row per slab
constexpr int kSlabRows = 64;     // rows of a transposed operand per slab (16-bit elements)
constexpr int kGroupM = 4;        // row tiles visited together, see find_task

__device__ __align__(16) const uint32_t zero_page[4] = {0, 0, 0, 0};

// 16 bytes per lane to LDS at lds_base + 16 * lane from base + voff (one
// scalar base for the wave, one 32-bit offset per lane).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_off(const void* base, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(voff), "s"(base), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

template <typename T>
__device__ __forceinline__ floatx4 mfma_step(const uint4& a, const uint4& b, const floatx4& c) {
  if constexpr (__is_same(T, F16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// 128 MXFP4 products per output: a lane's 32 codes are one block, scaled by
// byte kByte of its scale word.
template <int kByte>
__device__ __forceinline__ floatx4 mfma_step_fp4(const uint4& a, const uint4& b, const floatx4& c, int sa, int sb) {
  const intx8 av = {int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};
  const intx8 bv = {int(b.x), int(b.y), int(b.z), int(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, kByte, sa, kByte, sb);
}

// Start of expert e's rows: offsets clamped to [0, rows] and made
// non-decreasing, so that whatever the array holds, no row has two owners and
// no access leaves the operands.
struct Ranges {
  int first;   // first expert of this lane
  int start;   // start row of that expert
  int base;    // row tiles before this lane's experts
  int tiles;   // row tiles of this lane's experts
  int total;   // row tiles of all experts
};

__device__ __forceinline__ int clamp_row(int v, int lo, int rows) { return min(rows, max(lo, v)); }

// Each lane of a wave takes ceil(E / 64) consecutive experts.
template <int TB>
__device__ __forceinline__ Ranges scan_ranges(const int32_t* offsets, int E, int rows, int lane) {
  const int per = (E + 63) / 64;
  Ranges r;
  r.first = min(E, lane * per);
  const int last = min(E, r.first + per);
  int top = 0;
  for (int e = r.first; e < last; ++e) top = max(top, offsets[e]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(top, d, kWave);
    if (lane >= d) top = max(top, o);
  }
  const int before = __shfl_up(top, 1, kWave);
  const int floor0 = lane == 0 ? 0 : before;
  r.start = r.first < E ? clamp_row(offsets[r.first], floor0, rows) : rows;
  int cur = r.start, tiles = 0;
  for (int e = r.first; e < last; ++e) {
    const int nxt = clamp_row(offsets[e + 1], cur, rows);
    tiles += (nxt - cur + TB - 1) / TB;
    cur = nxt;
  }
  int incl = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += o;
  }
  r.tiles = tiles;
  r.base = incl - tiles;
  r.total = __builtin_amdgcn_readlane(incl, 63);
  return r;
}

struct Task {
  int e;       // expert
  int row0;    // first row of the tile
  int rows;    // valid rows of the tile (forward, input gradient) or of the expert (weight gradient)
  int a0;      // first output column of the tile (A operand's index)
  int b0;      // weight gradient: first index n of the tile
};

// Task L of total * NT (forward, input gradient). An expert's tasks are
// consecutive and go through kGroupM row tiles per column tile, so that the
// tasks running at one time on one XCD share weights and rows in its L2.
template <int TB>
__device__ __forceinline__ Task find_task(const Ranges& r, const int32_t* offsets, int E, int rows, int lane, int L,
                                          int NT, int TA) {
  const int t = L / NT;
  const uint64_t own = __ballot(t >= r.base && t < r.base + r.tiles);
  const int src = __ffsll(static_cast<unsigned long long>(own)) - 1;
  int e = r.first, cur = r.start, base = r.base, nxt = cur;
  if (lane == src) {
    for (;; ++e) {
      nxt = clamp_row(offsets[e + 1], cur, rows);
      const int n = (nxt - cur + TB - 1) / TB;
      if (t < base + n || e + 1 >= E) break;
      base += n;
      cur = nxt;
    }
  }
  e = __builtin_amdgcn_readlane(e, src);
  cur = __builtin_amdgcn_readlane(cur, src);
  nxt = __builtin_amdgcn_readlane(nxt, src);
  base = __builtin_amdgcn_readlane(base, src);
  const int mt = (nxt - cur + TB - 1) / TB;
  const int local = L - base * NT;
  const int grp = local / (kGroupM * NT);
  const int gm = min(kGroupM, mt - grp * kGroupM);
  const int in = local - grp * kGroupM * NT;
  const int n = in / gm;
  const int m = grp * kGroupM + (in - n * gm);
  Task k;
  k.e = e;
  k.row0 = cur + m * TB;
  k.rows = min(TB, nxt - k.row0);
  k.a0 = n * TA;
  k.b0 = 0;
  return k;
}

// Position of 16-byte chunk c of a direct tile row (eight chunks), and of the
// 32-byte unit u of a transposed tile row: an XOR with bits of the row spreads
// the lanes of one LDS read over the banks.
__device__ __forceinline__ int direct_pos(int row, int c) { return c ^ ((row >> 1) & 7); }

template <int T>   // tile width in 16-bit elements
__device__ __forceinline__ int trans_unit(int row, int u) {
  constexpr int units = T / 16;
  if constexpr (units >= 8)
    return u ^ ((row & 3) | ((row >> 1) & 4));
  else if constexpr (units == 4)
    return u ^ (((row >> 1) & 1) | ((row >> 2) & 2));
  else if constexpr (units == 2)
    return u ^ ((row >> 3) & 1);
  else
    return u;
}

// One operand's side of the data movement: which bytes this wave brings in.
// kTrans: the tile is [64 rows][T] (the rows are the summed index).
template <int T, int NW, bool kTrans>
struct Loader {
  static constexpr int kInstr = T / 8;                                 // 1 KB pieces per slab
  static constexpr int kPer = kInstr >= NW ? kInstr / NW : 1;          // pieces per wave (repeated ones when
                                                                       // there are fewer pieces than waves)
  const char* base;       // slab 0 of the tile
  int64_t step;           // bytes from slab to slab
  uint32_t voff[kPer];    // this lane's offset in each piece
  int where[kPer];        // its place along the summed index: byte within the slab (direct), row (transposed)

  // ld: bytes from row to row; limit: valid rows (direct) or valid 16-byte
  // chunks of a row (transposed) counted from the tile's first one.
  __device__ __forceinline__ void init(const void* p, int64_t ld, int limit, int wave, int lane) {
    base = static_cast<const char*>(p);
    step = kTrans ? ld * kSlabRows : kSlabBytes;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int q = ((wave + j * NW) % kInstr) * 64 + lane;   // 16-byte position in the tile
      if constexpr (!kTrans) {
        const int row = q >> 3;
        const int c = direct_pos(row, q & 7);                 // an XOR is its own inverse
        voff[j] = static_cast<uint32_t>(min(row, limit - 1) * ld) + c * 16;
        where[j] = c * 16;
      } else {
        const int row = q / (T / 8);
        const int pos = q % (T / 8);
        const int c = trans_unit<T>(row, pos >> 1) * 2 + (pos & 1);
        voff[j] = static_cast<uint32_t>(row * ld) + min(c, limit - 1) * 16;
        where[j] = row;
      }
    }
  }

  __device__ __forceinline__ void full(int slab, uint32_t lds, int wave) const {
    const char* b = base + slab * step;
#pragma unroll
    for (int j = 0; j < kPer; ++j) dma16_off(b, voff[j], lds + ((wave + j * NW) % kInstr) * 1024);
  }

  // The last slab: `left` is what remains of the summed index, in bytes
  // (direct) or rows (transposed).
  __device__ __forceinline__ void tail(int slab, int left, uint32_t lds, int wave) const {
    const char* b = base + slab * step;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const void* src = where[j] < left ? static_cast<const void*>(b + voff[j]) : static_cast<const void*>(zero_page);
      dma16(src, lds + ((wave + j * NW) % kInstr) * 1024);
    }
  }
};

// A lane's operand of one matrix step (step t of a slab) for the 16 tile rows
// (direct) or columns (transposed) from i0 on.
template <int T, bool kTrans, bool kFp4>
__device__ __forceinline__ uint4 fragment(const unsigned char* tile, int i0, int t, int lane) {
  const int g = lane >> 4;
  if constexpr (!kTrans) {
    const int row = i0 + (lane & 15);
    // 16-bit: the four lane groups take the step's 64 bytes in order. MXFP4:
    // group g takes blocks 2g and 2g + 1 of the slab, so that its two scales
    // are neighbours.
    const int c = kFp4 ? 2 * g + t : 4 * t + g;
    return *reinterpret_cast<const uint4*>(tile + row * kSlabBytes + direct_pos(row, c) * 16);
  } else {
    const int i = lane & 15;
    uint2 h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = 32 * t + 8 * g + 4 * k + (i >> 2);
      const unsigned char* p = tile + row * (2 * T) + trans_unit<T>(row, i0 >> 4) * 32 + (i & 3) * 8;
      const shortx4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)p);
      h[k] = __builtin_bit_cast(uint2, v);
    }
    return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
  }
}

// Waits until at most `later` slabs' loads of this wave are in flight.
template <int kPerSlab, int S>
__device__ __forceinline__ void wait_slab(int later) {
  if (S >= 4 && later >= 2)
    wait_vm<2 * kPerSlab>();
  else if (S >= 3 && later >= 1)
    wait_vm<kPerSlab>();
  else
    wait_vm<0>();
}

__device__ __forceinline__ void store4(void* out, int64_t i, const floatx4& v, int dtype) {
  if (dtype == MOE_DTYPE_F32) {
    *reinterpret_cast<floatx4*>(static_cast<float*>(out) + i) = v;
  } else if (dtype == MOE_DTYPE_BF16) {
    const bf16x4 h = __builtin_convertvector(v, bf16x4);
    *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(out) + i) = h;
  } else {
    const halfx4 h = __builtin_convertvector(v, halfx4);
    *reinterpret_cast<halfx4*>(static_cast<uint16_t*>(out) + i) = h;
  }
}

template <int TA, int TB, int S, bool kFp4>
constexpr int ring_bytes() {
  return S * (TA + TB) * (kSlabBytes + (kFp4 ? 8 : 0));
}

template <Kind kKind, typename T, int TA, int TB, int WA, int WB, int S>
__global__ __launch_bounds__(64 * WA * WB) void ragged_gemm(const RaggedArgs p) {
  constexpr bool kFp4 = __is_same(T, Fp4);
  constexpr bool kTransA = kKind != kForward;
  constexpr bool kTransB = kKind == kWeightGrad;
  constexpr int NW = WA * WB;
  constexpr int MA = TA / WA / 16, MB = TB / WB / 16;
  using LA = Loader<TA, NW, kTransA>;
  using LB = Loader<TB, NW, kTransB>;
  constexpr int kPerSlab = LA::kPer + LB::kPer;
  extern __shared__ __align__(16) unsigned char lds[];
  unsigned char* const tiles = lds;                                      // [S][A tile, B tile]
  constexpr int kSlot = (TA + TB) * kSlabBytes;
  unsigned char* const scales = lds + S * kSlot;                         // [S][TA + TB][8] (MXFP4)
  const uint32_t tiles_at = lds_addr(tiles);

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int wa = wave % WA, wb = wave / WA;
  const int E = p.E, N = p.N, K = p.K;
  // Output extents: OA along memory; the summed extent is K, N or the expert's rows.
  const int OA = kKind == kForward ? N : K;
  const int NT = (OA + TA - 1) / TA;
  const int MT = kKind == kWeightGrad ? (N + TB - 1) / TB : 0;

  Ranges r{};
  int total;
  if constexpr (kKind == kWeightGrad) {
    total = E * NT * MT;
  } else {
    r = scan_ranges<TB>(p.offsets, E, p.rows, lane);
    total = r.total * NT;
  }
  // Workgroups go to the eight XCDs in turn: XCD i takes the i-th eighth of
  // the tasks, so neighbouring tasks share an L2.
  const int per = (total + 7) / 8;
  for (int t = blockIdx.x; t < 8 * per; t += gridDim.x) {
    const int L = (t & 7) * per + (t >> 3);
    if (L >= total) continue;
    Task k;
    if constexpr (kKind == kWeightGrad) {
      k.e = L / (NT * MT);
      const int local = L - k.e * NT * MT;
      const int grp = local / (kGroupM * NT);
      const int gm = min(kGroupM, MT - grp * kGroupM);
      const int in = local - grp * kGroupM * NT;
      k.a0 = (in / gm) * TA;
      k.b0 = (grp * kGroupM + in % gm) * TB;
      int top = 0;                                        // the range as scan_ranges defines it
      for (int e = lane; e <= k.e; e += 64) top = max(top, p.offsets[e]);
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d, kWave));
      k.row0 = min(p.rows, uniform(top));
      k.rows = clamp_row(p.offsets[k.e + 1], k.row0, p.rows) - k.row0;
    } else {
      k = find_task<TB>(r, p.offsets, E, p.rows, lane, L, NT, TA);
    }

    // Operands of the tile.
    LA a;
    LB b;
    int ns, left;        // slabs, and what the last one holds (bytes, or rows)
    if constexpr (kKind == kForward) {
      const int64_t row_bytes = kFp4 ? K / 2 : int64_t(K) * 2;
      const int64_t x_bytes = kFp4 ? K / 2 : p.ldb * 2;
      a.init(static_cast<const char*>(p.a) + (int64_t(k.e) * N + k.a0) * row_bytes, row_bytes, min(TA, N - k.a0), wave,
             lane);
      b.init(static_cast<const char*>(p.b) + k.row0 * x_bytes, x_bytes, k.rows, wave, lane);
      ns = static_cast<int>((row_bytes + kSlabBytes - 1) / kSlabBytes);
      left = static_cast<int>(row_bytes) - (ns - 1) * kSlabBytes;
    } else if constexpr (kKind == kInputGrad) {
      a.init(static_cast<const uint16_t*>(p.a) + int64_t(k.e) * N * K + k.a0, int64_t(K) * 2, min(TA, K - k.a0) / 8, wave,
             lane);
      b.init(static_cast<const uint16_t*>(p.b) + k.row0 * p.ldb, p.ldb * 2, k.rows, wave, lane);
      ns = (N + kSlabRows - 1) / kSlabRows;
      left = N - (ns - 1) * kSlabRows;
    } else {
      a.init(static_cast<const uint16_t*>(p.a) + k.row0 * p.lda + k.a0, p.lda * 2, min(TA, K - k.a0) / 8, wave, lane);
      b.init(static_cast<const uint16_t*>(p.b) + k.row0 * p.ldb + k.b0, p.ldb * 2, min(TB, N - k.b0) / 8, wave, lane);
      ns = (k.rows + kSlabRows - 1) / kSlabRows;
      left = k.rows - (ns - 1) * kSlabRows;
    }
    const int left_b = kKind == kInputGrad ? left * 2 : left;   // dy is direct: bytes
    auto issue = [&](int s) {
      const uint32_t at = tiles_at + (s % S) * kSlot;
      if (s < ns - 1) {
        a.full(s, at, wave);
        b.full(s, at + TA * kSlabBytes, wave);
      } else {
        a.tail(s, left, at, wave);
        b.tail(s, left_b, at + TA * kSlabBytes, wave);
      }
    };
    // MXFP4 scales: each thread brings eight bytes (one slab) of a tile row.
    constexpr int kScaleRows = kFp4 ? (TA + TB + 64 * NW - 1) / (64 * NW) : 1;
    const uint8_t* srow[kScaleRows];
    uint64_t sval[kScaleRows];
    if constexpr (kFp4) {
      const int sb = K / 32;
#pragma unroll
      for (int j = 0; j < kScaleRows; ++j) {
        const int i = threadIdx.x + j * 64 * NW;
        const int an = min(k.a0 + i, N - 1), bn = k.row0 + min(i - TA, k.rows - 1);
        srow[j] = i < TA ? p.a_scale + (int64_t(k.e) * N + an) * sb : p.b_scale + int64_t(max(bn, k.row0)) * sb;
      }
    }
    auto load_scales = [&](int s) {
      if constexpr (kFp4) {
        const int n = K / 32 - s * 8;
#pragma unroll
        for (int j = 0; j < kScaleRows; ++j) {
          if (n >= 8) {
            __builtin_memcpy(&sval[j], srow[j] + s * 8, 8);
          } else {
            uint64_t v = 0;
            for (int i = 0; i < 8; ++i) v |= uint64_t(i < n ? srow[j][s * 8 + i] : 127) << (8 * i);
            sval[j] = v;
          }
        }
      }
    };
    auto keep_scales = [&](int s) {
      if constexpr (kFp4) {
#pragma unroll
        for (int j = 0; j < kScaleRows; ++j) {
          const int i = threadIdx.x + j * 64 * NW;
          if (i < TA + TB) *reinterpret_cast<uint64_t*>(scales + ((s % S) * (TA + TB) + i) * 8) = sval[j];
        }
      }
    };

    floatx4 acc[MA][MB];
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    lds_barrier();      // every wave is done with the ring of the task before
    wait_vm<0>();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
      if (s < ns) {
        load_scales(s);
        issue(s);
        keep_scales(s);
      }
    }
    for (int s = 0; s < ns; ++s) {
      wait_slab<kPerSlab, S>(min(S - 2, ns - 1 - s));
      lds_barrier();    // slab s is whole, and slab s - 1 has been read by every wave
      const bool more = s + S - 1 < ns;
      if (more) {
        load_scales(s + S - 1);
        issue(s + S - 1);
      }
      const unsigned char* const at = tiles + (s % S) * kSlot;
      const unsigned char* const bt = at + TA * kSlabBytes;
      int sa[MA], sb[MB];
      if constexpr (kFp4) {
        const unsigned char* sc = scales + (s % S) * (TA + TB) * 8;
#pragma unroll
        for (int i = 0; i < MA; ++i)
          sa[i] = *reinterpret_cast<const uint16_t*>(sc + ((wa * MA + i) * 16 + (lane & 15)) * 8 + 2 * (lane >> 4));
#pragma unroll
        for (int j = 0; j < MB; ++j)
          sb[j] = *reinterpret_cast<const uint16_t*>(sc + (TA + (wb * MB + j) * 16 + (lane & 15)) * 8 + 2 * (lane >> 4));
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint4 av[MA], bv[MB];
#pragma unroll
        for (int i = 0; i < MA; ++i) av[i] = fragment<TA, kTransA, kFp4>(at, (wa * MA + i) * 16, q, lane);
#pragma unroll
        for (int j = 0; j < MB; ++j) bv[j] = fragment<TB, kTransB, kFp4>(bt, (wb * MB + j) * 16, q, lane);
#pragma unroll
        for (int i = 0; i < MA; ++i)
#pragma unroll
          for (int j = 0; j < MB; ++j) {
            if constexpr (kFp4)
              acc[i][j] = q == 0 ? mfma_step_fp4<0>(av[i], bv[j], acc[i][j], sa[i], sb[j])
                                 : mfma_step_fp4<1>(av[i], bv[j], acc[i][j], sa[i], sb[j]);
            else
              acc[i][j] = mfma_step<T>(av[i], bv[j], acc[i][j]);
          }
      }
      if (more) keep_scales(s + S - 1);
    }

    // A lane holds four consecutive columns of one output row per 16 x 16 tile.
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int row = (wb * MB + j) * 16 + (lane & 15);
      const bool row_ok = kKind == kWeightGrad ? k.b0 + row < N : row < k.rows;
      const int64_t at = kKind == kWeightGrad ? (int64_t(k.e) * N + k.b0 + row) * K : (k.row0 + row) * p.ldo;
#pragma unroll
      for (int i = 0; i < MA; ++i) {
        const int col = k.a0 + (wa * MA + i) * 16 + 4 * (lane >> 4);
        if (row_ok && col < OA) store4(p.out, at + col, acc[i][j], p.out_dtype);
      }
    }
  }
}

template <Kind kKind, typename T, int TA, int TB, int WA, int WB, int S>
hipError_t run(const RaggedArgs& p, hipStream_t stream) {
  const int64_t OA = kKind == kForward ? p.N : p.K;
  const int64_t nt = (OA + TA - 1) / TA;
  const int64_t tasks = kKind == kWeightGrad
                            ? int64_t(p.E) * nt * ((p.N + TB - 1) / TB)
                            : (int64_t(p.rows) / TB + (p.E < p.rows ? p.E : p.rows)) * nt;
  launch(ragged_gemm<kKind, T, TA, TB, WA, WB, S>, dim3(grid_for((tasks + 7) & ~int64_t(7), 0)), dim3(64 * WA * WB),
         ring_bytes<TA, TB, S, __is_same(T, Fp4)>(), stream, p);
  return hipGetLastError();
}

template <Kind kKind, typename T>
hipError_t pick(const RaggedArgs& p, hipStream_t stream) {
  return run<kKind, T, 128, 128, 2, 2, 2>(p, stream);
}

}  // namespace

hipError_t launch_ragged_forward(const RaggedArgs& p, int dtype, hipStream_t stream) {
  if (dtype == MOE_DTYPE_MXFP4) return pick<kForward, Fp4>(p, stream);
  return dtype == MOE_DTYPE_F16 ? pick<kForward, F16>(p, stream) : pick<kForward, Bf16>(p, stream);
}

hipError_t launch_ragged_input_grad(const RaggedArgs& p, int dtype, hipStream_t stream) {
  return dtype == MOE_DTYPE_F16 ? pick<kInputGrad, F16>(p, stream) : pick<kInputGrad, Bf16>(p, stream);
}

hipError_t launch_ragged_weight_grad(const RaggedArgs& p, int dtype, hipStream_t stream) {
  return dtype == MOE_DTYPE_F16 ? pick<kWeightGrad, F16>(p, stream) : pick<kWeightGrad, Bf16>(p, stream);
}

}  // namespace moe
