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
// gradient). LDS-DMA brings a slab from global memory into a ring of two slots;
// direct tiles are read back 16 bytes a lane, transposed ones with gfx950's
// transposing LDS read, so neither operand needs a copy in another order.
//
// What is past the summed extent (the last slab's tail, rows after an expert's
// last one) is read from a zero page instead, in both operands, so that another
// expert's rows, whatever they hold, cannot reach a sum. What is past the
// output's extents re-reads the last valid row or chunk and is not stored.
#include <type_traits>

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
struct Fp4 {};      // K a multiple of 128, exponents aligned to 4 bytes: a slab's are aligned words
struct Fp4Odd {};   // any other K or alignment

enum Kind { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

constexpr int kSteps = 2;                      // matrix steps (32 16-bit elements or 128 codes) per slab
constexpr int kSlabBytes = 64 * kSteps;        // bytes of a direct row per slab
constexpr int kSlabRows = 32 * kSteps;         // rows of a transposed operand per slab (16-bit elements)
constexpr int kSlots = 2;                      // slabs in LDS: one read, one arriving
constexpr int kCus = 256;
constexpr int kLdsPerCu = 160 * 1024;
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

// A wave-uniform address made explicitly scalar.
__device__ __forceinline__ const char* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>(uint64_t(hi) << 32 | lo);
}

template <typename T>
__device__ __forceinline__ floatx4 mfma_step(const uint4& a, const uint4& b, const floatx4& c) {
  if constexpr (__is_same(T, F16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// 128 MXFP4 products per output: a lane's 32 codes are one block, whose
// exponent is byte ka (kb) of its word of exponents. Constants after inlining.
__device__ __forceinline__ floatx4 mfma_step_fp4(const uint4& a, const uint4& b, const floatx4& c, int sa, int ka, int sb,
                                                 int kb) {
  const intx8 av = {int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};
  const intx8 bv = {int(b.x), int(b.y), int(b.z), int(b.w), 0, 0, 0, 0};
#define MOE_FP4_CASE(A, B) \
  case 4 * A + B:          \
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, A, sa, B, sb);
  switch (4 * ka + kb) {
    MOE_FP4_CASE(0, 0) MOE_FP4_CASE(0, 2) MOE_FP4_CASE(2, 0) MOE_FP4_CASE(2, 2)
    MOE_FP4_CASE(1, 1) MOE_FP4_CASE(1, 3) MOE_FP4_CASE(3, 1) MOE_FP4_CASE(3, 3)
  }
#undef MOE_FP4_CASE
  return c;
}

__device__ __forceinline__ int clamp_row(int v, int lo, int rows) { return min(rows, max(lo, v)); }

// Inclusive scan over the wave's lanes of values >= 0 under an operation for
// which 0 is neutral: within rows of 16 lanes, then across them.
template <typename Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));   // row_bcast 15 into rows 1 and 3
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));   // row_bcast 31 into rows 2 and 3
  return v;
}

// Row tiles of the experts, by lane: lane l holds ceil(E / 64) consecutive ones.
struct Ranges {
  int first;   // first expert of this lane
  int base;    // row tiles before this lane's experts
  int tiles;   // row tiles of this lane's experts
  int total;   // row tiles of all experts
};

// Reads the offsets once: the start row of every expert goes to starts [E + 1]
// in LDS, clamped to [0, rows] and made non-decreasing, so that whatever the
// array holds, no row has two owners and no access leaves the operands. Every
// wave scans (and stores the same values); the caller puts a barrier behind.
template <int TB>
__device__ __forceinline__ Ranges scan_ranges(const int32_t* offsets, int E, int rows, int* starts, int lane) {
  constexpr int kHeld = 4;     // offsets a lane keeps in registers (up to 256 experts): one round trip
  const int per = (E + 63) / 64;
  Ranges r;
  r.first = min(E, lane * per);
  const int last = min(E, r.first + per);
  int held[kHeld + 1];
#pragma unroll
  for (int i = 0; i <= kHeld; ++i) held[i] = offsets[min(E, r.first + i)];
  auto offset = [&](int e) {
    const int i = e - r.first;
    return i == 0 ? held[0] : i == 1 ? held[1] : i == 2 ? held[2] : i == 3 ? held[3] : i == 4 ? held[4] : offsets[e];
  };
  int top = 0;
  for (int e = r.first; e < last; ++e) top = max(top, offset(e));
  top = wave_scan(top, [](int a, int b) { return max(a, b); });
  const int before = __builtin_amdgcn_update_dpp(0, top, 0x138, 0xF, 0xF, false);   // the lane below's; 0 for lane 0
  int cur = r.first < E ? clamp_row(offset(r.first), before, rows) : rows;
  int tiles = 0;
  for (int e = r.first; e < last; ++e) {
    const int nxt = clamp_row(offset(e + 1), cur, rows);
    starts[e] = cur;
    if (e + 1 == E) starts[E] = nxt;
    tiles += (nxt - cur + TB - 1) / TB;
    cur = nxt;
  }
  const int incl = wave_scan(tiles, [](int a, int b) { return a + b; });
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
__device__ __forceinline__ Task find_task(const Ranges& r, const int* starts, int E, int L, int NT, int TA) {
  const int t = L / NT;
  const uint64_t own = __ballot(t >= r.base && t < r.base + r.tiles);
  const int src = __ffsll(static_cast<unsigned long long>(own)) - 1;
  int e = __builtin_amdgcn_readlane(r.first, src);
  int base = __builtin_amdgcn_readlane(r.base, src);
  int cur = uniform(starts[e]), nxt, mt;
  for (;; ++e) {
    nxt = uniform(starts[e + 1]);
    mt = (nxt - cur + TB - 1) / TB;
    if (t < base + mt || e + 1 >= E) break;
    base += mt;
    cur = nxt;
  }
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
  static_assert(units == 4 || units >= 8, "rows of 128 bytes, or of 256 and more");
  if constexpr (units >= 8)
    return u ^ ((row & 3) | ((row >> 1) & 4));
  else
    return u ^ (((row >> 1) & 1) | ((row >> 2) & 2));
}

// One operand's side of the data movement: which bytes this wave brings in.
// kTrans: the tile is [64 rows][T] (the rows are the summed index).
// kSkip (direct): pieces without a valid row are left out; their LDS then holds
// whatever was there, which only reaches outputs that are not stored.
template <int T, int NW, bool kTrans, bool kSkip, bool kFp4>
struct Loader {
  static constexpr int kInstr = T * kSlabBytes / 1024;                 // 1 KB pieces per slab
  static constexpr int kPer = kInstr / NW;                             // pieces per wave
  static constexpr int kPieceRows = 1024 / kSlabBytes;                 // (direct)
  static_assert(kInstr % NW == 0, "every wave brings in as many pieces");
  const char* base;       // the next slab to bring in
  int64_t step;           // bytes from slab to slab
  uint32_t voff[kPer];    // this lane's offset in each piece
  int where[kPer];        // its place along the summed index: byte within the slab (direct), row (transposed)
  int have;               // kSkip: valid rows from this wave's first piece on

  // ld: bytes from row to row; limit: valid rows (direct) or valid 16-byte
  // chunks of a row (transposed) counted from the tile's first one.
  __device__ __forceinline__ void init(const void* p, int64_t ld, int limit, int wave, int lane) {
    base = uniform_ptr(p);
    step = kTrans ? ld * kSlabRows : kSlabBytes;
    have = uniform(limit - wave * kPieceRows);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int q = (wave + j * NW) * 64 + lane;   // 16-byte position in the tile
      if constexpr (!kTrans) {
        const int row = q / (kSlabBytes / 16);
        const int x = direct_pos(row, q % (kSlabBytes / 16));   // an XOR is its own inverse
        const int c = kFp4 ? (x & 3) * 2 + (x >> 2) : x;        // see Reader
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

  __device__ __forceinline__ void full(uint32_t lds, int wave) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (kSkip && have <= j * NW * kPieceRows) break;
      dma16_off(base, voff[j], lds + (wave + j * NW) * 1024);
    }
    base += step;
  }

  // The last slab: `left` is what remains of the summed index, in bytes
  // (direct) or rows (transposed).
  __device__ __forceinline__ void tail(int left, uint32_t lds, int wave) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const void* src =
          where[j] < left ? static_cast<const void*>(base + voff[j]) : static_cast<const void*>(zero_page);
      dma16(src, lds + (wave + j * NW) * 1024);
    }
  }
};

typedef __attribute__((address_space(3))) const unsigned char* LdsPtr;

// This lane's operands of the matrix steps from M groups of 16 tile rows
// (direct) or columns (transposed) of a tile of width T: group `first` and
// every kStride-th after it. In step q lane group g reads the direct tile's
// position 4q + g, which holds that chunk of a row; for MXFP4 it holds block
// 2g + q, so that a group's two exponents are neighbours.
template <int T, int M, int kStride, bool kTrans>
struct Reader {
  // Offset in the tile: of each step's first group, the others following
  // (direct), or of the first step's groups (transposed).
  uint32_t at[kTrans ? M : kSteps];

  __device__ __forceinline__ void init(int first, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!kTrans) {
#pragma unroll
      for (int q = 0; q < kSteps; ++q)
        at[q] = (first * 16 + i) * kSlabBytes + direct_pos(i, 4 * q + g) * 16;
    } else {
      const int row = 8 * g + (i >> 2);
#pragma unroll
      for (int m = 0; m < M; ++m) at[m] = row * (2 * T) + trans_unit<T>(row, first + m * kStride) * 32 + (i & 3) * 8;
    }
  }

  __device__ __forceinline__ uint4 get(LdsPtr tile, int q, int m) const {
    if constexpr (!kTrans) {
      const u32x4 v = *reinterpret_cast<__attribute__((address_space(3))) const u32x4*>(
          tile + at[q] + m * kStride * 16 * kSlabBytes);
      return make_uint4(v.x, v.y, v.z, v.w);
    } else {
      // Rows row .. row + 3 and, four further (the same units), row + 4 .. row + 7.
      LdsPtr p = tile + at[m] + q * 32 * 2 * T;
      const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)p);
      const shortx4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4*)(p + 4 * 2 * T));
      const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
      return make_uint4(l.x, l.y, h.x, h.y);
    }
  }
};

// One exponent byte per lane to the dword at lds_base + 4 * lane, and four
// (one aligned word) likewise.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma1(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off"
               :
               : "v"(src), "s"(lds_base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Exponents of a slab (eight blocks per row) of the A and then the B tile's
// rows, [row][block]. Where K is a multiple of 128 four bytes of a row are one
// aligned word and arrive as such; otherwise each comes by itself and takes a
// word. Blocks past K repeat earlier ones of their row (their codes are zeros,
// and a NaN there is a NaN of that row already).
template <int TA, int TB, int NW, bool kWords>
struct ScaleLoader {
  static constexpr int kBlocks = 4 * kSteps;                           // per row and slab
  static constexpr int kWordsPerRow = kWords ? kSteps : kBlocks;
  static constexpr int kRows = 64 / kWordsPerRow;                      // rows per piece
  static constexpr int kInstr = (TA + TB) / kRows;                     // pieces per slab
  static constexpr int kPer = kInstr / NW;
  static constexpr int kBytes = kInstr * 256;
  static_assert((TA + TB) % kRows == 0 && kInstr % NW == 0, "every wave brings in as many pieces");
  const uint8_t* src[kPer];
  int block;              // first block of this lane's next word

  __device__ __forceinline__ void init(const uint8_t* a, int a_rows, const uint8_t* b, int b_rows, int per_row, int wave,
                                       int lane) {
    block = (lane % kWordsPerRow) * (kWords ? 4 : 1);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int row = (wave + j * NW) * kRows + lane / kWordsPerRow;
      src[j] = row < TA ? a + int64_t(min(row, a_rows - 1)) * per_row : b + int64_t(min(row - TA, b_rows - 1)) * per_row;
    }
  }

  __device__ __forceinline__ void load(int per_row, uint32_t lds, int wave) {
    const int at = min(block, per_row - (kWords ? 4 : 1));
    block += kBlocks;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t to = lds + (wave + j * NW) * 256;
      if constexpr (kWords)
        dma4(src[j] + at, to);
      else
        dma1(src[j] + at, to);
    }
  }

  // The exponents of blocks 2g and 2g + 1 (g = lane >> 4) of tile row `row` (A's rows first).
  static __device__ __forceinline__ uint32_t read(LdsPtr scales, int row, int lane) {
    static_assert(kSteps == 2, "a lane group's blocks of a slab are a pair");
    if constexpr (kWords) {
      return *reinterpret_cast<__attribute__((address_space(3))) const uint16_t*>(scales + row * 8 + 2 * (lane >> 4));
    } else {
      LdsPtr p = scales + (row * 8 + 2 * (lane >> 4)) * 4;
      return uint32_t(p[0]) | uint32_t(p[4]) << 8;
    }
  }
};

struct NoScales {
  static constexpr int kPer = 0, kBytes = 0;
};

// Waits until at most N loads of this wave, and the stores issued behind them,
// are in flight: kA or kB stores, or none that are known of (0). Loads and
// stores of a wave finish in order, so what is issued behind only makes the
// wait longer.
template <int N, int kA, int kB>
__device__ __forceinline__ void wait_vm_and(int stores) {
  static_assert(N + kA < 64 && N + kB < 64, "vmcnt holds six bits");
  if (stores == kA)
    wait_vm<N + kA>();
  else if (stores == kB)
    wait_vm<N + kB>();
  else
    wait_vm<N>();
}

__device__ __forceinline__ uint2 pack16(const floatx4& v, int dtype) {
  return dtype == MOE_DTYPE_BF16 ? __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4))
                                 : __builtin_bit_cast(uint2, __builtin_convertvector(v, halfx4));
}

// Writes the M results of a lane's output row (four consecutive columns of
// each of M groups of 16 columns from col0 on; `at`: the row's first element).
// fp32: 16 bytes a lane, 64 contiguous ones per row and store. 16-bit: two
// groups change halves between lanes 16 apart, so that a lane holds eight
// consecutive columns and a store again writes 64 contiguous bytes of a row
// (stores of 32 bytes a row took up to 1.5 times as long: they go out by line).
// kAll: rows and columns are known to be valid, and each store is one instruction.
template <int M, bool kAll, typename Get>
__device__ __forceinline__ void store_row(void* out, int dtype, int64_t at, int col0, int cols, bool row_ok, int lane,
                                          Get get) {
  const int g = lane >> 4;
  if (dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int col = col0 + i * 16 + 4 * g;
      if (kAll || (row_ok && col < cols)) *reinterpret_cast<floatx4*>(static_cast<float*>(out) + at + col) = get(i);
    }
    return;
  }
  uint16_t* const o = static_cast<uint16_t*>(out) + at;
  if constexpr (M % 2 == 0) {
#pragma unroll
    for (int i = 0; i < M; i += 2) {
      const uint2 p = pack16(get(i), dtype), q = pack16(get(i + 1), dtype);
      // Lanes' rows of 16: {0, 2} of p with {1, 3} of p below them and the same of q.
      const auto lo = __builtin_amdgcn_permlane16_swap(p.x, q.x, false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(p.y, q.y, false, false);
      const int col = col0 + (i + (g & 1)) * 16 + (g >> 1) * 8;
      if (kAll || (row_ok && col < cols)) *reinterpret_cast<u32x4*>(o + col) = u32x4{lo[0], hi[0], lo[1], hi[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int col = col0 + i * 16 + 4 * g;
      if (kAll || (row_ok && col < cols)) *reinterpret_cast<uint2*>(o + col) = pack16(get(i), dtype);
    }
  }
}

template <typename T, int TA, int TB, int NW>
struct ScalesOf {
  using type = NoScales;
};
template <int TA, int TB, int NW>
struct ScalesOf<Fp4, TA, TB, NW> {
  using type = ScaleLoader<TA, TB, NW, true>;
};
template <int TA, int TB, int NW>
struct ScalesOf<Fp4Odd, TA, TB, NW> {
  using type = ScaleLoader<TA, TB, NW, false>;
};

// A TA x TB tile per task on WA x WB waves. Measured at 4096 tokens, top-8 of
// 128 experts, N = 1536, K = 2048 (128 x 128 tiles, two workgroups a CU):
//   forward 298 us (693 TFLOP/s; 1.2 GB of L2 misses at 4.2 TB/s; without loads
//   207 us, without stores 281), at 2.1 GHz; back to back the clock falls as far
//   as 1.7 GHz and the time rises to 330 us;
//   weight gradient 464 to 550 us by where the busiest experts come in the order
//   of tasks (805 MB written; a tile has four slabs, and its start and stores are
//   not hidden: without stores 299 to 344 us, without loads 288 to 320);
//   MXFP4 121 us (1.7 PFLOP/s; eight slabs per tile; without stores 120 us where
//   the whole takes 140, without loads 93 to 107).
// 8192^3 on one expert: 1210 TFLOP/s (256 x 256 tiles), where torch's product
// reaches 1382. Of 29 M cycles of LDS reads 8192 are bank conflicts; L2
// answers in 510 cycles on average. Two slots with the next step's operands held
// in registers beat more and thinner slots: 64-byte slabs, four deep, 369 us
// against 306 forward (half lines cost the direct operands twice the L2 requests).
// kSplit > 1: the summed index is shared by kSplit waves, each with a ring of
// its own and the whole tile's sums, which are added in wave order at the end;
// for products of few tiles, where a tile's slabs one after the other would be
// most of the time.
template <Kind kKind, typename T, int TA, int TB, int WA, int WB, int kSplit>
__global__ __launch_bounds__(64 * WA * WB * kSplit) __attribute__((amdgpu_waves_per_eu(2))) void
ragged_gemm(const RaggedArgs p) {
  static_assert(kSplit == 1 || WA * WB == 1, "waves that share the summed index keep whole tiles");
  constexpr bool kFp4 = __is_same(T, Fp4) || __is_same(T, Fp4Odd);
  constexpr bool kTransA = kKind != kForward;
  constexpr bool kTransB = kKind == kWeightGrad;
  constexpr int NW = WA * WB;
  constexpr int MA = TA / WA / 16, MB = TB / WB / 16;
  using LA = Loader<TA, NW, kTransA, false, kFp4>;
  using LB = Loader<TB, NW, kTransB, !kTransB, kFp4>;       // no wait counts B's loads, so some may be left out
  using LS = typename ScalesOf<T, TA, TB, NW>::type;
  constexpr int kSlot = (TA + TB) * kSlabBytes + LS::kBytes;    // A tile, B tile, exponents
  static_assert(kSteps == 2, "fb[q] holds step q of a slab");
  extern __shared__ __align__(16) unsigned char lds[];

  const int lane = threadIdx.x & 63;
  const int share = kSplit == 1 ? 0 : uniform(threadIdx.x >> 6);     // of the summed index
  const int wave = kSplit == 1 ? uniform(threadIdx.x >> 6) : 0;
  const int wa = wave % WA, wb = wave / WA;
  unsigned char* const ring = lds + share * kSlots * kSlot;
  const uint32_t ring_at = lds_addr(ring);
  // What the waves of a ring wait for before a slot is read or filled again.
  auto ring_barrier = [&]() {
    if constexpr (kSplit == 1)
      lds_barrier();
    else
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
  };
  const int E = p.E, N = p.N, K = p.K;
  const int OA = kKind == kForward ? N : K;              // output extent along memory
  const int NT = (OA + TA - 1) / TA;
  const int MT = kKind == kWeightGrad ? (N + TB - 1) / TB : 0;

  int* const starts = reinterpret_cast<int*>(lds + kSplit * kSlots * kSlot);
  const Ranges r = scan_ranges<TB>(p.offsets, E, p.rows, starts, lane);
  const int total = kKind == kWeightGrad ? E * NT * MT : r.total * NT;
  lds_barrier();
  // Workgroups go to the eight XCDs in turn: XCD i takes the i-th eighth of
  // the tasks, so neighbouring tasks share an L2.
  const int per = (total + 7) / 8;
  int t = blockIdx.x;
  Task k;
  LA a;
  LB b;
  LS sc;
  int ns = 0, left = 0;        // slabs, and what the last one holds (bytes, or rows)
  bool whole = false;          // ns are the first slabs of more: their last one is whole

  // The next task of this workgroup into k, if there is one.
  auto next = [&]() -> bool {
    for (;; t += gridDim.x) {
      if (t >= 8 * per) return false;
      const int L = (t & 7) * per + (t >> 3);
      if (L >= total) continue;
      t += gridDim.x;
      if constexpr (kKind == kWeightGrad) {
        k.e = L / (NT * MT);
        const int local = L - k.e * NT * MT;
        const int grp = local / (kGroupM * NT);
        const int gm = min(kGroupM, MT - grp * kGroupM);
        const int in = local - grp * kGroupM * NT;
        k.a0 = (in / gm) * TA;
        k.b0 = (grp * kGroupM + in % gm) * TB;
        k.row0 = uniform(starts[k.e]);
        k.rows = uniform(starts[k.e + 1]) - k.row0;
      } else {
        k = find_task<TB>(r, starts, E, L, NT, TA);
      }
      return true;
    }
  };

  // Slabs are brought in one after the other, into slots 0, 1, ..
  auto issue = [&](bool last, int slot) {
    const uint32_t at = ring_at + slot * kSlot;
    if (!last) {
      a.full(at, wave);
      b.full(at + TA * kSlabBytes, wave);
    } else {
      a.tail(left, at, wave);
      b.tail(kKind == kInputGrad ? left * 2 : left, at + TA * kSlabBytes, wave);   // dy is direct: bytes
    }
    if constexpr (kFp4) sc.load(K / 32, at + (TA + TB) * kSlabBytes, wave);
  };

  // Task k's operands, and its first slabs.
  auto begin = [&]() {
    if constexpr (kKind == kForward) {
      const int64_t row_bytes = kFp4 ? K / 2 : int64_t(K) * 2;
      const int64_t x_bytes = kFp4 ? K / 2 : p.ldb * 2;
      const int64_t wrow = int64_t(k.e) * N + k.a0;
      a.init(static_cast<const char*>(p.a) + wrow * row_bytes, row_bytes, min(TA, N - k.a0), wave, lane);
      b.init(static_cast<const char*>(p.b) + k.row0 * x_bytes, x_bytes, k.rows, wave, lane);
      if constexpr (kFp4)
        sc.init(p.a_scale + wrow * (K / 32), min(TA, N - k.a0), p.b_scale + int64_t(k.row0) * (K / 32), k.rows, K / 32,
                wave, lane);
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
    if constexpr (kSplit > 1) {
      const int from = ns * share / kSplit, to = ns * (share + 1) / kSplit;
      whole = to < ns;
      a.base += from * a.step;
      b.base += from * b.step;
      if constexpr (kFp4) sc.block += from * LS::kBlocks;
      ns = to - from;
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (s < ns) issue(!whole && s == ns - 1, s);
  };

  // Wave (wa, wb) takes MA neighbouring groups of 16 of the A tile and every
  // WB-th group of the B tile, so that a tile with few rows is shared evenly.
  // A matrix step's A operands are read in kHalves parts (two where all of
  // them would not fit the registers beside the sums).
  constexpr int kHalves = MA >= 8 ? 2 : 1;
  constexpr int kPart = MA / kHalves;
  Reader<TA, MA, 1, kTransA> ra;
  Reader<TB, MB, WB, kTransB> rb;
  ra.init(wa * MA, lane);
  rb.init(wb, lane);
  int nb = 0;              // groups of B with a row of the task, for this wave
  uint4 fa[2][kPart], fb[2][MB];
  struct {
    uint32_t a[(MA + 1) / 2], b[(MB + 1) / 2];   // exponents of two groups share a word
  } now, then;
  // Part h of step q of the slab in `slot`; `full`: the tile has all its B groups.
  auto read = [&](auto full, int slot, int q, int h) {
    const LdsPtr at = (LdsPtr)ring + slot * kSlot;
#pragma unroll
    for (int i = 0; i < kPart; ++i) fa[(q * kHalves + h) % 2][i] = ra.get(at, q, h * kPart + i);
    if (h == 0) {
#pragma unroll
      for (int j = 0; j < MB; ++j)
        if (decltype(full)::value || j < nb) fb[q][j] = rb.get(at + TA * kSlabBytes, q, j);
    }
    if constexpr (kFp4) {
      if (q == 0 && h == 0) {
        const LdsPtr st = at + (TA + TB) * kSlabBytes;
#pragma unroll
        for (int i = 0; i < MA; ++i) {
          const uint32_t v = LS::read(st, (wa * MA + i) * 16 + (lane & 15), lane);
          then.a[i / 2] = i % 2 ? then.a[i / 2] | v << 16 : v;
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const uint32_t v = LS::read(st, TA + (wb + j * WB) * 16 + (lane & 15), lane);
          then.b[j / 2] = j % 2 ? then.b[j / 2] | v << 16 : v;
        }
      }
    }
  };

  constexpr int kStores16 = MB * MA / 2, kStores32 = MB * MA;   // of a wave, for a tile that is all valid
  int stores = 0;          // issued behind the loads of this task's first slabs, where their number is known
  bool have = next();
  if (have) begin();
  while (have) {
    floatx4 acc[MA][MB];
#pragma unroll
    for (int i = 0; i < MA; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    // The compiler keeps the order of these blocks: it would sink the next
    // part's reads to their first use otherwise.
    auto multiply = [&](auto full, int q, int h) {
      if constexpr (kFp4) {
        if (q == 0 && h == 0) now = then;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        if (decltype(full)::value || j < nb) {
#pragma unroll
          for (int n = 0; n < kPart; ++n) {
            const int i = h * kPart + n;
            const uint4& av = fa[(q * kHalves + h) % 2][n];
            if constexpr (kFp4)
              acc[i][j] = mfma_step_fp4(av, fb[q][j], acc[i][j], now.a[i / 2], i % 2 * 2 + q, now.b[j / 2], j % 2 * 2 + q);
            else
              acc[i][j] = mfma_step<T>(av, fb[q][j], acc[i][j]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // The parts of the slab in slot i but the last product.
    auto inside = [&](auto full, int i) {
#pragma unroll
      for (int n = 1; n < 2 * kHalves; ++n) {
        read(full, i, n / kHalves, n % kHalves);
        multiply(full, (n - 1) / kHalves, (n - 1) % kHalves);
      }
    };
    {
      const int groups = ((kKind == kWeightGrad ? min(TB, N - k.b0) : k.rows) + 15) / 16;
      nb = uniform(max(0, (groups - wb + WB - 1) / WB));
    }
    // The next part is read into registers while this one is multiplied.
    // Behind a slab's barrier every wave has read that slab, and its slot takes
    // the one after the next. Slabs go in pairs, so that slots are constants.
    auto products = [&](auto full) {
      // Slab 0, while slab 1 (its A pieces and exponents at least) and the
      // stores of the task before, issued behind them, may be in flight; then
      // slab 1, while those stores may.
      if (ns > 1)
        wait_vm_and<LA::kPer + LS::kPer, kStores16, kStores32>(stores);
      else
        wait_vm<0>();
      ring_barrier();
      read(full, 0, 0, 0);
      auto wait_next = [&](int s) {
        if (s == 0)
          wait_vm_and<0, kStores16, kStores32>(stores);
        else
          wait_vm<0>();
      };
      int s = 0;
      for (; s + 2 * kSlots < ns; s += kSlots) {       // every slab brought in here is whole
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          inside(full, i);
          wait_next(s + i);
          ring_barrier();
          issue(false, i);
          read(full, (i + 1) % kSlots, 0, 0);
          multiply(full, 1, kHalves - 1);
        }
      }
      for (; s < ns; s += kSlots) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if (s + i < ns) {
            inside(full, i);
            if (s + i + 1 < ns) {
              wait_next(s + i);
              ring_barrier();
              if (s + i + kSlots < ns) issue(!whole && s + i + kSlots == ns - 1, i);
              read(full, (i + 1) % kSlots, 0, 0);
            }
            multiply(full, 1, kHalves - 1);
          }
        }
      }
    };
    if (ns > 0) {
      // Absent groups are left out by a test at each; a weight gradient makes none (what a last tile
      // reads past N repeats its last chunk and is not stored): 514 -> 503 us for 4096 tokens. A
      // second copy of the loop without tests for forward tiles that are whole gains nothing.
      products(std::bool_constant<kKind == kWeightGrad>{});
    }
    const Task done = k;
    const int cols = nb;
    if constexpr (kSplit > 1) {
      // Wave w takes the sums of every kSplit-th group of B from group w on.
      floatx4* const sums = reinterpret_cast<floatx4*>(lds);
      static_assert(MA * MB * 64 * sizeof(floatx4) <= kSlots * kSlot, "the sums take the rings' place");
      lds_barrier();
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int i = 0; i < MA; ++i) sums[((share * MB + j) * MA + i) * 64 + lane] = acc[i][j];
      lds_barrier();
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        if (j % kSplit != share || j >= cols) continue;
#pragma unroll
        for (int i = 0; i < MA; ++i) {
          floatx4 v = sums[(j * MA + i) * 64 + lane];
#pragma unroll
          for (int n = 1; n < kSplit; ++n) {
            const floatx4 o = sums[((n * MB + j) * MA + i) * 64 + lane];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] += o[c];
          }
          acc[i][j] = v;
        }
      }
    }
    have = next();
    if (have) {
      lds_barrier();      // every wave has read the last slab
      begin();            // the next task's loads run under this one's stores
    }

    const bool all = kSplit == 1 && done.a0 + TA <= OA &&
                     (kKind == kWeightGrad ? done.b0 + TB <= N : done.rows == TB);
    auto store = [&](auto valid) {
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        if (kSplit > 1 && (j % kSplit != share || j >= cols)) continue;
        const int row = (wb + j * WB) * 16 + (lane & 15);
        const bool row_ok = kKind == kWeightGrad ? done.b0 + row < N : row < done.rows;
        const int64_t at = kKind == kWeightGrad ? (int64_t(done.e) * N + done.b0 + row) * K : (done.row0 + row) * p.ldo;
        store_row<MA, decltype(valid)::value>(p.out, p.out_dtype, at, done.a0 + wa * MA * 16, OA, row_ok, lane,
                                              [&](int i) { return acc[i][j]; });
      }
    };
    if (all) {
      store(std::true_type{});
      stores = p.out_dtype == MOE_DTYPE_F32 ? kStores32 : kStores16;
    } else {
      store(std::false_type{});
      stores = 0;
    }
  }
}

// The forward product for experts with few rows each (a token's or a small
// batch's routes): bound by reading each weight once. A workgroup owns 16 rows
// and 16 * G output columns of an expert, and its waves share the summed
// index, so that a single token's products spread over the chip; weights go
// from memory straight to the matrix instructions' registers, every load of two
// blocks in flight before the first product. The waves' sums are added in wave
// order through LDS. One token, eight experts, N = 1536, K = 2048: bf16 10.7 us
// (50 MB: 4.7 TB/s), MXFP4 6.0 us (13 MB; its start, one round trip to memory
// and the sums). 21 tokens in bf16: 104 us, 5.7 TB/s.
constexpr int kStreamWaves = 4;
constexpr int kBlockBytes = 256;      // of a row per wave and turn: four matrix steps

template <typename T, int G>
__global__ __launch_bounds__(64 * kStreamWaves) __attribute__((amdgpu_waves_per_eu(G == 1 ? 4 : 3))) void
ragged_stream(const RaggedArgs p) {
  constexpr bool kFp4 = __is_same(T, Fp4);
  extern __shared__ __align__(16) unsigned char lds[];      // the waves' sums, then the experts' start rows
  floatx4* const sums = reinterpret_cast<floatx4*>(lds);
  int* const starts = reinterpret_cast<int*>(lds + kStreamWaves * G * 64 * sizeof(floatx4));
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int E = p.E, N = p.N, K = p.K;
  const int NT = (N + (16 * G) - 1) / (16 * G);
  const Ranges r = scan_ranges<16>(p.offsets, E, p.rows, starts, lane);
  const int total = r.total * NT;
  lds_barrier();
  const int per = (total + 7) / 8;       // XCD i takes the i-th eighth of the tasks
  for (int t = blockIdx.x; t < 8 * per; t += gridDim.x) {
    const int L = (t & 7) * per + (t >> 3);
    if (L >= total) continue;
    const Task k = find_task<16>(r, starts, E, L, NT, (16 * G));
    const int64_t wld = kFp4 ? K / 2 : int64_t(K) * 2, xld = kFp4 ? K / 2 : p.ldb * 2;
    const int bytes = static_cast<int>(wld);
    const int sb = K / 32;                // exponents of a row
    const char* wrow[G];
    const uint8_t* wscale[G];
    const int64_t xr = k.row0 + min(lane & 15, k.rows - 1);
    const char* const xrow = static_cast<const char*>(p.b) + xr * xld;
    const uint8_t* const xscale = kFp4 ? p.b_scale + xr * sb : nullptr;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      const int64_t n = int64_t(k.e) * N + min(k.a0 + c * 16 + (lane & 15), N - 1);
      wrow[c] = static_cast<const char*>(p.a) + n * wld;
      wscale[c] = kFp4 ? p.a_scale + n * sb : nullptr;
    }
    floatx4 acc[G];
#pragma unroll
    for (int c = 0; c < G; ++c) acc[c] = floatx4{0.f, 0.f, 0.f, 0.f};

    // One block of a wave: 256 bytes of every row. 16-bit: matrix step s takes
    // bytes 64 s .. 64 s + 63. MXFP4: lane group g takes blocks 4g .. 4g + 3 of
    // the sixteen, one a step, so that its exponents are one word.
    struct Block {
      uint4 w[G][4], x[4];
      uint32_t ws[G], xs;
    };
    auto chunk = [&](int s) { return kFp4 ? 64 * g + 16 * s : 64 * s + 16 * g; };
    auto load = [&](Block& b, int at) {
      if (at + kBlockBytes <= bytes) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          b.x[s] = *reinterpret_cast<const uint4*>(xrow + at + chunk(s));
#pragma unroll
          for (int c = 0; c < G; ++c) b.w[c][s] = *reinterpret_cast<const uint4*>(wrow[c] + at + chunk(s));
        }
        if constexpr (kFp4) {
          __builtin_memcpy(&b.xs, xscale + at / 16 + 4 * g, 4);
#pragma unroll
          for (int c = 0; c < G; ++c) __builtin_memcpy(&b.ws[c], wscale[c] + at / 16 + 4 * g, 4);
        }
      } else {                            // the row ends inside: zeros, with the exponent of one
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const bool in = at + chunk(s) < bytes;
          const int from = in ? at + chunk(s) : 0;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          const uint4 xv = *reinterpret_cast<const uint4*>(xrow + from);
          b.x[s] = in ? xv : zero;
#pragma unroll
          for (int c = 0; c < G; ++c) {
            const uint4 wv = *reinterpret_cast<const uint4*>(wrow[c] + from);
            b.w[c][s] = in ? wv : zero;
          }
        }
        if constexpr (kFp4) {
          b.xs = 0;
#pragma unroll
          for (int c = 0; c < G; ++c) b.ws[c] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = at / 16 + 4 * g + i;
            const bool in = n < sb;
            b.xs |= uint32_t(in ? xscale[in ? n : 0] : 127) << (8 * i);
#pragma unroll
            for (int c = 0; c < G; ++c) b.ws[c] |= uint32_t(in ? wscale[c][in ? n : 0] : 127) << (8 * i);
          }
        }
      }
    };
    auto multiply = [&](const Block& b) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int c = 0; c < G; ++c) {
          if constexpr (kFp4)
            acc[c] = mfma_step_fp4(b.w[c][s], b.x[s], acc[c], b.ws[c], s, b.xs, s);
          else
            acc[c] = mfma_step<T>(b.w[c][s], b.x[s], acc[c]);
        }
    };
    constexpr int kTurn = kStreamWaves * kBlockBytes;
    for (int at = wave * kBlockBytes; at < bytes; at += 2 * kTurn) {
      Block b0, b1;
      load(b0, at);
      const bool two = at + kTurn < bytes;
      if (two) load(b1, at + kTurn);
      multiply(b0);
      if (two) multiply(b1);
    }
#pragma unroll
    for (int c = 0; c < G; ++c) sums[(wave * G + c) * 64 + lane] = acc[c];
    lds_barrier();
    if (wave < G) {
      floatx4 v = sums[wave * 64 + lane];
#pragma unroll
      for (int i = 1; i < kStreamWaves; ++i) {
        const floatx4 o = sums[(i * G + wave) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += o[j];
      }
      store_row<1, false>(p.out, p.out_dtype, (k.row0 + (lane & 15)) * p.ldo, k.a0 + wave * 16, N, (lane & 15) < k.rows, lane,
                   [&](int) { return v; });
    }
    lds_barrier();
  }
}

int64_t row_tiles(const RaggedArgs& p, int tile) {      // at most
  return int64_t(p.rows) / tile + (p.E < p.rows ? p.E : p.rows);
}

template <Kind kKind>
int64_t task_count(const RaggedArgs& p, int ta, int tb) {
  const int64_t nt = ((kKind == kForward ? p.N : p.K) + ta - 1) / ta;
  return nt * (kKind == kWeightGrad ? int64_t(p.E) * ((p.N + tb - 1) / tb) : row_tiles(p, tb));
}

template <Kind kKind, typename T, int TA, int TB, int WA, int WB, int kSplit = 1>
hipError_t run(const RaggedArgs& p, hipStream_t stream) {
  const int64_t tasks = task_count<kKind>(p, TA, TB);
  constexpr int ring = kSplit * kSlots * ((TA + TB) * kSlabBytes + ScalesOf<T, TA, TB, WA * WB>::type::kBytes);
  const int lds = ring + (p.E + 1) * 4;
  // As many workgroups as run at once (two waves per SIMD, and by LDS); each
  // takes tasks in turn and loads its next one's first slabs under its stores.
  constexpr int waves = WA * WB * kSplit;
  const int at_once = kCus * (8 / waves < kLdsPerCu / lds ? 8 / waves : kLdsPerCu / lds);
  launch(ragged_gemm<kKind, T, TA, TB, WA, WB, kSplit>, dim3(grid_for((tasks + 7) & ~int64_t(7), at_once)),
         dim3(64 * waves), lds, stream, p);
  return hipGetLastError();
}

template <typename T, int G>
hipError_t run_stream(const RaggedArgs& p, hipStream_t stream) {
  const int64_t tasks = row_tiles(p, 16) * ((p.N + 16 * G - 1) / (16 * G));
  const int lds = kStreamWaves * G * 64 * int(sizeof(floatx4)) + (p.E + 1) * 4;
  launch(ragged_stream<T, G>, dim3(grid_for((tasks + 7) & ~int64_t(7), 0)), dim3(64 * kStreamWaves), lds, stream, p);
  return hipGetLastError();
}

// Which kernel: ragged_stream fills the chip with few rows, ragged_gemm reads
// weights in whole 128-byte lines and shares them between the rows of a tile.
// Measured at N = 1536, K = 2048, 128 experts, top-8 (us per call, stream / tiles):
//   bf16, tokens 1: 11.9 / 12.4, 4: 38.0 / 41.9, 21: 104 / 124, 64: 142 / 158, 128: 155 / 171, 256: 210 / 174;
//   MXFP4, tokens 1: 9.2 / 9.1, 4: 16.6 / 14.3, 21: 51.5 / 37.7.
// So 16-bit operands stream up to eight rows per expert, MXFP4 (a stream's
// loads of a quarter of the bytes leave more of each line to the cache) only
// where the tiles would leave CUs idle. The host knows the average alone: 1024
// rows that all belong to one of the 128 experts stream too, sixteen rows to a
// task, in 78 us where tiles take 25.
bool few_rows(const RaggedArgs& p) { return p.rows <= 8 * int64_t(p.E < p.rows ? p.E : p.rows); }

// Columns per workgroup: 16 where 32 would give a CU fewer than four
// workgroups (bf16, 1 token: 11.6 / 12.9 us; 4 tokens: 38.7 / 37.7).
template <typename T>
hipError_t pick_stream(const RaggedArgs& p, hipStream_t stream) {
  if (row_tiles(p, 16) * ((p.N + 31) / 32) < 4 * kCus) return run_stream<T, 1>(p, stream);
  return run_stream<T, 2>(p, stream);
}

// Tile shapes. 128 x 128 on four waves, two workgroups a CU, is the common one.
// 64 x 64 with the summed index shared by four waves where those tiles (at
// most: experts end inside them) fill the CUs about once: 1024 rows of 8
// experts, N = K = 1024: 14.7 -> 10.4 us; N = 1024, K = 4096: 61.6 -> 26.1; but
// N = 1536, K = 1024: 15.4 -> 16.7, and a weight gradient of 512 such tiles
// 8.2 -> 9.5. 256 x 256 for a 16-bit forward product with many rows per expert
// and tasks for two rounds: 8192 tokens, top-8 of uneven experts, N = 1536, K =
// 1024: 64 experts 302 -> 278 us, 128 experts 320 -> 318; 32768 rows shared
// evenly by 16 experts, K = 2048: 261 -> 228. With 256 rows per expert nothing
// is sure: 4096 tokens of 128 experts, K = 2048: 352 -> 346 on one card, 301 ->
// 324 on another. The gradients gain or lose 4 % by it and do without.
template <Kind kKind, typename T>
hipError_t pick(const RaggedArgs& p, hipStream_t stream) {
  constexpr bool kOdd = __is_same(T, Fp4Odd);
  if (2 * task_count<kKind>(p, 64, 64) <= 3 * kCus) return run<kKind, T, 64, kOdd ? 32 : 64, 1, 1, 4>(p, stream);
  if constexpr (kKind == kForward && (__is_same(T, Bf16) || __is_same(T, F16))) {
    if (p.rows >= 512 * int64_t(p.E) && task_count<kKind>(p, 256, 256) >= 2 * kCus)
      return run<kKind, T, 256, 256, 2, 4>(p, stream);
  }
  return run<kKind, T, 128, 128, 2, 2>(p, stream);
}

}  // namespace

hipError_t launch_ragged_forward(const RaggedArgs& p, int dtype, hipStream_t stream) {
  if (dtype == MOE_DTYPE_MXFP4) {
    const bool words = p.K % 128 == 0 && reinterpret_cast<uintptr_t>(p.a_scale) % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(p.b_scale) % 4 == 0;
    if (few_rows(p) && task_count<kForward>(p, 128, 128) < kCus) return run_stream<Fp4, 1>(p, stream);
    return words ? pick<kForward, Fp4>(p, stream) : pick<kForward, Fp4Odd>(p, stream);
  }
  if (few_rows(p)) return dtype == MOE_DTYPE_F16 ? pick_stream<F16>(p, stream) : pick_stream<Bf16>(p, stream);
  return dtype == MOE_DTYPE_F16 ? pick<kForward, F16>(p, stream) : pick<kForward, Bf16>(p, stream);
}

hipError_t launch_ragged_input_grad(const RaggedArgs& p, int dtype, hipStream_t stream) {
  return dtype == MOE_DTYPE_F16 ? pick<kInputGrad, F16>(p, stream) : pick<kInputGrad, Bf16>(p, stream);
}

hipError_t launch_ragged_weight_grad(const RaggedArgs& p, int dtype, hipStream_t stream) {
  return dtype == MOE_DTYPE_F16 ? pick<kWeightGrad, F16>(p, stream) : pick<kWeightGrad, Bf16>(p, stream);
}

}  // namespace moe
