// Products of a few rows with packed 4-bit weights (gfx950):
//   y[r][n] = sum_k (q[e][n][k] - z[e][n][k / g]) s[e][n][k / g] x[r / per][k]
// with one matrix for every row, or the matrix of the row's expert.
//
// The weights are the right operand of 16x16x32 matrix instructions and x the
// left one, so up to sixteen rows cost the same unpacking, and a lane's results
// belong to the weight row that it loads: scale and zero are one value per lane.
// A nibble is OR-ed into the top of a 16-bit mantissa, which gives 16 + q exactly;
// a group's sum is then
//   s (sum (16 + q) x - (16 + z) sum x)
// in fp32, where sum x comes from a matrix instruction with ones. (An offset of
// 128, from the mantissa's low bits, would cancel eight times as much.)
//
// A wave's loads take whole lines (eight lanes to 128 bytes of a weight row) and
// pass through LDS into the operands' layout; a load with neighbouring lanes in
// different rows costs the cache four times as much. Loads go through buffer
// descriptors, whose bounds give zeros past the ends of rows, features and the
// wave's share of the summed index.
#include "common.hpp"
#include "kernels.hpp"
#include "matvec_shape.hpp"

namespace moe {

namespace {

constexpr int kMaxWaves = 8;   // of a workgroup: they share the summed index
constexpr int kTile = 16;      // weight rows, and rows of x, of a matrix instruction

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

template <bool kHalf>
constexpr uint32_t kMask = kHalf ? 0x03C003C0u : 0x00780078u;

// Eight 4-bit values of a word as 16 + q, in element order.
template <bool kHalf>
__device__ __forceinline__ u32x4 unpack8(uint32_t w, uint32_t m) {   // m: kMask in a VGPR (see in_vgpr)
  u32x4 v;
  if constexpr (kHalf) {
    const uint32_t c = 0x4C004C00u;
    v[0] = ((w << 6) & m) | c;
    v[1] = ((w << 2) & m) | c;
    v[2] = ((w >> 2) & m) | c;
    v[3] = ((w >> 6) & m) | c;
  } else {
    const uint32_t c = 0x41804180u;
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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  // Wave-uniform, which the compiler has to see: it loops over a descriptor that it takes for a lane's own.
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  const uint32_t lo = uniform(static_cast<int>(a)), hi = uniform(static_cast<int>(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uintptr_t(hi) << 32 | lo), 0,
                                           uniform(static_cast<int>(bytes)), 0x00020000);
}

constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer here

// A workgroup takes 16 kShare weight rows, 16 to a wave, and up to kRows rows of
// x; the groups of kShare waves share the summed index, their sums meet in LDS. A
// step takes kChunk elements of it, whose x a group's waves bring in together.
// kFlush: products of 32 elements after which a sum is scaled (what divides the
// group and 128 alike).
template <bool kHalf, int kChunk, int kRows, int kShare, int kFlush>
__global__ __launch_bounds__(kMaxWaves* kWave) void matvec(MatvecArgs p) {
  constexpr int kCols = (kRows + kTile - 1) / kTile;
  constexpr int kSteps = kChunk / 32;                // products of a chunk
  constexpr int kWPieces = kSteps, kXPieces = kChunk / 8;   // 16-byte pieces of a chunk of a row
  constexpr int kWLoads = kTile * kWPieces / kWave;
  constexpr int kXLoads = kRows * kXPieces / kWave / kShare;
  constexpr int kSLoads = kTile * kSteps / kWave;
  // Chunks whose loads are in flight. Loads return in order, so x is as far ahead as the weights.
  constexpr int kAhead = kXLoads * kChunk <= 512 ? 4 : 2;
  constexpr int kUnroll = 4;                         // chunks of a batch of scales (kFlush), at most
  constexpr int kBatches = kAhead > kFlush ? kAhead / kFlush : 1;   // of scales in flight
  struct Stage {
    u32x4 w[kTile][kWPieces];
  };
  struct Mine {
    Stage stage[2];
    uint32_t sz[kTile][kSteps];                      // scale, and zero in the third byte, of kSteps flushes
  };
  struct Group {
    u32x4 x[2][kRows][kXPieces];
  };
  extern __shared__ u32x4 lds[];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int splits = blockDim.x / (kWave * kShare);
  const int split = wave / kShare, part_of = wave % kShare;
  Mine& mine = reinterpret_cast<Mine*>(lds)[wave];
  Group& shared = reinterpret_cast<Group*>(reinterpret_cast<Mine*>(lds) + splits * kShare)[split];
  const int r = lane & 15, q = lane >> 4;            // in operands: row, eight elements of a product's 32
  const int lr = lane / kWPieces, lp = lane % kWPieces;     // in loads of weights and scales
  const int tiles = (p.N + kTile * kShare - 1) / (kTile * kShare);
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int per = (chunks + splits - 1) / splits;
  const int c0 = per * split, c1 = min(c0 + per, chunks);
  const int groups = p.K / p.group;
  const uint32_t one = kHalf ? 0x3C003C00u : 0x3F803F80u;
  const u32x4 ones = {one, one, one, one};
  const uint32_t mask = in_vgpr(kMask<kHalf>);
  for (int64_t task = blockIdx.x; task < p.tasks; task += gridDim.x) {
    // (64-bit divisions are vector code: `uniform` keeps the descriptors scalar.)
    const int block = uniform(static_cast<int>(task / tiles));
    const int n0 = uniform(static_cast<int>(task - int64_t(block) * tiles)) * (kTile * kShare) + part_of * kTile;
    const int64_t row0 = p.ids != nullptr ? block : int64_t(block) * kRows;
    const int rows = p.ids != nullptr ? 1 : static_cast<int>(min(int64_t(kRows), p.rows - row0));
    const int e = p.ids != nullptr ? uniform(p.ids[row0]) : 0;
    floatx4 acc[kCols] = {};
    if (e >= 0 && e < p.E) {
      const int have = max(0, min(kTile, p.N - n0));
      const int64_t w0 = int64_t(e) * p.N + (have > 0 ? n0 : 0);
      const auto wbuf = buffer_of(static_cast<const uint8_t*>(p.w.q) + w0 * (p.K / 2), int64_t(have) * (p.K / 2));
      const auto sbuf = buffer_of(static_cast<const uint16_t*>(p.w.scale) + w0 * groups, int64_t(have) * groups * 2);
      const auto zbuf = buffer_of(p.w.zero != nullptr ? p.w.zero + w0 * groups : static_cast<const uint8_t*>(p.w.q),
                                  p.w.zero != nullptr ? int64_t(have) * groups : 0);
      const auto xbuf = buffer_of(static_cast<const uint16_t*>(p.x) + uniform(static_cast<int>(row0 / p.per)) * p.ldx,
                                  (int64_t(rows - 1) * p.ldx + p.K) * 2);
      const float zbase = p.w.zero != nullptr ? 16.0f : 24.0f;
      u32x4 w[kAhead][kWLoads], x[kAhead][kXLoads];
      const int xp = lane % kXPieces;                  // in loads of x
      const auto xrow = [&](int i) { return (i * kShare + part_of) * (kWave / kXPieces) + lane / kXPieces; };
      // Neighbouring tiles start at other batches of scales, so that the workgroups of a chip do not all want the
      // same lines of x at once: 64 rows, 4096 x 2048: 15.1 -> 13.5 us; 4096 rows: 203 -> 190.
      const int share = c1 - c0;
      const int turn = share > kUnroll && share % kUnroll == 0 ? n0 / (kTile * kShare) * kUnroll % share : 0;
      const auto turned = [&](int c) { return c >= c1 ? c : c + turn < c1 ? c + turn : c + turn - share; };
      const auto load = [&](int step, u32x4* wr, u32x4* xr) {
        const int c = turned(step);
        const uint32_t at = c < c1 ? c * (kChunk / 2) : kOutside;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
          wr[i] = __builtin_amdgcn_raw_buffer_load_b128(
              wbuf, uint32_t(i * (kWave / kWPieces) + lr) * (p.K / 2) + lp * 16 + at, 0, 0);
        // Past the sum's end x has to be zero; the weights there are another row's, and finite.
        const int left = c < c1 ? (p.K - c * kChunk) / 8 : 0;
        const uint32_t xat = xp < left ? c * (kChunk * 2) + xp * 16 : kOutside;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
          xr[i] = __builtin_amdgcn_raw_buffer_load_b128(
              xbuf, uint32_t(xrow(i)) * static_cast<uint32_t>(p.ldx) * 2 + xat, 0, 0);
      };
      const auto load_sz = [&](int step, uint16_t* sc, uint8_t* ze) {   // kSteps flushes from chunk `step` on
        const int c = turned(step);
        const int g = min(static_cast<int>(__umulhi(2 * (c * kSteps + lp * kFlush), p.group_inverse)), groups - 1);
#pragma unroll
        for (int i = 0; i < kSLoads; ++i) {
          const uint32_t at = uint32_t(i * (kWave / kWPieces) + lr) * groups + g;
          sc[i] = __builtin_amdgcn_raw_buffer_load_b16(sbuf, at * 2, 0, 0);
          ze[i] = __builtin_amdgcn_raw_buffer_load_b8(zbuf, at, 0, 0);
        }
      };
      // Pieces lie at an exclusive or with their row's number, so that eight rows' same piece is in other banks.
      constexpr int kTurn = kWPieces == 8 ? 1 : 2;
      const auto store = [&](int b, const u32x4* wr, const u32x4* xr) {
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) {
          const int row = i * (kWave / kWPieces) + lr;
          mine.stage[b].w[row][lp ^ (row >> kTurn)] = wr[i];
        }
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) shared.x[b][xrow(i)][xp ^ (xrow(i) & 15)] = xr[i];
      };
      const auto store_sz = [&](const uint16_t* sc, const uint8_t* ze) {
#pragma unroll
        for (int i = 0; i < kSLoads; ++i) {            // (not joined in a register: that would wait for the loads)
          char* at = reinterpret_cast<char*>(&mine.sz[i * (kWave / kWPieces) + lr][lp]);
          __builtin_memcpy(at, &sc[i], 2);
          __builtin_memcpy(at + 2, &ze[i], 1);
        }
      };
      uint32_t szs[kSteps];
      // A chunk in LDS: u-th of those that share a batch of scales.
      const auto multiply = [&](int b, int u) {
        u32x4 v[kWLoads];
#pragma unroll
        for (int h = 0; h < kWLoads; ++h) v[h] = transpose4(mine.stage[b].w[r][(h * 4 + q) ^ (r >> kTurn)]);
        floatx4 sum[kCols], xs[kCols];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          if (j % kFlush == 0) {
#pragma unroll
            for (int m = 0; m < kCols; ++m) sum[m] = xs[m] = floatx4{0, 0, 0, 0};
          }
          const u32x4 weights = unpack8<kHalf>(v[j / 4][j % 4], mask);
#pragma unroll
          for (int m = 0; m < kCols; ++m) {
            const int row = (m * kTile + r) % kRows;
            const u32x4 a = shared.x[b][row][(j * 4 + q) ^ (row & 15)];
            xs[m] = mfma<kHalf>(a, ones, xs[m]);
            sum[m] = mfma<kHalf>(a, weights, sum[m]);
          }
          if (j % kFlush == kFlush - 1) {
            const uint32_t h = szs[u * (kSteps / kFlush) + j / kFlush];
            const float sv = half_bits_to_float(h & 0xFFFF), z = zbase + static_cast<float>(h >> 16 & 0xFF);
#pragma unroll
            for (int m = 0; m < kCols; ++m) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][i] += sv * (sum[m][i] - z * xs[m][i]);
            }
          }
        }
      };
      uint16_t sc[kBatches][kSLoads];
      uint8_t ze[kBatches][kSLoads];
      // Step c: chunk c + 1 (in the order of `turned`) goes to LDS, chunk c + 1 + kAhead is requested, chunk c is multiplied.
      const auto step = [&](int c, int u, bool more) {
        __builtin_amdgcn_sched_barrier(0);   // or later chunks' loads move up and take registers
        if constexpr (kShare > 1)
          lds_barrier();
        else
          asm volatile("" ::: "memory");     // lanes read what others wrote: LDS accesses stay in this order
        if (u % kFlush == 0) {
#pragma unroll
          for (int f = 0; f < kSteps; ++f) szs[f] = mine.sz[r][f];
          asm volatile("" ::: "memory");
          const int next = (u / kFlush + 1) % kBatches;
          store_sz(sc[next], ze[next]);
          if (more || u + (1 + kBatches) * kFlush < kUnroll)
            load_sz(c + u + (1 + kBatches) * kFlush, sc[next], ze[next]);
        }
        store((u + 1) & 1, w[(u + 1) % kAhead], x[(u + 1) % kAhead]);
        if (more || u + 1 + kAhead < kUnroll) load(c + u + 1 + kAhead, w[(u + 1) % kAhead], x[(u + 1) % kAhead]);
        multiply(u & 1, u % kFlush);
      };
      // In the loop's order, or the waits at its head would be for these loads' order instead: chunk t is
      // requested by step t - 1 - kAhead.
      uint16_t sc0[kSLoads];
      uint8_t ze0[kSLoads];
      load_sz(c0, sc0, ze0);
      if constexpr (kAhead + 1 < kFlush) load_sz(c0 + kFlush, sc[0], ze[0]);
#pragma unroll
      for (int t = 0; t <= kAhead; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        if ((kAhead + 1 - t) % kFlush == 0) {
          const int batch = 1 + kBatches - (kAhead + 1 - t) / kFlush;
          if (batch > 0) load_sz(c0 + batch * kFlush, sc[batch % kBatches], ze[batch % kBatches]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t == kAhead) {
          store_sz(sc0, ze0);
          store(0, w[0], x[0]);
          asm volatile("" ::: "memory");
        }
        load(c0 + t, w[t % kAhead], x[t % kAhead]);
      }
      // Waves that meet at barriers take as many chunks; those past the sum's end are zeros.
      const int end = kShare > 1 ? c0 + per : c1;
      int c = c0;
      for (; c + kUnroll <= end; c += kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) step(c, u, true);
      }
      if (c < end) step(c, 0, false);
      if (c + 1 < end) step(c, 1, false);
      if (c + 2 < end) step(c, 2, false);
    }
    __syncthreads();
    floatx4* part = reinterpret_cast<floatx4*>(lds);
    if (split > 0) {
#pragma unroll
      for (int m = 0; m < kCols; ++m) part[((wave - kShare) * kCols + m) * kWave + lane] = acc[m];
    }
    __syncthreads();
    if (split == 0) {
      const int n = n0 + r;
#pragma unroll
      for (int m = 0; m < kCols; ++m) {
        for (int s = 1; s < splits; ++s) acc[m] += part[((wave + (s - 1) * kShare) * kCols + m) * kWave + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = m * kTile + q * 4 + i;
          if (col >= rows || n >= p.N) continue;
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

template <bool kHalf, int kChunk, int kRows, int kShare>
void start(MatvecArgs p, const MatvecShape& c, hipStream_t stream) {
  const int64_t tiles = (p.N + kTile * kShare - 1) / (kTile * kShare);
  const int64_t blocks = p.ids != nullptr ? p.rows : (p.rows + kRows - 1) / kRows;
  p.tasks = tiles * blocks;
  // Products of 32 elements to their group: exact for the 2^15 + 2^7 that are asked for at most.
  p.group_inverse = static_cast<uint32_t>(((uint64_t(1) << 31) + p.group / 32 - 1) / (p.group / 32));
  const int waves = c.splits * kShare;
  const dim3 grid(grid_for(p.tasks, 0)), block(waves * kWave);
  uint32_t lds = waves * (2 * kTile * kChunk / 2 + kTile * kChunk / 8) + c.splits * 2 * kRows * kChunk * 2;
  const uint32_t sums = (c.splits - 1) * kShare * ((kRows + kTile - 1) / kTile) * kWave * 16;
  lds = lds > sums ? lds : sums;
  if (c.flush == 4)
    launch(matvec<kHalf, kChunk, kRows, kShare, 4>, grid, block, lds, stream, p);
  else if (c.flush == 2)
    launch(matvec<kHalf, kChunk, kRows, kShare, 2>, grid, block, lds, stream, p);
  else
    launch(matvec<kHalf, kChunk, kRows, kShare, 1>, grid, block, lds, stream, p);
}

template <bool kHalf, int kRows>
void by_share(const MatvecArgs& p, const MatvecShape& c, hipStream_t stream) {
  if (c.share == 2)
    start<kHalf, 128, kRows, 2>(p, c, stream);
  else
    start<kHalf, 128, kRows, 4>(p, c, stream);
}

template <bool kHalf>
void by_shape(const MatvecArgs& p, hipStream_t stream) {
  const MatvecShape c = matvec_shape(p.ids != nullptr, p.rows, p.N, p.K, p.group);
  if (c.chunk == 256)
    start<kHalf, 256, 4, 1>(p, c, stream);
  else if (c.rows == 4)
    start<kHalf, 128, 4, 1>(p, c, stream);
  else if (c.rows == 16 && c.share == 1)
    start<kHalf, 128, 16, 1>(p, c, stream);
  else if (c.rows == 16)
    by_share<kHalf, 16>(p, c, stream);
  else if (c.rows == 32)
    by_share<kHalf, 32>(p, c, stream);
  else if (c.rows == 48)
    by_share<kHalf, 48>(p, c, stream);
  else
    by_share<kHalf, 64>(p, c, stream);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& p, int dtype, hipStream_t stream) {
  if (dtype == MOE_DTYPE_F16)
    by_shape<true>(p, stream);
  else
    by_shape<false>(p, stream);
  return hipGetLastError();
}

}  // namespace moe
