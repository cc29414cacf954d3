// Which kernel shape serves a product with packed 4-bit weights: plain host code,
// so that the tests' sizes can be held to reach every one.
#pragma once

#include <stdint.h>

namespace moe {

struct MatvecShape {
  int chunk, rows, share;   // elements of a step, rows of x, waves that share x (template arguments of the kernel)
  int splits;               // of the summed index
  int flush;                // products of 32 elements after which a sum is scaled (a template argument, too)
};

// Few workgroups share the summed index among more waves, many share x among more.
// Times in us (bf16, groups of 128), N x K, rows, and share x splits:
//   rows <= 4: 512 x 8192, 1 row: 1x8 6.5, 1x4 7.2, 1x2 11.1; 4096 x 2048: 1x4 4.2, 1x8 4.3, 1x2 5.0;
//     32 routes of 1536 x 2048: 1x2 17.0, 1x4 20.1; 32768 x 2048: 1x2 11.0, 1x4 12.0, x 768: 6.5, 9.2;
//     768 to 1024 tiles: 12288 x 768: 1x2 4.8, 1x4 5.2, 14336 x 768: 4.9, 5.9, 16384 x 512: 4.2, 5.3, x 1024: 5.8, 6.1,
//     8 routes of 2048 x 768: 5.3, 6.2; but 12288 x 2048: 7.4, 6.7, 16384 x 1536: 6.9, 6.6, x 2560: 8.6, 8.4;
//     16384 x 8192: chunks of 256, 1x2 18.9, of 128: 1x4 21.0, 1x2 22.3
//   16 rows: 4096 x 2048: 1x4 5.3, 2x4 6.2, 4x2 7.7; 8192 x 2048: 2x2 6.9, 1x4 7.5, 4x2 8.1;
//     8192 x 8192: 2x4 14.1, 2x2 15.2, 1x4 15.7; 16384 x 8192: 4x2 21.1, 2x4 29.9, 1x4 33.7
//   64 rows: 512 x 8192: 2x4 30, 2x2 34, 4x2 43; 8192 x 2048: 2x2 15.5, 2x4 18.1, 4x2 20.8;
//     16384 x 8192: 4x2 54.5, 4x1 59.9, 2x2 61.5; 200 rows, 8192 x 2048: 4x1 28.7, 2x2 39.3, 4x2 41.7;
//     37 rows, 5001 x 4064, groups of 32: 2x4 16.7, 2x2 18.2, 4x2 24.3
inline MatvecShape matvec_shape(bool routed, int64_t rows, int N, int K, int group) {
  const int flush = group % 128 == 0 ? 4 : group % 64 == 0 ? 2 : 1;
  const int64_t tiles = (int64_t(N) + 15) / 16 * (routed ? rows : (rows + 63) / 64);
  if (routed || rows <= 4) {
    if (tiles >= 1024 && K >= 4096) return {256, 4, 1, 2, flush};
    const bool filled = tiles > 1024 || (tiles >= 768 && K <= 1024);   // two waves a workgroup fill the chip
    return {128, 4, 1, filled ? 2 : tiles <= 256 && K >= 4096 ? 8 : 4, flush};
  }
  if (rows <= 16) {
    if (tiles < 512) return {128, 16, 1, 4, flush};
    if (tiles < 1024) return {128, 16, 2, K >= 8192 ? 4 : 2, flush};
    return {128, 16, 4, 2, flush};
  }
  const int held = rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  if (tiles < 1024) return {128, held, 2, K > 2048 ? 4 : 2, flush};
  return {128, held, 4, tiles < 2048 ? 2 : 1, flush};
}

}  // namespace moe
