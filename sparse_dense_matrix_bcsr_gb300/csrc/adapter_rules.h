// adapter_rules.h -- which kernels and tiles a batch with adapters takes, from
// its sizes alone.  Plain C++, so that the rules are tested without a GPU.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace spmm {

constexpr int kAdapterDecodeRows = 64;  // most rows of a tile of the row kernels
constexpr int kGroupRows = 1024;        // longest batch whose rows are sorted by adapter

// Rows of a tile of the row kernels: h and y leave room for two stages or more.
inline int32_t decode_tile_rows(int64_t N, int32_t rank) {
  return N <= 16 ? 16 : N <= 32 || rank > 64 ? 32 : kAdapterDecodeRows;
}

// Whether a batch takes the row kernels (adapter_decode_kernel.cu) or the tiled
// ones.  The row kernels' time grows with the rows, N * (a + b * rank) (every row
// meets its U on the CUDA cores), the tiled ones' with the segments (one more
// stage or more in every tile a segment touches).  Fitted to GPU times through 18944 x
// 3584 (us, rows / tiles): 64 rows of one adapter, rank 16: 13.9 / 15.9, rank 64: 23.6 / 17.1;
// 100 in 10 of rank 128: 70.9 / 44.1; 128 rows, rank 16, in 1 segment: 22.9 / 17.2, in 16: 23.7 /
// 33.9, in 128: 30.0 / 150; 200 in 20 of rank 32: 48.2 / 38.5; 256 rows in 4: 39.0 / 26.8, in 64:
// 41.6 / 69.1; 512 rows of rank 64 in 64: 169 / 135; 1024 rows of rank 16 in 128: 153 / 150; 300
// rows of rank 128 in 300 (3584 x 18944): 282 / 817.  Missed: 64 in 8 of rank 64: 24.6 / 28.4, and
// smaller layers favour the rows more (4096 x 4096, 128 in 16 of rank 64: 24.1 / 38.4).
inline bool rows_path(int64_t N, int32_t rank, int64_t n_seg) {
  return N <= 65535ll * decode_tile_rows(N, rank)  // the launch grid's second dimension
         && N * (rank + 24) < 2300 + 290 * n_seg;
}

// As many segments as the sorted rows can have.
inline int64_t most_groups(int64_t n_adapters, int64_t N, int64_t n_seg) {
  return std::min({N, n_seg, n_adapters});
}

// Whether the gradients sort the batch's rows by adapter first.  A segment less saves
// 0.5 us or more, sorting costs ~6 us and 0.5 ps for each of the m + 2 k columns of a
// row.  Gradients (us) as the rows come / sorted: 432 rows in 432 segments of 4 adapters,
// 3880 x 16048: 849 / 65; 500 in 500 of 64, 4096 x 4096: 347 / 81; 16 in 16 of 4,
// 18944 x 3584: 61 / 43; 1000 in 100 of 20, 4096 x 4096: 89 / 64, in 40: 58 / 64; 300 in 32
// of 8, 18944 x 3584: 84 / 63; 300 in 16 of 8, 3584 x 18944: 71 / 72.
inline bool sorting_pays(int64_t m, int64_t k, int64_t N, int64_t n_seg, int64_t groups) {
  return N <= kGroupRows && (n_seg - groups) * 550 > 6000 + N * (m + 2 * k) / 2000;  // ns
}

// Whether the projection sorts them and takes the tiled path.  Against the row kernels
// (us as they come / sorted): 160 single rows of 2 adapters of rank 128, 12424 x 2904: 122 /
// 37; 421 of 3 of rank 64, 7728 x 3048: 110 / 33; 433 of 25 of rank 24, 12336 x 1056: 90 / 54;
// 256 of 8 of rank 16, 18944 x 3584: 51 / 37, 3584 x 18944: 34 / 43; 128 of 8: 26 / 35; 512 of
// 64: 100 / 89 (missed).  Against tiles as they come: 1000 rows of rank 64 in 200 segments of 4,
// 18944 x 3584: 375 / 77; in 100 of 20, rank 32: 141 / 88, 4096 x 4096: 50 / 42; 412 of rank
// 128 in 109 of 6, 2168 x 624: 159 / 36; 402 in 55 of 9, 584 x 8712: 86 / 47; 392 of rank 128 in 14
// of 8, 6208 x 7408: 62 / 53 (missed); 777 in 40 of 24: 137 / 131 (missed).  The terms are ns.
inline bool sorting_pays_forward(int64_t m, int64_t k, int32_t rank, int64_t N, int64_t n_seg, int64_t groups) {
  if (N > kGroupRows || n_seg <= groups) return false;
  if (rows_path(N, rank, n_seg))
    return 26000 + 20 * N + groups * m * 7 / 100 < N * (rank + 24) * (800 + m * 21 / 100) / 1000;
  return (n_seg - groups) * (300 + 12 * rank) > 14000 + N * (k + m) / 2000;
}

// Tiles of the projection with adapters: 256 rows by one CTA per SM (as without
// adapters) or by two, or 512 rows by one.
constexpr int kMaxTileRows = 512;
enum class LinearTile : int32_t { k256, k256x2, k512 };
inline int linear_tile_rows(LinearTile t) { return t == LinearTile::k512 ? 512 : 256; }
// Blocks after which the tensor cores hand an accumulator over; a tile of 512 rows takes
// no longer block rows.
constexpr int kTurnF32 = 8, kTurnBf16 = 64;

// The tile with adapters.  GPU times (us) of 256 rows by one CTA per SM / by two /
// 512 rows, rank 16 where no other is given:
//   no more tiles than SMs (300 rows, 9 segments, 3584 x 18944):       34.2 / 30.7 / 42.8
//   more segments than row tiles, whose stages hide behind the other
//   CTA's blocks (777 rows of 8192 x 8192 in 40, 75 % zero blocks):     102 /   75 /   88
//   (the same of rank 64):                                              160 /  113 /  118
//   (2048 rows, 18944 x 3584, in 128):                                  258 /  159 /  249
//   fewer, short block rows, many tiles (65536 rows, 18944 x 3584, 9): 1531 / 1467 / 1328
//   (the same of rank 48):                                             2008 / 1870 / 1642
//   (16384 rows of rank 16):                                                /  377 /  378
//   (16384 rows of rank 64):                                            582 /  470 /  524
//   few tiles (2048 rows in 4):                                        87.5 / 68.1 / 75.2
//   fewer, block rows of 16 blocks or more (16384 rows, 3584 x 18944):  392 /  431 /  405
// (bf16 outputs; 512-row tiles need a longest block row of one turn, and fp16 inputs have
// none, see the kernel.)
// longest: blocks of the longest block row.
inline LinearTile linear_adapters_tile(int64_t n_block_rows, int64_t n_blocks, int64_t longest, int64_t N, int64_t n_seg,
                                       int32_t rank, bool in_bf16, bool out_bf16, int num_sms) {
  const int64_t row_tiles = (N + 255) / 256;
  if (n_block_rows * row_tiles <= num_sms) return LinearTile::k256;
  if (n_seg >= row_tiles) return LinearTile::k256x2;
  if (n_blocks >= 16 * n_block_rows) return LinearTile::k256;
  if (n_block_rows * ((N + 511) / 512) < 8ll * num_sms) return LinearTile::k256x2;
  if (rank > 16 && N < 32768) return LinearTile::k256x2;
  return in_bf16 && longest <= (out_bf16 ? kTurnBf16 : kTurnF32) ? LinearTile::k512 : LinearTile::k256x2;
}

}  // namespace spmm
