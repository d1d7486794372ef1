// Which kernel a call of moe_mx_linear takes, from its sizes, the format of its
// rows and whether their products are wanted exactly. Plain C++, so that it can be asked
// without a GPU.
#pragma once

#include <cstdint>

namespace moe {
namespace mxl {

enum class Kernel {
  // k_skinny: waves that share K, fragments of 16 columns, of 16 rows
  SKINNY_8_1_1_LITE, SKINNY_4_1_1_LITE, SKINNY_8_1_1, SKINNY_4_2_1, SKINNY_4_1_2,
  SKINNY_X_2_2,  // two waves for MXFP8, four for MXFP4
  // k_tile
  TILE_LARGEST,  // 128 x 256 MXFP8, 256 x 256 MXFP4
  TILE_128_128, TILE_64_128, TILE_64_64
};

// f8: MXFP8 rows. exact: with two instructions a product (MXFP8 only).
constexpr Kernel choose(bool f8, bool exact, int M, int N, int K) {
  auto tiles = [&](int bm, int bn) { return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  // Few rows: k_skinny; four waves, eight where that gives a compute unit at most
  // one workgroup. us at M = 1: 2048 x 7168 (N x K) 5.6 with eight, 6.3 with four, 7168 x 2048 6.2 and 5.1. M = 16:
  // 14336 x 4096 9.9 with 32 columns to a workgroup, 10.6 with 16; 2880 x 2880 6.8 and 5.2.
  const bool few = N <= 16 * 256;
  if (M <= (f8 ? 4 : 8)) return few ? Kernel::SKINNY_8_1_1_LITE : Kernel::SKINNY_4_1_1_LITE;
  if (M <= 16) return few ? Kernel::SKINNY_8_1_1 : Kernel::SKINNY_4_2_1;
  // More of them while such workgroups of 32 x 16 find place on the chip at once (88 KiB of LDS
  // for MXFP8, 56 for MXFP4): 32 x 4096 x 14336 MXFP8 15 where 32 columns to a workgroup take 17, 128 x 1024 x 7168 9.4
  // where tiles of 64 x 64 take 13.5; MXFP4 7.9 and 11.1, with 512 workgroups 64 x 4096 x 14336 19.5 and 24,
  // 128 x 2048 x 7168 10.9 and 11.2. MXFP8 with 512: 128 x 2048 x 7168 17 and 13.6.
  if (tiles(32, 16) <= (f8 ? 256 : 512)) return Kernel::SKINNY_4_1_2;
  // 24 x 7168 x 7168 MXFP8 12.3 where 16 columns take 17.7; 64 x 7168 x 7168 17 where tiles of 64 x 64 take 21,
  // but 33 x 7168 x 2048 8.3 and 6.3, 64 x 14336 x 4096 21 and 14; MXFP4 33 x 6000 x 6016 14.8 and 13.1.
  if (M <= 32 || (f8 && M <= 64 && K > 4096 && tiles(64, 64) <= 128)) return Kernel::SKINNY_X_2_2;
  // The largest tile that still gives most compute units one. Measured at 160-256
  // tiles (us, the tile taken against the next smaller): 300 x 7168 x 7168 MXFP8 29
  // against 33, 1024 x 4096 x 4096 MXFP8 21 against 22, MXFP4 16 against 21; below: 512 x 4096 x 4096
  // with 128 tiles of 128 x 128 17 against 13, 128 x 7168 x 7168 MXFP4 with 112 of 64 x 128 16 against 13.
  // The largest has no registers for an exact product's split codes.
  if (tiles(f8 ? 128 : 256, 256) >= 192 && !exact) return Kernel::TILE_LARGEST;
  if (tiles(128, 128) >= 160) return Kernel::TILE_128_128;
  if (tiles(64, 128) >= 160) return Kernel::TILE_64_128;
  return Kernel::TILE_64_64;
}

}  // namespace mxl
}  // namespace moe
