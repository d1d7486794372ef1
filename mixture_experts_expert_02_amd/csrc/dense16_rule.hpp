// Which tiles and how many K ranges a dense 16-bit product takes, from its kind and sizes. Plain C++, so that it can be
// asked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

namespace moe {
namespace d16 {

// GATED: gate and up products of the same rows; DX: two products added; DW: two products of the same columns;
// LORA: one product, with adapters.
enum Mode { GATED, DX, DW, LORA };

struct Plan {
  int bm;        // rows of a tile: 256 or 128 (256 columns; GATED: 128 gate and 128 up columns)
  int splits;    // K ranges, each in workgroups of their own, joined by a second kernel
  size_t part;   // bytes of their partial results
};

// M rows and N columns out, K values of one product. The plan of least time by this account (us), fitted to the
// kernels alone: a workgroup has a compute unit to itself, so tiles go in rounds of 256; a stage of 64 K values takes
// `idle` where few units work and `busy` where all do (the clock gives way), a round 10 us around its stages (7 with
// 128 rows), a join its launch and the partial results written and read.
//   1024 x 2048 x 7168 gated (M, N, K): 256 rows 115, in two ranges 78 with the join, 128 rows 93, in two ranges 69
//   77 x 2880 x 2880 DX: 128 rows 71, in 2, 4 and 8 ranges 43, 27 and 20; 256 rows 102, 59, 36 and 25
//   1023 x 7168 x 2048 DX: 128 rows 65, in two ranges 87; 256 rows 87 and 73
//   2880 x 2880 x 2048 DW: 256 rows 99, 128 rows 96; 7168 x 2048 x 1023 DW: 65 and 81
inline Plan plan_of(int mode, int64_t M, int64_t N, int64_t K) {
  constexpr double kIdle[2][4] = {{0.88, 0.90, 0.92, 0.86}, {0.50, 0.71, 0.54, 0.51}};
  constexpr double kBusy[2][4] = {{1.45, 1.71, 1.66, 1.47}, {0.81, 1.06, 0.92, 0.81}};
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int planes = mode == GATED || mode == DW ? 2 : 1, tn = mode == GATED ? 128 : 256;
  const int64_t stages = up(K, 64) * (mode == DX ? 2 : 1);
  Plan best{256, 1, 0};
  double least = 1e30;
  for (int small = 0; small < 2; ++small) {
    const int64_t tiles = up(M, small ? 128 : 256) * up(N, tn) * (mode == DW ? 2 : 1);
    for (int s = 1; s <= 16 && (s == 1 || s * 4 <= stages); ++s) {
      const int64_t rounds = up(tiles * s, 256);
      const double full = (double)(tiles * s) / (double)(rounds * 256), bytes = s > 1 ? (double)s * planes * M * N * 4 : 0;
      if (bytes > 256e6) break;
      const double us = rounds * (up(stages, s) * (kIdle[small][mode] + (kBusy[small][mode] - kIdle[small][mode]) * full) + (small ? 7 : 10)) +
                        (s > 1 ? 4 + bytes / 3.5e6 : 0);
      if (us < least) {
        least = us;
        best = {small ? 128 : 256, s, s > 1 ? ((size_t)s * planes * M * (size_t)((N + 7) & ~7) * 4 + 255) & ~(size_t)255 : 0};
      }
    }
  }
  return best;
}

// K of a product whose dg or du is two parts: whole stages of each.
inline int64_t parts_k(int64_t K) { return (K + 63) / 64 * 64 * 2; }

// The first product of adapters: 16-row fragments of a workgroup, and K ranges: at most one workgroup to a compute unit,
// at least 16 steps of 32 to a range (us of the kernel: 1000 rows of 4096, rank 24, 64 adapters 31, 17, 8.7, 12.5 and 17
// with 1, 2, 4, 8 and 16 ranges; 256 of 7168, rank 64, 34, 19, 11.6, 7.6 and 6.0; 8192 of 2048 18.6, 21 and 28 with 1, 2
// and 4). Two fragments share the factor's loads (us of a call without a projection, 512 columns, rank 64, one fragment second: 2049 of
// 4096 45.3 and 61.3, 8192 of 2048 54.6 and 60.4; rank 16 39.8 and 39.5). Both limits are on the cautious side: 1100 to 2048 rows of 4096 would
// gain 4, and rank 128 with two 2100 of 4096 101 -> 71, 8192 of 2048 95 -> 82.
constexpr int kMaxRanges = 16;
inline int shrink_frags(int64_t M, int R) { return R <= 64 && M > 2048 ? 2 : 1; }
inline int shrink_ranges(int64_t M, int K, int R) {
  const int64_t groups = (M + 16 * shrink_frags(M, R) - 1) / (16 * shrink_frags(M, R));
  const int64_t by_units = 256 / groups, by_k = (K + 31) / 32 / 16, r = by_units < by_k ? by_units : by_k;
  return r < 1 ? 1 : r > kMaxRanges ? kMaxRanges : (int)r;
}

// 16-row fragments of a workgroup of k_lora_expand; with one it joins the first product's K ranges itself. us of a call, rank 64, this
// and the other number: one 512 x 2048 x 7168 31.8 and 31.9, 1000 x 4096 x 2048 29.5 and 36.8, but 2040 x 2048 x 7168 75.6 and 61.7; four 2048 x 2048 x
// 7168 61.6 and 75.5, 8192 x 2048 x 7168 173 and 197, 2100 x 4096 x 2048 50.2 and 46.8.
inline int expand_frags(int64_t M) { return M >= 2048 ? 4 : 1; }

}  // namespace d16
}  // namespace moe
