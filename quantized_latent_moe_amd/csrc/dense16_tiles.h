// Choice of the tile of a 16-bit product: host code without any GPU header, so
// that it can be compiled and looked at by itself.
#pragma once

#include <stdint.h>

namespace latmoe {

// Large tiles move fewer bytes for a product, small ones fill the chip with few
// rows and leave less of its last pass idle.  The time of a variant is
// estimated from what a K step of 64 was measured to take (us): on every CU at
// once, each with all the tiles that it holds, and with one tile a CU on part of
// the chip; and from what a tile costs beside its steps.
struct Dense16Tile {
  int rows, tokens;  // weight rows (gated: half of them gate rows) and tokens
  int per_cu;        // tiles a CU holds (LDS)
  float full, alone, tile;
  int64_t count(int64_t T, int64_t weight_rows) const {
    return (T + tokens - 1) / tokens * ((weight_rows + rows - 1) / rows);
  }
};

constexpr Dense16Tile kDense16Tiles[] = {
    // 21000 x 4096 by 4096 | 5268 x 4096 by 1024 | 517 x 2056 by 4100 | 512 x 4096 by 4096, bf16 (us):
    {256, 256, 1, 1.47f, 1.07f, 4.f},  // 593 | 74 | 52 | 71
    {256, 192, 1, 1.24f, 0.88f, 4.f},  // 602 | 61 | 45 | 59
    {256, 128, 1, 0.84f, 0.64f, 4.f},  // 637 | 49 | 33 | 43
    {128, 128, 1, 0.52f, 0.39f, 3.f},  // 777 | 60 | 24 | 28
    {128, 64, 2, 0.62f, 0.29f, 4.f},   // 920 | 56 | 30 | 23
    {64, 64, 2, 0.33f, 0.19f, 3.f},    // 1024 | 70 | 29 | 27
    // K dealt to four slices of waves: 512 x 4096 by 1024 takes 11.6 us (64 x 64: 15)
    {64, 32, 1, 0.145f, 0.12f, 3.f},   // 1641 | 114 | 40 | 43
};
constexpr int kDense16Variants = 7;
// Short K, where a tile's beginning and end are most of it and the estimate
// knows neither: what it picks against the seven tiles in their order (us).
//   12994 x 64 by 2984  36 | 36 38 36 45 37 48 233    5268 x 64 by 4096  16 | 17 16 18 23 20 26 128
//   12994 x 264 by 2984 50 | 50 53 51 61 57 73 267    5268 x 264 by 4096 25 | 27 25 27 36 31 42 146
//   5268 x 264 by 1024  10 | 13 13 10 13 10 13 39     517 x 264 by 4100 9.1 | 23 18 14 9.1 7.9 8.8 20
// Few tokens with short K could save a microsecond; the rest is the best there is.

// Estimated time of a launch; steps: of K; weight_rows: gated ones counted twice.
inline float dense16_time(int variant, int64_t T, int64_t weight_rows, int steps, int num_cus) {
  const Dense16Tile& v = kDense16Tiles[variant];
  const int64_t tiles = v.count(T, weight_rows), slots = (int64_t)num_cus * v.per_cu;
  const int64_t passes = tiles / slots, rest = tiles % slots;
  float t = (float)passes * (v.full * (float)steps + v.tile);
  if (rest) t += (rest <= num_cus ? v.alone : v.full) * (float)steps + v.tile;
  return t;
}
inline int dense16_pick_tile(int64_t T, int64_t weight_rows, int steps, int num_cus) {
  int best = 0;
  for (int i = 1; i < kDense16Variants; ++i)
    if (dense16_time(i, T, weight_rows, steps, num_cus) < dense16_time(best, T, weight_rows, steps, num_cus)) best = i;
  return best;
}

// The first launch of a product: a tile, and for how many tokens.  Where large
// tiles would leave most CUs idle in their last pass, they take the whole
// passes, and the tokens that remain come in a launch of their own with the
// tile that suits them (21000 x 4096 by 4096: five passes of 256 x 256 and 520
// tokens in tiles of 128 x 128).
struct Dense16Launch {
  int variant;
  int64_t tokens;
};
inline Dense16Launch dense16_plan(int64_t T, int64_t weight_rows, int steps, int num_cus) {
  // What a second launch costs, so that it is made where it gains for certain
  // (us with it | without): 21000 x 4096 by 4096 566 | 605, 5268 x 4096 by 16384
  // 543 | 569, but 5268 x 4096 by 4096 149 | 143.
  constexpr float kLaunch = 8.f;
  Dense16Launch plan{dense16_pick_tile(T, weight_rows, steps, num_cus), T};
  float least = dense16_time(plan.variant, T, weight_rows, steps, num_cus);
  for (int i = 0; i < kDense16Variants; ++i) {
    const Dense16Tile& v = kDense16Tiles[i];
    if (v.per_cu != 1) continue;
    const int64_t columns = v.count(1, weight_rows), passes = v.count(T, weight_rows) / num_cus;
    const int64_t tokens = passes * num_cus / columns * v.tokens;
    if (tokens <= 0 || tokens >= T) continue;
    const float t = (float)passes * (v.full * (float)steps + v.tile) + kLaunch +
                    dense16_time(dense16_pick_tile(T - tokens, weight_rows, steps, num_cus), T - tokens, weight_rows,
                                 steps, num_cus);
    if (t < least) {
      least = t;
      plan = Dense16Launch{i, tokens};
    }
  }
  return plan;
}

// The kernel that streams the weights takes 4, 8 or 16 of them to a workgroup
// (gated at least 8) and 4, 8 or 16 tokens.  It beats the tiles as long as each
// workgroup has a CU (us here | in tiles, K = 4096): 16 x 4096 6.9 | 13, 64 x 1024 6.1 | 10.1, 512 x 128 6.8 | 10.2; with two
// on a CU no longer: 128 x 1024 10.4 | 10.1, 64 x 4096 22 | 12.5.
inline bool dense16_small(int64_t T, int64_t weight_rows, int num_cus) {
  return T <= 16 || (T + 15) / 16 * ((weight_rows + 15) / 16) <= num_cus;
}
// As few rows as leave a workgroup for each CU.
inline int dense16_small_rows(int64_t T, int64_t weight_rows, int num_cus) {
  const int64_t groups = (T + 15) / 16;
  if (weight_rows * groups <= 4 * (int64_t)num_cus) return 4;
  if (weight_rows * groups <= 8 * (int64_t)num_cus || T <= 8) return 8;
  return 16;
}

}  // namespace latmoe
