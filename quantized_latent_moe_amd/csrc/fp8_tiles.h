// Choice of the tile of an e4m3 product: host code without any GPU header, so
// that it can be compiled and looked at by itself.
#pragma once

#include <stdint.h>

namespace latmoe {

// Gated blocks of up to this many values of H may take the way through fp32 H
// in memory: with more, tiles of 128 columns and 64 tokens are on half of the
// CUs and their rounding costs no launch.
constexpr int64_t kFp8H32 = (int64_t)1 << 20;

// Large tiles move fewer bytes through LDS for a product, small ones fill the
// chip with few rows and leave less of its last pass idle.  The time of a
// variant is estimated from what one CU was measured to take for a K step while
// it holds 1, 2, ... of the variant's tiles (us; the launch has 256 CUs busy),
// for what a tile costs beside its steps, and for the start: passes with every
// CU full, then one with the tiles that remain.
struct Fp8Tile {
  int rows, tokens;  // weight rows (gated: half of them gate rows) and tokens
  bool gated;
  int per_cu;        // tiles a CU holds (LDS)
  float start, tile, step[2];
  constexpr int cols() const { return gated ? rows / 2 : rows; }
  // The workgroups of large tiles, of which a CU holds one, stay and take one
  // tile after the other: the next tile's loads run while the last one's
  // results are stored.  21000 tokens, bf16: 4096 x 1024 weights 119 us (142 with
  // a workgroup a tile, timed in turn), 8192 x 2048 370 (434), 4096 x 4096 336
  // (353); exact products to fp32 655 (682).  Smaller tiles overlap with the CU's
  // other workgroup, and gain nothing.
  constexpr bool stays() const { return rows * tokens >= 128 * 128; }
  int64_t count(int64_t T, int N) const { return (T + tokens - 1) / tokens * (((int64_t)N + cols() - 1) / cols()); }
};

// Projections with e4m3 and with exact products; gated pairs likewise.
enum Fp8Product : int { kFp8Dense = 0, kFp8DenseExact = 1, kFp8GatedPair = 2, kFp8GatedPairExact = 3 };

constexpr Fp8Tile kFp8Tiles[4][4] = {
    {{256, 128, false, 1, 3.f, 3.f, {0.86f}},
     {128, 128, false, 1, 3.f, 2.f, {0.46f}},
     {128, 64, false, 2, 0.f, 4.f, {0.32f, 0.65f}},
     {64, 64, false, 2, 0.f, 3.f, {0.20f, 0.39f}}},
    {{128, 192, false, 1, 5.f, 2.f, {1.40f}},
     {128, 128, false, 1, 4.f, 2.f, {0.92f}},
     {64, 64, false, 2, 0.f, 4.f, {0.35f, 0.57f}}},
    {{256, 128, true, 1, 4.f, 3.f, {0.86f}},
     {256, 64, true, 1, 3.f, 2.f, {0.50f}},
     // with fp32 H and its rounding in a launch of its own
     {128, 64, true, 2, 3.f, 4.f, {0.32f, 0.65f}},
     {64, 64, true, 2, 3.f, 3.f, {0.20f, 0.39f}}},
    // 512 tokens of C = 4096, F = 2048 take 37.4 us for the whole block (27.5
    // with e4m3 products), 5268 with F = 8192 913 us (553)
    {{256, 64, true, 1, 4.f, 3.f, {0.95f}},
     // with fp32 H
     {64, 64, true, 2, 3.f, 4.f, {0.35f, 0.57f}}}};

// Variants that can compute a product [T] x [N] (gated: N columns of H); those
// of a gated pair that round H themselves come first.  128 columns of H are one
// scale's, so these fill the chip only where T F is large: 65 tokens of
// C = 4096, F = 2048 (16 tiles of 128 columns x 64 tokens) took 24.0 us for the
// whole block, and take 16.9 us with tiles of 32 columns, fp32 H and a launch
// that rounds it.
inline int fp8_tile_variants(int product, int64_t T, int N) {
  const bool h32 = T * N <= kFp8H32;
  switch (product) {
    case kFp8Dense: return 4;
    case kFp8DenseExact: return 3;
    case kFp8GatedPair: return h32 ? 4 : 2;
    default: return h32 ? 2 : 1;
  }
}

// The variant with the least estimated time; nb: steps of K.
inline int fp8_pick_tile(int product, int64_t T, int N, int nb, int num_cus) {
  const Fp8Tile* v = kFp8Tiles[product];
  const int count = fp8_tile_variants(product, T, N);
  int best = 0;
  float least = 0.f;
  for (int i = 0; i < count; ++i) {
    const int64_t tiles = v[i].count(T, N);
    const int64_t slots = (int64_t)num_cus * v[i].per_cu, passes = tiles / slots, rest = tiles % slots;
    float t = v[i].start + (float)passes * (v[i].step[v[i].per_cu - 1] * (float)nb + v[i].tile);
    if (rest) t += v[i].step[(rest + num_cus - 1) / num_cus - 1] * (float)nb + v[i].tile;
    if (i == 0 || t < least) {
      best = i;
      least = t;
    }
  }
  return best;
}

}  // namespace latmoe
