// Host side of the tiled products: tile shape, split of K, workgroups.  Internal header.
#pragma once

#include <algorithm>

#include "moe_gemm_device.h"

namespace moeq4 {

// Tile shapes, tokens x rows.
constexpr int kGemm256x256 = 0, kGemm256x192 = 1, kGemm128x256 = 2, kGemm128x192 = 3, kGemm128x128 = 4, kGemm64x128 = 5, kGemmShapes = 6;

struct GemmPlan {
  int shape, workgroups;
  GemmTiles tiles;
};

// What a tile of each shape takes, in us: a step of 128 bytes of K where a
// compute unit has one workgroup, what each further one adds to it, the tile's
// beginning and end; and how many workgroups a unit holds (0: no such shape).
struct GemmCosts {
  float step[kGemmShapes], more[kGemmShapes], end[kGemmShapes];
  int held[kGemmShapes];
};
// 16-bit products, measured with 256 and 1024 tiles of 8, 32 and 128 steps (the
// mean of the forward's and of dx's, which are up to a tenth apart).
constexpr GemmCosts kGemmCosts16 = {{1.55f, 1.27f, 0.91f, 0.67f, 0.484f, 0.325f}, {}, {4.5f, 3.4f, 4.4f, 3.9f, 2.8f, 2.1f}, {1, 1, 1, 1, 1, 1}};

// For M x N results over `steps` steps: the shape and the split of K with the
// least sum.  Splits fill the card where the tiles do not; their sums go
// through memory (8 bytes a result and split at 5 TB/s) and another launch
// (6 us: 64 x 2832 results of 2056 inputs 12.8 us in 8 parts, 10 in one).
inline GemmPlan gemm_plan(const GemmCosts& costs, int M, int N, int steps) {
  static const int kTok[kGemmShapes] = {256, 256, 128, 128, 128, 64}, kRows[kGemmShapes] = {256, 192, 256, 192, 128, 128};
  GemmPlan best{};
  float least = 0.0f;
  for (int i = 0; i < kGemmShapes; ++i) {
    const int held = costs.held[i];
    if (!held) continue;
    const long tt = (M + kTok[i] - 1) / kTok[i], rt = (N + kRows[i] - 1) / kRows[i], tiles = tt * rt;
    long tried = 0;
    for (int fill = 0; fill <= held; ++fill) {
      const long s = std::max(1L, std::min<long>(std::min(16, steps / 4), 256L * fill / tiles));
      if (s == tried) continue;
      tried = s;
      const int per = (int)((steps + s - 1) / s), splits = (steps + per - 1) / per;
      const long n = tiles * splits, rounds = n / (256L * held), rest = (n - rounds * 256 * held + 255) / 256;
      const auto round = [&](long together) { return together ? (float)per * (costs.step[i] + (float)(together - 1) * costs.more[i]) + costs.end[i] : 0.0f; };
      float us = (float)rounds * round(held) + round(rest);
      if (splits > 1) us += 6.0f + (float)splits * (float)M * (float)N * (8.0f / 5e6f);
      if (least == 0.0f || us < least) {
        least = us;
        best = GemmPlan{i, (int)std::min<long>(n, 256L * held), GemmTiles{(int)tt, (int)rt, splits, per, steps}};
      }
    }
  }
  return best;
}

}  // namespace moeq4
