// Host side of the tiled products: tile shape, split of K, workgroups.  Internal header.
#pragma once

#include <algorithm>

#include "moe_gemm_device.h"

namespace moeq4 {

constexpr int kGemm256x256 = 0, kGemm256x192 = 1, kGemm128x128 = 2, kGemm64x128 = 3;

struct GemmPlan {
  int shape, workgroups;
  GemmTiles tiles;
};

// For M x N results over `steps` steps, with the shapes of `mask` (bits by number).
inline GemmPlan gemm_plan(int M, int N, int steps, int mask) {
  static const int kTok[4] = {256, 256, 128, 64}, kRows[4] = {256, 192, 128, 128};
  static const float kStep[4] = {1.3f, 1.05f, 0.8f, 0.6f};  // us of a step, workgroups that run at once
  static const int kAtOnce[4] = {256, 256, 512, 768};
  GemmPlan best{};
  float least = 0.0f;
  for (int i = 0; i < 4; ++i) {
    if (!(mask >> i & 1)) continue;
    const long tt = (M + kTok[i] - 1) / kTok[i], rt = (N + kRows[i] - 1) / kRows[i], tiles = tt * rt;
    int tried = 0;
    for (int fill = 0; fill <= kAtOnce[i]; fill += 256) {
      const int s = (int)std::max(1L, std::min<long>(std::min(16, steps / 4), fill / tiles));
      if (s == tried) continue;
      tried = s;
      const int per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
      const long n = tiles * splits, rounds = (n + kAtOnce[i] - 1) / kAtOnce[i];
      float us = (float)rounds * ((float)per * kStep[i] + 3.0f);
      if (splits > 1) us += 2.5f + (float)splits * (float)M * (float)N * (8.0f / 6e6f);
      if (least == 0.0f || us < least) {
        least = us;
        best = GemmPlan{i, (int)std::min<long>(n, kAtOnce[i]), GemmTiles{(int)tt, (int)rt, splits, per, steps}};
      }
    }
  }
  return best;
}

}  // namespace moeq4
