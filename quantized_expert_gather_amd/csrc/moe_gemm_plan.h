// Host side of the tiled products: tile shape and split of K.  Internal header.
#pragma once

#include <algorithm>

namespace moeq4 {

constexpr int kGemm256x256 = 0, kGemm128x128 = 1, kGemm64x128 = 2;

struct GemmPlan {
  int shape, tok_tiles, row_tiles, splits, steps_per;
};

// For M x N results over `steps` steps, from shape `first` on.
inline GemmPlan gemm_plan(int M, int N, int steps, int first = 0) {
  static const int kTok[3] = {256, 128, 64}, kRows[3] = {256, 128, 128};
  static const float kStep[3] = {1.1f, 0.42f, 0.3f};  // us of a step, workgroups that run at once
  static const int kAtOnce[3] = {256, 512, 768};
  GemmPlan best{};
  float least = 0.0f;
  for (int i = first; i < 3; ++i) {
    const long tt = (M + kTok[i] - 1) / kTok[i], rt = (N + kRows[i] - 1) / kRows[i], tiles = tt * rt;
    int tried = 0;
    for (int fill = 0; fill <= kAtOnce[i]; fill += 256) {
      const int s = (int)std::max(1L, std::min<long>(std::min(16, steps / 4), fill / tiles));
      if (s == tried) continue;
      tried = s;
      const int per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
      const long n = tiles * splits, rounds = (n + kAtOnce[i] - 1) / kAtOnce[i];
      float us = (float)rounds * ((float)per * kStep[i] + 2.0f);
      if (splits > 1) us += 2.5f + (float)splits * (float)M * (float)N * (8.0f / 6e6f);
      if (least == 0.0f || us < least) {
        least = us;
        best = GemmPlan{i, (int)tt, (int)rt, splits, per};
      }
    }
  }
  return best;
}

}  // namespace moeq4
