// Host side of the dense 4-bit product: plans, workspace layout and launches.
// Each format's kernels are instantiated in a source of their own
// (moe_linear_inst_*.hip).  Internal header.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "moe_linear_rows.h"
#include "moe_linear_tiles.h"
#include "moe_q4.h"

namespace moeq4 {

// Enqueues a checked call; returns a MOE_Q4_* status.
template <int FMT>
int linear_launch(bool f16, const LinearArgs& a, unsigned char* workspace, hipStream_t stream);

// Whether the tiles take a call.  The rows' kernel takes 16 tokens at a time,
// reading all weights for each 16, but needs neither a preparation (affine)
// nor splits of K to fill the card, so it keeps small products of any number
// of tokens (us, rows against tiles: affine4_g64 128 x 256 x 4096 7.4 and
// 15.7, 32 x 4096 x 4096 13.8 and 16.2, 32 x 8192 x 4096 19.0 and 18.4, 128 x
// 4096 x 4096 47 and 23; mxfp4 64 x 1024 x 4096 6.3 and 10.1, 64 x 8192 x 512
// 5.7 and 5.1, 32 x 4096 x 4096 12.0 and 10.3).
inline bool linear_by_tiles(int fmt, int L, int N, int K) {
  if (L <= 16) return false;
  const bool affine = lin_affine(fmt);
  const long read = (long)((L + 15) / 16) * N * K;  // codes of all passes
  return K < (affine ? kLinStep : 1024) || read > (affine ? 1L << 25 : 1L << 24);
}

// Tile shape and split of K.  A compute unit holds two workgroups, so they
// run in rounds of 512, and what a round takes per 1024 inputs was measured
// (us; 4096 x 4096 weights and other shapes of exactly 256 and 512 workgroups,
// the formats' mean): wide tiles do more per byte of LDS, narrow ones leave
// fewer compute units idle in the last round.  Splits add their partial sums'
// way through memory and a launch.  The plan is the one with the least sum;
// against the widest tiles that give 256 workgroups, mxfp4 1536 x 4096 x 4096
// goes from 84 to 60 us and 16384 outputs of 24 tokens from 24 to 17.
struct TilesPlan {
  int mt, nt, row_tiles, tok_tiles, splits, steps_per;
};
inline TilesPlan tiles_plan(int L, int N, int K) {
  static const float kFull[3][3] = {{6.0f, 9.5f, 13.5f}, {7.5f, 12.0f, 16.5f}, {13.0f, 18.0f, 26.0f}};
  static const float kHalf[3][3] = {{5.5f, 7.5f, 9.8f}, {6.5f, 8.7f, 11.5f}, {9.5f, 12.5f, 17.0f}};
  const int steps = (K + kLinStep - 1) / kLinStep;
  const float out_us = (float)L * (float)N * (8.0f / 6e6f);  // a split's sums written and read
  TilesPlan best{};
  float least = 0.0f;
  for (int m = 0; m < 3; ++m) {
    const int mt = 2 << m, tok_tiles = (L + 16 * mt - 1) / (16 * mt);
    if (m && 8 * mt >= (L + 15) / 16 * 16) break;  // half the tile would be empty
    for (int nt = 3; nt >= 1; --nt) {
      const int row_tiles = (N + 64 * nt - 1) / (64 * nt);
      const long tiles = (long)row_tiles * tok_tiles;
      int tried = 0;
      for (int fill = 0; fill <= 512; fill += 256) {
        const int s = (int)std::max(1L, std::min<long>(std::min(16, steps / 4), fill / tiles));
        if (s == tried) continue;
        tried = s;
        const int per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
        const long n = tiles * splits, rounds = n / 512, rest = n % 512;
        const float k = (float)per / 8.0f, end = 0.6f * (float)(mt * nt);
        float us = (float)rounds * (k * kFull[m][nt - 1] + end);
        if (rest) us += k * (rest > 256 ? kFull : kHalf)[m][nt - 1] + end;
        if (splits > 1) us += 2.5f + (float)splits * out_us;
        if (best.mt == 0 || us < least) {
          best = TilesPlan{mt, nt, row_tiles, tok_tiles, splits, per};
          least = us;
        }
      }
    }
  }
  return best;
}

struct TilesWorkspace {
  size_t xq, xsum, tsum, xexp, sh, wexp, part, total;
};
inline size_t lin_round256(size_t v) { return (v + 255) & ~size_t(255); }
inline TilesWorkspace tiles_layout(int fmt, int L, int N, int K) {
  TilesWorkspace w{};
  const TilesPlan p = tiles_plan(L, N, K);
  const size_t G = K / lin_group(fmt), Gp = (G + 31) / 32 * 32;
  const bool affine = lin_affine(fmt);
  size_t off = 0;
  w.xq = off;   off = lin_round256(off + (affine ? (size_t)p.tok_tiles * p.mt * 16 * ((K + kLinStep - 1) / kLinStep * kLinStep) * 2 : 0));
  w.xsum = off; off = lin_round256(off + (affine ? 3 * (size_t)L * Gp * 2 : 0));
  w.tsum = off; off = lin_round256(off + (affine ? 2 * (size_t)N * Gp * 2 : 0));
  w.xexp = off; off = lin_round256(off + (affine ? (size_t)L * 4 : 0));
  w.sh = off;   off = lin_round256(off + (affine ? (size_t)N * Gp * 2 : 0));
  w.wexp = off; off = lin_round256(off + (affine || fmt == kLinMxfp4 ? (size_t)N * 4 : 0));
  w.part = off; off = lin_round256(off + (p.splits > 1 ? (size_t)p.splits * L * N * 4 : 0));
  w.total = off;
  return w;
}

// Whether the scale arrays can be read by words.
inline bool linear_words(const LinearArgs& a) { return (uintptr_t)a.s % 4 == 0 && (uintptr_t)a.b % 4 == 0; }

// Bytes of partial sums of a call with few tokens, whatever its x.
inline size_t rows_workspace(int fmt, int L, int N, int K) {
  if (K < kLinStep) return 0;
  const int s = std::max(rows_plan(fmt, false, N, K, true).splits, rows_plan(fmt, true, N, K, true).splits);
  return s > 1 ? lin_round256((size_t)s * L * N * 4) : 0;
}

#ifdef MOE_LINEAR_INST
inline void launch_linear_join(const LinearArgs& l, const float* part, int splits, hipStream_t stream) {
  const size_t all = (size_t)l.L * l.N;
  hipLaunchKernelGGL(k_linear_join, dim3((unsigned)std::min<size_t>((all + 255) / 256, 4096)), dim3(256), 0, stream, part,
                     l.bias, l.out, l.ldo, l.L, l.N, splits, l.out_dtype);
}

template <int FMT, bool F16, int MT>
void launch_tiles_mt(const TilesArgs& a, const TilesPlan& p, hipStream_t stream) {
  const dim3 grid(p.row_tiles * p.tok_tiles, p.splits), block(256);
  switch (p.nt) {
    case 3: hipLaunchKernelGGL((k_linear_tiles<FMT, F16, MT, 3>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_linear_tiles<FMT, F16, MT, 2>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((k_linear_tiles<FMT, F16, MT, 1>), grid, block, 0, stream, a); break;
  }
}

template <int FMT, bool F16>
int launch_tiles(const LinearArgs& l, unsigned char* ws, hipStream_t stream) {
  const TilesPlan p = tiles_plan(l.L, l.N, l.K);
  const TilesWorkspace lay = tiles_layout(FMT, l.L, l.N, l.K);
  TilesArgs a{};
  a.x = a.xraw = l.x; a.w = l.w; a.s = l.s; a.b = l.b;
  a.bias = l.bias; a.out = l.out;
  a.ldx = l.ldx; a.ldo = l.ldo;
  a.L = l.L; a.N = l.N; a.K = l.K;
  a.G = l.K / lin_group(FMT);
  a.Gp = (a.G + 31) / 32 * 32;
  a.out_dtype = l.out_dtype;
  a.splits = p.splits; a.steps_per = p.steps_per;
  a.stagger = std::max(1, p.steps_per / p.tok_tiles);
  a.row_tiles = p.row_tiles; a.tok_tiles = p.tok_tiles;
  a.part = reinterpret_cast<float*>(ws + lay.part);
  constexpr bool kRowsScaled = lin_affine(FMT) || (FMT == kLinMxfp4 && F16);
  if constexpr (kRowsScaled) {
    a.wexp = reinterpret_cast<int32_t*>(ws + lay.wexp);
    PrepareArgs q{};
    q.x = l.x; q.w = l.w; q.s = l.s; q.b = l.b;
    q.wexp = reinterpret_cast<int32_t*>(ws + lay.wexp);
    q.ldx = l.ldx;
    q.L = l.L; q.N = l.N; q.K = l.K; q.G = a.G; q.Gp = a.Gp;
    q.row_lanes = 4;
    // (a launch holds fewer than 2^32 threads)
    while (q.row_lanes < 64 && 8 * q.row_lanes < a.G && (size_t)l.N * q.row_lanes <= size_t(1) << 30) q.row_lanes *= 2;
    const int row_blocks = (int)(((size_t)l.N * q.row_lanes + 255) / 256);
    if constexpr (lin_affine(FMT)) {
      q.xq = reinterpret_cast<uint16_t*>(ws + lay.xq);
      q.xsum = reinterpret_cast<uint16_t*>(ws + lay.xsum);
      q.xexp = reinterpret_cast<int32_t*>(ws + lay.xexp);
      q.sh = reinterpret_cast<uint16_t*>(ws + lay.sh);
      q.tok_blocks = l.L;
      a.x = q.xq;
      a.xsum = q.xsum;
      a.xexp = q.xexp;
      a.sh = q.sh;
      q.tsum = reinterpret_cast<uint16_t*>(ws + lay.tsum);
      a.tsum = q.tsum;
    }
    hipLaunchKernelGGL((k_linear_prepare<FMT, F16>), dim3(q.tok_blocks + row_blocks), dim3(256), 0, stream, q);
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  switch (p.mt) {
    case 2: launch_tiles_mt<FMT, F16, 2>(a, p, stream); break;
    case 4: launch_tiles_mt<FMT, F16, 4>(a, p, stream); break;
    default: launch_tiles_mt<FMT, F16, 8>(a, p, stream); break;
  }
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.splits > 1) launch_linear_join(l, a.part, p.splits, stream);
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

template <int FMT>
int linear_launch(bool f16, const LinearArgs& a, unsigned char* ws, hipStream_t stream) {
  if (linear_by_tiles(FMT, a.L, a.N, a.K)) return f16 ? launch_tiles<FMT, true>(a, ws, stream) : launch_tiles<FMT, false>(a, ws, stream);
  if (a.K < kLinStep) {
    const int most = (int)std::min<size_t>(a.L, (size_t(1) << 31) / a.N);  // tokens whose outputs fit a launch's threads
    LinearArgs l = a;
    for (int t = 0; t < a.L; t += most) {
      l.L = std::min(most, a.L - t);
      l.x = a.x + (size_t)t * a.ldx;
      l.out = static_cast<unsigned char*>(a.out) + (size_t)t * a.ldo * (a.out_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2);
      const dim3 grid((unsigned)(((size_t)l.L * l.N + 255) / 256));
      if (f16)
        hipLaunchKernelGGL((k_linear_short<FMT, true>), grid, dim3(256), 0, stream, l);
      else
        hipLaunchKernelGGL((k_linear_short<FMT, false>), grid, dim3(256), 0, stream, l);
      if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
    }
    return MOE_Q4_OK;
  }
  const RowsPlan p = rows_plan(FMT, f16, a.N, a.K, linear_words(a));
  LinearArgs l = a;
  if (p.splits > 1) l.part = reinterpret_cast<float*>(ws);
  f16 ? launch_linear_rows<FMT, true>(l, p, stream) : launch_linear_rows<FMT, false>(l, p, stream);
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.splits > 1) launch_linear_join(l, l.part, p.splits, stream);
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
#endif

}  // namespace moeq4
