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

// Tokens from which the tiles take over.
constexpr int kTilesFrom = 17;

struct TilesPlan {
  int mt, nt, row_tiles, tok_tiles, splits, steps_per;
};
inline TilesPlan tiles_plan(int L, int N, int K) {
  TilesPlan p{};
  p.mt = L <= 32 ? 2 : L <= 64 ? 4 : 8;
  p.tok_tiles = (L + 16 * p.mt - 1) / (16 * p.mt);
  const int steps = (K + kLinStep - 1) / kLinStep;
  for (p.nt = 3;; --p.nt) {
    p.row_tiles = (N + 64 * p.nt - 1) / (64 * p.nt);
    if (p.nt == 1 || (long)p.row_tiles * p.tok_tiles >= 256) break;
  }
  const long tiles = (long)p.row_tiles * p.tok_tiles;
  p.splits = 1;
  if (tiles < 256) p.splits = (int)std::max(1L, std::min<long>(std::min(16, steps / 4), 512 / tiles));
  p.steps_per = (steps + p.splits - 1) / p.splits;
  p.splits = (steps + p.steps_per - 1) / p.steps_per;
  return p;
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
  w.tsum = off; off = lin_round256(off + (affine ? 3 * (size_t)N * Gp * 2 : 0));
  w.xexp = off; off = lin_round256(off + (affine ? (size_t)L * 4 : 0));
  w.sh = off;   off = lin_round256(off + (affine ? (size_t)N * G * 2 : 0));
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
  const int s = std::max(rows_plan(fmt, false, K, true).splits, rows_plan(fmt, true, K, true).splits);
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
  a.x = l.x; a.w = l.w; a.s = l.s;
  a.bias = l.bias; a.out = l.out;
  a.ldx = l.ldx; a.ldo = l.ldo;
  a.L = l.L; a.N = l.N; a.K = l.K;
  a.G = l.K / lin_group(FMT);
  a.Gp = (a.G + 31) / 32 * 32;
  a.out_dtype = l.out_dtype;
  a.terms = l.out_dtype == MOE_Q4_DTYPE_F32 ? 3 : 2;
  a.splits = p.splits; a.steps_per = p.steps_per;
  a.stagger = std::max(1, p.steps_per / p.tok_tiles);
  a.row_tiles = p.row_tiles; a.tok_tiles = p.tok_tiles;
  a.part = reinterpret_cast<float*>(ws + lay.part);
  constexpr bool kRowsScaled = lin_affine(FMT) || (FMT == kLinMxfp4 && F16);
  if constexpr (kRowsScaled) {
    a.wexp = reinterpret_cast<int32_t*>(ws + lay.wexp);
    PrepareArgs q{};
    q.x = l.x; q.s = l.s; q.b = l.b;
    q.wexp = reinterpret_cast<int32_t*>(ws + lay.wexp);
    q.ldx = l.ldx;
    q.L = l.L; q.N = l.N; q.K = l.K; q.G = a.G; q.Gp = a.Gp;
    if constexpr (lin_affine(FMT)) {
      q.xq = reinterpret_cast<uint16_t*>(ws + lay.xq);
      q.xsum = reinterpret_cast<uint16_t*>(ws + lay.xsum);
      q.xexp = reinterpret_cast<int32_t*>(ws + lay.xexp);
      q.sh = reinterpret_cast<uint16_t*>(ws + lay.sh);
      q.tok_blocks = l.L;
      a.x = q.xq;
      a.xsum = q.xsum;
      a.xexp = F16 ? nullptr : q.xexp;
      a.sh = q.sh;
      q.tsum = reinterpret_cast<uint16_t*>(ws + lay.tsum);
      a.tsum = q.tsum;
    }
    hipLaunchKernelGGL((k_linear_prepare<FMT, F16>), dim3(q.tok_blocks + (l.N + 3) / 4), dim3(256), 0, stream, q);
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
  if (a.L >= kTilesFrom) return f16 ? launch_tiles<FMT, true>(a, ws, stream) : launch_tiles<FMT, false>(a, ws, stream);
  if (a.K < kLinStep) {
    const dim3 grid((unsigned)(((size_t)a.L * a.N + 255) / 256));
    if (f16)
      hipLaunchKernelGGL((k_linear_short<FMT, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_linear_short<FMT, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
  }
  const RowsPlan p = rows_plan(FMT, f16, a.K, linear_words(a));
  LinearArgs l = a;
  if (p.splits > 1) l.part = reinterpret_cast<float*>(ws);
  f16 ? launch_linear_rows<FMT, true>(l, p, stream) : launch_linear_rows<FMT, false>(l, p, stream);
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.splits > 1) launch_linear_join(l, l.part, p.splits, stream);
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
#endif

}  // namespace moeq4
