// Dense product with 4-bit weights: out[t, n] = sum_c x[t, c] W[n, c] + bias[n]
// over the expert banks' codecs.
//
// Affine: W = s q + b per group, so the sum over a group is s * sum x q + b *
// sum x; the matrix cores form sum x (16 + q) exactly from 16-bit operands
// with fp32 accumulation, and sum x by a product with ones.  mxfp4: the
// block's power of two multiplies the sum.  nvfp4: scale and element multiply
// exactly into the operand.  No weight is rounded.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "moe_linear_device.h"
#include "moe_linear_tiles.h"
#include "moe_q4.h"

namespace moeq4 {
namespace {

struct LinearArgs {
  const uint16_t* x;
  const uint32_t* w;
  const unsigned char* s;
  const unsigned char* b;
  const float* bias;
  void* out;
  long long ldx, ldo;
  int L, N, K;
  int out_dtype;
  int svec;    // scale rows can be read a step at a time
  int chunks;  // passes over K that the waves' registers take
};

__device__ __forceinline__ void lin_store(void* out, size_t at, int dtype, float v) {
  if (dtype == MOE_Q4_DTYPE_F32)
    static_cast<float*>(out)[at] = v;
  else if (dtype == MOE_Q4_DTYPE_BF16)
    static_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_rne(v);
  else
    static_cast<_Float16*>(out)[at] = (_Float16)v;
}

// A step's scales (or biases) of one row, as raw words.  Without `vec`
// single elements are read, clamped to the row.
template <int FMT>
__device__ __forceinline__ void load_scales(const unsigned char* p, size_t row, int step, int kb, int G, bool vec,
                                            uint32_t (&v)[lin_scale_words(FMT)]) {
  if constexpr (FMT == kLinNvfp4) {  // the lane's own two groups
    const int g = min(8 * step + 2 * kb, G - 2);
    v[0] = *reinterpret_cast<const uint16_t*>(p + row * G + g);
  } else if constexpr (FMT == kLinMxfp4) {
    if (vec) {
      v[0] = *reinterpret_cast<const uint32_t*>(p + row * G + 4 * step);
    } else {
      v[0] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0] |= (uint32_t)p[row * G + min(4 * step + i, G - 1)] << (8 * i);
    }
  } else {
    constexpr int kPer = kLinStep / lin_group(FMT);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + row * G;
    if (vec) {
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) v[i] = *reinterpret_cast<const uint32_t*>(q + kPer * step + 2 * i);
    } else {
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i)
        v[i] = (uint32_t)q[min(kPer * step + 2 * i, G - 1)] | (uint32_t)q[min(kPer * step + 2 * i + 1, G - 1)] << 16;
    }
  }
}

// Few tokens: a workgroup of W waves takes 16 weight rows at a time, its
// waves splitting K; wave w's S steps of x stay in its registers over all
// the rows it meets.  The waves' sums meet in LDS.
template <int FMT, bool F16, int S, int W>
__global__ __launch_bounds__(64 * W) void k_linear_rows(LinearArgs a) {
  __shared__ lin_f32x4 red[2][W][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = lane & 15, kb = lane >> 4;
  const int t0 = blockIdx.y * 16;
  const int steps = (a.K + kLinStep - 1) / kLinStep;
  const int G = a.K / lin_group(FMT);
  const int tiles = (a.N + 15) / 16;
  constexpr int kGroups = lin_affine(FMT) ? kLinStep / lin_group(FMT) : 1;
  const uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
  const uint4 ones = make_uint4(one, one, one, one);

  uint4 xf[S][4];
  lin_f32x4 xs[S][kGroups];
  auto load_x = [&](int chunk) {
#pragma unroll
    for (int st = 0; st < S; ++st) {
      const int step = (chunk * W + wave) * S + st;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = step * kLinStep + lin_input<FMT>(g, kb);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < a.K && t0 + n16 < a.L) v = *reinterpret_cast<const uint4*>(a.x + (size_t)(t0 + n16) * a.ldx + c);
        xf[st][g] = lin_affine(FMT) ? lin_pair_order(v) : v;
      }
      if constexpr (lin_affine(FMT)) {
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
          for (int g = q * 4 / kGroups; g < (q + 1) * 4 / kGroups; ++g) c = lin_mfma<F16>(xf[st][g], ones, c);
          xs[st][q] = c;
        }
      }
    }
  };
  const LinCode code = lin_code<F16>();
  if (a.chunks == 1) load_x(0);

  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const size_t row = min(tile * 16 + n16, a.N - 1);
    lin_f32x4 acc = {0, 0, 0, 0};
    for (int chunk = 0; chunk < a.chunks; ++chunk) {
      if (a.chunks > 1) load_x(chunk);
      uint4 cw[S];
      uint32_t sw[S][lin_scale_words(FMT)], bw[S][lin_scale_words(FMT)];
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int step = (chunk * W + wave) * S + st;
        if (step < steps) {
          const int c = min(step * kLinStep + 32 * kb, a.K - 32);
          cw[st] = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(a.w) +
                                                   row * ((size_t)a.K / 2) + c / 2);
          load_scales<FMT>(a.s, row, step, kb, G, a.svec, sw[st]);
          if constexpr (lin_affine(FMT)) load_scales<FMT>(a.b, row, step, kb, G, a.svec, bw[st]);
        }
      }
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int step = (chunk * W + wave) * S + st;
        if (step >= steps) break;
        uint32_t w4[4] = {cw[st].x, cw[st].y, cw[st].z, cw[st].w};
        const int left = a.K - step * kLinStep;  // inputs from here on
        if constexpr (FMT == kLinNvfp4) {
          // past the row's end x is zero and the codes and scales are the row's own last ones
          const float s0 = e4m3_to_f32(sw[st][0] & 255u), s1 = e4m3_to_f32(sw[st][0] >> 8);
#pragma unroll
          for (int g = 0; g < 4; ++g) acc = lin_mfma<F16>(xf[st][g], lin_fp4_scaled<F16>(w4[g], g < 2 ? s0 : s1), acc);
        } else {
          lin_transpose(w4);
          if constexpr (FMT == kLinMxfp4) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (32 * g >= left) break;
              lin_f32x4 c = {0, 0, 0, 0};
              c = lin_mfma<F16>(xf[st][g], lin_fp4<F16>(w4[g]), c);
              const float s = lin_e8m0((sw[st][0] >> (8 * g)) & 255u);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s, c[i], acc[i]);
            }
          } else {
            constexpr int kPer = 4 / kGroups;  // operand registers of a group
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
              if (32 * kPer * q >= left) break;
              lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
              for (int g = q * kPer; g < (q + 1) * kPer; ++g) c = lin_mfma<F16>(xf[st][g], lin_codes16<F16>(w4[g], code), c);
              const float s = q & 1 ? bf16_hi_to_f32(sw[st][q / 2]) : bf16_lo_to_f32(sw[st][q / 2]);
              const float b = q & 1 ? bf16_hi_to_f32(bw[st][q / 2]) : bf16_lo_to_f32(bw[st][q / 2]);
              const float off = __builtin_fmaf(-16.0f, s, b);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(off, xs[st][q][i], __builtin_fmaf(s, c[i], acc[i]));
            }
          }
        }
      }
    }
    // buffers alternate: a wave is at most one barrier ahead of the readers
    red[buf][wave][lane] = acc;
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += 64 * W) {
      const int i = o & 3, l = o >> 2;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += red[buf][w][l][i];
      const int t = t0 + 4 * (l >> 4) + i, n = tile * 16 + (l & 15);
      if (t < a.L && n < a.N) {
        if (a.bias) v += a.bias[n];
        lin_store(a.out, (size_t)t * a.ldo + n, a.out_dtype, v);
      }
    }
  }
}

template <int FMT, bool F16>
void launch_rows(const LinearArgs& args, hipStream_t stream) {
  LinearArgs a = args;
  constexpr int W = 8;
  const int steps = (a.K + kLinStep - 1) / kLinStep;
  a.chunks = (steps + 4 * W - 1) / (4 * W);
  const int S = (steps + a.chunks * W - 1) / (a.chunks * W);
  const int tiles = (a.N + 15) / 16;
  const dim3 grid(std::min(tiles, 512), (a.L + 15) / 16), block(64 * W);
  switch (S) {
    case 1: hipLaunchKernelGGL((k_linear_rows<FMT, F16, 1, W>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_linear_rows<FMT, F16, 2, W>), grid, block, 0, stream, a); break;
    case 3: hipLaunchKernelGGL((k_linear_rows<FMT, F16, 3, W>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((k_linear_rows<FMT, F16, 4, W>), grid, block, 0, stream, a); break;
  }
}

// Tokens from which the tiles take over.
constexpr int kTilesFrom = 17;

struct TilesPlan {
  int mt, nt, row_tiles, tok_tiles, splits, steps_per;
};
TilesPlan tiles_plan(int L, int N, int K) {
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
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
TilesWorkspace tiles_layout(int fmt, int L, int N, int K) {
  TilesWorkspace w{};
  const TilesPlan p = tiles_plan(L, N, K);
  const size_t G = K / lin_group(fmt), Gp = (G + 31) / 32 * 32;
  const bool affine = lin_affine(fmt);
  size_t off = 0;
  w.xq = off;   off = round256(off + (affine ? (size_t)p.tok_tiles * p.mt * 16 * ((K + kLinStep - 1) / kLinStep * kLinStep) * 2 : 0));
  w.xsum = off; off = round256(off + (affine ? 3 * (size_t)L * Gp * 2 : 0));
  w.tsum = off; off = round256(off + (affine ? 3 * (size_t)N * Gp * 2 : 0));
  w.xexp = off; off = round256(off + (affine ? (size_t)L * 4 : 0));
  w.sh = off;   off = round256(off + (affine ? (size_t)N * G * 2 : 0));
  w.wexp = off; off = round256(off + (affine || fmt == kLinMxfp4 ? (size_t)N * 4 : 0));
  w.part = off; off = round256(off + (p.splits > 1 ? (size_t)p.splits * L * N * 4 : 0));
  w.total = off;
  return w;
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
  if (p.splits > 1) {
    const size_t all = (size_t)l.L * l.N;
    hipLaunchKernelGGL(k_linear_join, dim3((unsigned)std::min<size_t>((all + 255) / 256, 4096)), dim3(256), 0, stream, a.part,
                       l.bias, l.out, l.ldo, l.L, l.N, p.splits, l.out_dtype);
  }
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

int linear_fmt(int codec) {
  switch (codec) {
    case MOE_Q4_CODEC_AFFINE4_G64: return kLinAffine64;
    case MOE_Q4_CODEC_AFFINE4_G32: return kLinAffine32;
    case MOE_Q4_CODEC_MXFP4: return kLinMxfp4;
    case MOE_Q4_CODEC_NVFP4: return kLinNvfp4;
  }
  return -1;
}

int linear_shape_status(int fmt, int L, int N, int K) {
  if (L < 0 || N < 1 || K < 1) return MOE_Q4_ERR_SHAPE;
  const int grp = fmt == kLinAffine64 ? 64 : 32;
  if (fmt < 0 || K % grp || L > MOE_Q4_LINEAR_MAX_L || K > MOE_Q4_LINEAR_MAX_K) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

bool aligned_to(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}
size_t span(int rows, long long ld, int cols, size_t es) {
  return rows ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0;
}

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" size_t moe_linear_codec_workspace_bytes(int codec, int L, int N, int K) {
  const int fmt = linear_fmt(codec);
  if (linear_shape_status(fmt, L, N, K) || L < kTilesFrom) return 0;
  return tiles_layout(fmt, L, N, K).total;
}

extern "C" int moe_linear_codec_forward(int codec, const void* x, int x_dtype, long long ldx, const uint32_t* w,
                                        const void* s, const void* b, const float* bias, int L, int N, int K, void* out,
                                        int out_dtype, long long ldo, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream) {
  const int fmt = linear_fmt(codec);
  const int st = linear_shape_status(fmt, L, N, K);
  if (st) return st;
  if (ldx < K || ldo < N) return MOE_Q4_ERR_SHAPE;
  if (x_dtype != MOE_Q4_DTYPE_BF16 && x_dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (out_dtype != MOE_Q4_DTYPE_BF16 && out_dtype != MOE_Q4_DTYPE_F32 && out_dtype != MOE_Q4_DTYPE_F16)
    return MOE_Q4_ERR_UNSUPPORTED;
  if (L == 0) return MOE_Q4_OK;
  const bool affine = lin_affine(fmt);
  if (!x || !w || !s || !out || (affine && !b)) return MOE_Q4_ERR_NULL;
  const size_t os = out_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2, sa = fmt == kLinMxfp4 ? 1 : 2;
  if (!aligned_to(x, 16) || (L > 1 && ldx % 8) || !aligned_to(w, 16) || !aligned_to(s, sa) || (affine && !aligned_to(b, 2)) ||
      !aligned_to(bias, 4) || !aligned_to(out, os))
    return MOE_Q4_ERR_ALIGN;
  const size_t need = moe_linear_codec_workspace_bytes(codec, L, N, K);
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (need && !aligned_to(workspace, 256)) return MOE_Q4_ERR_ALIGN;
  const size_t gs = lin_group(fmt), sb = (size_t)N * (K / gs) * (affine ? 2 : 1);
  const struct { const void* p; size_t n; } ins[] = {{x, span(L, ldx, K, 2)}, {w, (size_t)N * K / 2}, {s, sb},
                                                     {affine ? b : nullptr, affine ? sb : 0},
                                                     {bias, bias ? (size_t)N * 4 : 0}, {workspace, need}};
  const size_t on = span(L, ldo, N, os);
  for (const auto& in : ins)
    if (overlap(out, on, in.p, in.n)) return MOE_Q4_ERR_ALIAS;
  LinearArgs a{static_cast<const uint16_t*>(x), w, static_cast<const unsigned char*>(s),
               static_cast<const unsigned char*>(b), bias, out, ldx, ldo, L, N, K, out_dtype, 0, 1};
  // whole steps, and rows of scales that start on words
  a.svec = K % kLinStep == 0 && aligned_to(s, 4) && (!affine || aligned_to(b, 4));
  const bool f16 = x_dtype == MOE_Q4_DTYPE_F16;
  unsigned char* wsb = static_cast<unsigned char*>(workspace);
#define MOE_LINEAR_CALL(FMT)                                                                          \
  if (L >= kTilesFrom) return f16 ? launch_tiles<FMT, true>(a, wsb, stream) : launch_tiles<FMT, false>(a, wsb, stream); \
  f16 ? launch_rows<FMT, true>(a, stream) : launch_rows<FMT, false>(a, stream);                      \
  break
  switch (fmt) {
    case kLinAffine64: MOE_LINEAR_CALL(kLinAffine64);
    case kLinAffine32: MOE_LINEAR_CALL(kLinAffine32);
    case kLinMxfp4: MOE_LINEAR_CALL(kLinMxfp4);
    default: MOE_LINEAR_CALL(kLinNvfp4);
  }
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
