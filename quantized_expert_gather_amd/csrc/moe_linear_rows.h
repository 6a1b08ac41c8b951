// Dense 4-bit product for few tokens.  Internal header.
//
// A workgroup takes 16 weight rows at a time, its W waves splitting K; wave
// w's S steps of 128 inputs of x stay in its registers over all the rows it
// meets (longer K is taken in passes), and the next rows' codes are on their
// way while these are multiplied.  A lane (n, kb) loads 16 bytes of row n, the
// 32 codes from input 32 kb of the step; a matrix product of their words with
// x sums over n's four lanes, which hold different scale groups.  So
//   mxfp4       the block's power of two goes into the bf16 operand, exact
//               (fp16 x is split into two bf16 terms, exact too);
//   nvfp4       element times scale goes into the operand, exact;
//   affine      scales 16-bit operands cannot hold: the words are transposed
//               over the four lanes first, so each product is one group's, and
//               scale and bias multiply its fp32 sums.
// With at most four tokens (kFew) affine and nvfp4 words need none of this:
// token t takes operand rows 4 t .. 4 t + 3, row 4 t + b holding its x in
// lanes kb = b only, so a lane (n, t) receives the four blocks' sums of row n
// and token t separately, and multiplies them by the row's scales.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_linear_device.h"
#include "moe_q4.h"

namespace moeq4 {

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
  int passes;  // passes over K that the waves' registers take
};

__device__ __forceinline__ void lin_store(void* out, size_t at, int dtype, float v) {
  if (dtype == MOE_Q4_DTYPE_F32)
    static_cast<float*>(out)[at] = v;
  else if (dtype == MOE_Q4_DTYPE_BF16)
    static_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_rne(v);
  else
    static_cast<_Float16*>(out)[at] = (_Float16)v;
}

// Bytes of a row's scales in a step, and of those a lane reads: all of them
// where it scales sums, its own block's where it scales operands.
template <int FMT, bool FEW>
struct LinScales {
  static constexpr bool kOwn = FMT == kLinMxfp4 || (FMT == kLinNvfp4 && !FEW);
  static constexpr int kStep = FMT == kLinAffine64 ? 4 : FMT == kLinMxfp4 ? 4 : 8;
  static constexpr int kWords = !kOwn && kStep == 8 ? 2 : 1;
};

// Reads them.  A row's scales may start at any byte, and the last step of a
// row may be short: it is read from its end back (K >= 128) and shifted down,
// which leaves zeros for what is not there.
template <int FMT, bool FEW>
__device__ __forceinline__ void lin_scales(const unsigned char* row, int step, int kb, int row_bytes, bool ragged,
                                           uint32_t (&v)[LinScales<FMT, FEW>::kWords]) {
  typedef LinScales<FMT, FEW> Sc;
  if constexpr (Sc::kOwn) {
    constexpr int kBytes = Sc::kStep / 4;
    const int at = min(step * Sc::kStep + kb * kBytes, row_bytes - kBytes);
    if constexpr (kBytes == 1)
      v[0] = row[at];
    else
      v[0] = *reinterpret_cast<const uint16_t*>(row + at);
  } else {
    int at = step * Sc::kStep, shift = 0;
    if (ragged) {
      const int last = row_bytes - Sc::kStep;
      shift = 8 * max(at - last, 0);
      at = min(at, last);
    }
    if constexpr (Sc::kStep == 4) {
      uint32_t u;
      __builtin_memcpy(&u, row + at, 4);
      v[0] = u >> shift;
    } else {
      uint64_t u;
      __builtin_memcpy(&u, row + at, 8);
      u >>= shift;
      v[0] = (uint32_t)u;
      v[1] = (uint32_t)(u >> 32);
    }
  }
}

template <int FMT, bool F16, bool FEW, int S, int W>
__global__ __launch_bounds__(64 * W) void k_linear_rows(LinearArgs a) {
  typedef LinScales<FMT, FEW> Sc;
  constexpr bool kAffine = lin_affine(FMT);
  constexpr bool kSep = FEW && FMT != kLinMxfp4;       // blocks' sums kept apart
  constexpr bool kTurn = kAffine && !FEW;              // words transposed
  constexpr bool kTerms = FMT == kLinMxfp4 && F16;     // x as two bf16 terms
  constexpr int kX = kTerms ? 2 : 1;
  constexpr int kGroups = FMT == kLinAffine64 ? 2 : 4;  // group sums of x a step (affine)
  constexpr int kAcc = kSep ? 1 : 4;
  __shared__ float red[2][W][kAcc * 64];
  __shared__ __attribute__((aligned(16))) float xsum[kAffine ? W * S * kGroups * 16 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n16 = lane & 15, kb = lane >> 4;
  const int t0 = blockIdx.y * 16;
  const int steps = (a.K + kLinStep - 1) / kLinStep;
  const bool ragged = a.K % kLinStep != 0;
  const int tiles = (a.N + 15) / 16;
  const int wrow = a.K / 2, srow = a.K / lin_group(FMT) * (kAffine ? 2 : 1);
  const LinCode code = lin_code<F16>();

  struct Rows {  // a pass over 16 rows, as loaded
    uint4 c[S];
    uint32_t s[S][Sc::kWords], b[kAffine ? S : 1][Sc::kWords];
  };
  auto load = [&](int tile, int pass, Rows& r) __attribute__((always_inline)) {
    const size_t row = min(tile * 16 + n16, a.N - 1);
    const int first = (pass * W + wave) * S;
    const unsigned char* w = reinterpret_cast<const unsigned char*>(a.w) + row * wrow;
#pragma unroll
    for (int st = 0; st < S; ++st) {
      if (first + st >= steps) break;
      const int at = (first + st) * (kLinStep / 2) + 16 * kb;
      r.c[st] = *reinterpret_cast<const uint4*>(w + (ragged ? min(at, wrow - 16) : at));
    }
#pragma unroll
    for (int st = 0; st < S; ++st) {
      if (first + st >= steps) break;
      lin_scales<FMT, FEW>(a.s + row * srow, first + st, kb, srow, ragged, r.s[st]);
      if constexpr (kAffine) lin_scales<FMT, FEW>(a.b + row * srow, first + st, kb, srow, ragged, r.b[st]);
    }
  };

  uint4 xf[S][4][kX];
  auto load_x = [&](int pass) __attribute__((always_inline)) {
    const int first = (pass * W + wave) * S;
    const int t = t0 + (kSep ? n16 >> 2 : n16);
    const bool live = t < a.L && (!kSep || (n16 & 3) == kb);
    const uint16_t* x = a.x + (size_t)min(t, a.L - 1) * a.ldx + first * kLinStep;
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int j = 0; j < 4; ++j) xf[st][j][0] = make_uint4(0, 0, 0, 0);
    if (live) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        if (first + st >= steps) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // operand register j: after the transpose block j's inputs, else word j of block kb
          const int c = st * kLinStep + (kTurn ? 32 * j + 8 * kb : 32 * kb + 8 * j);
          if (!ragged || first * kLinStep + c < a.K) xf[st][j][0] = *reinterpret_cast<const uint4*>(x + c);
        }
      }
    }
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kAffine) xf[st][j][0] = lin_pair_order(xf[st][j][0]);
        if constexpr (kTerms) {
          uint32_t q[4] = {xf[st][j][0].x, xf[st][j][0].y, xf[st][j][0].z, xf[st][j][0].w}, hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // 11 bits as 8 + 3, both exact
            const lin_f16x2 h = __builtin_bit_cast(lin_f16x2, q[i]);
            const float f0 = (float)h.x, f1 = (float)h.y;
            const uint32_t h0 = __float_as_uint(f0) & 0xFFFF0000u, h1 = __float_as_uint(f1) & 0xFFFF0000u;
            hi[i] = h0 >> 16 | h1;
            // (an infinite or NaN x has no second term)
            const float r0 = f0 - __uint_as_float(h0), r1 = f1 - __uint_as_float(h1);
            lo[i] = (r0 == r0 ? __float_as_uint(r0) >> 16 : 0u) | (r1 == r1 ? __float_as_uint(r1) & 0xFFFF0000u : 0u);
          }
          xf[st][j][0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          xf[st][j][kX - 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    if constexpr (kAffine) {  // x times ones is the group sums, in the layout of the products
      const uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
      const uint4 ones = make_uint4(one, one, one, one);
#pragma unroll
      for (int st = 0; st < S; ++st) {
        float* to = xsum + (wave * S + st) * kGroups * 16;
        if constexpr (kSep) {  // [step][token][group]
          lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j) c = lin_mfma<F16>(xf[st][j][0], ones, c);
          if (n16 == 0) {
            if constexpr (kGroups == 2)
              *reinterpret_cast<lin_f32x2*>(to + 2 * kb) = lin_f32x2{c[0] + c[1], c[2] + c[3]};
            else
              *reinterpret_cast<lin_f32x4*>(to + 4 * kb) = c;
          }
        } else {  // [step][group][token]
          constexpr int kPer = 4 / kGroups;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
            for (int j = g * kPer; j < (g + 1) * kPer; ++j) c = lin_mfma<F16>(xf[st][j][0], ones, c);
            if (n16 == 0) *reinterpret_cast<lin_f32x4*>(to + g * 16 + 4 * kb) = c;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // read by this wave's other lanes
    }
  };

  lin_f32x4 acc = {0, 0, 0, 0};
  auto multiply = [&](const Rows& r, int pass) __attribute__((always_inline)) {
    const int first = (pass * W + wave) * S;
#pragma unroll
    for (int st = 0; st < S; ++st) {
      if (first + st >= steps) break;
      uint32_t w4[4] = {r.c[st].x, r.c[st].y, r.c[st].z, r.c[st].w};
      const float* xs = xsum + (wave * S + st) * kGroups * 16;
      if constexpr (FMT == kLinMxfp4) {
        // past a row's end x is zero, and the codes and scales are the row's own last ones
        const float s = lin_e8m0(r.s[st][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = lin_fp4_pow2<false>(w4[j], s);
#pragma unroll
          for (int i = 0; i < kX; ++i) acc = lin_mfma<false>(xf[st][j][i], w, acc);
        }
      } else if constexpr (FMT == kLinNvfp4 && !FEW) {
        const float s0 = lin_e4m3<0>(r.s[st][0]), s1 = lin_e4m3<1>(r.s[st][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = lin_mfma<F16>(xf[st][j][0], lin_fp4_scaled<F16>(w4[j], j < 2 ? s0 : s1), acc);
      } else if constexpr (FMT == kLinNvfp4) {
        lin_f32x4 c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0};  // the first and the second 16 inputs of the blocks
        c0 = lin_mfma<F16>(xf[st][0][0], lin_fp4<F16>(w4[0]), c0);
        c1 = lin_mfma<F16>(xf[st][2][0], lin_fp4<F16>(w4[2]), c1);
        c0 = lin_mfma<F16>(xf[st][1][0], lin_fp4<F16>(w4[1]), c0);
        c1 = lin_mfma<F16>(xf[st][3][0], lin_fp4<F16>(w4[3]), c1);
        const uint32_t s0 = r.s[st][0], s1 = r.s[st][1];
        acc[0] = __builtin_fmaf(lin_e4m3<0>(s0), c0[0], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<1>(s0), c1[0], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<2>(s0), c0[1], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<3>(s0), c1[1], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<0>(s1), c0[2], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<1>(s1), c1[2], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<2>(s1), c0[3], acc[0]);
        acc[0] = __builtin_fmaf(lin_e4m3<3>(s1), c1[3], acc[0]);
      } else {
        auto half = [](const uint32_t (&v)[Sc::kWords], int g) { return g & 1 ? bf16_hi_to_f32(v[g / 2]) : bf16_lo_to_f32(v[g / 2]); };
        if constexpr (FEW) {
          lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j) c = lin_mfma<F16>(xf[st][j][0], lin_codes16<F16>(w4[j], code), c);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float s = half(r.s[st], g), off = __builtin_fmaf(-16.0f, s, half(r.b[st], g));
            const float v = kGroups == 2 ? c[2 * g] + c[2 * g + 1] : c[g];
            acc[0] = __builtin_fmaf(off, xs[kGroups * kb + g], __builtin_fmaf(s, v, acc[0]));
          }
        } else {
          constexpr int kPer = 4 / kGroups;
          lin_transpose(w4);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            lin_f32x4 c = {0, 0, 0, 0};
#pragma unroll
            for (int j = g * kPer; j < (g + 1) * kPer; ++j) c = lin_mfma<F16>(xf[st][j][0], lin_codes16<F16>(w4[j], code), c);
            const float s = half(r.s[st], g), off = __builtin_fmaf(-16.0f, s, half(r.b[st], g));
            const lin_f32x4 x4 = *reinterpret_cast<const lin_f32x4*>(xs + g * 16 + 4 * kb);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(off, x4[i], __builtin_fmaf(s, c[i], acc[i]));
          }
        }
      }
    }
  };

  // The waves' sums of a tile, in ascending order of the waves.  The two
  // buffers alternate: a wave is at most one barrier ahead of the readers.
  auto finish = [&](int tile, int buf) __attribute__((always_inline)) {
    if constexpr (kSep)
      red[buf][wave][lane] = acc[0];
    else
      *reinterpret_cast<lin_f32x4*>(&red[buf][wave][4 * lane]) = acc;
    acc = lin_f32x4{0, 0, 0, 0};
    __syncthreads();
    constexpr int kParts = W / 4;  // threads of an output, four waves' sums each
    const int o = threadIdx.x / kParts, part = threadIdx.x % kParts;
    const int n = tile * 16 + (o & 15), t = t0 + (o >> 4);
    if (kSep && o >= 64) return;  // whole waves
    const float* r = &red[buf][4 * part][kSep ? o : 4 * ((o & 15) + 16 * (o >> 6)) + ((o >> 4) & 3)];
    constexpr int kWave = kAcc * 64;
    float v = (r[0] + r[kWave]) + (r[2 * kWave] + r[3 * kWave]);
    if constexpr (kParts >= 2) v += dpp_f32<0xB1>(v);  // lane ^ 1
    if constexpr (kParts >= 4) v += dpp_f32<0x4E>(v);  // lane ^ 2
    if (part == 0 && t < a.L && n < a.N) {
      if (a.bias) v += a.bias[n];
      lin_store(a.out, (size_t)t * a.ldo + n, a.out_dtype, v);
    }
  };

  int tile = blockIdx.x, pass = 0, buf = 0;
  auto body = [&](Rows& cur, Rows& nxt) __attribute__((always_inline)) {
    int tile2 = tile, pass2 = pass + 1;
    if (pass2 == a.passes) {
      pass2 = 0;
      tile2 += gridDim.x;
    }
    if (tile2 < tiles) load(tile2, pass2, nxt);
    multiply(cur, pass);
    if (pass2 == 0) {
      finish(tile, buf);
      buf ^= 1;
    }
    if (a.passes > 1 && tile2 < tiles) load_x(pass2);
    tile = tile2;
    pass = pass2;
  };
  Rows one, two;
  load(tile, 0, one);
  load_x(0);
  while (true) {
    body(one, two);
    if (tile >= tiles) break;
    body(two, one);
    if (tile >= tiles) break;
  }
}

template <int FMT, bool F16>
void launch_linear_rows(const LinearArgs& args, hipStream_t stream) {
  LinearArgs a = args;
  const int steps = (a.K + kLinStep - 1) / kLinStep;
  const bool wide = steps > 12;  // 16 waves, else 8
  const int W = wide ? 16 : 8;
  constexpr int kMost = FMT == kLinMxfp4 && F16 ? 2 : 3;  // steps of x that fit a wave's registers
  a.passes = (steps + kMost * W - 1) / (kMost * W);
  const int S = (steps + a.passes * W - 1) / (a.passes * W);
  const int tiles = (a.N + 15) / 16;
  const int most = wide ? 256 : 512;  // workgroups that run at once
  const int rounds = (tiles + most - 1) / most;
  const dim3 grid((tiles + rounds - 1) / rounds, (a.L + 15) / 16), block(64 * W);
  const bool few = a.L <= 4 && FMT != kLinMxfp4;
#define MOE_LINEAR_ROWS(FEW, S)                                                                         \
  if (wide)                                                                                             \
    hipLaunchKernelGGL((k_linear_rows<FMT, F16, FEW, S, 16>), grid, block, 0, stream, a);               \
  else                                                                                                  \
    hipLaunchKernelGGL((k_linear_rows<FMT, F16, FEW, S, 8>), grid, block, 0, stream, a)
  if constexpr (FMT != kLinMxfp4) {
    if (few) {
      switch (S) {
        case 1: MOE_LINEAR_ROWS(true, 1); break;
        case 2: MOE_LINEAR_ROWS(true, 2); break;
        default: MOE_LINEAR_ROWS(true, 3); break;
      }
      return;
    }
  }
  switch (S) {
    case 1: MOE_LINEAR_ROWS(false, 1); break;
    case 2: MOE_LINEAR_ROWS(false, 2); break;
    default:
      if constexpr (kMost >= 3) {
        MOE_LINEAR_ROWS(false, 3);
      }
      break;
  }
#undef MOE_LINEAR_ROWS
}

// Inputs shorter than a step: one thread an output.
template <int FMT, bool F16>
__global__ __launch_bounds__(256) void k_linear_short(LinearArgs a) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)a.L * a.N) return;
  const int t = (int)(i / a.N), n = (int)(i - (size_t)t * a.N);
  const uint16_t* x = a.x + (size_t)t * a.ldx;
  const unsigned char* w = reinterpret_cast<const unsigned char*>(a.w) + (size_t)n * (a.K / 2);
  const int G = a.K / lin_group(FMT);
  float acc = 0.0f;
  for (int g = 0; g < G; ++g) {
    const size_t at = (size_t)n * G + g;
    float sum = 0.0f, xs = 0.0f;
    for (int c = g * lin_group(FMT); c < (g + 1) * lin_group(FMT); ++c) {
      float v;
      if constexpr (F16)
        v = (float)__builtin_bit_cast(_Float16, x[c]);
      else
        v = bf16_to_f32(x[c]);
      const uint32_t q = (w[c / 2] >> (4 * (c & 1))) & 15u;
      float e = (float)q;
      if constexpr (!lin_affine(FMT)) {  // E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6
        const uint32_t ex = (q >> 1) & 3u, m = q & 1u;
        e = ex ? (float)((2u + m) << (ex - 1)) * 0.5f : 0.5f * (float)m;
        e = q & 8u ? -e : e;
      }
      sum = __builtin_fmaf(v, e, sum);
      xs += v;
    }
    float s;
    if constexpr (FMT == kLinMxfp4)
      s = lin_e8m0(a.s[at]);
    else if constexpr (FMT == kLinNvfp4)
      s = e4m3_to_f32(a.s[at]);
    else
      s = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.s)[at]);
    acc = __builtin_fmaf(s, sum, acc);
    if constexpr (lin_affine(FMT)) acc = __builtin_fmaf(bf16_to_f32(reinterpret_cast<const uint16_t*>(a.b)[at]), xs, acc);
  }
  if (a.bias) acc += a.bias[n];
  lin_store(a.out, (size_t)t * a.ldo + n, a.out_dtype, acc);
}

}  // namespace moeq4
