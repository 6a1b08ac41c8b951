// Dense 4-bit product for few tokens.  Internal header.
//
// A workgroup takes 16 weight rows at a time, its W waves splitting K; wave
// w's S steps of 128 inputs of x stay in its registers over all the rows it
// meets, and D tiles of rows are on their way at a time (K beyond W S steps
// is split over workgroups).  A lane (n, kb) loads 16 bytes of row n, the
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
//
// What it has to move is the weights.  Large ones stream at 5.2 TB/s (mxfp4 4
// x 131072 x 4096: 54 us for 287 MB; affine4_g64 1 x 131072 x 6144: 88 us; a
// kernel that only reads reaches 7.1): neighbouring lanes hold different rows,
// as the operand wants them, so a load touches 16 pieces of 64 bytes and takes
// 30 to 50 cycles to issue, and 16 waves a compute unit share that pipe.  A
// tile's codes are one load a step and its scales one a tile for that reason.
// Loads with a streaming hint were slower (60 us).  Small products take what a
// launch, x's way through LDS to registers, one round of weights and the
// waves' reduction take in sequence: 1 x 256 x 6144 5.9 us, 1 x 6144 x 6144 (21
// MB) 10.0, 7 x 4099 x 4096 9.2, 16 x 4096 x 4096 6.3 (mxfp4) to 8.0
// (affine4_g64).
#pragma once

#include <hip/hip_runtime.h>
#include <algorithm>
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
  float* part;        // K split over workgroups: [splits][L][N] partial sums, else NULL
  int split_steps;    // steps of each
};

__device__ __forceinline__ void lin_store(void* out, size_t at, int dtype, float v) {
  if (dtype == MOE_Q4_DTYPE_F32)
    static_cast<float*>(out)[at] = v;
  else if (dtype == MOE_Q4_DTYPE_BF16)
    static_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_rne(v);
  else
    static_cast<_Float16*>(out)[at] = (_Float16)v;
}

// Bytes of a row's scales in a step, and the words of those a lane reads: all
// of them where it scales sums, its own block's where it scales operands.
template <int FMT, bool FEW>
struct LinScales {
  static constexpr bool kOwn = FMT == kLinMxfp4 || (FMT == kLinNvfp4 && !FEW);
  static constexpr int kStep = FMT == kLinAffine64 ? 4 : FMT == kLinMxfp4 ? 4 : 8;
  static constexpr int kWords = !kOwn && kStep == 8 ? 2 : 1;
};

// A row's scales of a step where rows of scales may start at any byte or end
// inside a step: a short last step is read from its end back (K >= 128) and
// shifted down, which leaves zeros for what is not there.
template <int WORDS>
__device__ __forceinline__ void lin_scales_any(const unsigned char* row, int step, int row_bytes, uint32_t (&v)[WORDS]) {
  const int last = row_bytes - 4 * WORDS, at = min(step * 4 * WORDS, last);
  const int shift = 8 * (step * 4 * WORDS - at);
  if constexpr (WORDS == 1) {
    uint32_t u;
    __builtin_memcpy(&u, row + at, 4);
    v[0] = shift > 31 ? 0u : u >> shift;
  } else {
    uint64_t u;
    __builtin_memcpy(&u, row + at, 8);
    u = shift > 63 ? 0u : u >> shift;
    v[0] = (uint32_t)u;
    v[1] = (uint32_t)(u >> 32);
  }
}

// PLAIN: K in whole steps, scale arrays on words.
template <int FMT, bool F16, bool FEW, bool PLAIN, int S, int W>
__global__ __launch_bounds__(64 * W) void k_linear_rows(LinearArgs a) {
  typedef LinScales<FMT, FEW> Sc;
  constexpr bool kAffine = lin_affine(FMT);
  constexpr bool kSep = FEW && FMT != kLinMxfp4;       // blocks' sums kept apart
  constexpr bool kTurn = kAffine && !FEW;              // words transposed
  constexpr bool kTerms = FMT == kLinMxfp4 && F16;     // x as two bf16 terms
  constexpr int kX = kTerms ? 2 : 1;
  constexpr int kGroups = FMT == kLinAffine64 ? 2 : 4;  // group sums of x a step (affine)
  constexpr int kAcc = kSep ? 1 : 4;
  // Tiles on their way, in 128 registers a lane (which 16 waves a compute unit
  // have) with x and the scales.  Deeper rings change little: two tiles instead
  // of four at S = 1 take 38.3 us for 39.5 (mxfp4 4 x 131072 x 2048, 16 waves).
  constexpr int kDeep = S == 1 ? 4 : S == 2 ? 3 : 2;
  __shared__ float red[2][W][kAcc * 64];
  __shared__ __attribute__((aligned(16))) float xsum[kAffine ? W * S * kGroups * 16 : 1];
  constexpr int kStageSteps = kSep ? S : 1, kStageTokens = kSep ? 4 : 16;  // of x in LDS at a time
  __shared__ lin_u32x4 xstage[W][kStageTokens * kStageSteps * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n16 = lane & 15, kb = lane >> 4;
  const int t0 = blockIdx.y * 16;
  const int steps = min((a.K + kLinStep - 1) / kLinStep, ((int)blockIdx.z + 1) * a.split_steps);
  const int first = blockIdx.z * a.split_steps + wave * S;  // this wave's first step
  const int tiles = (a.N + 15) / 16;
  const int wrow = a.K / 2, srow = a.K / lin_group(FMT) * (kAffine ? 2 : 1);
  const LinCode code = lin_code<F16>();

  // Scales: one load a tile, lane (n, kb) taking those of row n and step kb
  // (every load of 16 rows' few bytes costs as much as one of their codes);
  // row moves spread them when they are used.
  constexpr int kRec = Sc::kStep / 4;
  struct Rows {  // 16 rows, as loaded
    lin_u32x4 c[S];
    uint32_t s[kRec], b[kAffine ? kRec : 1];
  };
  // Rows past N lie past the buffers' ranges and read as zero.
  const uint32_t woff = n16 * wrow + 16 * kb, soff = n16 * srow + min(kb, S - 1) * Sc::kStep;
  auto load = [&](int tile, Rows& r) __attribute__((always_inline)) {
    const int rows = min(a.N - tile * 16, 16);
    const rsrc_t wr = make_rsrc(reinterpret_cast<const unsigned char*>(a.w) + (size_t)tile * 16 * wrow, rows * wrow);
#pragma unroll
    for (int st = 0; st < S; ++st) {
      if (first + st >= steps) break;
      // a short last step's missing codes are those of the row's end: x is zero there
      const uint32_t at = PLAIN ? woff : woff + min(0, wrow - 64 - (first + st) * 64 + 48 - 16 * kb);
      r.c[st] = __builtin_bit_cast(lin_u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, at + st * 64, first * 64, 0));
    }
    if (first >= steps) return;
    if constexpr (PLAIN) {
      const rsrc_t sr = make_rsrc(a.s + (size_t)tile * 16 * srow, rows * srow);
      const rsrc_t br = make_rsrc(a.b + (kAffine ? (size_t)tile * 16 * srow : 0), kAffine ? rows * srow : 0);
      auto get = [&](rsrc_t p, uint32_t* v) __attribute__((always_inline)) {
        if constexpr (kRec == 1) {
          v[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(p, soff, first * Sc::kStep, 0);
        } else {
          const auto u = __builtin_amdgcn_raw_buffer_load_b64(p, soff, first * Sc::kStep, 0);
          v[0] = (uint32_t)u[0];
          v[1] = (uint32_t)u[1];
        }
      };
      get(sr, r.s);
      if constexpr (kAffine) get(br, r.b);
    } else {
      const size_t row = min(tile * 16 + n16, a.N - 1);
      const int step = first + min(kb, S - 1);
      lin_scales_any<kRec>(a.s + row * srow, step, srow, r.s);
      if constexpr (kAffine) lin_scales_any<kRec>(a.b + row * srow, step, srow, r.b);
    }
  };

  // x comes through LDS: contiguous 16-byte pieces in, operands out (each
  // wave its own inputs).
  lin_u32x4 xf[S][4][kX];
  auto load_x = [&]() __attribute__((always_inline)) {
    // reads past the range give zeros: inputs past the row's end or this split's lie there
    const int rows = min(a.L - t0, kSep ? 4 : 16);
    const rsrc_t xr = make_rsrc(a.x + (size_t)t0 * a.ldx, (uint32_t)((rows - 1) * (uint32_t)a.ldx + a.K) * 2u);
    const int room = min(a.K, steps * kLinStep) - first * kLinStep;  // inputs of this wave's steps that count
    lin_u32x4* const mine = xstage[wave];
    constexpr int kPieces = kStageSteps * 16;  // of a token
#pragma unroll
    for (int s0 = 0; s0 < S; s0 += kStageSteps) {
      constexpr int kLoads = (kStageTokens * kPieces + 63) / 64;
      lin_u32x4 in[kLoads];  // all on their way before the first is used
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const int i = 64 * l + lane, t = i / kPieces, c = s0 * kLinStep + (i - t * kPieces) * 8;
        const uint32_t at = t < rows && c < room ? ((uint32_t)t * (uint32_t)a.ldx + c) * 2u : 0x80000000u;
        in[l] = __builtin_bit_cast(lin_u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, at, first * kLinStep * 2, 0));
      }
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        lin_u32x4 v = in[l];
        if constexpr (kAffine)  // the codes' pair order
          v = lin_u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                        __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
        if (64 * l + lane < kStageTokens * kPieces) mine[64 * l + lane] = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int t = kSep ? n16 >> 2 : n16;
      const bool live = t < rows && (!kSep || (n16 & 3) == kb);
#pragma unroll
      for (int st = s0; st < s0 + kStageSteps; ++st)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // operand register j: after the transpose block j's inputs, else word j of block kb
          const int piece = t * kPieces + (st - s0) * 16 + (kTurn ? 4 * j + kb : 4 * kb + j);
          xf[st][j][0] = live ? mine[piece] : lin_u32x4{0, 0, 0, 0};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int st = 0; st < S; ++st)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kTerms) lin_two_terms(xf[st][j][0], xf[st][j][0], xf[st][j][kX - 1]);
      }
    if constexpr (kAffine) {  // x times ones is the group sums, in the layout of the products
      const uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
      const lin_u32x4 ones = {one, one, one, one};
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
  auto multiply = [&](const Rows& r) __attribute__((always_inline)) {
    // this lane's scales of each step
    uint32_t sv[S][Sc::kWords], bv[kAffine ? S : 1][Sc::kWords];
    auto spread = [&](const uint32_t* rec, uint32_t (*v)[Sc::kWords]) __attribute__((always_inline)) {
      uint32_t u[S][kRec];
#pragma unroll
      for (int w = 0; w < kRec; ++w) {
        uint32_t one[S];
        lin_spread<S>(rec[w], one);
#pragma unroll
        for (int st = 0; st < S; ++st) u[st][w] = one[st];
      }
#pragma unroll
      for (int st = 0; st < S; ++st) {
        if constexpr (!Sc::kOwn) {
#pragma unroll
          for (int w = 0; w < Sc::kWords; ++w) v[st][w] = u[st][w];
        } else if constexpr (kRec == 1) {
          v[st][0] = (u[st][0] >> (8 * kb)) & 255u;
        } else {
          // (a selection between the two would become an indexed array in memory)
          const uint32_t upper = 0u - (uint32_t)(kb >> 1);
          v[st][0] = ((u[st][kRec - 1] & upper) | (u[st][0] & ~upper)) >> (16 * (kb & 1));
        }
      }
    };
    if (first < steps) {
      spread(r.s, sv);
      if constexpr (kAffine) spread(r.b, bv);
    }
#pragma unroll
    for (int st = 0; st < S; ++st) {
      if (first + st >= steps) break;
      uint32_t w4[4] = {r.c[st][0], r.c[st][1], r.c[st][2], r.c[st][3]};
      const float* xs = xsum + (wave * S + st) * kGroups * 16;
      if constexpr (FMT == kLinMxfp4) {
        const float s = lin_e8m0(sv[st][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = lin_fp4_pow2<false>(w4[j], s);
#pragma unroll
          for (int i = 0; i < kX; ++i) acc = lin_mfma<false>(xf[st][j][i], w, acc);
        }
      } else if constexpr (FMT == kLinNvfp4 && !FEW) {
        const float s0 = lin_e4m3<0>(sv[st][0]), s1 = lin_e4m3<1>(sv[st][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = lin_mfma<F16>(xf[st][j][0], lin_fp4_scaled<F16>(w4[j], j < 2 ? s0 : s1), acc);
      } else if constexpr (FMT == kLinNvfp4) {
        lin_f32x4 c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0};  // the first and the second 16 inputs of the blocks
        c0 = lin_mfma<F16>(xf[st][0][0], lin_fp4<F16>(w4[0]), c0);
        c1 = lin_mfma<F16>(xf[st][2][0], lin_fp4<F16>(w4[2]), c1);
        c0 = lin_mfma<F16>(xf[st][1][0], lin_fp4<F16>(w4[1]), c0);
        c1 = lin_mfma<F16>(xf[st][3][0], lin_fp4<F16>(w4[3]), c1);
        const uint32_t s0 = sv[st][0], s1 = sv[st][1];
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
            const float s = half(sv[st], g), off = __builtin_fmaf(-16.0f, s, half(bv[st], g));
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
            const float s = half(sv[st], g), off = __builtin_fmaf(-16.0f, s, half(bv[st], g));
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
  constexpr int kParts = W / 4;  // threads of an output, four waves' sums each
  const int o = threadIdx.x / kParts, part = threadIdx.x % kParts;
  const int at = 4 * part * kAcc * 64 + (kSep ? o : 4 * ((o & 15) + 16 * (o >> 6)) + ((o >> 4) & 3));
  const int ot = t0 + (o >> 4);
  const bool writes = part == 0 && ot < a.L;
  auto finish = [&](int tile, float* buf) __attribute__((always_inline)) {
    if constexpr (kSep)
      buf[wave * 64 + lane] = acc[0];
    else
      *reinterpret_cast<lin_f32x4*>(buf + wave * 256 + 4 * lane) = acc;
    acc = lin_f32x4{0, 0, 0, 0};
    __syncthreads();
    if (kSep && o >= 64) return;  // whole waves
    const float* r = buf + at;
    constexpr int kWave = kAcc * 64;
    float v = (r[0] + r[kWave]) + (r[2 * kWave] + r[3 * kWave]);
    if constexpr (kParts >= 2) v += dpp_f32<0xB1>(v);  // lane ^ 1
    if constexpr (kParts >= 4) v += dpp_f32<0x4E>(v);  // lane ^ 2
    const int n = tile * 16 + (o & 15);
    if (writes && n < a.N) {
      if (a.part) {
        a.part[((size_t)blockIdx.z * a.L + ot) * a.N + n] = v;
      } else {
        if (a.bias) v += a.bias[n];
        lin_store(a.out, (size_t)ot * a.ldo + n, a.out_dtype, v);
      }
    }
  };

  Rows ring[kDeep];
  int tile = blockIdx.x;
#pragma unroll
  for (int d = 0; d < kDeep; ++d)
    if (tile + d * (int)gridDim.x < tiles) load(tile + d * gridDim.x, ring[d]);
  load_x();
  float *buf = &red[0][0][0], *other = &red[1][0][0];
  while (true) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      multiply(ring[d]);
      if (tile + kDeep * (int)gridDim.x < tiles) load(tile + kDeep * gridDim.x, ring[d]);
      finish(tile, buf);
      float* const t = buf;
      buf = other;
      other = t;
      tile += gridDim.x;
      if (tile >= tiles) return;
    }
  }
}

struct RowsPlan {
  int W, S, splits, split_steps;
  bool plain;
};
// The longest K of one workgroup is 16 waves x 3 steps (2 where x takes two
// operands), longer ones are split evenly.  Where a workgroup has a tile of
// rows or two, as many waves as there are steps; where it has many, so few
// that each wave has two or three steps, and several workgroups share a
// compute unit, whose barriers then overlap (mxfp4 1 x 131072 x 2048 28.8 us,
// 37.0 with 16 waves; 9000 rows of 2944 inputs 8.2 with three steps a wave,
// 7.1 with 16 waves of two).
inline RowsPlan rows_plan(int fmt, bool f16, int N, int K, bool words) {
  RowsPlan p{};
  p.plain = K % kLinStep == 0 && words;
  const int steps = (K + kLinStep - 1) / kLinStep;
  const int most = fmt == kLinMxfp4 && f16 ? 2 : 3;
  const int per = N <= 12288 ? 1 : N <= 32768 ? 2 : most;  // steps of a wave
  p.W = steps <= 4 * per ? 4 : steps <= 8 * per && p.plain ? 8 : 16;
  p.splits = (steps + 16 * most - 1) / (16 * most);
  p.split_steps = (steps + p.splits - 1) / p.splits;
  p.splits = (steps + p.split_steps - 1) / p.split_steps;
  p.S = (p.split_steps + p.W - 1) / p.W;
  return p;
}

template <int FMT, bool F16>
void launch_linear_rows(const LinearArgs& args, const RowsPlan& p, hipStream_t stream) {
  LinearArgs a = args;
  a.split_steps = p.split_steps;
  const int tiles = (a.N + 15) / 16;
  // As many workgroups as run at once, also where their shares of the tiles
  // then differ by one (against even shares on fewer: 7 x 4099 x 4096, 257
  // tiles, 9.4 us and 10.5; 1 x 4096 x 14336 15.2 and 18.7; 1 x 6144 x 6144,
  // 384 tiles, 9.9 and 9.8).
  const int most = 4096 / p.W / p.splits;
  const dim3 grid(std::max(1, std::min(tiles, most)), (a.L + 15) / 16, p.splits), block(64 * p.W);
  const bool few = a.L <= 4;
#define MOE_LINEAR_ROWS(FEW, PLAIN, S, W) \
  hipLaunchKernelGGL((k_linear_rows<FMT, F16, FEW, PLAIN, S, W>), grid, block, 0, stream, a)
#define MOE_LINEAR_ROWS_W(FEW, PLAIN, W)               \
  if (p.S == 1) {                                      \
    MOE_LINEAR_ROWS(FEW, PLAIN, 1, W);                 \
  } else if (p.S == 2) {                               \
    MOE_LINEAR_ROWS(FEW, PLAIN, 2, W);                 \
  } else if constexpr (!(FMT == kLinMxfp4 && F16)) {   \
    MOE_LINEAR_ROWS(FEW, PLAIN, 3, W);                 \
  }
#define MOE_LINEAR_ROWS_S(FEW, PLAIN)                  \
  if (p.W == 4) {                                      \
    MOE_LINEAR_ROWS_W(FEW, PLAIN, 4)                   \
  } else if (PLAIN && p.W == 8) {                      \
    MOE_LINEAR_ROWS_W(FEW, true, 8)                    \
  } else {                                             \
    MOE_LINEAR_ROWS_W(FEW, PLAIN, 16)                  \
  }
  if constexpr (FMT != kLinMxfp4) {
    if (few) {
      if (p.plain) {
        MOE_LINEAR_ROWS_S(true, true)
      } else {
        MOE_LINEAR_ROWS_S(true, false)
      }
      return;
    }
  }
  if (p.plain) {
    MOE_LINEAR_ROWS_S(false, true)
  } else {
    MOE_LINEAR_ROWS_S(false, false)
  }
#undef MOE_LINEAR_ROWS_S
#undef MOE_LINEAR_ROWS_W
#undef MOE_LINEAR_ROWS
}

// Inputs shorter than a step: one thread an output (1 x 16 x 64 4.9 us, 16 x
// 4096 x 64 6.0; 16 x 65536 x 64 67, bound by its vector instructions).
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
