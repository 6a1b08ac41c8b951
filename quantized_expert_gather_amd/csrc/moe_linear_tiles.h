// Dense 4-bit product for many tokens: tiles of 16 MT tokens x 64 NT weight
// rows on the matrix cores, K in steps of 128.  Internal header.
//
// Every weight is made one exact 16-bit operand, so the products add up over
// all of K in the accumulators with no work per scale group:
//   nvfp4    e2m1 * e4m3, exact in both types;
//   mxfp4    e2m1 * 2^e: exact in bf16; in fp16 with e counted from the row's
//            largest, whose power of two multiplies the row's result (exact
//            for the 35 powers of two below it; tiles with a wide row, one
//            with other codes than 0 below these, see `wide`);
//   affine   s * (q - 8): 8 + 3 significant bits, exact in fp16's 11, with s
//            divided by a power of two near its row's largest (down to 2^-26
//            of that; rows with smaller scales are wide too).  bf16 tokens
//            are divided by a power of two near their largest value likewise
//            and held in fp16.  Their values 2^-32 below it lose bits, 2^-25
//            each where the largest is at least 2^14: with the operands' 8 s
//            2^-39 of what a row's largest scale gives the largest value.  In
//            rows whose scales lie within 2^12 of one another that is 2^-27
//            of what the largest value does give, below fp32's own rounding;
//            tiles with another row and such a token go the wide rows' way.
// The affine rest, sum over groups of (b + 8 s) X with X = sum of the group's
// x, is a product over K / group columns in bf16 terms; it starts the
// accumulators.  b + 8 s is two terms, exact to fp32's rounding: of two
// numbers of 8 bits, d powers of two apart, the sum has at most 9 + d bits
// and what is left of it beside its first 8 at most 8, or, further apart, is
// the smaller one.  X is three terms, fp32's 24 bits (two would leave it 16
// and save 6 of 110 us for affine4_g32 2048 x 4096 x 4096, bf16, and at most
// 1 of 134 for affine4_g64 2048 x 6144 x 4096).
//
// Bound by matrix instructions with the decoding beside them: in a row of
// calls 2048 x 6144 x 4096 takes 97 us for mxfp4 (1065 TFLOP/s; 4 conversions
// per 8 weights), 117 for nvfp4 (880; 16 more multiplications and packings),
// 134 to 139 from card to card for affine4_g64 (11 instructions per 8 weights,
// 10 of these us the preparation); a bf16 library product of these sizes takes
// 87.  With few tiles the latency of a step's loads, one step ahead, bounds
// it: 96 x 2050 x 4096 nvfp4 11.3 us and 3.9 for joining the splits (12.4 in a
// row of calls).
//
// A wave holds 16 NT rows' codes in registers, one step ahead; the tokens'
// step (of affine weights: blocks of 16 tokens x 128 inputs, laid out first)
// is copied into LDS without passing registers, 16-byte pieces of a row
// XORed with the row so that the 16 rows of an operand read fall in
// different banks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_linear_device.h"
#include "moe_q4.h"

namespace moeq4 {

struct TilesArgs {
  const uint16_t* x;       // tokens in operand type and order
  const uint16_t* xraw;    // tokens as given, ldx apart
  const uint32_t* w;
  const unsigned char* s;  // scales as given
  const unsigned char* b;  // biases as given (affine)
  const uint16_t* sh;      // affine: fp16 scales over their row's power of two [N][Gp]
  const uint16_t* tsum;    // affine: bf16 terms of b + 8 s [2][N][Gp]
  const uint16_t* xsum;    // affine: bf16 terms of the group sums [3][L][Gp]
  const int32_t* xexp;     // power of two of each token (affine with bf16 tokens) and kLinWide, or NULL
  const int32_t* wexp;     // power of two of each row (affine; mxfp4 with fp16 tokens), kLinWide and kLinUneven, or NULL
  const float* bias;
  void* out;
  float* part;             // split K: [splits][L][N] partial sums
  long long ldx, ldo;
  int L, N, K, G, Gp;
  int out_dtype;
  int splits, steps_per;   // steps of 128 inputs of each split
  int stagger;             // steps between the token tiles' first ones
  int row_tiles, tok_tiles;
};

// A row's power of two is the low half of its word, the marks lie above.
constexpr int kLinWide = 1 << 16;    // one fp16 power of two does not fit the row (or token)
constexpr int kLinUneven = 1 << 17;  // scales 2^-12 and more below the row's largest
__device__ __forceinline__ int lin_exponent(int v) { return (int)(int16_t)v; }

__device__ __forceinline__ lin_f16x2 lin_h2(uint32_t v) { return __builtin_bit_cast(lin_f16x2, v); }
__device__ __forceinline__ uint32_t lin_u(lin_f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// s * (q - 8) of a word's codes in fp16: one fused multiply-add a pair, its
// addend -24 s exact (10 significant bits) and its result too.
__device__ __forceinline__ uint4 lin_affine_f16(uint32_t w, LinCode code, lin_f16x2 s, lin_f16x2 m24s) {
  const uint4 c = lin_codes16<true>(w, code);
  return make_uint4(lin_u(__builtin_elementwise_fma(lin_h2(c.x), s, m24s)), lin_u(__builtin_elementwise_fma(lin_h2(c.y), s, m24s)),
                    lin_u(__builtin_elementwise_fma(lin_h2(c.z), s, m24s)), lin_u(__builtin_elementwise_fma(lin_h2(c.w), s, m24s)));
}

// q - 8 of a word's codes, exact, in lin_codes16's order.
template <bool F16>
__device__ __forceinline__ uint4 lin_centred(uint32_t w, LinCode code) {
  if constexpr (F16) {
    const lin_f16x2 one = {(_Float16)1.0f, (_Float16)1.0f}, m24 = {(_Float16)-24.0f, (_Float16)-24.0f};
    return lin_affine_f16(w, code, one, m24);
  } else {
    const uint4 c = lin_codes16<false>(w, code);
    auto two = [](uint32_t v) {
      return __builtin_amdgcn_perm(__float_as_uint(bf16_hi_to_f32(v) - 24.0f), __float_as_uint(bf16_lo_to_f32(v) - 24.0f), 0x07060302u);
    };
    return make_uint4(two(c.x), two(c.y), two(c.z), two(c.w));
  }
}

// The scale of a row's 32 inputs from k on (nvfp4: two scales), as stored.
template <int FMT>
__device__ __forceinline__ uint32_t tile_scale(const unsigned char* base, uint32_t row, int k) {
  if constexpr (FMT == kLinMxfp4)
    return base[row + (uint32_t)(k / 32)];
  else if constexpr (FMT == kLinNvfp4)
    return *reinterpret_cast<const uint16_t*>(base + (row + (uint32_t)(k / 16)));
  else
    return *reinterpret_cast<const uint16_t*>(base + (row + 2u * (uint32_t)(k / lin_group(FMT))));
}

// Stores the first `left` (at least one) of four neighbours.
template <class T>
__device__ __forceinline__ void store4(T* p, int left, T a, T b, T c, T d) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  if (left >= 4 && ((uintptr_t)p & (sizeof(t4) - 1)) == 0) {
    *reinterpret_cast<t4*>(p) = t4{a, b, c, d};
  } else {
    p[0] = a;
    if (left > 1) p[1] = b;
    if (left > 2) p[2] = c;
    if (left > 3) p[3] = d;
  }
}

template <int FMT, bool F16, int MT, int NT>
__global__ __launch_bounds__(256, 2) void k_linear_tiles(TilesArgs a) {
  constexpr int kTok = 16 * MT, kRows = 64 * NT;
  constexpr bool kTiledX = lin_affine(FMT);  // the laid-out copy
  __shared__ int wide_waves[4];
  // Two objects, each named where it is used: the compiler then knows that
  // reads of one do not wait for the copies into the other.
  __shared__ __attribute__((aligned(1024))) unsigned char lds0[kTok * 256], lds1[kTok * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n16 = lane & 15, kb = lane >> 4;

  // Workgroups b, b + 8, ... share an XCD (and its L2): each XCD takes a
  // contiguous run of the tiles, tokens fastest, so it reads an eighth of the
  // weights.
  const int tiles = a.row_tiles * a.tok_tiles;
  int tile = blockIdx.x;
  {
    const int per = tiles / 8, rest = tiles % 8, xcd = tile & 7, at = tile >> 3;
    tile = xcd * per + min(xcd, rest) + at;
  }
  const int tok0 = (tile % a.tok_tiles) * kTok;
  const int row0 = (tile / a.tok_tiles) * kRows + wave * 16 * NT;
  const int split = blockIdx.y;
  const int all = (a.K + kLinStep - 1) / kLinStep;
  const int step0 = split * a.steps_per, step1 = min(all, step0 + a.steps_per);

  size_t row[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) row[nt] = min(row0 + 16 * nt + n16, a.N - 1);

  lin_f32x4 acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = lin_f32x4{0, 0, 0, 0};

  if constexpr (!lin_affine(FMT)) {
    // hides the zeros: as known constants the compiler carries them through the loop in registers of their own
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) asm volatile("" : "+v"(acc[mt][nt]));
  }
  // whether rows, and tokens, have powers of two
  constexpr bool kScaled = lin_affine(FMT) || (FMT == kLinMxfp4 && F16), kTokens = lin_affine(FMT) && !F16;
  int wexp[NT], marks = 0;
  if constexpr (kScaled) {  // the same lanes' rows as the codes'
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      wexp[nt] = a.wexp[row[nt]];
      marks |= wexp[nt];
      wexp[nt] = lin_exponent(wexp[nt]);
    }
  }

  if constexpr (lin_affine(FMT)) {
    // This split's share of the groups (all of them in the first split: 262 x
    // 728 x 12288 takes 42 us, the shares 31).
    const int chunks = a.Gp / 32;
    const int g0 = 32 * (int)((long)chunks * split / a.splits), g1 = 32 * (int)((long)chunks * (split + 1) / a.splits);
    if (g0 < g1) {
      // sum over groups of t X, t = b + 8 s, by their bf16 terms (the last of
      // t times the last of X is below fp32's rounding)
#pragma unroll 1
      for (int g = g0 + 8 * kb; g < g1; g += 32) {
        uint4 tf[2][NT], xf[3][MT];
        auto load_t = [&](int i) __attribute__((always_inline)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) tf[i][nt] = *reinterpret_cast<const uint4*>(a.tsum + ((size_t)i * a.N + row[nt]) * a.Gp + g);
        };
        auto load_x = [&](int i) __attribute__((always_inline)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            xf[i][mt] = *reinterpret_cast<const uint4*>(a.xsum + ((size_t)i * a.L + min(tok0 + 16 * mt + n16, a.L - 1)) * a.Gp + g);
        };
        auto add = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = lin_mfma<false>(tf[i][nt], xf[j][mt], acc[mt][nt]);
        };
        load_t(0); load_t(1); load_x(0);
        add(0, 0); add(1, 0);
        load_x(1);
        add(0, 1);
        add(1, 1);
        __builtin_amdgcn_sched_barrier(0);  // all of X at once would not fit the registers
        load_x(2);
        add(0, 2);
      }
      // into the operands' units
      int we[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) we[nt][i] = __shfl(wexp[nt], 4 * kb + i, 64);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        int xe = 0;
        if constexpr (kTokens) xe = lin_exponent(a.xexp[min(tok0 + 16 * mt + n16, a.L - 1)]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[mt][nt][i] = __builtin_amdgcn_ldexpf(acc[mt][nt][i], -xe - we[nt][i]);
      }
    }
  }

  // Pieces of a step's tokens: LDS slot i holds piece (i % 16) ^ (row % 16) of
  // token i / 16.  Addresses are a base that the wave shares and 32-bit
  // offsets, which take half the registers of pointers.
  constexpr int kCopies = kTok / 16;
  const int piece = (tid & 15) ^ ((tid >> 4) & 15);
  const unsigned char* xbase = reinterpret_cast<const unsigned char*>(a.x) +
                               (kTiledX ? (size_t)(tok0 / 16) * all * (16 * kLinStep * 2) : (size_t)tok0 * a.ldx * 2);
  uint32_t xoff[kTiledX ? 1 : kCopies];
  if constexpr (kTiledX) {
    xoff[0] = (tid >> 4) * (kLinStep * 2) + piece * 16;
  } else {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) xoff[c] = (uint32_t)(min(tok0 + 16 * c + (tid >> 4), a.L - 1) - tok0) * (uint32_t)(2 * a.ldx);
  }
  auto stage = [&](int step, unsigned char* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const unsigned char* src;
      if constexpr (kTiledX)
        src = xbase + ((size_t)c * all + step) * (16 * kLinStep * 2) + xoff[0];
      else
        src = xbase + (xoff[c] + 2u * (uint32_t)min(step * kLinStep + piece * 8, a.K - 8));
      // a wave's 64 pieces go to 1 KB of LDS from its first slot on
      unsigned char* dst = buf + (c * 256 + wave * 64) * 16;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                       (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
    }
  };
  const int rows0 = __builtin_amdgcn_readfirstlane(min(row0, a.N - 1));
  const uint32_t scale_row = lin_affine(FMT) ? 2 * a.Gp : a.G;  // bytes
  const unsigned char* wbase = reinterpret_cast<const unsigned char*>(a.w) + (size_t)rows0 * ((size_t)a.K / 2);
  const unsigned char* sbase = (lin_affine(FMT) ? reinterpret_cast<const unsigned char*>(a.sh) : a.s) + (size_t)rows0 * scale_row;
  uint32_t woff[NT], soff[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    woff[nt] = (uint32_t)((int)row[nt] - rows0) * (uint32_t)(a.K / 2);
    soff[nt] = (uint32_t)((int)row[nt] - rows0) * scale_row;
  }
  auto load = [&](int step, lin_u32x4 (&cw)[NT], uint32_t (&sw)[NT]) __attribute__((always_inline)) {
    const int k = min(step * kLinStep + 32 * kb, a.K - 32);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      cw[nt] = *reinterpret_cast<const lin_u32x4*>(wbase + (woff[nt] + (uint32_t)(k / 2)));
      sw[nt] = tile_scale<FMT>(sbase, soff[nt], k);
    }
  };

  lin_u32x4 cw[NT];
  uint32_t sw[NT];
  // Rows whose length is a power of two put one step's pieces of all rows on
  // a few memory channels: token tiles start at different steps, round the
  // end to the beginning, so the tiles that run together read different ones.
  const int count = step1 - step0;
  int step = count > 0 ? step0 + (tile % a.tok_tiles) * a.stagger % count : 0;
  int token_marks = 0, more_marks = 0;
  if constexpr (kTokens) {
    token_marks = a.xexp[min(tok0 + lane, a.L - 1)];
    if constexpr (kTok > 64) more_marks = a.xexp[min(tok0 + 64 + lane, a.L - 1)];
  }
  if (count > 0) {
    stage(step, lds0);
    load(step, cw, sw);
  }

  __builtin_amdgcn_s_waitcnt(0);
  if constexpr (kScaled) {
    const int wide_wave = __any(marks & kLinWide) || (__any(marks & kLinUneven) && __any((token_marks | more_marks) & kLinWide));
    if (lane == 0) wide_waves[wave] = wide_wave;
    __builtin_amdgcn_s_waitcnt(0);
  }
  __syncthreads();
  const LinCode code = lin_code<true>();
  int i = 0;
  auto body = [&](unsigned char* xb, unsigned char* other) __attribute__((always_inline)) {
    lin_u32x4 cn[NT];
    uint32_t sn[NT];
    const int next = step + 1 < step1 ? step + 1 : step0;
    if (i + 1 < count) {
      stage(next, other);
      load(next, cn, sn);
    }
    const bool dead = step * kLinStep + 32 * kb >= a.K;  // past the row's end
    float sf[NT][2];
    lin_f16x2 sv[NT], sm[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (FMT == kLinNvfp4) {
        sf[nt][0] = dead ? 0.0f : e4m3_to_f32(sw[nt] & 255u);
        sf[nt][1] = dead ? 0.0f : e4m3_to_f32(sw[nt] >> 8);
      } else if constexpr (FMT == kLinMxfp4) {
        if (dead) cw[nt] = lin_u32x4{0, 0, 0, 0};
        if constexpr (F16) {  // counted from the row's largest exponent; 255 stands for NaN
          const int e = max((int)sw[nt] - 127 - wexp[nt], -126);
          sf[nt][0] = sw[nt] == 255u ? __builtin_nanf("") : __int_as_float((e + 127) << 23);
        } else {
          sf[nt][0] = lin_e8m0(sw[nt]);
        }
      } else {
        sv[nt] = lin_h2(dead ? 0u : sw[nt] | sw[nt] << 16);
        sm[nt] = sv[nt] * lin_f16x2{(_Float16)-24.0f, (_Float16)-24.0f};
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 wf[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (FMT == kLinNvfp4)
          wf[nt] = lin_fp4_scaled<F16>(cw[nt][j], sf[nt][j >> 1]);
        else if constexpr (FMT == kLinMxfp4)
          wf[nt] = lin_fp4_pow2<F16>(cw[nt][j], sf[nt][0]);
        else
          wf[nt] = lin_affine_f16(cw[nt][j], code, sv[nt], sm[nt]);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const uint4 xf = *reinterpret_cast<const uint4*>(xb + (16 * mt + n16) * 256 + (((4 * kb + j) ^ n16) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = lin_mfma<lin_affine(FMT) || F16>(wf[nt], xf, acc[mt][nt]);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    step = next;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      cw[nt] = cn[nt];
      sw[nt] = sn[nt];
    }
    ++i;
  };
  while (i < count) {
    body(lds0, lds1);
    if (i >= count) break;
    body(lds1, lds0);
  }

  // A workgroup with a wide row, or an uneven row and a wide token, starts
  // again: its tokens from memory as they are, every product exact, and the
  // sums in their own units.  mxfp4: the blocks' powers of two in bf16
  // operands, x as two bf16 terms.  Affine: the words transposed over the
  // lanes, so that a product is one group's, and its fp32 sum times the scale,
  // plus b + 8 s times the group's sum of x.  Here and not in place of the
  // loop above, whose registers it would share.  (2048 x 6144 x 4096 with such
  // a row in every tile: mxfp4 476 us, 102 with none; affine4_g64 826 and 137,
  // 128 tokens x 4096 x 4096 53 and 23.)
  bool wide = false;
  if constexpr (kScaled) {
    wide = (wide_waves[0] | wide_waves[1] | wide_waves[2] | wide_waves[3]) != 0;
    if (wide) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[mt][nt] = lin_f32x4{0, 0, 0, 0};
          asm volatile("" : "+v"(acc[mt][nt]));  // (hides the zeros, as above)
        }
      uint32_t from[MT];  // (the last token's rows stand for those past it)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) from[mt] = (uint32_t)(min(tok0 + 16 * mt + n16, a.L - 1) - tok0) * (uint32_t)(2 * a.ldx);
      const unsigned char* xrow = reinterpret_cast<const unsigned char*>(a.xraw) + (size_t)tok0 * a.ldx * 2;
      auto piece_at = [&](int mt, int k) __attribute__((always_inline)) {  // eight inputs of token n16 of a tile
        return *reinterpret_cast<const lin_u32x4*>(xrow + (from[mt] + 2u * (uint32_t)k));
      };
      if constexpr (lin_affine(FMT)) {
        constexpr int kPer = lin_group(FMT) / 32, kGroups = 4 / kPer;  // blocks of a group, groups of a step
        const LinCode own = lin_code<F16>();
        const uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
        const uint4 ones = make_uint4(one, one, one, one);
#pragma unroll 1
        for (int s = step0; s < step1; ++s) {
          load(s, cw, sw);
          // one row tile at a time, and its tokens again: what that takes fits the registers beside the sums
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t words[4] = {cw[nt][0], cw[nt][1], cw[nt][2], cw[nt][3]};
            lin_transpose(words);
#pragma unroll 1
            for (int g = 0; g < kGroups; ++g) {
              const int group = s * kGroups + g;
              if (group >= a.G) break;
              uint4 wf[kPer];
#pragma unroll
              for (int p = 0; p < kPer; ++p) wf[p] = lin_centred<F16>(words[p], own);
#pragma unroll
              for (int j = 0; j + kPer < 4; ++j) words[j] = words[j + kPer];  // the next group's
              float scale[4], rest[4];  // s and b + 8 s of the rows whose sums the lane holds
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const size_t at = (size_t)min(row0 + 16 * nt + 4 * kb + e, a.N - 1) * a.G + group;
                scale[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.s)[at]);
                rest[e] = __builtin_fmaf(8.0f, scale[e], bf16_to_f32(reinterpret_cast<const uint16_t*>(a.b)[at]));
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                lin_f32x4 c = {0, 0, 0, 0}, sum = {0, 0, 0, 0};  // sum: of the token's x, the same in all four
#pragma unroll
                for (int p = 0; p < kPer; ++p) {
                  const uint4 xf = lin_pair_order(__builtin_bit_cast(uint4, piece_at(mt, s * kLinStep + 32 * (g * kPer + p) + 8 * kb)));
                  c = lin_mfma<F16>(wf[p], xf, c);
                  sum = lin_mfma<F16>(ones, xf, sum);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  acc[mt][nt][e] = __builtin_fmaf(scale[e], c[e], __builtin_fmaf(rest[e], sum[e], acc[mt][nt][e]));
                if (mt % 2) __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
        }
      } else {
#pragma unroll 1
        for (int s = step0; s < step1; ++s) {
          load(s, cw, sw);
          const int k = s * kLinStep + 32 * kb;
          const bool dead = k >= a.K;
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint4 wf[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t c01 = j & 1 ? cw[nt][1] : cw[nt][0], c23 = j & 1 ? cw[nt][3] : cw[nt][2];
              wf[nt] = lin_fp4_pow2<false>(dead ? 0u : j & 2 ? c23 : c01, lin_e8m0(sw[nt]));
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              lin_u32x4 x = {0, 0, 0, 0}, hi, lo;
              if (!dead) x = piece_at(mt, k + 8 * j);
              lin_two_terms(x, hi, lo);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                acc[mt][nt] = lin_mfma<false>(wf[nt], hi, acc[mt][nt]);
                acc[mt][nt] = lin_mfma<false>(wf[nt], lo, acc[mt][nt]);
              }
            }
          }
        }
      }
    }
  }

  // Lane (n16, kb) holds token n16 of each token tile and rows 4 kb .. + 3 of
  // each row tile.  Through LDS (the waves' own shares, some token tiles at
  // a time) it comes to hold four neighbouring rows of a token whose other
  // rows the next lanes hold.
  // token tiles of a pass, 16-byte pieces of a token's rows; two waves' share fits each buffer
  constexpr int kHalf = NT > 2 ? MT / 2 : MT, kPass = kHalf < 4 ? kHalf : 4, kQuads = 4 * NT;
  static_assert(2 * kPass * 16 * kQuads * 16 <= kTok * 256, "the waves' output fits the token buffers");
  const int units = wide ? 0 : -1;  // (a mask: a branch here would part the loads below)
  unsigned char* mine = (wave < 2 ? lds0 : lds1) + (wave & 1) * (kPass * 16 * kQuads * 16);
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += kPass) {
#pragma unroll
    for (int mt = 0; mt < kPass; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<lin_f32x4*>(mine + ((16 * mt + n16) * kQuads + (4 * nt + kb + n16) % kQuads) * 16) =
            acc[m0 + mt][nt];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
    for (int i = lane; i < kPass * 16 * kQuads; i += 64) {
      const int tt = i / kQuads, quad = i % kQuads;
      const int t = tok0 + 16 * m0 + tt, n = row0 + 4 * quad;
      const lin_f32x4 v4 = *reinterpret_cast<const lin_f32x4*>(mine + (tt * kQuads + (quad + (tt & 15)) % kQuads) * 16);
      if (t >= a.L || n >= a.N) continue;
      float v[4] = {v4[0], v4[1], v4[2], v4[3]};
      if constexpr (kScaled) {
        int xe = 0;
        if constexpr (kTokens) xe = lin_exponent(a.xexp[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = __builtin_amdgcn_ldexpf(v[e], (xe + lin_exponent(a.wexp[min(n + e, a.N - 1)])) & units);
      }
      if (a.splits > 1) {
        store4<float>(a.part + ((size_t)split * a.L + t) * a.N + n, a.N - n, v[0], v[1], v[2], v[3]);
        continue;
      }
      if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += a.bias[min(n + e, a.N - 1)];
      }
      const size_t at = (size_t)t * a.ldo + n;
      if (a.out_dtype == MOE_Q4_DTYPE_F32)
        store4<float>(static_cast<float*>(a.out) + at, a.N - n, v[0], v[1], v[2], v[3]);
      else if (a.out_dtype == MOE_Q4_DTYPE_BF16)
        store4<uint16_t>(static_cast<uint16_t*>(a.out) + at, a.N - n, (uint16_t)f32_to_bf16_rne(v[0]),
                         (uint16_t)f32_to_bf16_rne(v[1]), (uint16_t)f32_to_bf16_rne(v[2]), (uint16_t)f32_to_bf16_rne(v[3]));
      else
        store4<_Float16>(static_cast<_Float16*>(a.out) + at, a.N - n, (_Float16)v[0], (_Float16)v[1], (_Float16)v[2],
                         (_Float16)v[3]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// v as bf16 terms, each the nearest to what the ones before leave.
template <int N>
__device__ __forceinline__ void split_terms(float v, uint32_t (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = f32_to_bf16_rne(v);
    v -= bf16_lo_to_f32(t[i]);
  }
}

// Largest and smallest of pairs of 16-bit numbers.
typedef unsigned short lin_u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t lin_max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(lin_u16x2, a), __builtin_bit_cast(lin_u16x2, b)));
}
__device__ __forceinline__ uint32_t lin_min2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(lin_u16x2, a), __builtin_bit_cast(lin_u16x2, b)));
}
__device__ __forceinline__ uint32_t lin_sub2(uint32_t a, uint32_t b) {  // each wraps for itself
  return __builtin_bit_cast(uint32_t, (lin_u16x2)(__builtin_bit_cast(lin_u16x2, a) - __builtin_bit_cast(lin_u16x2, b)));
}
// A pair's largest and the inverse of another's smallest as one pair, whose
// reduction by lin_max2 serves both.
__device__ __forceinline__ uint32_t lin_ends(uint32_t most, uint32_t least) {
  return max(most & 0xFFFFu, most >> 16) << 16 | (0xFFFFu - min(least & 0xFFFFu, least >> 16));
}

// Lays out what the tiles read besides codes and tokens.  One workgroup a
// token (affine): its power of two, the fp16 copy in the codes' pair order
// and the group sums' bf16 terms.  row_lanes threads a weight row (affine, and
// mxfp4 with fp16 tokens), eight groups each at a time: its power of two, the
// fp16 scales and b + 8 s in bf16 terms (112843 rows of 24 groups: 9.7 us;
// of 12 groups, with a wave a row and a group a lane, 29.8).
struct PrepareArgs {
  const uint16_t* x;
  const uint32_t* w;
  const unsigned char* s;
  const unsigned char* b;
  uint16_t* xq;
  uint16_t* xsum;
  uint16_t* tsum;
  int32_t* xexp;
  uint16_t* sh;
  int32_t* wexp;
  long long ldx;
  int L, N, K, G, Gp;
  int row_lanes;  // a power of two, 64 at most
  int tok_blocks;
};

template <int FMT, bool F16>
__global__ __launch_bounds__(256) void k_linear_prepare(PrepareArgs a) {
  __shared__ uint32_t red[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x < a.tok_blocks) {
    if constexpr (lin_affine(FMT)) {
      const int t = blockIdx.x;
      const uint16_t* x = a.x + (size_t)t * a.ldx;
      int e = 0;
      if constexpr (!F16) {
        uint32_t most = 0, lows = ~0u;  // the largest, and the least but 0, each less 1 (0 itself wraps)
        for (int c = 8 * tid; c < a.K; c += 2048) {
          const uint4 v = *reinterpret_cast<const uint4*>(x + c);
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            most = lin_max2(most, q[i] & 0x7FFF7FFFu);
            lows = lin_min2(lows, lin_sub2(q[i] & 0x7FFF7FFFu, 0x00010001u));
          }
        }
        uint32_t ends = lin_ends(most, lows);
        for (int o = 32; o > 0; o >>= 1) ends = lin_max2(ends, (uint32_t)__shfl_xor((int)ends, o, 64));
        if (lane == 0) red[wave] = ends;
        __syncthreads();
        ends = lin_max2(lin_max2(red[0], red[1]), lin_max2(red[2], red[3]));
        const uint32_t m = ends >> 16, least = (0x10000u - (ends & 0xFFFFu)) & 0xFFFFu;  // 0 where all are
        e = m ? min(max((int)(m >> 7), 1), 254) - 127 - 14 : 0;  // the largest falls in [2^14, 2^15)
        // the last of a value's eight bits has to reach fp16's smallest number, 2^-24 (an infinity's token is lost anyway)
        const bool wide = least && m < 0x7F80u && max((int)(least >> 7), 1) - 127 - 7 < e - 24;
        if (tid == 0) a.xexp[t] = (e & 0xFFFF) | (wide ? kLinWide : 0);
      }
      constexpr int kLanes = lin_group(FMT) / 8;  // lanes of a group
      uint4 next = make_uint4(0, 0, 0, 0);  // a step ahead
      if (8 * tid < a.K) next = *reinterpret_cast<const uint4*>(x + 8 * tid);
      for (int c0 = 0; c0 < a.K; c0 += 2048) {
        const int c = c0 + 8 * tid;
        uint4 v = next;
        next = make_uint4(0, 0, 0, 0);
        if (c + 2048 < a.K) next = *reinterpret_cast<const uint4*>(x + c + 2048);
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (F16) {
            const lin_f16x2 h = lin_h2(q[i]);
            f[2 * i] = (float)h.x;
            f[2 * i + 1] = (float)h.y;
          } else {
            f[2 * i] = bf16_lo_to_f32(q[i]);
            f[2 * i + 1] = bf16_hi_to_f32(q[i]);
          }
        }
        float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        if constexpr (!F16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const lin_f16x2 h = {(_Float16)__builtin_amdgcn_ldexpf(f[2 * i], -e), (_Float16)__builtin_amdgcn_ldexpf(f[2 * i + 1], -e)};
            (&v.x)[i] = lin_u(h);
          }
        }
        // zeros past the row's end fill its last step
        if (c < (a.K + kLinStep - 1) / kLinStep * kLinStep)
          *reinterpret_cast<uint4*>(a.xq + (((size_t)(t >> 4) * ((a.K + kLinStep - 1) / kLinStep) + c / kLinStep) * 16 + (t & 15)) * kLinStep +
                                    c % kLinStep) = lin_pair_order(v);
        sum += __shfl_xor(sum, 1, 64);
        sum += __shfl_xor(sum, 2, 64);
        if constexpr (kLanes == 8) sum += __shfl_xor(sum, 4, 64);
        if (c < a.K && (tid & (kLanes - 1)) == 0) {
          uint32_t term[3];
          split_terms(sum, term);
          uint16_t* to = a.xsum + (size_t)t * a.Gp + c / lin_group(FMT);
#pragma unroll
          for (int p = 0; p < 3; ++p) to[(size_t)p * a.L * a.Gp] = (uint16_t)term[p];
        }
      }
      if (a.G + tid < a.Gp) {
        for (int p = 0; p < 3; ++p) a.xsum[((size_t)p * a.L + t) * a.Gp + a.G + tid] = 0;
      }
    }
    return;
  }
  const int P = a.row_lanes, sub = tid & (P - 1);
  const size_t n = ((size_t)(blockIdx.x - a.tok_blocks) * 256 + tid) / P;
  if (n >= (size_t)a.N) return;  // a row's threads together
  int m = 0;
  if constexpr (FMT == kLinMxfp4) {
    int least = 255;
    for (int g = sub; g < a.G; g += P) {
      const int e = a.s[n * a.G + g];
      m = max(m, e == 255 ? 0 : e);
      least = min(least, e);
    }
    for (int o = P / 2; o > 0; o >>= 1) m = max(m, __shfl_xor(m, o, 64));
    // The largest block's elements reach 6 * 2^12, the smallest, 0.5 of a
    // block 2^35 below, fp16's smallest number 2^-24; further down only zeros are exact.
    int wide = 0;
    if (least < m - 35) {
      for (int g = sub; g < a.G; g += P) {
        if (a.s[n * a.G + g] >= m - 35) continue;
        const uint4 c = *reinterpret_cast<const uint4*>(a.w + n * (a.K / 8) + 4 * (size_t)g);
        wide |= ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0;
      }
    }
    for (int o = P / 2; o > 0; o >>= 1) wide |= __shfl_xor(wide, o, 64);
    if (sub == 0) a.wexp[n] = ((m - 127 - 12) & 0xFFFF) | (wide ? kLinWide : 0);
  } else if constexpr (lin_affine(FMT)) {
    // eight bf16 from group g on, zeros past the row (whose start has any alignment)
    auto eight = [&](const unsigned char* base, int g, uint16_t (&v)[8]) __attribute__((always_inline)) {
      const uint16_t* from = reinterpret_cast<const uint16_t*>(base) + n * a.G + g;
      if (g + 8 <= a.G) {
        __builtin_memcpy(v, from, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = g + i < a.G ? from[i] : (uint16_t)0;
      }
    };
    uint16_t s[8], b[8];
    constexpr uint32_t kFloor = (127 - 96) << 7;  // 2^-96
    // the largest scale and bias; the least scale, and the least from kFloor on (less kFloor: those below wrap)
    uint32_t most_s = 0, most_b = 0, lows = ~0u, floored = ~0u;
    for (int g = 8 * sub; g < a.Gp; g += 8 * P) {
      eight(a.s, g, s);
      eight(a.b, g, b);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t u = (s[i] | (uint32_t)s[i + 1] << 16) & 0x7FFF7FFFu;
        most_s = lin_max2(most_s, u);
        most_b = lin_max2(most_b, (b[i] | (uint32_t)b[i + 1] << 16) & 0x7FFF7FFFu);
        lows = lin_min2(lows, u | (g + i < a.G ? 0u : 0x7FFFu) | (g + i + 1 < a.G ? 0u : 0x7FFF0000u));
        floored = lin_min2(floored, lin_sub2(u, kFloor << 16 | kFloor));
      }
    }
    uint32_t ends_s = lin_ends(most_s, lows), ends_b = lin_ends(most_b, floored);
    for (int o = P / 2; o > 0; o >>= 1) {
      ends_s = lin_max2(ends_s, (uint32_t)__shfl_xor((int)ends_s, o, 64));
      ends_b = lin_max2(ends_b, (uint32_t)__shfl_xor((int)ends_b, o, 64));
    }
    m = ends_s >> 16;
    const int mb = ends_b >> 16, lowest = 0xFFFF - (ends_s & 0xFFFFu), least = 0xFFFF - (int)(ends_b & 0xFFFFu) + (int)kFloor;
    // The largest scale falls in [2^8, 2^9), 24 s in 2^14; with biases 2^68 and
    // more above the scales, lower: the rest, at most K 2^16 (|b| + 8 |s|) in its
    // token's units, then stays below 2^110 in the row's.
    const int es = min(max(m >> 7, 1), 254) - 127 - 8, eb = (mb >> 7) - 127 - 68;
    const int e = m == 0 ? max(eb, 0) : max(es, eb);
    const bool again = a.Gp > 8 * P;  // else they are at hand
    for (int g = 8 * sub; g < a.Gp; g += 8 * P) {
      if (again) {
        eight(a.s, g, s);
        eight(a.b, g, b);
      }
      uint32_t h[4], t[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t term[2][2];
        const float s0 = bf16_to_f32(s[2 * i]), s1 = bf16_to_f32(s[2 * i + 1]);
        h[i] = lin_u(lin_f16x2{(_Float16)__builtin_amdgcn_ldexpf(s0, -e), (_Float16)__builtin_amdgcn_ldexpf(s1, -e)});
        split_terms(__builtin_fmaf(8.0f, s0, bf16_to_f32(b[2 * i])), term[0]);
        split_terms(__builtin_fmaf(8.0f, s1, bf16_to_f32(b[2 * i + 1])), term[1]);
#pragma unroll
        for (int p = 0; p < 2; ++p) t[p][i] = term[0][p] | term[1][p] << 16;
      }
      *reinterpret_cast<uint4*>(a.sh + n * a.Gp + g) = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int p = 0; p < 2; ++p)
        *reinterpret_cast<uint4*>(a.tsum + ((size_t)p * a.N + n) * a.Gp + g) = make_uint4(t[p][0], t[p][1], t[p][2], t[p][3]);
    }
    // the last of a scale's eight bits has to reach fp16's smallest number, 2^-24
    // (a row with an infinity or NaN is lost anyway)
    const bool wide = m < 0x7F80 && mb < 0x7F80 && (least >> 7) - 127 - 7 < e - 24;
    const bool uneven = (lowest >> 7) < (m >> 7) - 12;
    if (sub == 0) a.wexp[n] = (e & 0xFFFF) | (wide ? kLinWide : 0) | (uneven ? kLinUneven : 0);
  }
}

// Adds the splits of K in ascending order, the bias, and rounds (bound by a
// launch, or by the partial sums: 5 x 636 x 1219 in 5.5 us).
static __global__ __launch_bounds__(256) void k_linear_join(const float* __restrict__ part, const float* __restrict__ bias,
                                                     void* out, long long ldo, int L, int N, int splits, int dtype) {
  const size_t all = (size_t)L * N;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (size_t)gridDim.x * 256) {
    float v = part[i];
    for (int z = 1; z < splits; ++z) v += part[(size_t)z * all + i];
    const size_t t = i / N, n = i - t * N;
    if (bias) v += bias[n];
    const size_t at = t * ldo + n;
    if (dtype == MOE_Q4_DTYPE_F32)
      static_cast<float*>(out)[at] = v;
    else if (dtype == MOE_Q4_DTYPE_BF16)
      static_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_rne(v);
    else
      static_cast<_Float16*>(out)[at] = (_Float16)v;
  }
}

}  // namespace moeq4
