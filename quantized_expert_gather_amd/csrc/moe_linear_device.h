// Device helpers of the dense 4-bit product: matrix-core operands out of
// packed codes.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_q4_device.h"

namespace moeq4 {

constexpr int kLinAffine64 = 0, kLinAffine32 = 1, kLinMxfp4 = 2, kLinNvfp4 = 3;
__host__ __device__ constexpr bool lin_affine(int f) { return f == kLinAffine64 || f == kLinAffine32; }
__host__ __device__ constexpr int lin_group(int f) { return f == kLinAffine64 ? 64 : f == kLinNvfp4 ? 16 : 32; }
// A wave takes weights 128 inputs (a step) of 16 rows at a time: lane (n, kb) =
// (lane % 16, lane / 16) loads 16 bytes of row n, the 32 codes from input 32 kb,
// so a row's 64 bytes are contiguous.  v_mfma_f32_16x16x32 sums the eight
// inputs of a word over the four kb.
constexpr int kLinStep = 128;

typedef __bf16 lin_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 lin_f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 lin_f16x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x4 __attribute__((ext_vector_type(4)));

typedef unsigned int lin_u32x4 __attribute__((ext_vector_type(4)));

template <bool F16, class A, class B>
__device__ __forceinline__ lin_f32x4 lin_mfma(A a, B b, lin_f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(lin_f16x8, a), __builtin_bit_cast(lin_f16x8, b), c,
                                                  0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(lin_bf16x8, a), __builtin_bit_cast(lin_bf16x8, b),
                                                   c, 0, 0, 0);
}

// 16 + q for the eight codes of a word, as pairs (q0,q4) (q1,q5) (q2,q6)
// (q3,q7): a code in the top mantissa bits under the exponent of 16.  The
// smallest offset that one mask and one or can give keeps the fp32 sums
// near the size of the codes' own (128 + q would cost three more bits).
// Mask and base come in registers (one scalar, one vector: what a
// three-operand instruction may read), so each pair is a shift and one
// v_and_or; as literals they would be two instructions.
struct LinCode {
  uint32_t mask, base;
};
template <bool F16>
__device__ __forceinline__ LinCode lin_code() {
  LinCode c;
  asm("s_mov_b32 %0, %1" : "=s"(c.mask) : "i"(F16 ? 0x03C003C0 : 0x00780078));
  c.base = F16 ? 0x4C004C00u : 0x41804180u;
  asm("" : "+v"(c.base));
  return c;
}
template <bool F16>
__device__ __forceinline__ uint4 lin_codes16(uint32_t w, LinCode c) {
  constexpr int kUp = F16 ? 6 : 3;  // from a word's lowest code to the mantissa's top
  return make_uint4(((w << kUp) & c.mask) | c.base, ((F16 ? w << 2 : w >> 1) & c.mask) | c.base,
                    ((w >> (8 - kUp)) & c.mask) | c.base, ((w >> (12 - kUp)) & c.mask) | c.base);
}

// Eight activations in the order lin_codes16 gives the codes.
__device__ __forceinline__ uint4 lin_pair_order(uint4 v) {
  return make_uint4((v.x & 0xFFFFu) | (v.z << 16), (v.x >> 16) | (v.z & 0xFFFF0000u), (v.y & 0xFFFFu) | (v.w << 16),
                    (v.y >> 16) | (v.w & 0xFFFF0000u));
}

// E2M1 values of a word's codes, natural order, exact.
template <bool F16>
__device__ __forceinline__ uint4 lin_fp4(uint32_t w) {
  if constexpr (F16)
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3)));
  else
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3)));
}

// mxfp4 codes times the power of two in the exponent of `s`.
template <bool F16>
__device__ __forceinline__ uint4 lin_fp4_pow2(uint32_t w, float s) {
  if constexpr (F16)
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3)));
  else
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3)));
}

// fp16 values as two bf16 terms, hi + lo: 11 bits as 8 + 3, both exact.
__device__ __forceinline__ void lin_two_terms(lin_u32x4 v, lin_u32x4& hi, lin_u32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = v[i];
    const lin_f16x2 h = __builtin_bit_cast(lin_f16x2, word);
    const float f0 = (float)h.x, f1 = (float)h.y;
    const uint32_t h0 = __float_as_uint(f0) & 0xFFFF0000u, h1 = __float_as_uint(f1) & 0xFFFF0000u;
    // (an infinite or NaN value has no second term)
    const float r0 = f0 - __uint_as_float(h0), r1 = f1 - __uint_as_float(h1);
    hi[i] = h0 >> 16 | h1;
    lo[i] = (r0 == r0 ? __float_as_uint(r0) >> 16 : 0u) | (r1 == r1 ? __float_as_uint(r1) & 0xFFFF0000u : 0u);
  }
}

// Value of byte B of a word of E4M3 bytes.
template <int B>
__device__ __forceinline__ float lin_e4m3(uint32_t w) {
  return __builtin_amdgcn_cvt_f32_fp8((int)w, B);
}

// E2M1 values times an E4M3 scale: at most 2 + 4 significant bits and an
// exponent both types hold, so the product is exact in bf16 and in fp16.
template <bool F16>
__device__ __forceinline__ uint4 lin_fp4_scaled(uint32_t w, float s) {
  if constexpr (F16) {
    const lin_f16x2 h = {(_Float16)s, (_Float16)s};
    uint4 v = lin_fp4<true>(w);
    v.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(lin_f16x2, v.x) * h);
    v.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(lin_f16x2, v.y) * h);
    v.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(lin_f16x2, v.z) * h);
    v.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(lin_f16x2, v.w) * h);
    return v;
  } else {
    auto two = [&](lin_f32x2 p) {  // the high halves of two fp32 are their exact bf16
      return __builtin_amdgcn_perm(__float_as_uint(p.y * s), __float_as_uint(p.x * s), 0x07060302u);
    };
    return make_uint4(two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)),
                      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3)));
  }
}

// 2^(e - 127) of an E8M0 byte: the byte in fp32's exponent field, the
// subnormal 2^-127 for 0 and NaN for 255.
__device__ __forceinline__ float lin_e8m0(uint32_t e) {
  const uint32_t v = e == 0 ? 0x00400000u : e << 23;
  return __uint_as_float(e == 255u ? 0x7FC00000u : v);
}

// The values of the first S 16-lane rows, each to all four rows.
template <int S>
__device__ __forceinline__ void lin_spread(uint32_t v, uint32_t (&out)[S]) {
  static_assert(S >= 1 && S <= 3, "steps of a wave");
  if constexpr (S == 1) {
    out[0] = v;
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // rows 0 1 0 1, rows 2 3 2 3
    const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    out[0] = lo[0];
    out[1] = lo[1];
    if constexpr (S > 2) {
      out[2] = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false)[0];
    }
  }
}

// Transposes the 4 x 4 words of four 16-lane rows: w[j] of row kb goes to
// w[kb] of row j.
__device__ __forceinline__ void lin_transpose(uint32_t (&w)[4]) {
  auto s = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  w[0] = s[0]; w[2] = s[1];
  s = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  w[1] = s[0]; w[3] = s[1];
  s = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
  w[0] = s[0]; w[1] = s[1];
  s = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
  w[2] = s[0]; w[3] = s[1];
}

}  // namespace moeq4
