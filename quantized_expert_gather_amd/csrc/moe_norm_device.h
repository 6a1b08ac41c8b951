// Device helpers of the norm and the quantization: chunks of 8 neighbours,
// sums over the threads of a row, E4M3 codes of a block.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_q4.h"

namespace moeq4 {

// Vectors as they lie: rows of any length put them at any element.
typedef __bf16 norm_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 norm_f16x8 __attribute__((ext_vector_type(8)));
typedef float norm_f32x8 __attribute__((ext_vector_type(8)));
template <class T> struct NormVec;
template <> struct NormVec<__bf16> { typedef norm_bf16x8 type __attribute__((aligned(2))); };
template <> struct NormVec<_Float16> { typedef norm_f16x8 type __attribute__((aligned(2))); };
template <> struct NormVec<float> { typedef norm_f32x8 type __attribute__((aligned(4))); };

// The first n of 8 neighbours, zeros for the others (n may be past 8, or negative).
template <class T>
__device__ __forceinline__ void norm_load8(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const typename NormVec<T>::type t = *reinterpret_cast<const typename NormVec<T>::type*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) v[i] = (float)p[i];
    }
  }
}
template <class T>
__device__ __forceinline__ void norm_store8(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    typename NormVec<T>::type t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (T)v[i];
    *reinterpret_cast<typename NormVec<T>::type*>(p) = t;
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (T)v[i];
  }
}
// The same at element `at` of an array of a MOE_Q4_DTYPE_*.
__device__ __forceinline__ void norm_load8_as(const void* p, int dtype, long at, int n, float (&v)[8]) {
  if (dtype == MOE_Q4_DTYPE_F32)
    norm_load8(static_cast<const float*>(p) + at, n, v);
  else if (dtype == MOE_Q4_DTYPE_BF16)
    norm_load8(static_cast<const __bf16*>(p) + at, n, v);
  else
    norm_load8(static_cast<const _Float16*>(p) + at, n, v);
}
__device__ __forceinline__ void norm_store8_as(void* p, int dtype, long at, int n, const float (&v)[8]) {
  if (dtype == MOE_Q4_DTYPE_F32)
    norm_store8(static_cast<float*>(p) + at, n, v);
  else if (dtype == MOE_Q4_DTYPE_BF16)
    norm_store8(static_cast<__bf16*>(p) + at, n, v);
  else
    norm_store8(static_cast<_Float16*>(p) + at, n, v);
}
template <class T>
__device__ __forceinline__ float norm_round(float v) {
  return (float)(T)v;
}

// v of the lane `ROT` places on in the 16 lanes of a row.
template <int ROT>
__device__ __forceinline__ float norm_rot(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + ROT, 0xf, 0xf, true));
}
__device__ __forceinline__ float norm_sum16(float v) {
  v += norm_rot<8>(v);
  v += norm_rot<4>(v);
  v += norm_rot<2>(v);
  return v + norm_rot<1>(v);
}
__device__ __forceinline__ float norm_max16(float v) {
  v = fmaxf(v, norm_rot<8>(v));
  v = fmaxf(v, norm_rot<4>(v));
  v = fmaxf(v, norm_rot<2>(v));
  return fmaxf(v, norm_rot<1>(v));
}
__device__ __forceinline__ float norm_sum64(float v) {
  v = norm_sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sums over the LANES threads of a row, the same in all of them (a workgroup
// is one row where LANES is more than a wave).
template <int LANES>
__device__ __forceinline__ void norm_row_sums(float& a, float& b) {
  if constexpr (LANES == 16) {
    a = norm_sum16(a);
    b = norm_sum16(b);
  } else {
    a = norm_sum64(a);
    b = norm_sum64(b);
    if constexpr (LANES > 64) {
      __shared__ float2 waves[LANES / 64];
      __syncthreads();  // (the row before may still be read)
      if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = make_float2(a, b);
      __syncthreads();
      float2 s = waves[0];
#pragma unroll
      for (int i = 1; i < LANES / 64; ++i) {
        s.x += waves[i].x;
        s.y += waves[i].y;
      }
      a = s.x;
      b = s.y;
    }
  }
}
template <int LANES>
__device__ __forceinline__ float norm_row_sum(float a) {
  float b = 0.0f;
  norm_row_sums<LANES>(a, b);
  return a;
}

// A block's scale: its largest magnitude over E4M3's largest number, and above
// zero.
__device__ __forceinline__ float norm_scale(float most) { return fmaxf(most / 448.0f, 0x1p-126f); }

// Eight values over the block's scale as E4M3, each a quotient rounded to fp32
// and then to nearest even.  A product with the reciprocal will not do: of
// 16-bit values one in 2000 is a tie, which that may put on its wrong side.  So
// the quotient's remainder, which is exact, corrects it (8192 x 6144 into codes
// 72.4 us with products, 78.6 with divisions, 73.9 so); where it would be
// subnormal, and is not exact, it is a division.
__device__ __forceinline__ uint2 norm_pack8(const float (&v)[8], float s) {
  float q[8];
  if (s < 0x1p-90f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / s;
  } else {
    const float y = __builtin_amdgcn_rcpf(s), m = s < __builtin_inff() ? s : 0.0f;  // (an infinite scale leaves zeros and NaN)
    const float inv = __builtin_fmaf(__builtin_fmaf(-m, y, 1.0f), y, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = v[i] * inv;
      q[i] = __builtin_fmaf(-__builtin_fmaf(q[i], m, -v[i]), inv, q[i]);  // (-0 stays)
    }
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Codes of this thread's 8 values of a block that 16 neighbours hold, and the block's scale.
__device__ __forceinline__ uint2 norm_codes(const float (&v)[8], float& s) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
  s = norm_scale(norm_max16(most));
  return norm_pack8(v, s);
}

__device__ __forceinline__ void norm_store_codes(uint8_t* p, int n, uint2 q) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef u32x2 u32x2_any __attribute__((aligned(1)));
  if (n >= 8) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{q.x, q.y};
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

}  // namespace moeq4
