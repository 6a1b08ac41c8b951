// Device helpers of the router's selection and of the balance loss: one row
// of E router values lies in the registers of one wave, or of one 16-wave
// workgroup where E is large.  Internal header.
//
// Layout: thread i of the row's threads holds the EPL consecutive values
// i * EPL .. i * EPL + EPL - 1, so a lower thread always holds lower experts
// and ties go to the lowest set bit of a ballot.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_q4_device.h"

namespace moeq4 {

constexpr int kRouterScoreSoftmax = 0;
constexpr int kRouterScoreSigmoid = 1;

// Element types of the logits and of their gradient (MOE_Q4_DTYPE_*).
struct LogitBf16 {
  typedef uint16_t mem;
  static __device__ __forceinline__ float load(mem v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ mem store(float v) { return (mem)f32_to_bf16_rne(v); }
};
struct LogitF32 {
  typedef float mem;
  static __device__ __forceinline__ float load(mem v) { return v; }
  static __device__ __forceinline__ mem store(float v) { return v; }
};
struct LogitF16 {
  typedef _Float16 mem;
  static __device__ __forceinline__ float load(mem v) { return (float)v; }
  static __device__ __forceinline__ mem store(float v) { return (mem)v; }
};

struct OpMaxF { __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct OpSumF { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };
struct OpMaxI { __device__ __forceinline__ int operator()(int a, int b) const { return a > b ? a : b; } };

template <int CTRL, class V>
__device__ __forceinline__ V dpp_move(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// op over the 64 lanes of a wave; every lane receives it.  Inside 16-lane
// rows the steps are DPP lane permutes, across rows gfx950's row swaps, so
// nothing goes through the LDS pipe.  The tree is fixed: sums are the same
// from run to run.
template <class OP, class V>
__device__ __forceinline__ V wave_all(V v, OP op) {
  v = op(v, dpp_move<0xB1>(v));   // lane ^ 1
  v = op(v, dpp_move<0x4E>(v));   // lane ^ 2
  v = op(v, dpp_move<0x141>(v));  // half-row mirror
  v = op(v, dpp_move<0x140>(v));  // row mirror
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto s16 = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  v = op(__builtin_bit_cast(V, (uint32_t)s16[0]), __builtin_bit_cast(V, (uint32_t)s16[1]));
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto s32 = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return op(__builtin_bit_cast(V, (uint32_t)s32[0]), __builtin_bit_cast(V, (uint32_t)s32[1]));
}

// op over all threads of a row: WPR waves, through `red` (LDS, 16 words)
// where WPR > 1.  Every thread of the workgroup must call it then.
template <int WPR, class OP, class V>
__device__ __forceinline__ V row_all(V v, OP op, V* red) {
  v = wave_all(v, op);
  if constexpr (WPR > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) v = op(v, red[w]);
  }
  return v;
}

template <int N>
struct alignas(N) Bytes {
  unsigned char b[N];
};

// Values base .. base + EPL - 1 of a row as fp32, `fill` past E.  `vec`: the
// row starts on a boundary of the widest load below and E is a multiple of
// EPL, so a thread's values are all inside the row or all outside.
template <class LT, int EPL>
__device__ __forceinline__ void load_row(const typename LT::mem* __restrict__ row, int base, int E, bool vec,
                                         float fill, float (&v)[EPL]) {
  typedef typename LT::mem mem;
  constexpr int kBytes = EPL * (int)sizeof(mem);
  constexpr int kLoad = kBytes < 16 ? kBytes : 16;
  constexpr int kPer = kLoad / (int)sizeof(mem);
  if (vec) {
    if (base < E) {
#pragma unroll
      for (int c = 0; c < EPL / kPer; ++c) {
        typedef mem vt __attribute__((ext_vector_type(kPer)));
        const vt x = *reinterpret_cast<const vt*>(row + base + c * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[c * kPer + j] = LT::load(x[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = fill;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = base + i < E ? LT::load(row[base + i]) : fill;
  }
}

template <class LT, int EPL>
__device__ __forceinline__ void store_row(typename LT::mem* __restrict__ row, int base, int E, bool vec,
                                          const float (&v)[EPL]) {
  typedef typename LT::mem mem;
  constexpr int kBytes = EPL * (int)sizeof(mem);
  constexpr int kStore = kBytes < 16 ? kBytes : 16;
  constexpr int kPer = kStore / (int)sizeof(mem);
  if (vec) {
    if (base < E) {
#pragma unroll
      for (int c = 0; c < EPL / kPer; ++c) {
        typedef mem vt __attribute__((ext_vector_type(kPer)));
        vt x;
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = LT::store(v[c * kPer + j]);
        *reinterpret_cast<vt*>(row + base + c * kPer) = x;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (base + i < E) row[base + i] = LT::store(v[i]);
  }
}

// 1 / v by the hardware's reciprocal (one step off at most) and one Newton
// step, for v >= 1 (infinity included).
__device__ __forceinline__ float recip_f32(float v) {
  const float r = __builtin_amdgcn_rcpf(v);
  const float e = __builtin_fmaf(-v, r, 1.0f);
  return v == __builtin_inff() ? r : __builtin_fmaf(e, r, r);
}

// exp(d) as 2^(d log2 e): the product is off by 2^-24 of itself and so, with
// the constant's own rounding, exp(d) by 2^-24 (1.5 |d|) and the two steps
// of v_exp_f32.  d = -inf gives 0.
__device__ __forceinline__ float exp_f32(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504f); }

// sigmoid(z) and 1 - sigmoid(z) = sigmoid(-z), each without cancellation.
__device__ __forceinline__ float sigmoid_f32(float z) { return recip_f32(1.0f + exp_f32(-z)); }

// exp(z - m) with exp of a masked value (-inf) 0 also where the whole row is
// masked (m = -inf), whose softmax is taken as zero.
__device__ __forceinline__ float exp_below(float z, float m) {
  return m == -__builtin_inff() ? 0.0f : exp_f32(z - m);
}

// Host side: values per thread and waves per row for E experts, and whether
// a row of this layout can be read and written with vector accesses.
struct RowPlan {
  int epl, wpr;
};
inline RowPlan row_plan(int E) {
  RowPlan p{1, 1};
  if (E > 1024) p.wpr = 16;
  while (64 * p.wpr * p.epl < E) p.epl *= 2;
  return p;
}
inline bool row_vec(const void* base, long long ld, int E, int epl, int elem) {
  const int bytes = epl * elem < 16 ? epl * elem : 16;
  return E % epl == 0 && (uintptr_t)base % bytes == 0 && (ld * elem) % bytes == 0;
}

}  // namespace moeq4

// Calls F<LT, EPL, WPR>(...) for a logits type and a RowPlan.
#define MOE_ROW_DISPATCH_EPL(LT, plan, CALL)                       \
  if ((plan).wpr == 1) {                                           \
    switch ((plan).epl) {                                          \
      case 1: CALL(LT, 1, 1); break;                               \
      case 2: CALL(LT, 2, 1); break;                               \
      case 4: CALL(LT, 4, 1); break;                               \
      case 8: CALL(LT, 8, 1); break;                               \
      default: CALL(LT, 16, 1); break;                             \
    }                                                              \
  } else {                                                         \
    switch ((plan).epl) {                                          \
      case 2: CALL(LT, 2, 16); break;                              \
      case 4: CALL(LT, 4, 16); break;                              \
      case 8: CALL(LT, 8, 16); break;                              \
      default: CALL(LT, 16, 16); break;                            \
    }                                                              \
  }
#define MOE_ROW_DISPATCH(dtype, plan, CALL)                        \
  if ((dtype) == MOE_Q4_DTYPE_BF16) {                              \
    MOE_ROW_DISPATCH_EPL(LogitBf16, plan, CALL)                    \
  } else if ((dtype) == MOE_Q4_DTYPE_F32) {                        \
    MOE_ROW_DISPATCH_EPL(LogitF32, plan, CALL)                     \
  } else {                                                         \
    MOE_ROW_DISPATCH_EPL(LogitF16, plan, CALL)                     \
  }
