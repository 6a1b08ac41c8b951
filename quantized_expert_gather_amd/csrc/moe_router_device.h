// Device helpers of the router's selection and of the balance loss.  Internal
// header.
//
// LPR threads hold one row of E router values in their registers: 16, 32 or
// 64 lanes of a wave (so a wave works on four, two or one rows at a time, and
// a reduction's steps serve all of them), or a workgroup of 1024 threads where
// E is large.  Thread i of a row holds EPL values, in chunks of V neighbours:
// value j is expert (j / V) * LPR * V + i * V + j % V, so that a load takes
// neighbouring bytes in neighbouring threads, and j rises with the expert.
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
  // gfx950 converts in hardware: to nearest even, NaN stays NaN
  static __device__ __forceinline__ mem store(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
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
struct OpMinI { __device__ __forceinline__ int operator()(int a, int b) const { return a < b ? a : b; } };
struct OpMaxI { __device__ __forceinline__ int operator()(int a, int b) const { return a > b ? a : b; } };

template <int CTRL, class V>
__device__ __forceinline__ V dpp_move(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// op over the LPR threads of each row; every thread receives its row's.
// Inside 16-lane rows the steps are DPP lane permutes, across them gfx950's
// row swaps, so nothing goes through the LDS pipe (but for LPR = 1024, whose
// waves meet in `red`, 16 words; all threads must call it then).  The tree is
// fixed: sums are the same from run to run.
template <int LPR, class OP, class V>
__device__ __forceinline__ V row_all(V v, OP op, V* red = nullptr) {
  v = op(v, dpp_move<0xB1>(v));   // lane ^ 1
  v = op(v, dpp_move<0x4E>(v));   // lane ^ 2
  v = op(v, dpp_move<0x141>(v));  // half-row mirror
  v = op(v, dpp_move<0x140>(v));  // row mirror
  if constexpr (LPR >= 32) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    v = op(__builtin_bit_cast(V, s0), __builtin_bit_cast(V, s1));
  }
  if constexpr (LPR >= 64) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    v = op(__builtin_bit_cast(V, s0), __builtin_bit_cast(V, s1));
  }
  if constexpr (LPR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < LPR / 64; ++w) v = op(v, red[w]);
  }
  return v;
}

// Neighbouring values of a thread: a 16-byte load's, or all of them.
template <class LT, int EPL>
constexpr int row_chunk() {
  return EPL < 16 / (int)sizeof(typename LT::mem) ? EPL : 16 / (int)sizeof(typename LT::mem);
}
// Expert of value j of thread `slot`.
template <class LT, int EPL, int LPR>
__device__ __forceinline__ int row_expert(int slot, int j) {
  constexpr int V = row_chunk<LT, EPL>();
  return (j / V) * (LPR * V) + slot * V + j % V;
}

// A thread's values of a row as fp32, `fill` past E.  Rows may start at any
// element: loads of a whole chunk need no alignment, and only the chunk that E
// ends in goes by elements (against elements throughout, 5 x 16525 rows of 93
// bf16 values went from 18.6 to 14.3 us in the balance loss, from 27.6 to 17.6
// in its gradient).
template <class LT, int EPL, int LPR>
__device__ __forceinline__ void load_row(const typename LT::mem* __restrict__ row, int slot, int E, float fill,
                                         float (&v)[EPL]) {
  typedef typename LT::mem mem;
  constexpr int V = row_chunk<LT, EPL>();
  typedef mem vt __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int c = 0; c < EPL / V; ++c) {
    const int e = row_expert<LT, EPL, LPR>(slot, c * V);
    if (e + V <= E) {
      vt x;
      __builtin_memcpy(&x, row + e, sizeof(vt));
#pragma unroll
      for (int j = 0; j < V; ++j) v[c * V + j] = LT::load(x[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[c * V + j] = e + j < E ? LT::load(row[e + j]) : fill;
    }
  }
}

template <class LT, int EPL, int LPR>
__device__ __forceinline__ void store_row(typename LT::mem* __restrict__ row, int slot, int E, const float (&v)[EPL]) {
  typedef typename LT::mem mem;
  constexpr int V = row_chunk<LT, EPL>();
  typedef mem vt __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int c = 0; c < EPL / V; ++c) {
    const int e = row_expert<LT, EPL, LPR>(slot, c * V);
    if (e + V <= E) {
      vt x;
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = LT::store(v[c * V + j]);
      __builtin_memcpy(row + e, &x, sizeof(vt));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e + j < E) row[e + j] = LT::store(v[c * V + j]);
    }
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

// sigmoid(z) and 1 - sigmoid(z) = e^-z sigmoid(z) together, neither by a
// difference; below -80 the second is 1 (and e^-z may be infinite).
__device__ __forceinline__ float sigmoid_pair(float z, float& rest) {
  const float e = exp_f32(-z), s = recip_f32(1.0f + e);
  rest = z < -80.0f ? 1.0f : e * s;
  return s;
}

// Scores whose row's sum is below this (every logit below -16) are formed
// again from the row's maximum where they are divided by that sum: fp32 holds
// no sigmoid below -87, the ratios of these are ordinary numbers.
constexpr float kLowSum = 0x1p-24f;
// sigmoid(z) e^-base, for z <= base <= 0.
__device__ __forceinline__ float sigmoid_from(float z, float base) { return exp_f32(z - base) * recip_f32(1.0f + exp_f32(z)); }

// What a row's exponentials count from: its maximum, or 0 where all of it is
// masked (-inf): exp(-inf - 0) = 0, a softmax of zeros.
__device__ __forceinline__ float exp_base(float row_max) { return row_max == -__builtin_inff() ? 0.0f : row_max; }

// Host side: threads per row and values per thread for E experts and k
// picks (one thread each).  Few threads a row share a reduction's steps among more
// rows; many (`wide`) have less to do one after the other.
struct RowPlan {
  int lpr, epl;
};
inline RowPlan row_plan(int E, int k, bool wide) {
  RowPlan p{wide ? 64 : 16, 0};
  if (E > 1024) {
    p.lpr = 1024;
  } else {
    while (16 * p.lpr < E || p.lpr < k) p.lpr *= 2;
  }
  const int need = (E + p.lpr - 1) / p.lpr;
  p.epl = need <= 4 ? 4 : need <= 8 && (p.lpr == 16 || p.lpr == 64) ? 8 : 16;
  return p;
}

// Rows of one launch: a grid holds fewer than 2^32 threads, so the longest
// inputs take several.
constexpr size_t kLaunchThreads = size_t(1) << 31;
inline int rows_of_launch(int lpr) { return (int)(kLaunchThreads / lpr); }
}  // namespace moeq4

// Expands CALL(LT, EPL, LPR) for a logits type and a RowPlan.
#define MOE_ROW_DISPATCH_EPL(LT, plan, CALL)         \
  if ((plan).lpr == 16) {                            \
    switch ((plan).epl) {                            \
      case 4: CALL(LT, 4, 16); break;                \
      case 8: CALL(LT, 8, 16); break;                \
      default: CALL(LT, 16, 16); break;              \
    }                                                \
  } else if ((plan).lpr == 32) {                     \
    if ((plan).epl == 4) {                           \
      CALL(LT, 4, 32);                               \
    } else {                                         \
      CALL(LT, 16, 32);                              \
    }                                                \
  } else if ((plan).lpr == 64) {                     \
    switch ((plan).epl) {                            \
      case 4: CALL(LT, 4, 64); break;                \
      case 8: CALL(LT, 8, 64); break;                \
      default: CALL(LT, 16, 64); break;              \
    }                                                \
  } else if ((plan).epl == 4) {                      \
    CALL(LT, 4, 1024);                               \
  } else {                                           \
    CALL(LT, 16, 1024);                              \
  }
#define MOE_ROW_DISPATCH(dtype, plan, CALL)          \
  if ((dtype) == MOE_Q4_DTYPE_BF16) {                \
    MOE_ROW_DISPATCH_EPL(LogitBf16, plan, CALL)      \
  } else if ((dtype) == MOE_Q4_DTYPE_F32) {          \
    MOE_ROW_DISPATCH_EPL(LogitF32, plan, CALL)       \
  } else {                                           \
    MOE_ROW_DISPATCH_EPL(LogitF16, plan, CALL)       \
  }
