// The router's selection: the k experts of each token from its router
// logits, their weights, and the weights' gradient.
//
//   p = softmax(z) or sigmoid(z); the k largest of z (or of p + select_bias);
//   w_j = scale * p_j / sum over the chosen (renormalised), or scale * p_j.
//
// One wave holds a row (16 waves above 1024 experts) and takes the largest
// value k times: a maximum over the thread's values, a DPP maximum over the
// lanes, a ballot for its owner.  z is read once.
#include <hip/hip_runtime.h>

#include <limits.h>
#include <stdint.h>

#include "moe_q4.h"
#include "moe_router_device.h"

namespace moeq4 {
namespace {

constexpr int kRowsPerBlock = 4;  // waves of a workgroup, one row each (E <= 1024)

struct TopkArgs {
  const void* z;
  const float* bias;
  int32_t* ids;
  float* w;
  long long ld;
  int T, k, E, score, norm, vec;
  float scale;
};

// Orders fp32 values as signed integers: -0 as +0, NaN below -inf.
constexpr int kKeyTaken = INT_MIN;      // chosen already, or past E
constexpr int kKeyNan = INT_MIN + 1;
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  const int key = b ^ ((b >> 31) & 0x7FFFFFFF);
  return v != v ? kKeyNan : key;
}
__device__ __forceinline__ float key_value(int key) {
  if (key <= kKeyNan) return __builtin_nanf("");
  return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF));
}

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// What one round of the selection found.
struct Pick {
  int key, id;
};

// The largest key among the row's threads, lowest expert first, and takes it
// out.
template <int EPL, int WPR>
__device__ __forceinline__ Pick take_largest(int (&key)[EPL], Pick* red) {
  const int lane = threadIdx.x & 63;
  int lm = key[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) lm = lm > key[i] ? lm : key[i];
  const int m = wave_all(lm, OpMaxI());
  const int owner = __ffsll((unsigned long long)__ballot(lm == m)) - 1;
  int at = 0;
#pragma unroll
  for (int i = EPL - 1; i >= 0; --i) at = key[i] == m ? i : at;
  Pick p;
  p.key = m;
  p.id = lane_value((WPR > 1 ? (int)threadIdx.x : lane) * EPL + at, owner);
  bool mine = lane == owner;
  if constexpr (WPR > 1) {
    __syncthreads();
    if (lane == 0) red[threadIdx.x >> 6] = p;
    __syncthreads();
    int best = 0;
#pragma unroll
    for (int w = 1; w < WPR; ++w)
      if (red[w].key > red[best].key) best = w;
    p = red[best];
    mine = mine && best == (int)(threadIdx.x >> 6);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (mine && at == i) key[i] = kKeyTaken;
  return p;
}

// 16-bit logits without a bias: order and expert fit one word, so keys differ
// and each thread can keep its own in falling order.  A round is a maximum
// over the threads' first keys; its owner moves up.
template <class LT>
__device__ __forceinline__ int packed_key(float v, int e) {
  const int b = (int)(int16_t)__builtin_bit_cast(uint16_t, LT::store(v + 0.0f));
  const int o = v != v ? -32767 : b ^ ((b >> 31) & 0x7FFF);  // NaN below -inf
  return (int)((uint32_t)o << 16) | (0xFFFF - e);
}
template <class LT>
__device__ __forceinline__ float packed_value(int key) {
  const int o = key >> 16;
  if (o == -32767) return __builtin_nanf("");
  return LT::load(__builtin_bit_cast(typename LT::mem, (uint16_t)(o ^ ((o >> 31) & 0x7FFF))));
}
template <int EPL>
__device__ __forceinline__ void sort_falling(int (&k)[EPL]) {  // odd-even merges
#pragma unroll
  for (int p = 1; p < EPL; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < EPL; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int x = i + j, y = i + j + q;
          if (y < EPL && x / (2 * p) == y / (2 * p)) {
            const int hi = k[x] > k[y] ? k[x] : k[y], lo = k[x] > k[y] ? k[y] : k[x];
            k[x] = hi;
            k[y] = lo;
          }
        }
}

// The same selection with the scores in 64 bits, for the rows whose 32-bit
// scores lie too close to be told apart: lane j keeps pick j.
template <int EPL, int WPR>
__device__ void select_in_64(const float (&z)[EPL], const float (&b)[EPL], int base, int E, int k, int score,
                             double* red, int* red_id, int& my_id, float& my_z) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slot = WPR > 1 ? (int)threadIdx.x : lane;
  double s[EPL];
  auto all = [&](double v, bool max) {
    for (int o = 32; o > 0; o >>= 1) {
      const double u = __shfl_xor(v, o, 64);
      v = max ? (u > v ? u : v) : v + u;
    }
    if constexpr (WPR > 1) {
      __syncthreads();
      if (lane == 0) red[wave] = v;
      __syncthreads();
      v = red[0];
      for (int w = 1; w < WPR; ++w) v = max ? (red[w] > v ? red[w] : v) : v + red[w];
    }
    return v;
  };
  if (score == kRouterScoreSoftmax) {
    double m = -__builtin_inf(), sum = 0.0;
    for (int i = 0; i < EPL; ++i)
      if (base + i < E && (double)z[i] > m) m = (double)z[i];
    m = all(m, true);
    for (int i = 0; i < EPL; ++i) {
      s[i] = base + i < E && m > -__builtin_inf() ? exp((double)z[i] - m) : 0.0;
      sum += s[i];
    }
    sum = all(sum, false);
    for (int i = 0; i < EPL; ++i) s[i] = (m > -__builtin_inf() ? s[i] / sum : 0.0) + (double)b[i];
  } else {
    for (int i = 0; i < EPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)z[i])) + (double)b[i];
  }
  uint32_t open = 0;  // bit i: value i not yet chosen
  for (int i = 0; i < EPL; ++i) open |= (base + i < E ? 1u : 0u) << i;
  for (int j = 0; j < k; ++j) {
    // best of the thread: numbers before NaN, then the larger, then the lower expert
    int id = INT_MAX, at = -1;
    double v = 0.0;
    for (int i = EPL - 1; i >= 0; --i) {
      if (!((open >> i) & 1u)) continue;
      const bool nan_i = s[i] != s[i], nan_v = at >= 0 && v != v;
      if (at < 0 || nan_v || (!nan_i && s[i] >= v)) {
        at = i;
        v = s[i];
        id = base + i;
      }
    }
    float zs = 0.0f;
    for (int i = 0; i < EPL; ++i) zs = at == i ? z[i] : zs;
    const int mine = id;
    auto better = [](double v1, int id1, double v0, int id0) {  // is (v1, id1) before (v0, id0)?
      if (id1 == INT_MAX) return false;
      if (id0 == INT_MAX) return true;
      const bool n1 = v1 != v1, n0 = v0 != v0;
      if (n1 != n0) return n0;
      if (!n1 && v1 != v0) return v1 > v0;
      return id1 < id0;
    };
    for (int o = 32; o > 0; o >>= 1) {
      const double u = __shfl_xor(v, o, 64);
      const int uid = __shfl_xor(id, o, 64);
      const float uz = __shfl_xor(zs, o, 64);
      if (better(u, uid, v, id)) {
        v = u;
        id = uid;
        zs = uz;
      }
    }
    if constexpr (WPR > 1) {
      __syncthreads();
      if (lane == 0) {
        red[wave] = v;
        red_id[wave] = id;
        red_id[WPR + wave] = __float_as_int(zs);
      }
      __syncthreads();
      int bw = 0;
      for (int w = 1; w < WPR; ++w)
        if (better(red[w], red_id[w], red[bw], red_id[bw])) bw = w;
      id = red_id[bw];
      zs = __int_as_float(red_id[WPR + bw]);
    }
    if (mine == id) open &= ~(1u << at);
    if (slot == j) {
      my_id = id;
      my_z = zs;
    }
  }
}

// Weights of the chosen: thread j < k of the row holds logit z of pick j.
// Every thread of the wave calls it; the sums run over the first wave.
__device__ __forceinline__ float chosen_weight(float z, bool live, int score, int norm, float scale, float row_max,
                                               float row_sum) {
  if (score == kRouterScoreSoftmax) {
    if (norm) {
      const float m = wave_all(live ? z : -__builtin_inff(), OpMaxF());
      const float e = live ? exp_below(z, m) : 0.0f;
      const float sum = wave_all(e, OpSumF());
      return sum == 0.0f ? 0.0f : scale * (e / sum);
    }
    return row_sum == 0.0f ? 0.0f : scale * (exp_below(z, row_max) / row_sum);
  }
  const float s = live ? sigmoid_f32(z) : 0.0f;
  if (!norm) return scale * s;
  const float sum = wave_all(s, OpSumF());
  return sum == 0.0f ? 0.0f : scale * (s / sum);
}

template <class LT, int EPL, int WPR, bool BIAS>
__global__ __launch_bounds__(WPR > 1 ? 64 * WPR : 64 * kRowsPerBlock) void k_router_topk(TopkArgs a) {
  constexpr bool kPacked = !BIAS && WPR == 1 && sizeof(typename LT::mem) == 2;
  typedef typename LT::mem mem;
  __shared__ Pick red[WPR];
  __shared__ float redf[WPR];
  __shared__ double redd[WPR];
  __shared__ int redi[2 * WPR];
  const int lane = threadIdx.x & 63;
  const int slot = WPR > 1 ? (int)threadIdx.x : lane;
  const int t = __builtin_amdgcn_readfirstlane(WPR > 1 ? (int)blockIdx.x : (int)blockIdx.x * kRowsPerBlock + (int)(threadIdx.x >> 6));
  if (t >= a.T) return;  // whole rows only
  const int base = slot * EPL;
  const mem* row = static_cast<const mem*>(a.z) + (size_t)t * a.ld;
  float z[EPL];
  load_row<LT, EPL>(row, base, a.E, a.vec, -__builtin_inff(), z);

  // softmax statistics, where the whole row counts
  float row_max = 0.0f, row_sum = 1.0f;
  float e[EPL];
  if (a.score == kRouterScoreSoftmax && (BIAS || !a.norm)) {
    row_max = z[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) row_max = fmaxf(row_max, z[i]);
    row_max = row_all<WPR>(row_max, OpMaxF(), redf);
    row_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      e[i] = exp_below(z[i], row_max);
      row_sum += e[i];
    }
    row_sum = row_all<WPR>(row_sum, OpSumF(), redf);
  }

  int my_id = 0;
  float my_z = 0.0f;
  int key[EPL];
  if constexpr (kPacked) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = base + i < a.E ? packed_key<LT>(z[i], base + i) : kKeyTaken;
    sort_falling<EPL>(key);
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
      const int m = wave_all(key[0], OpMaxI());
      if (lane == j) mine = m;
      const bool own = key[0] == m;
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = own ? (i + 1 < EPL ? key[i + 1] : kKeyTaken) : key[i];
    }
    my_id = 0xFFFF - (mine & 0xFFFF);
    my_z = packed_value<LT>(mine);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      float v = z[i];
      if constexpr (BIAS) {
        const float b = base + i < a.E ? a.bias[base + i] : 0.0f;
        v = (a.score == kRouterScoreSoftmax ? (row_sum == 0.0f ? 0.0f : e[i] / row_sum) : sigmoid_f32(z[i])) + b;
      }
      key[i] = base + i < a.E ? order_key(v) : kKeyTaken;
    }
    int my_key = 0, last_key = 0, last_id = 0;
    const int rounds = BIAS && a.k < a.E ? a.k + 1 : a.k;
    for (int j = 0; j < rounds; ++j) {
      const Pick p = take_largest<EPL, WPR>(key, red);
      if (slot == j) {
        my_id = p.id;
        my_key = p.key;
      }
      last_key = p.key;
      last_id = p.id;
    }
    if constexpr (BIAS) {
      // Two neighbours in the order of different logits or biases that fp32
      // cannot tell apart: a score is off by at most about 5e-6 p + 2^-24
      // |score| (the exponential, its sum, the quotient, the sum with the
      // bias), p <= 1.  The first wave holds the picks.
      bool close = false;
      if (WPR == 1 || threadIdx.x < 64) {
        const bool last = lane == rounds - 1 || lane == 63;
        const int id2 = lane == 63 ? last_id : __shfl_down(my_id, 1, 64);
        const int key2 = lane == 63 ? last_key : __shfl_down(my_key, 1, 64);
        const bool pair = lane < rounds - 1 && (!last || (lane == 63 && rounds == 65));
        if (lane < a.k) my_z = LT::load(row[my_id]);
        if (pair) {
          const float s1 = key_value(my_key), s0 = key_value(key2);
          if (!(s1 - s0 > 8e-6f + 5e-7f * fabsf(s1)))
            close = !(LT::load(row[id2]) == my_z && a.bias[id2] == a.bias[my_id]);
        }
        close = __any(close);
      }
      if constexpr (WPR > 1) {
        __syncthreads();
        if (threadIdx.x == 0) redi[0] = close;
        __syncthreads();
        close = redi[0];
        __syncthreads();
      }
      if (close) {
        float b[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) b[i] = base + i < a.E ? a.bias[base + i] : 0.0f;
        select_in_64<EPL, WPR>(z, b, base, a.E, a.k, a.score, redd, redi, my_id, my_z);
      }
    } else {
      my_z = key_value(my_key);
    }
  }

  if (WPR > 1 && threadIdx.x >= 64) return;  // k <= 64: the picks lie in the first wave
  const bool live = slot < a.k;
  const float w = chosen_weight(my_z, live, a.score, a.norm, a.scale, row_max, row_sum);
  if (live) {
    a.ids[(size_t)t * a.k + slot] = my_id;
    a.w[(size_t)t * a.k + slot] = w;
  }
}

struct TopkBackArgs {
  const void* z;
  const int32_t* ids;
  const float* dw;
  void* dz;
  long long ld, ldd;
  int T, k, E, score, norm, vec, vecd;
  float scale;
};

// dz of one row per wave (16 waves above 1024 experts): the first wave's
// lanes j < k form their pick's term; the terms reach the threads that hold
// their experts through an LDS row, in ascending j where an expert repeats.
template <class LT, int EPL, int WPR>
__global__ __launch_bounds__(WPR > 1 ? 64 * WPR : 64 * kRowsPerBlock) void k_router_topk_backward(TopkBackArgs a) {
  typedef typename LT::mem mem;
  __shared__ float redf[WPR];
  __shared__ __attribute__((aligned(16))) float rows[WPR > 1 ? 1 : kRowsPerBlock][WPR > 1 ? 4 : 64 * EPL];
  const int lane = threadIdx.x & 63;
  const int slot = WPR > 1 ? (int)threadIdx.x : lane;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int t = WPR > 1 ? (int)blockIdx.x : (int)blockIdx.x * kRowsPerBlock + wave;
  if (t >= a.T) return;
  const int base = slot * EPL;
  const mem* row = static_cast<const mem*>(a.z) + (size_t)t * a.ld;
  // every wave of the row forms the k terms for itself
  int id = -1;
  float g = 0.0f, z = 0.0f;
  if (lane < a.k) {
    id = a.ids[(size_t)t * a.k + lane];
    g = a.dw[(size_t)t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) z = LT::load(row[id]);
  }
  const bool live = id >= 0;
  float out[EPL], term;
  if (a.score == kRouterScoreSoftmax && !a.norm) {
    load_row<LT, EPL>(row, base, a.E, a.vec, -__builtin_inff(), out);
    float m = out[0], sum = 0.0f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, out[i]);
    m = row_all<WPR>(m, OpMaxF(), redf);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      out[i] = exp_below(out[i], m);
      sum += out[i];
    }
    sum = row_all<WPR>(sum, OpSumF(), redf);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    term = live ? a.scale * (exp_below(z, m) * inv) * g : 0.0f;
    const float dot = wave_all(term, OpSumF());
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = -(out[i] * inv) * dot;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
    float p, damp = 1.0f;
    if (a.score == kRouterScoreSoftmax) {
      const float m = wave_all(live ? z : -__builtin_inff(), OpMaxF());
      p = live ? exp_below(z, m) : 0.0f;
    } else {
      p = live ? sigmoid_f32(z) : 0.0f;
      damp = sigmoid_f32(-z);
    }
    if (a.norm) {
      const float sum = wave_all(p, OpSumF());
      p = sum == 0.0f ? 0.0f : p / sum;
      g -= wave_all(live ? p * g : 0.0f, OpSumF());
    }
    term = live ? a.scale * p * g * damp : 0.0f;
  }
  bool repeats = true;
  if constexpr (WPR == 1) {
    float* mine = rows[wave];
    // does an expert repeat?  each pick leaves its lane and looks whether it stayed
    if (live) mine[id] = __int_as_float(lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    repeats = __any(live && __float_as_int(mine[live ? id : 0]) != lane);
    if (!repeats) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < EPL; ++i) mine[base + i] = 0.0f;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (live) mine[id] = term;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] += mine[base + i];
    }
  }
  if (repeats) {
    for (int j = 0; j < a.k; ++j) {
      const int at = __builtin_amdgcn_readlane(id, j) - base;
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(term), j));
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] += at == i ? v : 0.0f;
    }
  }
  store_row<LT, EPL>(static_cast<mem*>(a.dz) + (size_t)t * a.ldd, base, a.E, a.vecd, out);
}

int check_router(int dtype, long long ld, int T, int k, int E, int score, int norm) {
  if (T < 0 || k < 1 || E < 1 || k > E || ld < E) return MOE_Q4_ERR_SHAPE;
  if (E > MOE_Q4_MAX_E || k > MOE_Q4_ROUTER_MAX_K) return MOE_Q4_ERR_UNSUPPORTED;
  if (dtype != MOE_Q4_DTYPE_BF16 && dtype != MOE_Q4_DTYPE_F32 && dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (score != MOE_Q4_SCORE_SOFTMAX && score != MOE_Q4_SCORE_SIGMOID) return MOE_Q4_ERR_UNSUPPORTED;
  if (norm != 0 && norm != 1) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

bool aligned_to(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

size_t span(int T, long long ld, int E, size_t es) { return T ? ((size_t)(T - 1) * (size_t)ld + (size_t)E) * es : 0; }

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" int moe_router_topk(const void* logits, int logits_dtype, long long ld, const float* select_bias, int T,
                               int k, int E, int score, int renormalize, float scale, int32_t* topk_ids,
                               float* topk_weights, hipStream_t stream) {
  const int st = check_router(logits_dtype, ld, T, k, E, score, renormalize);
  if (st) return st;
  if (T == 0) return MOE_Q4_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_Q4_ERR_NULL;
  const size_t es = logits_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4) || !aligned_to(select_bias, 4))
    return MOE_Q4_ERR_ALIGN;
  const size_t pairs = (size_t)T * k * 4, in = span(T, ld, E, es);
  if (overlap(topk_ids, pairs, logits, in) || overlap(topk_weights, pairs, logits, in) ||
      overlap(topk_ids, pairs, topk_weights, pairs) || overlap(topk_ids, pairs, select_bias, select_bias ? (size_t)E * 4 : 0) ||
      overlap(topk_weights, pairs, select_bias, select_bias ? (size_t)E * 4 : 0))
    return MOE_Q4_ERR_ALIAS;
  const RowPlan plan = row_plan(E);
  TopkArgs a{logits, select_bias, topk_ids, topk_weights, ld, T, k, E, score, renormalize, 0, scale};
  a.vec = row_vec(logits, ld, E, plan.epl, (int)es);
  const dim3 grid(plan.wpr > 1 ? T : (T + kRowsPerBlock - 1) / kRowsPerBlock);
  const dim3 block(plan.wpr > 1 ? 64 * plan.wpr : 64 * kRowsPerBlock);
#define MOE_TOPK_CALL(LT, EPL, WPR)                                                                    \
  if (select_bias)                                                                                     \
    hipLaunchKernelGGL((k_router_topk<LT, EPL, WPR, true>), grid, block, 0, stream, a);                \
  else                                                                                                 \
    hipLaunchKernelGGL((k_router_topk<LT, EPL, WPR, false>), grid, block, 0, stream, a)
  MOE_ROW_DISPATCH(logits_dtype, plan, MOE_TOPK_CALL)
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

extern "C" int moe_router_topk_backward(const void* logits, int logits_dtype, long long ld, const int32_t* topk_ids,
                                        const float* dweights, int T, int k, int E, int score, int renormalize,
                                        float scale, void* dlogits, long long ldd, hipStream_t stream) {
  const int st = check_router(logits_dtype, ld, T, k, E, score, renormalize);
  if (st) return st;
  if (ldd < E) return MOE_Q4_ERR_SHAPE;
  if (T == 0) return MOE_Q4_OK;
  if (!logits || !topk_ids || !dweights || !dlogits) return MOE_Q4_ERR_NULL;
  const size_t es = logits_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(topk_ids, 4) || !aligned_to(dweights, 4))
    return MOE_Q4_ERR_ALIGN;
  const size_t pairs = (size_t)T * k * 4, out = span(T, ldd, E, es);
  if (overlap(dlogits, out, logits, span(T, ld, E, es)) || overlap(dlogits, out, topk_ids, pairs) ||
      overlap(dlogits, out, dweights, pairs))
    return MOE_Q4_ERR_ALIAS;
  const RowPlan plan = row_plan(E);
  TopkBackArgs a{logits, topk_ids, dweights, dlogits, ld, ldd, T, k, E, score, renormalize, 0, 0, scale};
  a.vec = row_vec(logits, ld, E, plan.epl, (int)es);
  a.vecd = row_vec(dlogits, ldd, E, plan.epl, (int)es);
  const dim3 grid(plan.wpr > 1 ? T : (T + kRowsPerBlock - 1) / kRowsPerBlock);
  const dim3 block(plan.wpr > 1 ? 64 * plan.wpr : 64 * kRowsPerBlock);
#define MOE_TOPK_BACK_CALL(LT, EPL, WPR) \
  hipLaunchKernelGGL((k_router_topk_backward<LT, EPL, WPR>), grid, block, 0, stream, a)
  MOE_ROW_DISPATCH(logits_dtype, plan, MOE_TOPK_BACK_CALL)
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
