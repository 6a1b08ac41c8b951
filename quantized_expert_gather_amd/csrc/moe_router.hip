// The router's selection: the k experts of each token from its router
// logits, their weights, and the weights' gradient.
//
//   p = softmax(z) or sigmoid(z); the k largest of z (or of p + select_bias);
//   w_j = scale * p_j / sum over the chosen (renormalised), or scale * p_j.
//
// The threads of a row take its largest value k times: each thread's largest,
// the row's, and the lowest expert that has it.  z is read once.
//
// Bound by a launch where there are few tokens (4 x 256 fp32, k = 8, with a
// bias: 3.8 us) and by vector instructions where there are many: 16384 x 256
// bf16, k = 8 takes 9.0 us, its 8.4 MB two.  16-bit logits without a bias
// make order and expert one word, so a thread's keys can be sorted once and a
// round is one reduction and a shift (8.3 us of a captured run; 9.8 with a
// maximum, the lowest expert that has it and its removal each round); the
// reductions stay in registers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <limits.h>
#include <stdint.h>

#include "moe_q4.h"
#include "moe_router_device.h"

namespace moeq4 {
namespace {

constexpr int kTopkThreads = 256;  // of a workgroup, 256 / LPR rows each (E <= 1024)

struct TopkArgs {
  const void* z;
  const float* bias;
  int32_t* ids;
  float* w;
  long long ld;
  int T, k, E, score, norm;
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

// What one round of the selection found.
struct Pick {
  int key, id;
};

// The largest key among the row's threads, lowest expert first, and takes it
// out.
template <class LT, int EPL, int LPR>
__device__ __forceinline__ Pick take_largest(int (&key)[EPL], int slot, int* red) {
  int lm = key[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) lm = lm > key[i] ? lm : key[i];
  Pick p;
  p.key = row_all<LPR>(lm, OpMaxI(), red);
  int mine = INT_MAX, at = 0;
#pragma unroll
  for (int i = EPL - 1; i >= 0; --i) {
    const bool hit = key[i] == p.key;
    at = hit ? i : at;
    mine = hit ? row_expert<LT, EPL, LPR>(slot, i) : mine;
  }
  p.id = row_all<LPR>(mine, OpMinI(), red);
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (mine == p.id && at == i) key[i] = kKeyTaken;
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
template <int LO, int N, int STEP, int EPL>
__device__ __forceinline__ void merge_falling(int (&k)[EPL]) {
  auto order = [&](int x, int y) __attribute__((always_inline)) {
    const int hi = k[x] > k[y] ? k[x] : k[y], lo = k[x] > k[y] ? k[y] : k[x];
    k[x] = hi;
    k[y] = lo;
  };
  if constexpr (2 * STEP < N) {
    merge_falling<LO, N, 2 * STEP>(k);
    merge_falling<LO + STEP, N, 2 * STEP>(k);
#pragma unroll
    for (int i = LO + STEP; i + STEP < LO + N; i += 2 * STEP) order(i, i + STEP);
  } else {
    order(LO, LO + STEP);
  }
}
template <int LO, int N, int EPL>
__device__ __forceinline__ void sort_falling(int (&k)[EPL]) {  // by odd-even merges
  if constexpr (N > 1) {
    sort_falling<LO, N / 2>(k);
    sort_falling<LO + N / 2, N / 2>(k);
    merge_falling<LO, N, 1>(k);
  }
}

// The same selection with the scores in 64 bits, for the rows whose 32-bit
// scores lie too close to be told apart: lane j keeps pick j.
template <class LT, int EPL, int LPR>
__device__ void select_in_64(const float (&z)[EPL], const float (&b)[EPL], int slot, int E, int k, int score,
                             double* red, int* red_id, int& my_id, float& my_z) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kHalf = LPR > 64 ? 32 : LPR / 2, kWaves = LPR > 64 ? LPR / 64 : 1;
  double s[EPL];
  uint32_t open = 0;  // bit i: value i not yet chosen
  for (int i = 0; i < EPL; ++i) open |= (row_expert<LT, EPL, LPR>(slot, i) < E ? 1u : 0u) << i;
  auto all = [&](double v, bool max) {
    for (int o = kHalf; o > 0; o >>= 1) {
      const double u = __shfl_xor(v, o, 64);
      v = max ? (u > v ? u : v) : v + u;
    }
    if constexpr (kWaves > 1) {
      __syncthreads();
      if (lane == 0) red[wave] = v;
      __syncthreads();
      v = red[0];
      for (int w = 1; w < kWaves; ++w) v = max ? (red[w] > v ? red[w] : v) : v + red[w];
    }
    return v;
  };
  if (score == kRouterScoreSoftmax) {
    double m = -__builtin_inf(), sum = 0.0;
    for (int i = 0; i < EPL; ++i)
      if (((open >> i) & 1u) && (double)z[i] > m) m = (double)z[i];
    m = all(m, true);
    for (int i = 0; i < EPL; ++i) {
      // (NaN stays NaN, also in a row of nothing else)
      s[i] = !((open >> i) & 1u) ? 0.0 : z[i] != z[i] || m > -__builtin_inf() ? exp((double)z[i] - m) : 0.0;
      sum += s[i];
    }
    sum = all(sum, false);
    for (int i = 0; i < EPL; ++i) s[i] = (sum == 0.0 ? 0.0 : s[i] / sum) + (double)b[i];
  } else {
    for (int i = 0; i < EPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)z[i])) + (double)b[i];
  }
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
        id = row_expert<LT, EPL, LPR>(slot, i);
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
    for (int o = kHalf; o > 0; o >>= 1) {
      const double u = __shfl_xor(v, o, 64);
      const int uid = __shfl_xor(id, o, 64);
      const float uz = __shfl_xor(zs, o, 64);
      if (better(u, uid, v, id)) {
        v = u;
        id = uid;
        zs = uz;
      }
    }
    if constexpr (kWaves > 1) {
      __syncthreads();
      if (lane == 0) {
        red[wave] = v;
        red_id[wave] = id;
        red_id[kWaves + wave] = __float_as_int(zs);
      }
      __syncthreads();
      int bw = 0;
      for (int w = 1; w < kWaves; ++w)
        if (better(red[w], red_id[w], red[bw], red_id[bw])) bw = w;
      id = red_id[bw];
      zs = __int_as_float(red_id[kWaves + bw]);
    }
    if (mine == id) open &= ~(1u << at);
    if (slot == j) {
      my_id = id;
      my_z = zs;
    }
  }
}

// Puts the picks that lanes j < held hold in order by their scores in 64 bits
// (they are the row's first `held` already).  `base`: the row's exp_base.
// Every lane of the wave calls it.
template <int EPL, int LPR>
__device__ void order_in_64(const float (&z)[EPL], const float* bias, int slot, int held, int score, float base, int& my_id,
                            float& my_z) {
  double s = 0.0, sum = 0.0;
  if (score == kRouterScoreSoftmax) {
#pragma unroll 1
    for (int i = 0; i < EPL; ++i) {
      float zi = z[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) zi = i == j ? z[j] : zi;
      sum += exp((double)zi - (double)base);  // 0 past E
    }
    for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  }
  if (slot < held) {
    if (score == kRouterScoreSoftmax)
      s = sum > 0.0 ? exp((double)my_z - (double)base) / sum : 0.0;
    else
      s = 1.0 / (1.0 + exp(-(double)my_z));
    s += (double)bias[my_id];
  }
  // neighbours change places, even and odd pairs in turn, until none does
  int still = 0;
  for (int r = 0; r <= held + 1 && still < 2; ++r) {
    const int other = r & 1 ? ((slot + 1) ^ 1) - 1 : slot ^ 1;
    const bool pair = slot < held && other >= 0 && other < held;
    const int from = (threadIdx.x & 63) + (pair ? other - slot : 0);
    const double s2 = __shfl(s, from, 64);
    const int id2 = __shfl(my_id, from, 64);
    const float z2 = __shfl(my_z, from, 64);
    // numbers before NaN, the larger, the lower expert
    const bool n1 = s != s, n2 = s2 != s2;
    const bool first = n1 != n2 ? n2 : !n1 && s != s2 ? s > s2 : my_id < id2;
    const bool swap = pair && (slot < other) != first;
    if (swap) {
      s = s2;
      my_id = id2;
      my_z = z2;
    }
    still = __any(swap) ? 0 : still + 1;
  }
}

// Sigmoid scores of a row's picks (z of the lanes that are live) over their sum.
// Every lane of the wave calls it.
template <int LANES>
__device__ __forceinline__ float chosen_sigmoid(float z, bool live) {
  float s = live ? sigmoid_f32(z) : 0.0f, sum = row_all<LANES>(s, OpSumF());
  const bool low = sum < kLowSum;
  if (__any(low)) {
    const float base = exp_base(row_all<LANES>(live ? z : -__builtin_inff(), OpMaxF()));
    const float u = live ? sigmoid_from(z, low ? base : 0.0f) : 0.0f, all = row_all<LANES>(u, OpSumF());
    s = low ? u : s;
    sum = low ? all : sum;
  }
  return sum == 0.0f ? 0.0f : s / sum;
}

// Weights of the chosen: thread j < k of the row holds logit z of pick j.
// Every thread of the wave calls it; the sums run over the row's lanes (the
// first wave's).
template <int LPR>
__device__ __forceinline__ float chosen_weight(float z, bool live, int score, int norm, float scale, float row_base,
                                               float row_sum) {
  constexpr int kLanes = LPR > 64 ? 64 : LPR;
  if (score == kRouterScoreSoftmax) {
    if (norm) {
      const float m = exp_base(row_all<kLanes>(live ? z : -__builtin_inff(), OpMaxF()));
      const float e = live ? exp_f32(z - m) : 0.0f;
      const float sum = row_all<kLanes>(e, OpSumF());
      return sum == 0.0f ? 0.0f : scale * (e / sum);
    }
    return row_sum == 0.0f ? 0.0f : scale * (exp_f32(z - row_base) / row_sum);
  }
  if (!norm) return scale * (live ? sigmoid_f32(z) : 0.0f);
  return scale * chosen_sigmoid<kLanes>(z, live);
}

template <class LT, int EPL, int LPR, bool BIAS>
__global__ __launch_bounds__(LPR > 64 ? LPR : kTopkThreads) void k_router_topk(TopkArgs a) {
  constexpr bool kPacked = !BIAS && LPR <= 64 && sizeof(typename LT::mem) == 2;
  constexpr int kWaves = LPR > 64 ? LPR / 64 : 1, kGroups = (LPR > 64 ? LPR : kTopkThreads) / LPR;
  typedef typename LT::mem mem;
  __shared__ int red[kWaves];
  __shared__ float redf[kWaves];
  __shared__ double redd[kWaves];
  __shared__ int redi[2 * kWaves];
  const int tid = threadIdx.x, slot = tid % LPR;
  const int want = blockIdx.x * kGroups + tid / LPR, t = min(want, a.T - 1);  // rows past T do the last one's work
  const mem* row = static_cast<const mem*>(a.z) + (size_t)t * a.ld;
  float z[EPL];
  load_row<LT, EPL, LPR>(row, slot, a.E, -__builtin_inff(), z);

  // softmax statistics, where the whole row counts
  float row_base = 0.0f, row_sum = 1.0f;
  float e[EPL];
  if (a.score == kRouterScoreSoftmax && (BIAS || !a.norm)) {
    row_base = z[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) row_base = fmaxf(row_base, z[i]);
    row_base = exp_base(row_all<LPR>(row_base, OpMaxF(), redf));
    row_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      e[i] = exp_f32(z[i] - row_base);
      row_sum += e[i];
    }
    row_sum = row_all<LPR>(row_sum, OpSumF(), redf);
  }

  int my_id = 0;
  float my_z = 0.0f;
  int key[EPL];
  if constexpr (kPacked) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int ex = row_expert<LT, EPL, LPR>(slot, i);
      key[i] = ex < a.E ? packed_key<LT>(z[i], ex) : kKeyTaken;
    }
    sort_falling<0, EPL>(key);
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
      const int m = row_all<LPR>(key[0], OpMaxI());
      if (slot == j) mine = m;
      // by a mask: a selection between two elements becomes a computed index to the compiler
      const int own = key[0] == m ? -1 : 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = (key[i] & ~own) | ((i + 1 < EPL ? key[i + 1] : kKeyTaken) & own);
    }
    my_id = 0xFFFF - (mine & 0xFFFF);
    my_z = packed_value<LT>(mine);
  } else {
    float b[BIAS ? EPL : 1];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int ex = row_expert<LT, EPL, LPR>(slot, i);
      float v = z[i];
      if constexpr (BIAS) {
        b[i] = ex < a.E ? a.bias[ex] : 0.0f;
        v = (a.score == kRouterScoreSoftmax ? (row_sum == 0.0f ? 0.0f : e[i] / row_sum) : sigmoid_f32(z[i])) + b[i];
      }
      key[i] = ex < a.E ? order_key(v) : kKeyTaken;
    }
    int my_key = 0;
    Pick last{};
    // with a bias one pick more than the lanes hold, for the comparison; they
    // hold the pick after the k-th too where there is a lane for it
    const bool spare = BIAS && LPR <= 64 && a.k < LPR;
    const int held = BIAS ? min(a.E, a.k + spare) : a.k, rounds = BIAS ? min(a.E, a.k + spare + 1) : a.k;
    for (int j = 0; j < rounds; ++j) {
      last = take_largest<LT, EPL, LPR>(key, slot, red);
      if (slot == j) {
        my_id = last.id;
        my_key = last.key;
      }
    }
    if constexpr (BIAS) {
      // Two neighbours in the order of different logits or biases that fp32
      // cannot tell apart: with |d| the distance from the row's maximum, a
      // softmax p is off by at most 2^-24 (1.5 |d| + 80) p (the exponential,
      // its sum, the quotient), |d| <= 88 where p is not 0 and p |d| <= 0.4: by
      // 1.3e-5 p and by 4e-6 in any case.  A sigmoid is off by 2^-24 (1.5 |z|
      // (1 - p) + 5) p: by 8.2e-6 p and by 4e-7.  The sum with the bias adds
      // 2^-24 of itself.  Lanes hold the picks and compare with the next.  The
      // rest of the row, whose errors are at most those of its largest p, lies
      // at the last pick or below: the first k are among the picks held
      // unless that one is close to the k-th.
      bool close = false, open = false;
      if (LPR <= 64 || tid < 64) {
        const int id2 = __shfl_down(my_id, 1, 64), key2 = __shfl_down(my_key, 1, 64);
        const bool softmax = a.score == kRouterScoreSoftmax;
        if (slot < held) {
          my_z = LT::load(row[my_id]);
          const float s1 = key_value(my_key), s0 = key_value(key2), step = 5e-7f * fabsf(s1);
          if (slot + 1 < held && !(s1 - s0 > 8e-6f + step)) {
            const float b1 = a.bias[my_id], b0 = a.bias[id2], p = fabsf(s1 - b1) + fabsf(s0 - b0);
            const float off = softmax ? fminf(8e-6f, 1.3e-5f * p) : fminf(8e-7f, 8.2e-6f * p);
            close = !(s1 - s0 > off + step) && !(LT::load(row[id2]) == my_z && b0 == b1);
          }
          if (slot == a.k - 1 && rounds > held)
            open = !(s1 - key_value(last.key) > (softmax ? fminf(8e-6f, 2.6e-5f / row_sum) : 8e-7f) + step);
        }
        open = __any(open);
        close = __any(close);
      }
      if constexpr (LPR > 64) {
        __syncthreads();
        if (tid == 0) redi[0] = open || close;
        __syncthreads();
        open = redi[0];
        __syncthreads();
      }
      if (open)
        select_in_64<LT, EPL, LPR>(z, b, slot, a.E, a.k, a.score, redd, redi, my_id, my_z);
      else if constexpr (LPR <= 64) {
        if (close) order_in_64<EPL, LPR>(z, a.bias, slot, held, a.score, row_base, my_id, my_z);
      }
    } else {
      my_z = key_value(my_key);
    }
  }

  if (LPR > 64 && tid >= 64) return;  // k <= 64: the picks lie in the first wave
  const bool live = slot < a.k;
  const float w = chosen_weight<LPR>(my_z, live, a.score, a.norm, a.scale, row_base, row_sum);
  if (live && want < a.T) {
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
  int T, k, E, score, norm;
  float scale;
};

// w_j's gradient g_j, in the logits: renormalised p_j (g_j - sum_i p_i g_i)
// at the chosen only (times 1 - sigmoid(z_j) for sigmoid scores), else the
// softmax's over the whole row, which is read for that alone.  Bound by the
// gradient it writes: 16384 x 256 bf16, k = 8: 5.0 us for 9.5 MB, most of it
// zeros; 5003 x 288 fp32 over the whole row: 5.5 us for 11.8 MB.
//
// dz of rows as the selection holds them: a row's lanes j < k form their
// pick's term; the terms reach the threads that hold their experts through an
// LDS row, in ascending j where an expert repeats.
template <class LT, int EPL, int LPR>
__global__ __launch_bounds__(LPR > 64 ? LPR : kTopkThreads) void k_router_topk_backward(TopkBackArgs a) {
  typedef typename LT::mem mem;
  constexpr int kThreads = LPR > 64 ? LPR : kTopkThreads, kGroups = kThreads / LPR, kLanes = LPR > 64 ? 64 : LPR;
  __shared__ float redf[LPR > 64 ? LPR / 64 : 1];
  __shared__ __attribute__((aligned(16))) float rows[LPR > 64 ? 1 : kGroups][LPR > 64 ? 4 : LPR * EPL];
  const int tid = threadIdx.x, slot = tid % LPR, group = tid / LPR;
  const int pick = LPR > 64 ? (tid & 63) : slot;  // every wave of a large row forms the terms for itself
  const int want = blockIdx.x * kGroups + group, t = min(want, a.T - 1);
  const mem* row = static_cast<const mem*>(a.z) + (size_t)t * a.ld;
  int id = -1;
  float g = 0.0f, z = 0.0f;
  if (pick < a.k) {
    id = a.ids[(size_t)t * a.k + pick];
    g = a.dw[(size_t)t * a.k + pick];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) z = LT::load(row[id]);
  }
  const bool live = id >= 0;
  float out[EPL], term;
  if (a.score == kRouterScoreSoftmax && !a.norm) {
    load_row<LT, EPL, LPR>(row, slot, a.E, -__builtin_inff(), out);
    float m = out[0], sum = 0.0f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, out[i]);
    m = exp_base(row_all<LPR>(m, OpMaxF(), redf));
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      out[i] = exp_f32(out[i] - m);
      sum += out[i];
    }
    sum = row_all<LPR>(sum, OpSumF(), redf);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    term = live ? a.scale * (exp_f32(z - m) * inv) * g : 0.0f;
    const float dot = row_all<kLanes>(term, OpSumF());
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = -(out[i] * inv) * dot;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
    float p, damp = 1.0f;
    if (a.score == kRouterScoreSoftmax) {  // (renormalised: else above)
      const float m = exp_base(row_all<kLanes>(live ? z : -__builtin_inff(), OpMaxF()));
      p = live ? exp_f32(z - m) : 0.0f;
      const float sum = row_all<kLanes>(p, OpSumF());
      p = sum == 0.0f ? 0.0f : p / sum;
    } else {
      p = a.norm ? chosen_sigmoid<kLanes>(z, live) : live ? sigmoid_f32(z) : 0.0f;
      damp = sigmoid_f32(-z);
    }
    if (a.norm) g -= row_all<kLanes>(live ? p * g : 0.0f, OpSumF());
    term = live ? a.scale * p * g * damp : 0.0f;
  }
  bool repeats = true;
  if constexpr (LPR <= 64) {
    // thread slot's value i lies at i * LPR + slot; expert e's place follows
    constexpr int V = row_chunk<LT, EPL>();
    float* mine = rows[group];
    const int e = live ? id : 0, at = (e / (LPR * V) * V + e % V) * LPR + e / V % LPR;
    // does an expert repeat?  each pick leaves its slot and looks whether it stayed
    if (live) mine[at] = __int_as_float(slot);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    repeats = __any(live && __float_as_int(mine[at]) != slot);
    if (!repeats) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < EPL; ++i) mine[i * LPR + slot] = 0.0f;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (live) mine[at] = term;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] += mine[i * LPR + slot];
    }
  }
  if (repeats) {
    const int lane0 = (tid & 63) & ~(kLanes - 1);
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl(id, lane0 + j, 64);
      const float v = __shfl(term, lane0 + j, 64);
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] += row_expert<LT, EPL, LPR>(slot, i) == e ? v : 0.0f;
    }
  }
  if (want < a.T) store_row<LT, EPL, LPR>(static_cast<mem*>(a.dz) + (size_t)t * a.ldd, slot, a.E, out);
}

int check_router(int dtype, long long ld, int T, int k, int E, int score, int norm) {
  if (T < 0 || k < 1 || E < 1 || k > E || ld < E) return MOE_Q4_ERR_SHAPE;
  if (E > MOE_Q4_MAX_E || k > MOE_Q4_ROUTER_MAX_K || T > MOE_Q4_ROUTER_MAX_T) return MOE_Q4_ERR_UNSUPPORTED;
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
  // Few lanes a row where there are rows enough to fill the card with them
  // (k = 8 of 256, us over 16 lanes and over 64: 16384 fp32 rows 9.9 and 15.0,
  // with a bias 16.7 and 20.0, bf16 8.3 and 9.6; 8192 with a bias 9.5 and
  // 12.2, 4096 8.7 and 7.8, bf16 4.7 and 4.1; 1000 4.5 and 3.0).
  const RowPlan plan = row_plan(E, k, T <= 6144);
  const int threads = plan.lpr > 64 ? plan.lpr : kTopkThreads, per = threads / plan.lpr, most = rows_of_launch(plan.lpr);
#define MOE_TOPK_CALL(LT, EPL, LPR)                                                                    \
  if (select_bias)                                                                                     \
    hipLaunchKernelGGL((k_router_topk<LT, EPL, LPR, true>), grid, block, 0, stream, a);                \
  else                                                                                                 \
    hipLaunchKernelGGL((k_router_topk<LT, EPL, LPR, false>), grid, block, 0, stream, a)
  for (int t = 0; t < T; t += most) {
    const int n = std::min(most, T - t);
    const TopkArgs a{static_cast<const unsigned char*>(logits) + (size_t)t * ld * es, select_bias, topk_ids + (size_t)t * k,
                     topk_weights + (size_t)t * k, ld, n, k, E, score, renormalize, scale};
    const dim3 grid((n + per - 1) / per), block(threads);
    MOE_ROW_DISPATCH(logits_dtype, plan, MOE_TOPK_CALL)
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  return MOE_Q4_OK;
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
  // 2048 x 256 bf16: 2.9 us over 16 lanes a row, 2.7 over 64; 4096: 3.1 and 3.4
  const RowPlan plan = row_plan(E, k, T <= 2048);
  const int threads = plan.lpr > 64 ? plan.lpr : kTopkThreads, per = threads / plan.lpr, most = rows_of_launch(plan.lpr);
#define MOE_TOPK_BACK_CALL(LT, EPL, LPR) \
  hipLaunchKernelGGL((k_router_topk_backward<LT, EPL, LPR>), grid, block, 0, stream, a)
  for (int t = 0; t < T; t += most) {
    const int n = std::min(most, T - t);
    const TopkBackArgs a{static_cast<const unsigned char*>(logits) + (size_t)t * ld * es, topk_ids + (size_t)t * k,
                         dweights + (size_t)t * k, static_cast<unsigned char*>(dlogits) + (size_t)t * ldd * es, ld, ldd, n, k, E,
                         score, renormalize, scale};
    const dim3 grid((n + per - 1) / per), block(threads);
    MOE_ROW_DISPATCH(logits_dtype, plan, MOE_TOPK_BACK_CALL)
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  return MOE_Q4_OK;
}
