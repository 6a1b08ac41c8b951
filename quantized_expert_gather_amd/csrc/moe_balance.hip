// The router's balance loss and the per-expert route counts, with the loss's
// gradient.  Per sequence of n unmasked tokens:
//
//   p = softmax(z), or sigmoid(z) over its row sum;  P_e = sum_t p[t, e] / n;
//   c_e = number of routes to e;  loss = coef * E / (k * n) * sum_e c_e P_e;
//   dz = p (a - sum_e a_e p_e) (softmax; times 1 - sigmoid(z) for sigmoid),
//   a_e = dloss * coef * E * c_e / (k * n^2), the counts held fixed.
//
// What it has to move is z, once each way, and dz: 32768 x 256 bf16 takes
// 9.6 + 4.8 us forward (16.8 MB) and 10.5 us backward (33.6 MB).  A launch
// here takes about 3.5 us whatever it does; the rest is the exponentials'
// vector work and the latency of a workgroup's first rows, which 256
// workgroups of 16 waves, one a compute unit, pay once (128 of them: 12.9 us).
//
// Forward: a workgroup sums p over its run of tokens in registers (a wave
// holds whole rows) and its routes in an LDS histogram of integers, and
// leaves one row of partials in the workspace; a second launch adds the
// partials in a fixed order.  Nothing depends on an order of atomics.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "moe_q4.h"
#include "moe_router_device.h"

namespace moeq4 {
namespace {

// Waves of a workgroup, each thread group taking kRows rows at a time: their
// loads are all on their way before the first is used, and their reductions
// interleave.
constexpr int kPartialWaves = 16, kBackWaves = 4;
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <int EPL, int LPR>
constexpr int kRows = LPR > 64 ? 1 : EPL == 4 ? 4 : EPL == 8 ? 2 : 1;

struct BalanceArgs {
  const void* z;
  const int32_t* ids;
  const uint8_t* mask;
  float* psum;      // [S][blocks][E] partial sums of p
  int32_t* pcount;  // [S][blocks][E] partial route counts
  int32_t* ptok;    // [S][blocks] unmasked tokens
  float* pdot;      // [S][chunks] sums of c_e p_e over a chunk of experts
  int32_t* ticket;  // [S] chunks done
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  long long ld;
  int S, T, k, E, score;
  int blocks, per;  // workgroups of a sequence, tokens of each
  int chunks;
  float coef;
};

// p of R rows but for their factor `inv`, in place of their logits, and
// 1 - sigmoid(z) in `damp` (DAMP, sigmoid scores only).  reload(r, u) reads row
// r's logits again.
template <class LT, int EPL, int LPR, int R, bool DAMP, class RELOAD>
__device__ __forceinline__ void row_probabilities(float (&v)[R][EPL], float (&damp)[DAMP ? R : 1][EPL], float (&inv)[R],
                                                  int score, float* red, RELOAD reload) {
  float sum[R];
  if (score == kRouterScoreSoftmax) {
    float m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = v[r][0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m[r] = fmaxf(m[r], v[r][i]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = exp_base(row_all<LPR>(m[r], OpMaxF(), red));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        v[r][i] = exp_f32(v[r][i] - m[r]);
        sum[r] += v[r][i];
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {  // past E the logits are -inf, their sigmoid 0
        if constexpr (DAMP)
          v[r][i] = sigmoid_pair(v[r][i], damp[r][i]);
        else
          v[r][i] = sigmoid_f32(v[r][i]);
        sum[r] += v[r][i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) sum[r] = row_all<LPR>(sum[r], OpSumF(), red);
  if (score != kRouterScoreSoftmax) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool low = sum[r] < kLowSum;  // (the same in a workgroup that holds one row)
      if (!__any(low)) continue;
      float u[EPL];
      reload(r, u);
      float m = u[0], all = 0.0f;
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, u[i]);
      m = exp_base(row_all<LPR>(m, OpMaxF(), red));
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        u[i] = sigmoid_from(u[i], low ? m : 0.0f);
        all += u[i];
        v[r][i] = low ? u[i] : v[r][i];
      }
      all = row_all<LPR>(all, OpSumF(), red);
      sum[r] = low ? all : sum[r];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) inv[r] = sum[r] == 0.0f ? 0.0f : 1.0f / sum[r];
}

// dot = sum_e c_e sum_t p[t, e]
__device__ __forceinline__ void store_loss(const BalanceArgs& a, int seq, int n, float dot) {
  const float nf = (float)n;
  a.tokens[seq] = n;
  a.loss[seq] = n ? a.coef * (float)a.E / ((float)a.k * nf) * (dot / nf) : 0.0f;
}

template <class LT, int EPL, int LPR>
__global__ __launch_bounds__(64 * kPartialWaves) void k_balance_partial(BalanceArgs a) {
  typedef typename LT::mem mem;
  constexpr int R = kRows<EPL, LPR>, kGroups = 64 * kPartialWaves / LPR;  // rows at a time
  extern __shared__ unsigned char lds[];
  float* red = reinterpret_cast<float*>(lds);            // [16]
  int32_t* ntok = reinterpret_cast<int32_t*>(lds) + 16;  // [1], padded to 16
  int32_t* hist = reinterpret_cast<int32_t*>(lds) + 32;  // [E], padded to 4
  float* sums = reinterpret_cast<float*>(hist + (a.E + 3) / 4 * 4);  // [kPartialWaves][kWide] (LPR <= 64)
  constexpr int kWide = EPL * LPR;
  const int tid = threadIdx.x, nthr = 64 * kPartialWaves;
  const int wave = tid >> 6, group = tid / LPR, slot = tid % LPR;
  const int t0 = blockIdx.x * a.per, t1 = min(a.T, t0 + a.per);
  const size_t seq = (size_t)blockIdx.y * a.T;

  // the rows after the ones at hand are on their way
  float acc[EPL], v[R][EPL], next[R][EPL], none[1][EPL];
  auto load_one = [&](int t, int r, float (&to)[EPL]) __attribute__((always_inline)) {
    load_row<LT, EPL, LPR>(static_cast<const mem*>(a.z) + (seq + min(t + r * kGroups + group, t1 - 1)) * a.ld, slot, a.E, -__builtin_inff(), to);
  };
  auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_one(t, r, next[r]);
  };
  if (t0 < t1) load(t0);
  for (int e = tid; e < a.E; e += nthr) hist[e] = 0;
  if (tid == 0) ntok[0] = 0;
  __syncthreads();
  {
    const int32_t* ids = a.ids + (seq + t0) * a.k;
    const int n = max(t1 - t0, 0) * a.k;
    for (int i = tid; i < n; i += nthr) {
      const int e = ids[i];
      if (e >= 0 && e < a.E && !(a.mask && !a.mask[seq + t0 + i / a.k])) atomicAdd(&hist[e], 1);
    }
    int live = 0;
    for (int t = t0 + tid; t < t1; t += nthr) live += !(a.mask && !a.mask[seq + t]);
    for (int o = 32; o > 0; o >>= 1) live += __shfl_xor(live, o, 64);
    if ((tid & 63) == 0 && live) atomicAdd(ntok, live);
  }

#pragma unroll
  for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
  // whole waves go round as long as one of their rows is left
  for (int t = t0; t < t1; t += R * kGroups) {
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tr = t + r * kGroups + group;
      live[r] = tr < t1 && !(a.mask && !a.mask[seq + tr]);
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[r][i] = next[r][i];
    }
    if (t + R * kGroups < t1) load(t + R * kGroups);
    float inv[R];
    row_probabilities<LT, EPL, LPR, R, false>(v, none, inv, a.score, red, [&](int r, float (&u)[EPL]) { load_one(t, r, u); });
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (live[r]) {  // (a masked row may hold anything)
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = __builtin_fmaf(v[r][i], inv[r], acc[i]);
      }
  }

  // few tokens: one workgroup finishes by itself
  const bool alone = a.blocks == 1;
  float dot = 0.0f;
  auto leave = [&](int e, float s) __attribute__((always_inline)) {
    if (alone) {
      a.counts[(size_t)blockIdx.y * a.E + e] = hist[e];
      dot += (float)hist[e] * s;
    } else {
      const size_t part = ((size_t)blockIdx.y * a.blocks + blockIdx.x) * a.E;
      a.psum[part + e] = s;
      a.pcount[part + e] = hist[e];
    }
  };
  if constexpr (LPR <= 64) {
    // a wave's rows, then the waves', in a fixed order
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (LPR <= 16) {
        const uint32_t u = __float_as_uint(acc[i]);
        const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        acc[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
      }
      if constexpr (LPR <= 32) {
        const uint32_t u = __float_as_uint(acc[i]);
        const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        acc[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
      }
    }
    if ((tid & 63) < LPR) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4)
        *reinterpret_cast<f32x4*>(sums + wave * kWide + row_expert<LT, EPL, LPR>(slot, i)) =
            f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += nthr) {
      float s = sums[e];
#pragma unroll
      for (int w = 1; w < kPartialWaves; ++w) s += sums[w * kWide + e];
      leave(e, s);
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = row_expert<LT, EPL, LPR>(slot, i);
      if (e < a.E) leave(e, acc[i]);
    }
  }
  if (alone) {
    dot = row_all<1024>(dot, OpSumF(), red);
    if (tid == 0) store_loss(a, blockIdx.y, ntok[0], dot);
  } else if (tid == 0) {
    a.ptok[(size_t)blockIdx.y * a.blocks + blockIdx.x] = ntok[0];
    if (blockIdx.x == 0) a.ticket[blockIdx.y] = 0;
  }
}

// Adds a sequence's partials: counts, token count and loss.  A workgroup takes
// kCols experts, 1024 / kCols threads sharing an expert's partials; the last
// one to finish adds the workgroups' sums in ascending order (256 partials of
// 256 experts: 4.6 us, most of it the launch and the ordering of the last).
constexpr int kCols = 32;
__global__ __launch_bounds__(1024) void k_balance_finish(BalanceArgs a) {
  constexpr int kSlices = 1024 / kCols;
  __shared__ float redf[kSlices][kCols + 1];
  __shared__ int redi[kSlices][kCols + 1];
  __shared__ int redn[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int seq = blockIdx.y;
  const size_t part = (size_t)seq * a.blocks;
  const int slice = tid / kCols, col = tid % kCols;
  int n = 0;
  for (int b = tid; b < a.blocks; b += 1024) n += a.ptok[part + b];
  const int e = blockIdx.x * kCols + col;
  float s = 0.0f;
  int c = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int b = slice; b < a.blocks; b += kSlices) {
      s += a.psum[(part + b) * a.E + e];
      c += a.pcount[(part + b) * a.E + e];
    }
  }
  redf[slice][col] = s;
  redi[slice][col] = c;
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  if (lane == 0) redn[wave] = n;
  __syncthreads();
  if (wave > 0) return;
  // lanes 0..31 and 32..63 add half the slices each
  constexpr int kHalf = kSlices / 2;
  s = 0.0f;
  c = 0;
#pragma unroll
  for (int q = 0; q < kHalf; ++q) {
    s += redf[(lane / kCols) * kHalf + q][col];
    c += redi[(lane / kCols) * kHalf + q][col];
  }
  s += __shfl_xor(s, kCols, 64);
  c += __shfl_xor(c, kCols, 64);
  if (lane < kCols && e < a.E) a.counts[(size_t)seq * a.E + e] = c;
  float dot = row_all<64>(lane < kCols ? (float)c * s : 0.0f, OpSumF());
  n = row_all<64>(lane < 16 ? redn[lane & 15] : 0, [](int x, int y) { return x + y; });
  if (lane > 0) return;
  if (a.chunks > 1) {
    float* dots = a.pdot + (size_t)seq * a.chunks;
    __hip_atomic_store(dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(a.ticket + seq, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != a.chunks - 1) return;
    dot = 0.0f;
    for (int q = 0; q < a.chunks; ++q) dot += __hip_atomic_load(dots + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  store_loss(a, seq, n, dot);
}

struct BalanceBackArgs {
  const void* z;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float* dloss;
  void* dz;
  long long ld, ldd;
  int S, T, k, E, score;
  int per;
  float coef;
};

// Rows as in the forward; a row's p is formed again, which costs less than
// keeping it (four times the bytes of bf16 logits).  The counts are the same
// for all rows of a workgroup: through LDS once, then registers (read by each
// thread for itself from memory: 16.7 us instead of 10.5).
template <class LT, int EPL, int LPR>
__global__ __launch_bounds__(LPR > 64 ? LPR : 64 * kBackWaves) void k_balance_backward(BalanceBackArgs a) {
  typedef typename LT::mem mem;
  constexpr int R = kRows<EPL, LPR>, kGroups = (LPR > 64 ? LPR : 64 * kBackWaves) / LPR;
  __shared__ float red[16];
  __shared__ __attribute__((aligned(16))) float factors[EPL * LPR];
  const int tid = threadIdx.x, group = tid / LPR, slot = tid % LPR;
  const int t0 = blockIdx.x * a.per, t1 = min(a.T, t0 + a.per);
  const size_t seq = (size_t)blockIdx.y * a.T;
  float v[R][EPL], next[R][EPL], damp[R][EPL];
  auto load_one = [&](int t, int r, float (&to)[EPL]) __attribute__((always_inline)) {
    load_row<LT, EPL, LPR>(static_cast<const mem*>(a.z) + (seq + min(t + r * kGroups + group, t1 - 1)) * a.ld, slot, a.E, -__builtin_inff(), to);
  };
  auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_one(t, r, next[r]);
  };
  load(t0);
  const float n = (float)a.tokens[blockIdx.y];
  const float f = n > 0.0f ? a.dloss[blockIdx.y] * a.coef * ((float)a.E / ((float)a.k * n)) / n : 0.0f;
  // the counts through LDS: neighbouring threads read neighbouring ones, each then its own
  for (int e = tid; e < EPL * LPR; e += blockDim.x) factors[e] = e < a.E ? f * (float)a.counts[(size_t)blockIdx.y * a.E + e] : 0.0f;
  __syncthreads();
  float w[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i += 4) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(factors + row_expert<LT, EPL, LPR>(slot, i));
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i + j] = u[j];
  }
  for (int t = t0; t < t1; t += R * kGroups) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[r][i] = next[r][i];
    if (t + R * kGroups < t1) load(t + R * kGroups);
    float dot[R], inv[R];
    row_probabilities<LT, EPL, LPR, R, true>(v, damp, inv, a.score, red, [&](int r, float (&u)[EPL]) { load_one(t, r, u); });
#pragma unroll
    for (int r = 0; r < R; ++r) {
      dot[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[r][i] *= inv[r];
#pragma unroll
      for (int i = 0; i < EPL; ++i) dot[r] += w[i] * v[r][i];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = row_all<LPR>(dot[r], OpSumF(), red);
    if (a.score != kRouterScoreSoftmax) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[r][i] *= damp[r][i];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tr = t + r * kGroups + group;
      if (tr >= t1) continue;
      const bool live = !(a.mask && !a.mask[seq + tr]);
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[r][i] = live ? v[r][i] * (w[i] - dot[r]) : 0.0f;
      store_row<LT, EPL, LPR>(static_cast<mem*>(a.dz) + (seq + tr) * a.ldd, slot, a.E, v[r]);
    }
  }
}

// Workgroups of a sequence: enough of them to fill the card; one, which
// needs no second launch, where a sequence has few values (512 x 64 fp32:
// 7.5 us, against 9.2 with two launches; 1000 x 64: 12.3 against 8.7).
constexpr int kMaxBlocks = 256;
constexpr long kAloneValues = 32768;
int blocks_of(int S, int T, int E) {
  if ((long)T * std::max(E, 64) <= kAloneValues) return 1;
  const int rows = E > 1024 ? 1 : kPartialWaves;
  const int want = std::max(1, kMaxBlocks / std::max(1, S));
  return std::max(1, std::min(want, (T + rows - 1) / rows));
}

struct BalanceWorkspace {
  size_t psum, pcount, ptok, pdot, ticket, total;
};
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
BalanceWorkspace balance_layout(int S, int T, int E) {
  BalanceWorkspace w{};
  const size_t rows = (size_t)S * blocks_of(S, T, E);
  size_t off = 0;
  w.psum = off;   off = round256(off + rows * E * 4);
  w.pcount = off; off = round256(off + rows * E * 4);
  w.ptok = off;   off = round256(off + rows * 4);
  w.pdot = off;   off = round256(off + (size_t)S * ((E + kCols - 1) / kCols) * 4);
  w.ticket = off; off = round256(off + (size_t)S * 4);
  w.total = off;
  return w;
}

int check_balance(int dtype, long long ld, int S, int T, int k, int E, int score) {
  if (S < 0 || T < 0 || k < 1 || E < 1 || k > E || ld < E) return MOE_Q4_ERR_SHAPE;
  if (E > MOE_Q4_MAX_E || S > MOE_Q4_BALANCE_MAX_SEQS || T > MOE_Q4_ROUTER_MAX_T) return MOE_Q4_ERR_UNSUPPORTED;
  if (dtype != MOE_Q4_DTYPE_BF16 && dtype != MOE_Q4_DTYPE_F32 && dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (score != MOE_Q4_SCORE_SOFTMAX && score != MOE_Q4_SCORE_SIGMOID) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

bool aligned_to(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}
size_t span(size_t rows, long long ld, int E, size_t es) { return rows ? ((rows - 1) * (size_t)ld + (size_t)E) * es : 0; }

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" size_t moe_balance_loss_workspace_bytes(int S, int T, int E) {
  if (S < 1 || T < 0 || E < 1 || E > MOE_Q4_MAX_E || S > MOE_Q4_BALANCE_MAX_SEQS || T > MOE_Q4_ROUTER_MAX_T) return 0;
  return balance_layout(S, T, E).total;
}

extern "C" int moe_balance_loss(const void* logits, int logits_dtype, long long ld, const int32_t* topk_ids,
                                const uint8_t* token_mask, int S, int T, int k, int E, int score, float coef,
                                float* loss, int32_t* counts, int32_t* tokens, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  const int st = check_balance(logits_dtype, ld, S, T, k, E, score);
  if (st) return st;
  if (S == 0) return MOE_Q4_OK;
  if (!loss || !counts || !tokens || (T > 0 && (!logits || !topk_ids))) return MOE_Q4_ERR_NULL;
  if (!workspace) return MOE_Q4_ERR_WORKSPACE;
  const size_t es = logits_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(topk_ids, 4) || !aligned_to(loss, 4) || !aligned_to(counts, 4) ||
      !aligned_to(tokens, 4) || !aligned_to(workspace, 256))
    return MOE_Q4_ERR_ALIGN;
  const BalanceWorkspace lay = balance_layout(S, T, E);
  if (workspace_bytes < lay.total) return MOE_Q4_ERR_WORKSPACE;
  const size_t rows = (size_t)S * T;
  const struct { const void* p; size_t n; } ins[] = {{logits, span(rows, ld, E, es)}, {topk_ids, rows * k * 4},
                                                     {token_mask, token_mask ? rows : 0}, {workspace, lay.total}};
  const struct { const void* p; size_t n; } outs[] = {{loss, (size_t)S * 4}, {counts, (size_t)S * E * 4},
                                                      {tokens, (size_t)S * 4}};
  for (const auto& o : outs)
    for (const auto& in : ins)
      if (overlap(o.p, o.n, in.p, in.n)) return MOE_Q4_ERR_ALIAS;
  for (int i = 0; i < 3; ++i)
    if (overlap(workspace, lay.total, ins[i].p, ins[i].n)) return MOE_Q4_ERR_ALIAS;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return MOE_Q4_ERR_ALIAS;
  const RowPlan plan = row_plan(E, 1, false);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  BalanceArgs a{};
  a.z = logits;
  a.ids = topk_ids;
  a.mask = token_mask;
  a.psum = reinterpret_cast<float*>(ws + lay.psum);
  a.pcount = reinterpret_cast<int32_t*>(ws + lay.pcount);
  a.ptok = reinterpret_cast<int32_t*>(ws + lay.ptok);
  a.pdot = reinterpret_cast<float*>(ws + lay.pdot);
  a.ticket = reinterpret_cast<int32_t*>(ws + lay.ticket);
  a.chunks = (E + kCols - 1) / kCols;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.ld = ld;
  a.S = S; a.T = T; a.k = k; a.E = E;
  a.score = score;
  a.blocks = blocks_of(S, T, E);
  a.per = (T + a.blocks - 1) / a.blocks;
  a.coef = coef;
  const dim3 grid(a.blocks, S), block(64 * kPartialWaves);
  const size_t lds = 128 + ((size_t)E + 3) / 4 * 16 + (plan.lpr > 64 ? 0 : (size_t)kPartialWaves * plan.epl * plan.lpr * 4);
#define MOE_BALANCE_CALL(LT, EPL, LPR) hipLaunchKernelGGL((k_balance_partial<LT, EPL, LPR>), grid, block, lds, stream, a)
  MOE_ROW_DISPATCH(logits_dtype, plan, MOE_BALANCE_CALL)
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (a.blocks > 1) hipLaunchKernelGGL(k_balance_finish, dim3(a.chunks, S), dim3(1024), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

extern "C" int moe_balance_loss_backward(const void* logits, int logits_dtype, long long ld, const uint8_t* token_mask,
                                         const int32_t* counts, const int32_t* tokens, const float* dloss, int S,
                                         int T, int k, int E, int score, float coef, void* dlogits, long long ldd,
                                         hipStream_t stream) {
  const int st = check_balance(logits_dtype, ld, S, T, k, E, score);
  if (st) return st;
  if (ldd < E) return MOE_Q4_ERR_SHAPE;
  if (S == 0 || T == 0) return MOE_Q4_OK;
  if (!logits || !counts || !tokens || !dloss || !dlogits) return MOE_Q4_ERR_NULL;
  const size_t es = logits_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(counts, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(dloss, 4))
    return MOE_Q4_ERR_ALIGN;
  const size_t rows = (size_t)S * T, out = span(rows, ldd, E, es);
  if (overlap(dlogits, out, logits, span(rows, ld, E, es)) || overlap(dlogits, out, token_mask, token_mask ? rows : 0) ||
      overlap(dlogits, out, counts, (size_t)S * E * 4) || overlap(dlogits, out, tokens, (size_t)S * 4) ||
      overlap(dlogits, out, dloss, (size_t)S * 4))
    return MOE_Q4_ERR_ALIAS;
  const RowPlan plan = row_plan(E, 1, false);
  BalanceBackArgs a{logits, token_mask, counts, tokens, dloss, dlogits, ld, ldd, S, T, k, E, score, 0, coef};
  // a workgroup's rows at a time, and few enough workgroups that each goes round a few times
  const int threads = plan.lpr > 64 ? plan.lpr : 64 * kBackWaves;
  const int unit = threads / plan.lpr * (plan.lpr > 64 ? 1 : plan.epl == 4 ? 4 : plan.epl == 8 ? 2 : 1);
  const int want = std::max(1, 1024 / S);
  a.per = std::max((T + want - 1) / want, unit);
  a.per = (a.per + unit - 1) / unit * unit;
  const dim3 grid((T + a.per - 1) / a.per, S), block(threads);
#define MOE_BALANCE_BACK_CALL(LT, EPL, LPR) \
  hipLaunchKernelGGL((k_balance_backward<LT, EPL, LPR>), grid, block, 0, stream, a)
  MOE_ROW_DISPATCH(logits_dtype, plan, MOE_BALANCE_BACK_CALL)
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
