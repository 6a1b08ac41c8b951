// Kernels of the gated feed-forward block and its gradient, for 16-bit types.
// Each type is instantiated in a source of its own (moe_glu_inst_*.hip).
// Internal header.
//
//   forward   g = x Wg^T, u = x Wu^T, h = silu(g) u: one product whose tile takes
//             the same rows of Wg and Wu, so that a lane holds g and u of a result
//   backward  dg = dh u silu'(g), du = dh silu(g), side by side as D;
//             dx = D [Wg; Wu], [dWg; dWu] = D^T x
// The backward's products have their sums along the other axis of the weights,
// or of both D and x, which the tiles read as they are.
// 8192 x 6144 x 2048 bf16, each kernel by itself: forward with g and u kept 317
// us (1300 TFLOP/s), dg and du 40, dx 317, dw 320, a call of all four 1031; the
// forward alone, sustained, 274 to 281 (1470 to 1500), where a library product
// of its size reaches 1598; 4 tokens 8.2 us, 6.1 TB/s.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_gemm_device.h"
#include "moe_gemm_plan.h"
#include "moe_q4.h"

namespace moeq4 {

struct GluArgs {
  const unsigned char *x, *wg, *wu;  // rows ldx, ldw bytes apart
  void* h;                           // or NULL
  float* saved;                      // [2][T][I], or NULL
  float* part;                       // split K: [splits][2][T][I]
  long long ldx, ldw, ldh;           // ldh in elements
  int T, H, I;
  GemmTiles tiles;
};

// dx [M, N] = D [b0; b1], or out [M, N] = D^T b0 (K tokens), whose rows from
// `cut` on go to out1.
struct GluMmArgs {
  const unsigned char *a, *b0, *b1;  // rows lda, ldb bytes apart
  void *out0, *out1;
  float* part;                       // split K: [splits][M][N]
  long long lda, ldb, ldo;           // ldo in elements
  int M, N, K, steps, cut;           // K of b0, and its steps
  int ip;                            // of D: du lies ip elements behind dg
  const float* back;                 // fp16: what one of D's units is worth
  GemmTiles tiles;
};

// Launches for each type; MOE_Q4_* status.
int glu_forward_bf16(const GluArgs& a, bool rows, const GemmPlan& p, hipStream_t stream);
int glu_forward_f16(const GluArgs& a, bool rows, const GemmPlan& p, hipStream_t stream);
int glu_mm_bf16(const GluMmArgs& a, const GemmPlan& p, hipStream_t stream);
int glu_mm_f16(const GluMmArgs& a, const GemmPlan& p, hipStream_t stream);
// D [T][2 ip], dg and du of I each, from g, u and dh (lddh elements apart);
// `scale` is of fp16 (kGluScaleBytes): back, and the workgroups' largest.
int glu_grad_bf16(const float* saved, const void* dh, long long lddh, int T, int I, int ip, void* d, float* scale, hipStream_t stream);
int glu_grad_f16(const float* saved, const void* dh, long long lddh, int T, int I, int ip, void* d, float* scale, hipStream_t stream);
constexpr int kGluMost = 1024, kGluScaleBytes = 256 + 4 * kGluMost;

#ifdef MOE_GLU_INST

template <int KIND> struct GluType;
template <> struct GluType<kGemmBf16> { typedef __bf16 type; };
template <> struct GluType<kGemmF16> { typedef _Float16 type; };

// 1 / (1 + e^-g): the exponential of the hardware's 2^x is off by about
// 2^-24 |g| of itself, far below a 16-bit result's half step.
__device__ __forceinline__ float glu_sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// A tile of 32 of B's rows is 16 of Wg's and the same 16 of Wu's.
template <class S>
struct GluSource {
  const GluArgs& a;
  static constexpr bool kTokT = false, kRowT = false;
  const unsigned char *tok, *row;
  int toks, rows;
  __device__ __forceinline__ uint32_t k(int s) const { return (uint32_t)s * kGemmStep; }
  __device__ __forceinline__ int left(int s) const { return 2 * a.H - s * kGemmStep; }
  __device__ __forceinline__ void set(const GemmPlace& p) {
    tok = a.x + (size_t)p.tok * S::kTok * a.ldx;
    // a thread's rows are 32 apart, a wave's 8 threads of them side by side
    row = (__builtin_amdgcn_readfirstlane(threadIdx.x) / 8 % 32 < 16 ? a.wg : a.wu) + (size_t)p.row * (S::kRows / 2) * a.ldw;
    toks = a.T - 1 - p.tok * S::kTok;
    rows = a.I - 1 - p.row * (S::kRows / 2);
  }
  __device__ __forceinline__ uint32_t tok_off(int r) const { return (uint32_t)min(r, toks) * (uint32_t)a.ldx; }
  __device__ __forceinline__ const unsigned char* row_base(int) const { return row; }
  __device__ __forceinline__ uint32_t row_off(int r) const { return (uint32_t)min(r / 32 * 16 + r % 16, rows) * (uint32_t)a.ldw; }
};

template <int KIND, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_glu_tiles(GluArgs a) {
  using S = GemmShape<KIND, MT, NT, WM, WN>;
  typedef typename GluType<KIND>::type T16;
  static_assert(S::kThreads / 8 == 32, "GluSource's rows");
  GluSource<S> source{a};
  gemm_tiles<S>(a.tiles, source, [&](const GemmPlace& p, const gemm_f32x4 (&acc)[MT][NT]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = gemm_opaque(threadIdx.x & 63), kb = lane >> 4;
    const int t0 = p.tok * S::kTok + wave % WM * MT * 16 + (lane & 15), n0 = p.row * (S::kRows / 2) + wave / WM * NT * 8;
    const bool split = a.tiles.splits > 1;
    float* keep = split ? a.part + (size_t)p.split * 2 * a.T * a.I : a.saved;
    T16* h = split ? nullptr : static_cast<T16*>(a.h);
    // g and u are read again by a backward pass at the earliest (8192 x 6144 x 2048 309 us through the caches, 302 past
    // them; of rows that are no multiple of 64 bytes, 1537 x 2056 x 1416, 31 and 39)
    const bool past = !split && ((uintptr_t)a.saved | 4 * (uintptr_t)a.I) % 64 == 0;
    // (I is a multiple of 8: neighbours are all there or none)
    const auto keep4 = [&](size_t row, int t, int n, gemm_f32x4 v) __attribute__((always_inline)) {
      if (t >= a.T || n >= a.I) return;
      float* to = keep + (row + t) * a.I + n;
      if (past)
        gemm_put32_past(to, v);
      else
        gemm_put32(to, 4, v);
    };
    const auto put8 = [&](int t, int n, uint4 v) __attribute__((always_inline)) {
      if (t < a.T && n < a.I) gemm_put16(h + (size_t)t * a.ldh + n, 8, v);
    };
    uint2 alone = make_uint2(0, 0);  // of an odd number of pairs the last one's, for the next tokens
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int t = t0 + 16 * mt;
      uint2 before = make_uint2(0, 0);
#pragma unroll
      for (int q = 0; q < NT / 2; ++q) {
        const gemm_f32x4 gate = gemm_here(acc[mt][2 * q]), up = gemm_here(acc[mt][2 * q + 1]);
        if (keep) {
          keep4(0, t, n0 + 16 * q + 4 * kb, gate);
          keep4(a.T, t, n0 + 16 * q + 4 * kb, up);
        }
        gemm_f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = gate[i] * glu_sigmoid(gate[i]) * up[i];
        const uint2 out = gemm_pack4<T16>(v);
        if (q % 2) {
          const uint4 eight = gemm_eight16(before, out);
          if (h) put8(t, n0 + 16 * (q - 1) + 8 * kb, eight);
        } else if (q + 1 < NT / 2) {
          before = out;
        } else if (mt % 2) {
          const uint4 eight = gemm_eight16(alone, out);
          if (h) put8(t - 16 + 16 * (kb >> 1), n0 + 16 * q + 8 * (kb & 1), eight);
        } else {
          alone = out;
        }
      }
    }
  });
}

// Few tokens: 8 rows of Wg and the same of Wu a workgroup, their inputs spread
// over its waves; G x 8 tokens.
template <int KIND, int G, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void k_glu_rows(GluArgs a) {
  typedef typename GluType<KIND>::type T16;
  __shared__ float lds[WAVES][2][G][64];
  const int wave = threadIdx.x >> 6, row0 = blockIdx.x * 8, index = gemm_rows_index();
  // (I is a multiple of 8: every row is there)
  const unsigned char *tok[G], *const row[2] = {a.wg + (size_t)(row0 + index) * a.ldw, a.wu + (size_t)(row0 + index) * a.ldw};
  const float* none[G];
  gemm_f32x4 acc[2][G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    tok[g] = a.x + (size_t)min(8 * g + index, a.T - 1) * a.ldx;
    none[g] = nullptr;
    acc[0][g] = acc[1][g] = gemm_f32x4{0, 0, 0, 0};
  }
  gemm_rows<KIND, 2, G, U>(row, tok, 2 * a.H, wave, WAVES, a.tiles.steps, nullptr, none, acc);
  gemm_join_waves<2, G, WAVES>(lds, acc);
  for (int i = threadIdx.x; i < G * 8 * 8; i += 64 * WAVES) {  // 8 neighbours of a token to as many lanes
    const int t = i / 8, r = i % 8, n = row0 + r, at = r / 2 * 16 + t % 8 * 2 + r % 2;
    if (t >= a.T) continue;
    const float g = lds[0][0][t / 8][at], u = lds[0][1][t / 8][at];
    if (a.saved) {
      a.saved[(size_t)t * a.I + n] = g;
      a.saved[((size_t)a.T + t) * a.I + n] = u;
    }
    if (a.h) static_cast<T16*>(a.h)[(size_t)t * a.ldh + n] = (T16)(g * glu_sigmoid(g) * u);
  }
}

// Partial sums of a split K, added in their order: g and u, and h of them.
template <int KIND>
__global__ __launch_bounds__(256) void k_glu_join(GluArgs a, int splits) {
  typedef typename GluType<KIND>::type T16;
  const size_t all = (size_t)a.T * a.I / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (size_t)gridDim.x * 256) {
    float s[2][8], v[8];
#pragma unroll
    for (int up = 0; up < 2; ++up) {
      gemm_join8(a.part + up * all * 8 + i * 8, 2 * all * 8, splits, s[up]);
      if (a.saved) norm_store8(a.saved + up * all * 8 + i * 8, 8, s[up]);
    }
    if (a.h) {
      const size_t t = i * 8 / a.I;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = s[0][j] * glu_sigmoid(s[0][j]) * s[1][j];
      norm_store8(static_cast<T16*>(a.h) + t * a.ldh + (i * 8 - t * a.I), 8, v);
    }
  }
}

// dx: D's rows, and the weights across; steps of Wg's and then of Wu's rows.
template <class S>
struct GluDxSource {
  const GluMmArgs& a;
  static constexpr bool kTokT = false, kRowT = true;
  const unsigned char* tok;
  int toks, col;
  __device__ __forceinline__ void set(const GemmPlace& p) {
    tok = a.a + (size_t)p.tok * S::kTok * a.lda;
    toks = a.M - 1 - p.tok * S::kTok;
    col = p.row * S::kRows;
  }
  __device__ __forceinline__ int part(int s) const { return s >= a.steps ? s - a.steps : s; }
  __device__ __forceinline__ uint32_t k(int s) const { return (uint32_t)(part(s) * kGemmStep + (s >= a.steps ? 2 * a.ip : 0)); }
  __device__ __forceinline__ int left(int s) const { return 2 * a.K - part(s) * kGemmStep; }
  __device__ __forceinline__ uint32_t tok_off(int r) const { return (uint32_t)min(r, toks) * (uint32_t)a.lda; }
  __device__ __forceinline__ const unsigned char* row_at(int s) const { return (s >= a.steps ? a.b1 : a.b0) + (size_t)part(s) * 64 * a.ldb; }
  __device__ __forceinline__ long long row_ld() const { return a.ldb; }
  __device__ __forceinline__ uint32_t row_col(int c) const { return 2u * (uint32_t)min(col + 8 * c, a.N - 8); }
};

// dWg and dWu: D and x across, steps of tokens.
template <class S>
struct GluDwSource {
  const GluMmArgs& a;
  static constexpr bool kTokT = true, kRowT = true;
  int tok, col;
  __device__ __forceinline__ void set(const GemmPlace& p) {
    tok = p.tok * S::kTok;
    col = p.row * S::kRows;
  }
  __device__ __forceinline__ int left(int s) const { return 2 * a.K - s * kGemmStep; }
  __device__ __forceinline__ const unsigned char* tok_at(int s) const { return a.a + (size_t)s * 64 * a.lda; }
  __device__ __forceinline__ long long tok_ld() const { return a.lda; }
  __device__ __forceinline__ uint32_t tok_col(int c) const {
    const int m = min(tok + 8 * c, a.M - 8);
    return 2u * (uint32_t)(m < a.cut ? m : m - a.cut + a.ip);
  }
  __device__ __forceinline__ const unsigned char* row_at(int s) const { return a.b0 + (size_t)s * 64 * a.ldb; }
  __device__ __forceinline__ long long row_ld() const { return a.ldb; }
  __device__ __forceinline__ uint32_t row_col(int c) const { return 2u * (uint32_t)min(col + 8 * c, a.N - 8); }
};

template <int KIND>
__device__ __forceinline__ gemm_f32x4 glu_back(gemm_f32x4 v, float back) {
  if constexpr (KIND == kGemmF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= back;
  }
  return v;
}

template <int KIND, bool DW, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_glu_mm(GluMmArgs a) {
  using S = GemmShape<KIND, MT, NT, WM, WN>;
  typedef typename GluType<KIND>::type T16;
  std::conditional_t<DW, GluDwSource<S>, GluDxSource<S>> source{a};
  const float back = KIND == kGemmF16 ? *a.back : 1.0f;
  gemm_tiles<S>(a.tiles, source, [&](const GemmPlace& p, const gemm_f32x4 (&acc)[MT][NT]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = gemm_opaque(threadIdx.x & 63), kb = lane >> 4;
    const int m0 = p.tok * S::kTok + wave % WM * MT * 16 + (lane & 15), n0 = p.row * S::kRows + wave / WM * NT * 16;
    float* part = a.tiles.splits > 1 ? a.part + (size_t)p.split * a.M * a.N : nullptr;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int m = m0 + 16 * mt;
      const size_t row = (size_t)(m < a.cut ? m : m - a.cut) * a.ldo;
      T16* to = static_cast<T16*>(m < a.cut ? a.out0 : a.out1) + row;
      // (N is a multiple of 8: neighbours are all there or none)
#pragma unroll
      for (int nt = 0; nt < NT; nt += 2) {
        const gemm_f32x4 u = gemm_here(acc[mt][nt]), v = gemm_here(acc[mt][nt + 1]);
        if (part) {
          const int n = n0 + 16 * nt + 4 * kb;
          if (m < a.M && n < a.N) gemm_put32(part + (size_t)m * a.N + n, 4, u);
          if (m < a.M && n + 16 < a.N) gemm_put32(part + (size_t)m * a.N + n + 16, 4, v);
        } else {
          const int n = n0 + 16 * nt + 8 * kb;
          const uint4 q = gemm_eight16(gemm_pack4<T16>(glu_back<KIND>(u, back)), gemm_pack4<T16>(glu_back<KIND>(v, back)));
          if (m < a.M && n < a.N) gemm_put16(to + n, 8, q);
        }
      }
    }
  });
}

// (N is a multiple of 8)
template <int KIND>
__global__ __launch_bounds__(256) void k_glu_mm_join(GluMmArgs a, int splits) {
  typedef typename GluType<KIND>::type T16;
  const size_t all = (size_t)a.M * a.N / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (size_t)gridDim.x * 256) {
    float s[8];
    gemm_join8(a.part + i * 8, all * 8, splits, s);
    if constexpr (KIND == kGemmF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] *= *a.back;
    }
    const int m = (int)(i * 8 / a.N), n = (int)(i * 8 - (size_t)m * a.N);
    norm_store8(static_cast<T16*>(m < a.cut ? a.out0 : a.out1) + (size_t)(m < a.cut ? m : m - a.cut) * a.ldo + n, 8, s);
  }
}

// dg and du of 8 neighbours.
template <class T16>
struct GluGrad {
  float g[8], u[8], e[8], dg[8], du[8];
  __device__ __forceinline__ void load(const float* saved, const void* dh, long long lddh, size_t all, int I, size_t i) {
    const size_t t = i / I, n = i - t * I;
    norm_load8(saved + i, 8, g);
    norm_load8(saved + all + i, 8, u);
    norm_load8(static_cast<const T16*>(dh) + t * lddh + n, 8, e);
  }
  __device__ __forceinline__ void compute() {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = glu_sigmoid(g[j]);
      dg[j] = e[j] * u[j] * (s * __builtin_fmaf(g[j], 1.0f - s, 1.0f));
      du[j] = e[j] * (g[j] * s);
    }
  }
};

// dg and du enter the matrix cores as 16-bit numbers, rounded once: products of
// fp32 numbers run at a fraction of that rate, and the gradients' error is 1.4
// times that of their own rounding alone (bf16 2.35e-3 and 1.66e-3).
// fp16 has not the range for them, though dh, u and the gradients are of it:
// with a loss scale, dh = 10^4 and u = 20 give an infinity, and without one,
// 10^-6 and 0.02 nothing, where the sum over the tokens is an ordinary number.
// So they are kept over a power of two that puts the call's largest finite one
// between 2^14 and 2^15: those down to 2^-28 of it have all of fp16's bits.  The
// sums are multiplied by that power again, before their one rounding.  Finding
// the largest reads g, u and dh once more (1537 x 1416: 5 us of 99).
__device__ __forceinline__ float glu_most(float most, float v) { return fabsf(v) < __builtin_inff() ? fmaxf(most, fabsf(v)) : most; }
__device__ __forceinline__ float glu_most256(float v) {  // of the workgroup's 256 threads
  __shared__ float waves[4];
  v = norm_max16(v);
  v = fmaxf(v, __shfl_xor(v, 16));
  v = fmaxf(v, __shfl_xor(v, 32));
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(waves[0], waves[1]), fmaxf(waves[2], waves[3]));
}
template <int KIND>
__global__ __launch_bounds__(256) void k_glu_most(const float* saved, const void* dh, long long lddh, int T, int I, float* most) {
  const size_t all = (size_t)T * I;
  float m = 0.0f;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; i < all; i += (size_t)gridDim.x * 2048) {
    GluGrad<typename GluType<KIND>::type> v;
    v.load(saved, dh, lddh, all, I, i);
    v.compute();
#pragma unroll
    for (int j = 0; j < 8; ++j) m = glu_most(glu_most(m, v.dg[j]), v.du[j]);
  }
  m = glu_most256(m);
  if (threadIdx.x == 0) most[blockIdx.x] = m;
}

// 8 of a token's I a thread.
template <int KIND>
__global__ __launch_bounds__(256) void k_glu_grad(const float* saved, const void* dh, long long lddh, int T, int I, int ip, void* d,
                                                  float* scale, int groups) {
  typedef typename GluType<KIND>::type T16;
  const size_t all = (size_t)T * I;
  size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  GluGrad<T16> v;
  if (i < all) v.load(saved, dh, lddh, all, I, i);
  float up = 1.0f;
  if constexpr (KIND == kGemmF16) {
    float m = 0.0f;
    for (int k = threadIdx.x; k < groups; k += 256) m = fmaxf(m, scale[64 + k]);
    m = glu_most256(m);
    // (where the largest is below 2^-86, both gradients are 0 in fp16)
    up = m > 0.0f ? ldexpf(1.0f, min(14 - ilogbf(m), 100)) : 1.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) scale[0] = 1.0f / up;
  }
  while (i < all) {
    v.compute();
    if constexpr (KIND == kGemmF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v.dg[j] *= up;
        v.du[j] *= up;
      }
    }
    const size_t t = i / I, n = i - t * I;
    T16* to = static_cast<T16*>(d) + t * 2 * ip + n;
    norm_store8(to, 8, v.dg);
    norm_store8(to + ip, 8, v.du);
    i += (size_t)gridDim.x * 2048;
    if (i < all) v.load(saved, dh, lddh, all, I, i);
  }
}

template <int KIND>
int glu_forward_kind(const GluArgs& a, bool rows, const GemmPlan& p, hipStream_t stream) {
  if (rows) {  // as many loads on their way as the registers of 16 waves hold
    const dim3 grid(a.I / 8);
    if (a.T <= 8)
      hipLaunchKernelGGL((k_glu_rows<KIND, 1, 16, 6>), grid, dim3(1024), 0, stream, a);
    else if (a.T <= 16)
      hipLaunchKernelGGL((k_glu_rows<KIND, 2, 16, 4>), grid, dim3(1024), 0, stream, a);
    else
      hipLaunchKernelGGL((k_glu_rows<KIND, 4, 16, 3>), grid, dim3(1024), 0, stream, a);
    return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
  }
  const dim3 grid(p.workgroups);
  switch (p.shape) {
    case kGemm256x256: hipLaunchKernelGGL((k_glu_tiles<KIND, 8, 8, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm256x192: hipLaunchKernelGGL((k_glu_tiles<KIND, 8, 6, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x256: hipLaunchKernelGGL((k_glu_tiles<KIND, 4, 8, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x192: hipLaunchKernelGGL((k_glu_tiles<KIND, 4, 6, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x128: hipLaunchKernelGGL((k_glu_tiles<KIND, 4, 4, 2, 2>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((k_glu_tiles<KIND, 4, 2, 1, 4>), grid, dim3(256), 0, stream, a); break;
  }
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.tiles.splits > 1) {
    const size_t all = (size_t)a.T * a.I / 8;
    hipLaunchKernelGGL((k_glu_join<KIND>), dim3((unsigned)std::min<size_t>((all + 255) / 256, 4096)), dim3(256), 0, stream, a, p.tiles.splits);
  }
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

template <int KIND, bool DW>
void glu_mm_launch(const GluMmArgs& a, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid(p.workgroups);
  switch (p.shape) {
    case kGemm256x256: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 8, 8, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm256x192: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 8, 6, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x256: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 4, 8, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x192: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 4, 6, 2, 2>), grid, dim3(256), 0, stream, a); break;
    case kGemm128x128: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 4, 4, 2, 2>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((k_glu_mm<KIND, DW, 4, 2, 1, 4>), grid, dim3(256), 0, stream, a); break;
  }
}

template <int KIND>
int glu_mm_kind(const GluMmArgs& a, const GemmPlan& p, hipStream_t stream) {
  if (a.b1)
    glu_mm_launch<KIND, false>(a, p, stream);
  else
    glu_mm_launch<KIND, true>(a, p, stream);
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.tiles.splits > 1) {
    const size_t all = (size_t)a.M * a.N / 8;
    hipLaunchKernelGGL((k_glu_mm_join<KIND>), dim3((unsigned)std::min<size_t>((all + 255) / 256, 4096)), dim3(256), 0, stream, a, p.tiles.splits);
  }
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}

template <int KIND>
int glu_grad_kind(const float* saved, const void* dh, long long lddh, int T, int I, int ip, void* d, float* scale, hipStream_t stream) {
  const size_t all = ((size_t)T * I + 2047) / 2048;
  const int groups = (int)std::min<size_t>(all, kGluMost);
  if constexpr (KIND == kGemmF16) {
    hipLaunchKernelGGL((k_glu_most<KIND>), dim3((unsigned)groups), dim3(256), 0, stream, saved, dh, lddh, T, I, scale + 64);
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  const dim3 grid((unsigned)std::min<size_t>(all, 8192));
  hipLaunchKernelGGL((k_glu_grad<KIND>), grid, dim3(256), 0, stream, saved, dh, lddh, T, I, ip, d, scale, groups);
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
#endif

}  // namespace moeq4
