// Product in 8 bits with a scale for each block of 128:
//   out[t, n] = sum_b sx[t, b] sw[n / 128, b] (sum over c in block b of x[t, c] w[n, c]) + bias[n]
// A block of 128 inputs is one step of the matrix cores: its sum comes out of
// one instruction and enters the fp32 accumulator by one multiply-add with
// sx sw.  fp32 results, and those of few tokens, which memory bounds either
// way, multiply the codes as bf16 (kGemmFp8Wide).
// 8192 x 12288 x 6144: 530 to 545 us, 2300 TFLOP/s, sustained 502 (a library
// product with one scale 386), with fp32 results 1145; 1 x 6144 x 6144: 8.2 us, 4.6 TB/s;
// 16 tokens 11.6, 24 tokens 12.5 + 1.8; 96 x 2050 x 4096 in fp32: 10.4 + 2.2.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "moe_args.h"
#include "moe_gemm_device.h"
#include "moe_gemm_plan.h"
#include "moe_q4.h"

namespace moeq4 {
namespace {

struct Fp8Args {
  const unsigned char* x;
  const float* sx;
  const unsigned char* w;
  const float* sw;
  const float* bias;
  void* out;
  float* part;  // split K: [splits][L][N]
  long long ldx, ldo;
  int L, N, K, G, out_dtype;
  GemmTiles tiles;
  int row0;  // by rows: the launch's first
};

template <class S>
struct Fp8Source {
  const Fp8Args& a;
  const unsigned char *tok, *row;
  const float* scales;
  int toks, rows;  // the tile's last token and row
  __device__ __forceinline__ void set(const GemmPlace& p) {
    const int tok0 = p.tok * S::kTok, row0 = p.row * S::kRows, tid = threadIdx.x;
    tok = a.x + (size_t)tok0 * a.ldx;
    row = a.w + (size_t)row0 * a.K;
    toks = a.L - 1 - tok0;
    rows = a.N - 1 - row0;
    scales = tid < S::kTok ? a.sx + (size_t)min(tok0 + tid, a.L - 1) * a.G
                           : a.sw + (size_t)min(row0 / 128 + tid - S::kTok, (a.N - 1) / 128) * a.G;
  }
  __device__ __forceinline__ uint32_t tok_off(int r) const { return (uint32_t)min(r, toks) * (uint32_t)a.ldx; }
  __device__ __forceinline__ const unsigned char* row_base(int) const { return row; }
  __device__ __forceinline__ uint32_t row_off(int r) const { return (uint32_t)min(r, rows) * (uint32_t)a.K; }
};

template <int KIND, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_tiles(Fp8Args a) {
  using S = GemmShape<KIND, MT, NT, WM, WN>;
  Fp8Source<S> source{a};
  gemm_tiles_scaled<S>(a.tiles, a.K, source, [&](const GemmPlace& p, const gemm_f32x4 (&acc)[MT][NT]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = p.tok * S::kTok + wave % WM * MT * 16, n0 = p.row * S::kRows + wave / WM * NT * 16;
    const int lane = gemm_opaque(threadIdx.x & 63), n16 = lane & 15, kb = lane >> 4;
    const bool fp32 = a.part || a.out_dtype == MOE_Q4_DTYPE_F32, bf16 = a.out_dtype == MOE_Q4_DTYPE_BF16;
    float* to = a.part ? a.part + (size_t)p.split * a.L * a.N : static_cast<float*>(a.out);
    const long long ld = a.part ? a.N : a.ldo;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int t = t0 + 16 * mt + n16;
      const bool row = t < a.L;
      float* to32 = to + t * ld + n0 + 4 * kb;
      uint16_t* to16 = static_cast<uint16_t*>(a.out) + t * ld + n0 + 8 * kb;
#pragma unroll
      for (int nt = 0; nt < NT; nt += 2) {
        gemm_f32x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + 16 * (nt + h) + 4 * kb;
          v[h] = gemm_here(acc[mt][nt + h]);
          if (a.bias && !a.part) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] += a.bias[min(n + i, a.N - 1)];
          }
          if (fp32 && row) gemm_put32(to32 + 16 * (nt + h), a.N - n, v[h]);
        }
        if (!fp32) {
          const uint4 q = bf16 ? gemm_eight16(gemm_pack4<__bf16>(v[0]), gemm_pack4<__bf16>(v[1]))
                               : gemm_eight16(gemm_pack4<_Float16>(v[0]), gemm_pack4<_Float16>(v[1]));
          if (row) gemm_put16(to16 + 16 * nt, a.N - n0 - 16 * nt - 8 * kb, q);
        }
      }
    }
  });
}

// 8 J rows of w a workgroup, their inputs spread over its waves; G x 8 tokens.
template <int J, int G, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void k_fp8_rows(Fp8Args a) {
  __shared__ float lds[WAVES][J][G][64];
  const int wave = threadIdx.x >> 6, row0 = a.row0 + blockIdx.x * 8 * J, index = gemm_rows_index();
  const unsigned char *tok[G], *row[J];
  const float* sx[G];
  gemm_f32x4 acc[J][G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const size_t t = min(8 * g + index, a.L - 1);
    tok[g] = a.x + t * a.ldx;
    sx[g] = a.sx + t * a.G;
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j][g] = gemm_f32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int j = 0; j < J; ++j) row[j] = a.w + (size_t)min(row0 + 8 * j + index, a.N - 1) * a.K;
  gemm_rows<kGemmFp8Wide, J, G, U>(row, tok, a.K, wave, WAVES, a.G, a.sw + (size_t)(row0 / 128) * a.G, sx, acc);
  gemm_join_waves<J, G, WAVES>(lds, acc);
  // neighbours of a token to as many lanes
  for (int i = threadIdx.x; i < G * 8 * J * 8; i += 64 * WAVES) {
    const int t = i / (8 * J), r = i % (8 * J), n = row0 + r;
    if (t >= a.L || n >= a.N) continue;
    float v = lds[0][r / 8][t / 8][r % 8 / 2 * 16 + t % 8 * 2 + r % 2];
    if (a.bias) v += a.bias[n];
    const size_t at = (size_t)t * a.ldo + n;
    if (a.out_dtype == MOE_Q4_DTYPE_F32)
      static_cast<float*>(a.out)[at] = v;
    else if (a.out_dtype == MOE_Q4_DTYPE_BF16)
      static_cast<__bf16*>(a.out)[at] = (__bf16)v;
    else
      static_cast<_Float16*>(a.out)[at] = (_Float16)v;
  }
}

// Partial sums of a split K, added in their order.
__global__ __launch_bounds__(256) void k_fp8_join(const float* part, const float* bias, void* out, long long ldo, int L, int N,
                                                  int splits, int dtype) {
  const size_t all = (size_t)L * N;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (size_t)gridDim.x * 256) {
    const size_t t = i / N;
    const int n = (int)(i - t * N);
    float s = part[i];
    for (int p = 1; p < splits; p += 4) {  // four parts' loads on their way together
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = part[(size_t)min(p + u, splits - 1) * all + i];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p + u < splits) s += v[u];
    }
    if (bias) s += bias[n];
    const size_t at = t * ldo + n;
    if (dtype == MOE_Q4_DTYPE_F32)
      static_cast<float*>(out)[at] = s;
    else if (dtype == MOE_Q4_DTYPE_BF16)
      static_cast<__bf16*>(out)[at] = (__bf16)s;
    else
      static_cast<_Float16*>(out)[at] = (_Float16)s;
  }
}

int fp8_status(int L, int N, int K) {
  if (L < 0 || N < 1 || K < 1) return MOE_Q4_ERR_SHAPE;
  if (K % 16 || L > MOE_Q4_LINEAR_MAX_L || N > MOE_Q4_LINEAR_MAX_N || K > MOE_Q4_LINEAR_MAX_K) return MOE_Q4_ERR_UNSUPPORTED;
  if ((long)L * N > 1L << 40) return MOE_Q4_ERR_UNSUPPORTED;  // (2^31 tiles and more)
  return MOE_Q4_OK;
}

// Measured with 256 tiles and with as many as are held at once, of 8, 32 and
// 128 steps.
constexpr GemmCosts kFp8Costs = {{1.62f, 0, 0, 0, 0.64f, 0.41f}, {0, 0, 0, 0, 0.47f, 0.32f}, {8.5f, 0, 0, 0, 4.3f, 3.5f}, {1, 0, 0, 0, 2, 3}};
// (tiles of 256 x 256 were not built for it)
constexpr GemmCosts kFp8WideCosts = {{0, 0, 0, 0, 1.02f, 0.69f}, {0, 0, 0, 0, 0.83f, 0.465f}, {0, 0, 0, 0, 7.0f, 5.0f}, {0, 0, 0, 0, 2, 3}};
// Few tokens by rows, whose weights then pass the card once at the memory's
// rate; from 17 tokens on the tiles' matrix instructions are the faster for
// large weights (us by rows and by tiles, 24 tokens: 2050 x 4096 9.7 and 10.7,
// 6144 x 6144 17.1 and 14.9, 12288 x 6144 32 and 22; 16 tokens 7.5 and 10.7,
// 12.5 and 14.9, 23.5 and 21.7).
bool fp8_by_rows(int L, int N, int K) { return L <= 16 || (L <= 32 && (long)N * K < 1L << 24); }
// Up to 32 tokens, and fp32 results, with the codes as bf16.
bool fp8_wide(int L, int out_dtype) { return L <= 32 || out_dtype == MOE_Q4_DTYPE_F32; }
GemmPlan fp8_plan(int L, int N, int K, bool wide) { return gemm_plan(wide ? kFp8WideCosts : kFp8Costs, L, N, (K + 127) / 128); }
size_t fp8_part(int L, int N, int K, bool wide) {
  const GemmPlan p = fp8_plan(L, N, K, wide);
  return p.tiles.splits > 1 ? ((size_t)p.tiles.splits * L * N * 4 + 255) & ~size_t(255) : 0;
}

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" size_t moe_linear_fp8_workspace_bytes(int L, int N, int K) {
  if (fp8_status(L, N, K) || L == 0 || fp8_by_rows(L, N, K)) return 0;
  return std::max(fp8_part(L, N, K, false), fp8_part(L, N, K, true));
}

extern "C" int moe_linear_fp8_forward(const uint8_t* x, long long ldx, const float* sx, const uint8_t* w, const float* sw,
                                      const float* bias, int L, int N, int K, void* out, int out_dtype, long long ldo,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = fp8_status(L, N, K);
  if (st) return st;
  if (ldx < K || ldo < N) return MOE_Q4_ERR_SHAPE;
  const size_t os = args_size(out_dtype);
  if (!os || (L > 1 && ldx > MOE_Q4_LINEAR_MAX_LDX)) return MOE_Q4_ERR_UNSUPPORTED;
  if (L == 0) return MOE_Q4_OK;
  if (!x || !sx || !w || !sw || !out) return MOE_Q4_ERR_NULL;
  if (!args_aligned(x, 16) || (L > 1 && ldx % 16) || !args_aligned(w, 16) || !args_aligned(sx, 4) || !args_aligned(sw, 4) ||
      !args_aligned(bias, 4) || !args_aligned(out, os))
    return MOE_Q4_ERR_ALIGN;
  const size_t need = moe_linear_fp8_workspace_bytes(L, N, K);
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (need && !args_aligned(workspace, 256)) return MOE_Q4_ERR_ALIGN;
  const int G = (K + 127) / 128;
  const ArgSpan ins[] = {{x, args_span(L, ldx, K, 1)}, {sx, (size_t)L * G * 4}, {w, (size_t)N * K},
                         {sw, ((size_t)N + 127) / 128 * G * 4}, {bias, bias ? (size_t)N * 4 : 0}};
  const ArgSpan outs[] = {{out, args_span(L, ldo, N, os)}, {need ? workspace : nullptr, need}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  Fp8Args a{x, sx, w, sw, bias, out, nullptr, ldx, ldo, L, N, K, G, out_dtype, {}, 0};
  if (fp8_by_rows(L, N, K)) {
    // 32 rows of w share a workgroup's reads of x where that leaves most compute units one (us, 16 and 32 rows:
    // 16 tokens 6144 x 6144 15.1 and 12.6, 4099 x 4112 9.4 and 10.6; 32 tokens 27 and 19, 16.1 and 13.8)
    const bool wide = L > 8 && N >= (L > 16 ? 4096 : 6144);
    const int most = 1 << 26;  // rows of a launch, which holds fewer than 2^32 threads
    for (; a.row0 < N; a.row0 += most) {
      const int n = std::min(most, N - a.row0);
      const dim3 grid(wide ? (n + 31) / 32 : (n + 15) / 16);
      if (L <= 8)
        hipLaunchKernelGGL((k_fp8_rows<2, 1, 8, 6>), grid, dim3(512), 0, stream, a);
      else if (L <= 16 && wide)
        hipLaunchKernelGGL((k_fp8_rows<4, 2, 8, 6>), grid, dim3(512), 0, stream, a);
      else if (L <= 16)
        hipLaunchKernelGGL((k_fp8_rows<2, 2, 8, 3>), grid, dim3(512), 0, stream, a);
      else if (wide)
        hipLaunchKernelGGL((k_fp8_rows<4, 4, 8, 2>), grid, dim3(512), 0, stream, a);
      else
        hipLaunchKernelGGL((k_fp8_rows<2, 4, 8, 2>), grid, dim3(512), 0, stream, a);
      if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
    }
    return MOE_Q4_OK;
  }
  const bool codes_bf16 = fp8_wide(L, out_dtype);
  const GemmPlan p = fp8_plan(L, N, K, codes_bf16);
  a.tiles = p.tiles;
  if (p.tiles.splits > 1) a.part = static_cast<float*>(workspace);
  const dim3 grid(p.workgroups);
  if (codes_bf16) {
    if (p.shape == kGemm128x128)
      hipLaunchKernelGGL((k_fp8_tiles<kGemmFp8Wide, 4, 4, 2, 2>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_fp8_tiles<kGemmFp8Wide, 4, 2, 1, 4>), grid, dim3(256), 0, stream, a);
  } else {
    switch (p.shape) {
      case kGemm256x256: hipLaunchKernelGGL((k_fp8_tiles<kGemmFp8, 8, 4, 2, 4>), grid, dim3(512), 0, stream, a); break;
      case kGemm128x128: hipLaunchKernelGGL((k_fp8_tiles<kGemmFp8, 4, 4, 2, 2>), grid, dim3(256), 0, stream, a); break;
      default: hipLaunchKernelGGL((k_fp8_tiles<kGemmFp8, 4, 2, 1, 4>), grid, dim3(256), 0, stream, a); break;
    }
  }
  if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  if (p.tiles.splits > 1) {
    const size_t all = (size_t)L * N;
    hipLaunchKernelGGL(k_fp8_join, dim3((unsigned)std::min<size_t>((all + 255) / 256, 4096)), dim3(256), 0, stream, a.part,
                       bias, out, ldo, L, N, p.tiles.splits, out_dtype);
  }
  return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
}
