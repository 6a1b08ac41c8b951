// Root-mean-square norm with the residual's addition, its gradient, and the
// quantization into 8 bits with a scale per block.
//
//   r = x + residual (rounded to the residual's type), v = 1 / sqrt(mean(r^2) + eps)
//   y = r v w, or 8-bit codes q = e4m3(y / s) with s = max(max |y| / 448, 2^-126)
//       for each 128 channels of a token
//   backward: n = r v, a = w dy: dr = v (a - n mean(a n)) + dtotal, dw = sum over tokens of dy n
//
// Bound by memory: a row is read once, held in registers as fp32 (8 channels a
// chunk, up to 2 chunks a thread) through the reduction and written once.
// 8192 x 6144 bf16 with a residual into codes: 354 MB in 73.9 us, 4.8 TB/s, as
// a large copy; 5003 x 2050 with an fp32 residual 21 us, its gradient 28 and 4;
// one row of 6144 3.1 us; 12288 x 6144 fp32 in blocks of 128 x 128 69 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "moe_args.h"
#include "moe_norm_device.h"
#include "moe_q4.h"

namespace moeq4 {
namespace {

struct NormArgs {
  const void* x;
  const void* res;   // or NULL
  const void* w;     // or NULL: ones
  void* total;       // where res is given
  void* y;           // or NULL
  uint8_t* codes;    // or NULL
  float* scales;
  long long ldx, ldr, ldt, ldy, ldc;
  int T, H, G;       // G: blocks of 128 channels of a row
  int res_f32;       // residual and total are fp32 (else x's type)
  int w_dtype, y_dtype;
  float eps;
  long row0;         // the launch's first row
};

// LANES threads share a row, each with up to C chunks of 8 channels; chunk j
// of thread l begins at channel 8 (j LANES + l), so 16 neighbours hold a block
// of 128 and a wave's loads are contiguous.
template <class TX, int LANES, int C>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void k_rms_norm(NormArgs a) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kRows = kThreads / LANES;
  const int l = threadIdx.x % LANES;
  const long row = a.row0 + (long)blockIdx.x * kRows + threadIdx.x / LANES;
  const bool live = row < a.T;
  const long at = live ? row : 0;
  float r[C][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
    norm_load8(static_cast<const TX*>(a.x) + at * a.ldx + c, n, r[j]);
  }
  if (a.res) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
      float b[8];
      if (a.res_f32)
        norm_load8(static_cast<const float*>(a.res) + at * a.ldr + c, n, b);
      else
        norm_load8(static_cast<const TX*>(a.res) + at * a.ldr + c, n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] += b[i];
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
      // the sum as it is carried on: what the norm, and a backward pass, take
      if (a.res_f32) {
        norm_store8(static_cast<float*>(a.total) + at * a.ldt + c, n, r[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = norm_round<TX>(r[j][i]);
        norm_store8(static_cast<TX*>(a.total) + at * a.ldt + c, n, r[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(r[j][i], r[j][i], sum);
  sum = norm_row_sum<LANES>(sum);
  const float v = 1.0f / sqrtf(sum / (float)a.H + a.eps);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[j][i] *= v;
    if (a.w) {
      float w[8];
      norm_load8_as(a.w, a.w_dtype, c, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] *= w[i];
    }
    if (a.y) norm_store8_as(a.y, a.y_dtype, at * a.ldy + c, n, r[j]);
    if (a.codes) {
      float s;
      const uint2 q = norm_codes(r[j], s);
      norm_store_codes(a.codes + at * a.ldc + c, n, q);
      if (n > 0 && (l & 15) == 0) a.scales[at * a.G + (c >> 7)] = s;
    }
  }
}

struct NormBackArgs {
  const void* r;
  const void* w;        // or NULL
  const void* dy;
  const void* dtotal;   // or NULL
  void* dx;
  float* part;          // [workgroups][H] sums of dy n, or NULL
  long long ldr, ldy, ldt, ldd;
  int T, H;
  int dy_dtype, w_dtype;
  float eps;
};

// As above; LANES threads take one row after another and keep their sums of dy
// n in registers.  All of a row's reads are on their way before its
// sums (dtotal read behind them: 37 and not 34 us of 5003 x 2050).
template <class TR, int LANES, int C>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void k_rms_norm_back(NormBackArgs a) {
  constexpr int kThreads = LANES > 256 ? LANES : 256, kRows = kThreads / LANES;
  const int l = threadIdx.x % LANES;
  const long first = (long)blockIdx.x * kRows + threadIdx.x / LANES, step = (long)gridDim.x * kRows;
  const int rounds = (int)((a.T + step - 1) / step);  // as many for every thread: the sums have barriers
  float w[C][8], dw[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = 8 * (j * LANES + l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[j][i] = 1.0f;
      dw[j][i] = 0.0f;
    }
    if (a.w) norm_load8_as(a.w, a.w_dtype, c, a.H - c, w[j]);
  }
  for (int round = 0; round < rounds; ++round) {
    const long row = first + round * step;
    const bool live = row < a.T;
    const long at = live ? row : 0;
    float r[C][8], dy[C][8], d[C][8], ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
      norm_load8(static_cast<const TR*>(a.r) + at * a.ldr + c, n, r[j]);
      norm_load8_as(a.dy, a.dy_dtype, at * a.ldy + c, n, dy[j]);
      if (a.dtotal) norm_load8(static_cast<const TR*>(a.dtotal) + at * a.ldt + c, n, d[j]);
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = __builtin_fmaf(r[j][i], r[j][i], ss);
        dot = __builtin_fmaf(dy[j][i] * w[j][i], r[j][i], dot);
      }
    norm_row_sums<LANES>(ss, dot);
    const float v = 1.0f / sqrtf(ss / (float)a.H + a.eps);
    const float m = dot * v / (float)a.H;  // mean(a n)
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = 8 * (j * LANES + l), n = live ? a.H - c : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float nn = r[j][i] * v;
        const float g = v * (dy[j][i] * w[j][i] - nn * m);
        d[j][i] = a.dtotal ? g + d[j][i] : g;
        if (live) dw[j][i] = __builtin_fmaf(dy[j][i], nn, dw[j][i]);
      }
      norm_store8(static_cast<TR*>(a.dx) + at * a.ldd + c, n, d[j]);
    }
  }
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * a.H;
  if constexpr (kRows > 1) {  // the rows' sums added in their order
    __shared__ float sums[kRows][LANES * 8];
    norm_store8(&sums[threadIdx.x / LANES][8 * l], 8, dw[0]);
    __syncthreads();
    for (int c = threadIdx.x; c < LANES * 8 && c < a.H; c += kThreads) {
      float s = sums[0][c];
      for (int r = 1; r < kRows; ++r) s += sums[r][c];
      part[c] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = 8 * (j * LANES + l);
      norm_store8(part + c, a.H - c, dw[j]);
    }
  }
}

// dw: the workgroups' sums added in a fixed order, 64 channels a workgroup here.
__global__ __launch_bounds__(1024) void k_rms_norm_dw(const float* part, int groups, int H, void* dw, int dtype) {
  __shared__ float waves[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) s += part[(size_t)g * H + c];
  }
  waves[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < H) {
    for (int i = 1; i < 16; ++i) s += waves[i][lane];
    if (dtype == MOE_Q4_DTYPE_F32)
      static_cast<float*>(dw)[c] = s;
    else if (dtype == MOE_Q4_DTYPE_BF16)
      static_cast<__bf16*>(dw)[c] = (__bf16)s;
    else
      static_cast<_Float16*>(dw)[c] = (_Float16)s;
  }
}

// Codes and scales of blocks of 1 x 128: 16 threads a block.
template <class TX>
__global__ __launch_bounds__(256) void k_quant_rows(const TX* x, long long ldx, int K, int G, size_t chunks, uint8_t* codes,
                                                    long long ldc, float* scales) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const bool live = i < chunks;
  const size_t at = live ? i : chunks - 1;
  const size_t row = at / ((size_t)G * 16);
  const int c = 8 * (int)(at % ((size_t)G * 16)), n = live ? K - c : 0;
  float v[8], s;
  norm_load8(x + row * ldx + c, n, v);
  const uint2 q = norm_codes(v, s);
  norm_store_codes(codes + row * ldc + c, n, q);
  if (n > 0 && (threadIdx.x & 15) == 0) scales[row * G + (c >> 7)] = s;
}

// Codes and scales of blocks of 128 x 128, one a workgroup.
template <class TX>
__global__ __launch_bounds__(256) void k_quant_blocks(const TX* x, long long ldx, int T, int K, int G, uint8_t* codes,
                                                      long long ldc, float* scales) {
  __shared__ float waves[4];
  const int g = blockIdx.x % G, t0 = (blockIdx.x / G) * 128;
  const int c = g * 128 + 8 * (threadIdx.x & 15), row0 = t0 + (threadIdx.x >> 4);
  float v[8][8], most = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) norm_load8(x + (size_t)min(row0 + 16 * j, T - 1) * ldx + c, row0 + 16 * j < T ? K - c : 0, v[j]);
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[j][i]));
  most = norm_max16(most);
  most = fmaxf(most, __shfl_xor(most, 16));
  most = fmaxf(most, __shfl_xor(most, 32));
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = most;
  __syncthreads();
  most = fmaxf(fmaxf(waves[0], waves[1]), fmaxf(waves[2], waves[3]));
  const float s = norm_scale(most);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = row0 + 16 * j;
    if (row < T) norm_store_codes(codes + (size_t)row * ldc + c, K - c, norm_pack8(v[j], s));
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

// Threads of a row and chunks of each.  1024 threads for more than 4096
// channels, since 256 with four chunks hold fewer rows in flight (us, 1024 and
// 256: norm into codes 8192 x 8192 83 and 97, x 6144 72 and 74, x 4104 50 and
// 46, 1 x 6144 3.1 and 6.9; gradient 8192 x 6144 110 and 127), and with few rows
// for more than 2048 (1 x 4096 2.9 and 4.8 with two chunks, 256 x 4096 3.9 and
// 4.2; 1024 x 4096 8.4 and 6.4).
struct NormPlan {
  int lanes, chunks;
};
NormPlan norm_plan(int T, int H) {
  const int n = (H + 7) / 8;
  if (n <= 16) return {16, 1};
  if (n <= 64) return {64, 1};
  if (n <= 256) return {256, 1};
  if (n > 1024) return {1024, 2};
  return n > 512 || T <= 512 ? NormPlan{1024, 1} : NormPlan{256, 2};
}

#define NORM_SWITCH(KERNEL, TYPE, PLAN, GRID, STREAM, ARGS)                                                       \
  switch ((PLAN).lanes * 8 + (PLAN).chunks) {                                                                     \
    case 16 * 8 + 1: hipLaunchKernelGGL((KERNEL<TYPE, 16, 1>), GRID, dim3(256), 0, STREAM, ARGS); break;          \
    case 64 * 8 + 1: hipLaunchKernelGGL((KERNEL<TYPE, 64, 1>), GRID, dim3(256), 0, STREAM, ARGS); break;          \
    case 256 * 8 + 1: hipLaunchKernelGGL((KERNEL<TYPE, 256, 1>), GRID, dim3(256), 0, STREAM, ARGS); break;        \
    case 256 * 8 + 2: hipLaunchKernelGGL((KERNEL<TYPE, 256, 2>), GRID, dim3(256), 0, STREAM, ARGS); break;        \
    case 1024 * 8 + 1: hipLaunchKernelGGL((KERNEL<TYPE, 1024, 1>), GRID, dim3(1024), 0, STREAM, ARGS); break;     \
    default: hipLaunchKernelGGL((KERNEL<TYPE, 1024, 2>), GRID, dim3(1024), 0, STREAM, ARGS); break;               \
  }

int rows_of(const NormPlan& p) { return p.lanes >= 256 ? 1 : 256 / p.lanes; }

// Workgroups of the backward pass, each with a row of sums: as many as the
// compute units hold at once, by their registers (us with 512, 768 and 1024:
// 5003 x 2050 fp32 33.2 28.3 35.7, 8192 x 2048 31 26 24; 8192 x 6144, a unit
// holds one, 110 with 256 and 111 with 512).
int norm_back_groups(int T, int H) {
  const NormPlan p = norm_plan(T, H);
  const int rows = rows_of(p), blocks = (T + rows - 1) / rows;
  return std::min(blocks, p.lanes == 1024 ? 256 : p.chunks == 2 ? 768 : 1024);
}

int norm_status(int T, int H) {
  if (T < 0 || H < 1) return MOE_Q4_ERR_SHAPE;
  if (H > MOE_Q4_NORM_MAX_H || T > MOE_Q4_ROUTER_MAX_T) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

int launched() { return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH; }

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" int moe_rms_norm(const void* x, int x_dtype, long long ldx, const void* residual, int residual_dtype,
                            long long ldr, const void* weight, int weight_dtype, int T, int H, float eps, void* total,
                            long long ldt, void* y, int y_dtype, long long ldy, uint8_t* codes, long long ldc,
                            float* scales, hipStream_t stream) {
  const int st = norm_status(T, H);
  if (st) return st;
  if (!(eps >= 0.0f) || ldx < H || (residual && (ldr < H || ldt < H)) || (y && ldy < H) || (codes && ldc < H))
    return MOE_Q4_ERR_SHAPE;
  const size_t xs = args_size(x_dtype);
  if (!xs || (residual && residual_dtype != x_dtype && residual_dtype != MOE_Q4_DTYPE_F32) ||
      (weight && !args_size(weight_dtype)) || (y && !args_size(y_dtype)))
    return MOE_Q4_ERR_UNSUPPORTED;
  if (T == 0) return MOE_Q4_OK;
  if (!x || (!y && !codes) || (codes && !scales) || (residual && !total)) return MOE_Q4_ERR_NULL;
  const size_t rs = args_size(residual_dtype), wsz = args_size(weight_dtype), ys = args_size(y_dtype);
  if (!args_aligned(x, xs) || (residual && (!args_aligned(residual, rs) || !args_aligned(total, rs))) ||
      (weight && !args_aligned(weight, wsz)) || (y && !args_aligned(y, ys)) || (codes && !args_aligned(scales, 4)))
    return MOE_Q4_ERR_ALIGN;
  const int G = (H + 127) / 128;
  // total may be the residual itself: a thread reads its channels before it writes them
  const bool in_place = residual && total == residual && ldt == ldr;
  const ArgSpan ins[] = {{x, args_span(T, ldx, H, xs)},
                         {in_place ? nullptr : residual, residual ? args_span(T, ldr, H, rs) : 0},
                         {weight, weight ? (size_t)H * wsz : 0}};
  const ArgSpan outs[] = {{residual ? total : nullptr, residual ? args_span(T, ldt, H, rs) : 0},
                          {y, y ? args_span(T, ldy, H, ys) : 0},
                          {codes, codes ? args_span(T, ldc, H, 1) : 0},
                          {codes ? scales : nullptr, codes ? (size_t)T * G * 4 : 0}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  NormArgs a{x, residual, weight, total, y, codes, scales, ldx, ldr, ldt, ldy, ldc, T, H, G,
             residual && residual_dtype == MOE_Q4_DTYPE_F32, weight_dtype, y_dtype, eps, 0};
  const NormPlan p = norm_plan(T, H);
  const int rows = rows_of(p);
  const long most = 1L << 21;  // workgroups of a launch, which holds fewer than 2^32 threads
  for (; a.row0 < T; a.row0 += most * rows) {
    const dim3 grid((unsigned)std::min(most, (T - a.row0 + rows - 1) / rows));
    switch (x_dtype) {
      case MOE_Q4_DTYPE_BF16: NORM_SWITCH(k_rms_norm, __bf16, p, grid, stream, a) break;
      case MOE_Q4_DTYPE_F16: NORM_SWITCH(k_rms_norm, _Float16, p, grid, stream, a) break;
      default: NORM_SWITCH(k_rms_norm, float, p, grid, stream, a) break;
    }
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  return MOE_Q4_OK;
}

extern "C" size_t moe_rms_norm_backward_workspace_bytes(int T, int H) {
  if (norm_status(T, H) || T == 0) return 0;
  return ((size_t)norm_back_groups(T, H) * H * 4 + 255) & ~size_t(255);
}

extern "C" int moe_rms_norm_backward(const void* total, int total_dtype, long long ldr, const void* weight,
                                     int weight_dtype, const void* dy, int dy_dtype, long long ldy, const void* dtotal,
                                     long long ldt, int T, int H, float eps, void* dx, long long ldd, void* dweight,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = norm_status(T, H);
  if (st) return st;
  if (!(eps >= 0.0f) || ldr < H || ldy < H || ldd < H || (dtotal && ldt < H)) return MOE_Q4_ERR_SHAPE;
  const size_t rs = args_size(total_dtype), ys = args_size(dy_dtype), wsz = args_size(weight_dtype);
  if (!rs || !ys || ((weight || dweight) && !wsz)) return MOE_Q4_ERR_UNSUPPORTED;
  if ((T && (!total || !dy || !dx)) || (dweight && !weight)) return MOE_Q4_ERR_NULL;
  const size_t need = dweight ? moe_rms_norm_backward_workspace_bytes(T, H) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (!args_aligned(total, rs) || !args_aligned(dy, ys) || !args_aligned(dtotal, rs) || !args_aligned(dx, rs) ||
      (weight && !args_aligned(weight, wsz)) || (dweight && !args_aligned(dweight, wsz)) ||
      (need && !args_aligned(workspace, 256)))
    return MOE_Q4_ERR_ALIGN;
  const ArgSpan ins[] = {{total, args_span(T, ldr, H, rs)},
                         {weight, weight ? (size_t)H * wsz : 0},
                         {dy, args_span(T, ldy, H, ys)},
                         {dtotal, dtotal ? args_span(T, ldt, H, rs) : 0}};
  const ArgSpan outs[] = {{dx, args_span(T, ldd, H, rs)}, {dweight, dweight ? (size_t)H * wsz : 0}, {need ? workspace : nullptr, need}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  const int groups = T ? norm_back_groups(T, H) : 0;
  if (T) {
    const NormPlan p = norm_plan(T, H);
    NormBackArgs a{total, weight, dy, dtotal, dx, dweight ? static_cast<float*>(workspace) : nullptr, ldr, ldy, ldt, ldd,
                   T, H, dy_dtype, weight_dtype, eps};
    const dim3 grid((unsigned)groups);
    switch (total_dtype) {
      case MOE_Q4_DTYPE_BF16: NORM_SWITCH(k_rms_norm_back, __bf16, p, grid, stream, a) break;
      case MOE_Q4_DTYPE_F16: NORM_SWITCH(k_rms_norm_back, _Float16, p, grid, stream, a) break;
      default: NORM_SWITCH(k_rms_norm_back, float, p, grid, stream, a) break;
    }
    if (hipGetLastError() != hipSuccess) return MOE_Q4_ERR_LAUNCH;
  }
  if (dweight)
    hipLaunchKernelGGL(k_rms_norm_dw, dim3((H + 63) / 64), dim3(1024), 0, stream, static_cast<const float*>(workspace),
                       groups, H, dweight, weight_dtype);
  return launched();
}

extern "C" int moe_quantize_fp8(const void* x, int x_dtype, long long ldx, int T, int K, int block_rows, uint8_t* codes,
                                long long ldc, float* scales, hipStream_t stream) {
  if (T < 0 || K < 1 || ldx < K || ldc < K) return MOE_Q4_ERR_SHAPE;
  const size_t xs = args_size(x_dtype);
  if (!xs || (block_rows != 1 && block_rows != 128)) return MOE_Q4_ERR_UNSUPPORTED;
  const long G = ((long)K + 127) / 128, R = ((long)T + block_rows - 1) / block_rows;
  // (a launch holds fewer than 2^31 workgroups of 256 threads and 2^32 threads)
  if (block_rows == 1 ? T * G > (1L << 27) : R * G > (1L << 23)) return MOE_Q4_ERR_UNSUPPORTED;
  if (T == 0) return MOE_Q4_OK;
  if (!x || !codes || !scales) return MOE_Q4_ERR_NULL;
  if (!args_aligned(x, xs) || !args_aligned(scales, 4)) return MOE_Q4_ERR_ALIGN;
  const ArgSpan ins[] = {{x, args_span(T, ldx, K, xs)}};
  const ArgSpan outs[] = {{codes, args_span(T, ldc, K, 1)}, {scales, (size_t)R * G * 4}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  if (block_rows == 1) {
    const size_t chunks = (size_t)T * G * 16;
    const dim3 grid((unsigned)((chunks + 255) / 256));
    switch (x_dtype) {
      case MOE_Q4_DTYPE_BF16: hipLaunchKernelGGL((k_quant_rows<__bf16>), grid, dim3(256), 0, stream, static_cast<const __bf16*>(x), ldx, K, (int)G, chunks, codes, ldc, scales); break;
      case MOE_Q4_DTYPE_F16: hipLaunchKernelGGL((k_quant_rows<_Float16>), grid, dim3(256), 0, stream, static_cast<const _Float16*>(x), ldx, K, (int)G, chunks, codes, ldc, scales); break;
      default: hipLaunchKernelGGL((k_quant_rows<float>), grid, dim3(256), 0, stream, static_cast<const float*>(x), ldx, K, (int)G, chunks, codes, ldc, scales); break;
    }
  } else {
    const dim3 grid((unsigned)(R * G));
    switch (x_dtype) {
      case MOE_Q4_DTYPE_BF16: hipLaunchKernelGGL((k_quant_blocks<__bf16>), grid, dim3(256), 0, stream, static_cast<const __bf16*>(x), ldx, T, K, (int)G, codes, ldc, scales); break;
      case MOE_Q4_DTYPE_F16: hipLaunchKernelGGL((k_quant_blocks<_Float16>), grid, dim3(256), 0, stream, static_cast<const _Float16*>(x), ldx, T, K, (int)G, codes, ldc, scales); break;
      default: hipLaunchKernelGGL((k_quant_blocks<float>), grid, dim3(256), 0, stream, static_cast<const float*>(x), ldx, T, K, (int)G, codes, ldc, scales); break;
    }
  }
  return launched();
}
