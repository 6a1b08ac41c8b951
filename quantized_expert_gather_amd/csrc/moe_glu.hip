// Gated feed-forward block of dense weights and its gradient: argument checks,
// plans and workspaces.  The kernels are in moe_glu_kernels.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "moe_args.h"
#include "moe_glu_kernels.h"
#include "moe_q4.h"

namespace moeq4 {
namespace {

int glu_status(int T, int H, int I) {
  if (T < 0 || H < 1 || I < 1) return MOE_Q4_ERR_SHAPE;
  if (H % 8 || I % 8 || T > MOE_Q4_LINEAR_MAX_L || H > MOE_Q4_LINEAR_MAX_K || I > MOE_Q4_LINEAR_MAX_K) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

// Few tokens by rows (us by rows with 32 tokens, by tiles with 33: 2056 x 1416 6.9
// and 11.2, 6144 x 2048 14.2 and 16.9, 4096 x 4096 19.0 and 17.7: with
// such weights the tiles would be the faster before that; their size is not looked
// at).
bool glu_by_rows(int T) { return T <= 32; }
int glu_steps(long k) { return (int)((2 * k + kGemmStep - 1) / kGemmStep); }
GemmPlan glu_forward_plan(int T, int H, int I) { return gemm_plan(kGemmCosts16, T, 2 * I, glu_steps(H)); }
size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

size_t glu_forward_part(int T, int H, int I) {
  if (glu_by_rows(T)) return 0;
  const GemmPlan p = glu_forward_plan(T, H, I);
  return p.tiles.splits > 1 ? round256((size_t)p.tiles.splits * 2 * T * I * 4) : 0;
}

struct GluBackLayout {
  size_t gu, d, scale, part, total;
  int ip;  // dg's and du's places in a row of D: whole lines, since tiles of other rows' read twice as many
  GemmPlan dx, dw;
};
GluBackLayout glu_back_layout(int T, int H, int I, bool saved) {
  GluBackLayout w{};
  w.ip = (I + 63) / 64 * 64;
  w.dx = gemm_plan(kGemmCosts16, T, H, 2 * glu_steps(I));
  w.dw = gemm_plan(kGemmCosts16, 2 * I, H, glu_steps(T));
  size_t off = 0;
  w.gu = off; off = round256(off + (saved ? 0 : (size_t)2 * T * I * 4));
  w.d = off; off = round256(off + (size_t)T * 2 * w.ip * 2);
  w.scale = off; off = round256(off + kGluScaleBytes);
  w.part = off;
  size_t part = saved ? 0 : glu_forward_part(T, H, I);
  if (w.dx.tiles.splits > 1) part = std::max(part, (size_t)w.dx.tiles.splits * T * H * 4);
  if (w.dw.tiles.splits > 1) part = std::max(part, (size_t)w.dw.tiles.splits * 2 * I * H * 4);
  w.total = round256(off + part);
  return w;
}

int glu_forward(bool f16, const GluArgs& given, void* part, hipStream_t stream) {
  GluArgs a = given;
  const bool rows = glu_by_rows(a.T);
  const GemmPlan p = glu_forward_plan(a.T, a.H, a.I);
  a.tiles = p.tiles;
  if (!rows && p.tiles.splits > 1) a.part = static_cast<float*>(part);
  return f16 ? glu_forward_f16(a, rows, p, stream) : glu_forward_bf16(a, rows, p, stream);
}

int glu_mm(bool f16, GluMmArgs a, const GemmPlan& p, void* part, hipStream_t stream) {
  a.tiles = p.tiles;
  a.part = p.tiles.splits > 1 ? static_cast<float*>(part) : nullptr;
  return f16 ? glu_mm_f16(a, p, stream) : glu_mm_bf16(a, p, stream);
}

__global__ __launch_bounds__(256) void k_glu_zero(uint4* a, uint4* b, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) a[i] = b[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" size_t moe_glu_workspace_bytes(int T, int H, int I) {
  if (glu_status(T, H, I) || T == 0) return 0;
  return glu_forward_part(T, H, I);
}

extern "C" int moe_glu_forward(int dtype, const void* x, long long ldx, const void* wg, const void* wu, long long ldw, int T,
                               int H, int I, void* h, long long ldh, float* saved, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  const int st = glu_status(T, H, I);
  if (st) return st;
  if (ldx < H || ldw < H || ldh < I) return MOE_Q4_ERR_SHAPE;
  if (dtype != MOE_Q4_DTYPE_BF16 && dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (ldx > MOE_Q4_GLU_MAX_LD || ldw > MOE_Q4_GLU_MAX_LD) return MOE_Q4_ERR_UNSUPPORTED;
  if (T == 0) return MOE_Q4_OK;
  if (!x || !wg || !wu || !h) return MOE_Q4_ERR_NULL;
  if (!args_aligned(x, 16) || !args_aligned(wg, 16) || !args_aligned(wu, 16) || (T > 1 && ldx % 8) || (I > 1 && ldw % 8) ||
      !args_aligned(h, 2) || !args_aligned(saved, 16))
    return MOE_Q4_ERR_ALIGN;
  const size_t need = moe_glu_workspace_bytes(T, H, I);
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (need && !args_aligned(workspace, 256)) return MOE_Q4_ERR_ALIGN;
  const ArgSpan ins[] = {{x, args_span(T, ldx, H, 2)}, {wg, args_span(I, ldw, H, 2)}, {wu, args_span(I, ldw, H, 2)}};
  const ArgSpan outs[] = {{h, args_span(T, ldh, I, 2)}, {saved, saved ? (size_t)2 * T * I * 4 : 0}, {need ? workspace : nullptr, need}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  GluArgs a{};
  a.x = static_cast<const unsigned char*>(x);
  a.wg = static_cast<const unsigned char*>(wg);
  a.wu = static_cast<const unsigned char*>(wu);
  a.h = h;
  a.saved = saved;
  a.ldx = 2 * ldx;
  a.ldw = 2 * ldw;
  a.ldh = ldh;
  a.T = T; a.H = H; a.I = I;
  return glu_forward(dtype == MOE_Q4_DTYPE_F16, a, workspace, stream);
}

extern "C" size_t moe_glu_backward_workspace_bytes(int T, int H, int I, int have_saved) {
  if (glu_status(T, H, I) || T == 0) return 0;
  return glu_back_layout(T, H, I, have_saved != 0).total;
}

extern "C" int moe_glu_backward(int dtype, const void* x, long long ldx, const void* wg, const void* wu, long long ldw,
                                const void* dh, long long lddh, const float* saved, int T, int H, int I, void* dx,
                                long long lddx, void* dwg, void* dwu, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  int st = glu_status(T, H, I);
  if (st) return st;
  if (ldx < H || ldw < H || lddh < I || (dx && lddx < H)) return MOE_Q4_ERR_SHAPE;
  if (dtype != MOE_Q4_DTYPE_BF16 && dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (ldx > MOE_Q4_GLU_MAX_LD || ldw > MOE_Q4_GLU_MAX_LD) return MOE_Q4_ERR_UNSUPPORTED;
  if (!dwg != !dwu || (T && (!x || !wg || !wu || !dh))) return MOE_Q4_ERR_NULL;
  if (!args_aligned(x, 16) || !args_aligned(wg, 16) || !args_aligned(wu, 16) || (T > 1 && ldx % 8) || (I > 1 && ldw % 8) ||
      !args_aligned(dh, 2) || !args_aligned(saved, 16) || !args_aligned(dx, 2) || !args_aligned(dwg, 16) || !args_aligned(dwu, 16))
    return MOE_Q4_ERR_ALIGN;
  const size_t need = dx || dwg ? moe_glu_backward_workspace_bytes(T, H, I, saved != nullptr) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (need && !args_aligned(workspace, 256)) return MOE_Q4_ERR_ALIGN;
  const ArgSpan ins[] = {{x, args_span(T, ldx, H, 2)}, {wg, args_span(I, ldw, H, 2)}, {wu, args_span(I, ldw, H, 2)},
                         {dh, args_span(T, lddh, I, 2)}, {saved, saved ? (size_t)2 * T * I * 4 : 0}};
  const size_t wn = dwg ? (size_t)I * H * 2 : 0;
  const ArgSpan outs[] = {{dx, dx ? args_span(T, lddx, H, 2) : 0}, {dwg, wn}, {dwu, wn}, {need ? workspace : nullptr, need}};
  if (args_alias(outs, ins)) return MOE_Q4_ERR_ALIAS;
  if (T == 0) {
    if (dwg) hipLaunchKernelGGL(k_glu_zero, dim3((unsigned)std::min<size_t>((wn / 16 + 255) / 256, 4096)), dim3(256), 0, stream,
                                static_cast<uint4*>(dwg), static_cast<uint4*>(dwu), wn / 16);
    return hipGetLastError() == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_LAUNCH;
  }
  if (!dx && !dwg) return MOE_Q4_OK;
  const bool f16 = dtype == MOE_Q4_DTYPE_F16;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const GluBackLayout w = glu_back_layout(T, H, I, saved != nullptr);
  if (!saved) {
    GluArgs a{};
    a.x = static_cast<const unsigned char*>(x);
    a.wg = static_cast<const unsigned char*>(wg);
    a.wu = static_cast<const unsigned char*>(wu);
    a.saved = reinterpret_cast<float*>(ws + w.gu);
    a.ldx = 2 * ldx;
    a.ldw = 2 * ldw;
    a.T = T; a.H = H; a.I = I;
    if ((st = glu_forward(f16, a, ws + w.part, stream))) return st;
    saved = a.saved;
  }
  float* scale = reinterpret_cast<float*>(ws + w.scale);
  if ((st = (f16 ? glu_grad_f16 : glu_grad_bf16)(saved, dh, lddh, T, I, w.ip, ws + w.d, scale, stream))) return st;
  GluMmArgs m{};
  m.a = ws + w.d;
  m.lda = 4LL * w.ip;
  m.ip = w.ip;
  m.back = scale;
  m.N = H;
  if (dx) {  // dx = D [Wg; Wu]
    m.b0 = static_cast<const unsigned char*>(wg);
    m.b1 = static_cast<const unsigned char*>(wu);
    m.out0 = m.out1 = dx;
    m.ldb = 2 * ldw;
    m.ldo = lddx;
    m.M = m.cut = T;
    m.K = I;
    m.steps = glu_steps(I);
    if ((st = glu_mm(f16, m, w.dx, ws + w.part, stream))) return st;
  }
  if (dwg) {  // [dWg; dWu] = D^T x
    m.b0 = static_cast<const unsigned char*>(x);
    m.b1 = nullptr;
    m.out0 = dwg;
    m.out1 = dwu;
    m.ldb = 2 * ldx;
    m.ldo = H;
    m.M = 2 * I;
    m.cut = I;
    m.K = T;
    m.steps = glu_steps(T);
    if ((st = glu_mm(f16, m, w.dw, ws + w.part, stream))) return st;
  }
  return MOE_Q4_OK;
}
