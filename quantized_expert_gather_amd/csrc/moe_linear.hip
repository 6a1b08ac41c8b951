// Dense product with 4-bit weights: out[t, n] = sum_c x[t, c] W[n, c] + bias[n]
// over the expert banks' codecs.  Argument checks; the kernels for few tokens
// are in moe_linear_rows.h, those for many in moe_linear_tiles.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "moe_linear_launch.h"
#include "moe_q4.h"

namespace moeq4 {
namespace {

int linear_fmt(int codec) {
  switch (codec) {
    case MOE_Q4_CODEC_AFFINE4_G64: return kLinAffine64;
    case MOE_Q4_CODEC_AFFINE4_G32: return kLinAffine32;
    case MOE_Q4_CODEC_MXFP4: return kLinMxfp4;
    case MOE_Q4_CODEC_NVFP4: return kLinNvfp4;
  }
  return -1;
}

int linear_shape_status(int fmt, int L, int N, int K) {
  if (L < 0 || N < 1 || K < 1) return MOE_Q4_ERR_SHAPE;
  const int grp = fmt == kLinAffine64 ? 64 : 32;
  if (fmt < 0 || K % grp || L > MOE_Q4_LINEAR_MAX_L || N > MOE_Q4_LINEAR_MAX_N || K > MOE_Q4_LINEAR_MAX_K) return MOE_Q4_ERR_UNSUPPORTED;
  return MOE_Q4_OK;
}

bool aligned_to(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}
size_t span(int rows, long long ld, int cols, size_t es) {
  return rows ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0;
}

}  // namespace
}  // namespace moeq4

using namespace moeq4;

extern "C" size_t moe_linear_codec_workspace_bytes(int codec, int L, int N, int K) {
  const int fmt = linear_fmt(codec);
  if (linear_shape_status(fmt, L, N, K) || L == 0) return 0;
  return linear_by_tiles(fmt, L, N, K) ? tiles_layout(fmt, L, N, K).total : rows_workspace(fmt, L, N, K);
}

extern "C" int moe_linear_codec_forward(int codec, const void* x, int x_dtype, long long ldx, const uint32_t* w,
                                        const void* s, const void* b, const float* bias, int L, int N, int K, void* out,
                                        int out_dtype, long long ldo, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream) {
  const int fmt = linear_fmt(codec);
  const int st = linear_shape_status(fmt, L, N, K);
  if (st) return st;
  if (ldx < K || ldo < N) return MOE_Q4_ERR_SHAPE;
  if (L > 1 && ldx > MOE_Q4_LINEAR_MAX_LDX) return MOE_Q4_ERR_UNSUPPORTED;
  if (x_dtype != MOE_Q4_DTYPE_BF16 && x_dtype != MOE_Q4_DTYPE_F16) return MOE_Q4_ERR_UNSUPPORTED;
  if (out_dtype != MOE_Q4_DTYPE_BF16 && out_dtype != MOE_Q4_DTYPE_F32 && out_dtype != MOE_Q4_DTYPE_F16)
    return MOE_Q4_ERR_UNSUPPORTED;
  if (L == 0) return MOE_Q4_OK;
  const bool affine = lin_affine(fmt);
  if (!x || !w || !s || !out || (affine && !b)) return MOE_Q4_ERR_NULL;
  const size_t os = out_dtype == MOE_Q4_DTYPE_F32 ? 4 : 2, sa = fmt == kLinMxfp4 ? 1 : 2;
  if (!aligned_to(x, 16) || (L > 1 && ldx % 8) || !aligned_to(w, 16) || !aligned_to(s, sa) || (affine && !aligned_to(b, 2)) ||
      !aligned_to(bias, 4) || !aligned_to(out, os))
    return MOE_Q4_ERR_ALIGN;
  const size_t need = moe_linear_codec_workspace_bytes(codec, L, N, K);
  if (need && (!workspace || workspace_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
  if (need && !aligned_to(workspace, 256)) return MOE_Q4_ERR_ALIGN;
  const size_t gs = lin_group(fmt), sb = (size_t)N * (K / gs) * (affine ? 2 : 1);
  const struct { const void* p; size_t n; } ins[] = {{x, span(L, ldx, K, 2)}, {w, (size_t)N * K / 2}, {s, sb},
                                                     {affine ? b : nullptr, affine ? sb : 0},
                                                     {bias, bias ? (size_t)N * 4 : 0}, {workspace, need}};
  const size_t on = span(L, ldo, N, os);
  for (const auto& in : ins)
    if (overlap(out, on, in.p, in.n) || (&in != &ins[5] && overlap(workspace, need, in.p, in.n))) return MOE_Q4_ERR_ALIAS;
  const LinearArgs a{static_cast<const uint16_t*>(x), w, static_cast<const unsigned char*>(s),
               affine ? static_cast<const unsigned char*>(b) : nullptr, bias, out, ldx, ldo, L, N, K, out_dtype, nullptr, 0};
  const bool f16 = x_dtype == MOE_Q4_DTYPE_F16;
  unsigned char* wsb = static_cast<unsigned char*>(workspace);
  switch (fmt) {
    case kLinAffine64: return linear_launch<kLinAffine64>(f16, a, wsb, stream);
    case kLinAffine32: return linear_launch<kLinAffine32>(f16, a, wsb, stream);
    case kLinMxfp4: return linear_launch<kLinMxfp4>(f16, a, wsb, stream);
    default: return linear_launch<kLinNvfp4>(f16, a, wsb, stream);
  }
}
