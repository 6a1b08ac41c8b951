// The gated block's kernels for bf16 operands.
#define MOE_GLU_INST
#include "moe_glu_kernels.h"

namespace moeq4 {
int glu_forward_bf16(const GluArgs& a, bool rows, const GemmPlan& p, hipStream_t s) { return glu_forward_kind<kGemmBf16>(a, rows, p, s); }
int glu_mm_bf16(const GluMmArgs& a, const GemmPlan& p, hipStream_t s) { return glu_mm_kind<kGemmBf16>(a, p, s); }
int glu_grad_bf16(const float* saved, const void* dh, long long lddh, int T, int I, int ip, void* d, float* scale,
                 hipStream_t s) {
  return glu_grad_kind<kGemmBf16>(saved, dh, lddh, T, I, ip, d, scale, s);
}
}  // namespace moeq4
