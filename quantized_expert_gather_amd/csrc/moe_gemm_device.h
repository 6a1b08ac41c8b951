// Products C[t, n] = sum_k A[t, k] B[n, k] on the matrix cores, both operands
// with their rows along k: 16-bit numbers, or E4M3 codes with a scale per
// 128.  A step is 128 bytes of every row (64 or 128 elements).  Internal header.
//
//   gemm_tile   many tokens: A's and B's steps are copied into LDS
//   gemm_rows   few tokens: B is read once, straight into the operands
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_norm_device.h"
#include "moe_q4.h"

namespace moeq4 {

// kGemmFp8 multiplies E4M3 as it is: the matrix cores add 8 neighbouring
// products after cutting each at 2^-13 of the largest one's power of two, and
// these sums in fp32 (measured; 1.4e-5 of a result of normal values: enough
// for 16-bit results).  kGemmFp8Wide makes the codes bf16, which is exact, and
// adds all of them in fp32, at half the rate.
constexpr int kGemmBf16 = 0, kGemmF16 = 1, kGemmFp8 = 2, kGemmFp8Wide = 3;
__host__ __device__ constexpr bool gemm_scaled(int kind) { return kind == kGemmFp8 || kind == kGemmFp8Wide; }
constexpr int kGemmStep = 128;  // bytes

typedef __bf16 gemm_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 gemm_f16x8 __attribute__((ext_vector_type(8)));
typedef float gemm_f32x4 __attribute__((ext_vector_type(4)));
typedef int gemm_i32x4 __attribute__((ext_vector_type(4)));
typedef int gemm_i32x8 __attribute__((ext_vector_type(8)));

// A lane's part of 16 rows of a step: row lane % 16, 16-byte chunks kb and
// kb + 4 with kb = lane / 16.  (Any order of k will do that both operands share.)
struct GemmFrag {
  gemm_i32x4 v[2];
};

// Eight E4M3 codes as bf16, exact.
__device__ __forceinline__ gemm_bf16x8 gemm_e4m3_bf16(int lo, int hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return gemm_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// acc (+)= a b over a step, a's rows along the result's rows (4 kb + i), b's
// along its columns (lane % 16).  E4M3: the step's sum times f.
template <int KIND>
__device__ __forceinline__ void gemm_mfma(const GemmFrag& a, const GemmFrag& b, float f, gemm_f32x4& acc) {
  if constexpr (KIND == kGemmFp8) {
    const gemm_i32x8 x = {a.v[0][0], a.v[0][1], a.v[0][2], a.v[0][3], a.v[1][0], a.v[1][1], a.v[1][2], a.v[1][3]};
    const gemm_i32x8 y = {b.v[0][0], b.v[0][1], b.v[0][2], b.v[0][3], b.v[1][0], b.v[1][1], b.v[1][2], b.v[1][3]};
    const gemm_f32x4 zero = {0, 0, 0, 0};
    const gemm_f32x4 s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s[i], f, acc[i]);
  } else if constexpr (KIND == kGemmFp8Wide) {
    gemm_f32x4 s = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gemm_e4m3_bf16(a.v[j >> 1][2 * (j & 1)], a.v[j >> 1][2 * (j & 1) + 1]),
                                                  gemm_e4m3_bf16(b.v[j >> 1][2 * (j & 1)], b.v[j >> 1][2 * (j & 1) + 1]), s, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s[i], f, acc[i]);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (KIND == kGemmBf16)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gemm_bf16x8, a.v[j]),
                                                      __builtin_bit_cast(gemm_bf16x8, b.v[j]), acc, 0, 0, 0);
      else
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(gemm_f16x8, a.v[j]),
                                                     __builtin_bit_cast(gemm_f16x8, b.v[j]), acc, 0, 0, 0);
    }
  }
}

// Zeros that the compiler does not know: as constants it would carry them
// through a loop in registers of their own.
__device__ __forceinline__ gemm_f32x4 gemm_zero() {
  gemm_f32x4 z = {0, 0, 0, 0};
  asm volatile("" : "+v"(z));
  return z;
}

// ---- many tokens ----

// MT x NT tiles of 16 x 16 a wave, WM x WN waves: 16 MT WM tokens x 16 NT WN rows of B.
template <int KIND_, int MT_, int NT_, int WM_, int WN_>
struct GemmShape {
  static constexpr int KIND = KIND_, MT = MT_, NT = NT_, WM = WM_, WN = WN_;
  static constexpr int kThreads = 64 * WM * WN, kTok = 16 * MT * WM, kRows = 16 * NT * WN;
  static constexpr int kBuffer = (kTok + kRows) * kGemmStep;
};

// Tile of a workgroup.  Workgroups b, b + 8, ... share an XCD (and its L2):
// each XCD takes a contiguous run, which goes through 8 token tiles at a time,
// so the 32 tiles it works on together read 8 + 4 tiles of the operands.
__device__ __forceinline__ void gemm_place(int block, int tok_tiles, int row_tiles, int& tok, int& row) {
  const int tiles = tok_tiles * row_tiles;
  const int per = tiles / 8, rest = tiles % 8, xcd = block & 7, at = block >> 3;
  const int id = xcd * per + min(xcd, rest) + at;
  const int group = id / (8 * row_tiles), in = id % (8 * row_tiles), first = group * 8;
  const int size = min(tok_tiles - first, 8);
  tok = first + in % size;
  row = in / size;
}

// Steps step0 .. step1 of a tile into acc.  Row r of the tile begins at
// tok_base + tok_off(r) in A, row_base(r) + row_off(r) in B (some row within
// the operand for those past its end); offsets have 32 bits.  kbytes, a
// multiple of 16, is a row's length.  E4M3: sx_row is the scales of this
// thread's token tid of the tile, sw those of the wave's rows.
//
// LDS holds a step of all rows, 128 bytes each, copied without passing
// registers; chunk c of row r lies at place c ^ (r % 8), so that the 8 rows
// that are read together fall in different banks.
template <class S, class TokOff, class RowBase, class RowOff>
__device__ __forceinline__ void gemm_tile(unsigned char* lds0, unsigned char* lds1, float* scl0, float* scl1, int kbytes,
                                          int step0, int step1, const unsigned char* tok_base, TokOff tok_off,
                                          RowBase row_base, RowOff row_off, const float* sx_row, const float* sw,
                                          gemm_f32x4 (&acc)[S::MT][S::NT]) {
  constexpr int MT = S::MT, NT = S::NT, KIND = S::KIND;
  constexpr int kPass = S::kThreads / 8, kTokCopies = S::kTok / kPass, kCopies = (S::kTok + S::kRows) / kPass;
  static_assert(S::kTok % kPass == 0 && S::kRows % kPass == 0 && S::kTok <= S::kThreads, "copies of whole passes");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n16 = lane & 15, kb = lane >> 4;
  const int wm = wave % S::WM, wn = wave / S::WM;

  uint32_t off[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int r = c * kPass + tid / 8;
    off[c] = c < kTokCopies ? tok_off(r) : row_off(r - S::kTok);
  }
  const int chunk = ((tid & 7) ^ ((tid >> 3) & 7)) * 16;
  auto stage = [&](int step, unsigned char* buf) __attribute__((always_inline)) {
    const uint32_t k = min(step * kGemmStep + chunk, kbytes - 16);  // (past the end: never used)
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const unsigned char* base = c < kTokCopies ? tok_base : row_base(c * kPass + tid / 8 - S::kTok);
      // a wave's 64 chunks go to 1 KB of LDS from its first place on
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + (off[c] + k)),
                                       (__attribute__((address_space(3))) void*)(buf + (c * S::kThreads + wave * 64) * 16), 16, 0, 0);
    }
  };
  const int tok_at = (wm * MT * 16 + n16) * kGemmStep + ((kb ^ (n16 & 7)) << 4);
  const int row_at = (S::kTok + wn * NT * 16 + n16) * kGemmStep + ((kb ^ (n16 & 7)) << 4);
  auto read = [&](const unsigned char* buf, int at, int more) __attribute__((always_inline)) {
    GemmFrag r;  // (chunk kb + 4 lies at the place with bit 2 flipped)
    r.v[0] = *reinterpret_cast<const gemm_i32x4*>(buf + at + more);
    r.v[1] = *reinterpret_cast<const gemm_i32x4*>(buf + (at ^ 64) + more);
    return r;
  };
  auto compute = [&](const unsigned char* buf, const float* scl, float wscale, int left) __attribute__((always_inline)) {
    GemmFrag w[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      w[nt] = read(buf, row_at, nt * 16 * kGemmStep);
      if (left < kGemmStep) {  // past the rows' end: one operand's zeros
        if (kb * 16 >= left) w[nt].v[0] = gemm_i32x4{0, 0, 0, 0};
        if (kb * 16 + 64 >= left) w[nt].v[1] = gemm_i32x4{0, 0, 0, 0};
      }
    }
    GemmFrag x = read(buf, tok_at, 0);
    float f = 0.0f;
    if constexpr (gemm_scaled(KIND)) f = scl[wm * MT * 16 + n16] * wscale;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      GemmFrag xn;
      float fn = 0.0f;
      if (mt + 1 < MT) {
        xn = read(buf, tok_at, (mt + 1) * 16 * kGemmStep);
        if constexpr (gemm_scaled(KIND)) fn = scl[(wm * MT + mt + 1) * 16 + n16] * wscale;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) gemm_mfma<KIND>(w[nt], x, f, acc[mt][nt]);
      if constexpr (gemm_scaled(KIND)) {  // the sums stay here: sunk below, each would hold registers of its own
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) asm volatile("" : "+v"(acc[mt][nt]));
      }
      x = xn;
      f = fn;
    }
  };

  const int count = step1 - step0;
  if (count <= 0) return;
  const int left = kbytes - (step1 - 1) * kGemmStep;   // bytes of the last step
  const int full = left < kGemmStep ? count - 1 : count;
  stage(step0, lds0);
  float wscale = 0.0f, wnext = 0.0f;
  if constexpr (gemm_scaled(KIND)) {
    wscale = sw[step0];
    if (tid < S::kTok) scl0[tid] = sx_row[step0];
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  int i = 0;
  auto body = [&](unsigned char* buf, unsigned char* other, float* scl, float* scl_other) __attribute__((always_inline)) {
    float s = 0.0f;
    if (i + 1 < count) {
      stage(step0 + i + 1, other);
      if constexpr (gemm_scaled(KIND)) {
        wnext = sw[step0 + i + 1];
        if (tid < S::kTok) s = sx_row[step0 + i + 1];
      }
    }
    compute(buf, scl, wscale, kGemmStep);
    __builtin_amdgcn_s_waitcnt(0);
    if constexpr (gemm_scaled(KIND)) {
      if (tid < S::kTok) scl_other[tid] = s;
      wscale = wnext;
    }
    __syncthreads();
    ++i;
  };
  while (i < full) {
    body(lds0, lds1, scl0, scl1);
    if (i >= full) break;
    body(lds1, lds0, scl1, scl0);
  }
  if (full < count) compute(full & 1 ? lds1 : lds0, full & 1 ? scl1 : scl0, wscale, left);
}

// ---- few tokens ----

// One tile of 16 rows of B (row_ptr gives this lane's) against MT x 16 tokens,
// steps first, first + stride, ... below `steps`, into acc; U steps' loads are
// issued together.
template <int KIND, int MT, int U>
__device__ __forceinline__ void gemm_rows(const unsigned char* row, const unsigned char* const (&tok)[MT], int kbytes,
                                          int first, int stride, int steps, const float* sw, const float* const (&sx)[MT],
                                          gemm_f32x4 (&acc)[MT]) {
  const int kb = (threadIdx.x & 63) >> 4;
  for (int s = first; s < steps; s += U * stride) {
    GemmFrag w[U], x[U][MT];
    float f[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = s + u * stride;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = min(step * kGemmStep + (kb + 4 * j) * 16, kbytes - 16);
        w[u].v[j] = __builtin_nontemporal_load(reinterpret_cast<const gemm_i32x4*>(row + k));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) x[u][mt].v[j] = *reinterpret_cast<const gemm_i32x4*>(tok[mt] + k);
      }
      if constexpr (gemm_scaled(KIND)) {
        const int g = min(step, steps - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) f[u][mt] = sx[mt][g] * sw[g];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int left = kbytes - (s + u * stride) * kGemmStep;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if ((kb + 4 * j) * 16 >= left) w[u].v[j] = gemm_i32x4{0, 0, 0, 0};
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) gemm_mfma<KIND>(w[u], x[u][mt], f[u][mt], acc[mt]);
    }
  }
}

// Sums of the workgroup's waves, in their order: thread i < 64 MT holds lane i
// % 64's part of token tile i / 64.
template <int MT, int WAVES>
__device__ __forceinline__ gemm_f32x4 gemm_join_waves(gemm_f32x4 (&lds)[WAVES][MT][64], const gemm_f32x4 (&acc)[MT]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) lds[wave][mt][lane] = acc[mt];
  __syncthreads();
  gemm_f32x4 s = {0, 0, 0, 0};
  if (wave < MT) {
    s = lds[0][wave][lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) s += lds[i][wave][lane];
  }
  return s;
}

// ---- results ----

// Hands a wave's tile, rows of 16 NT results with get(mt, nt) the lanes' parts,
// to store(t, n, v) by 8 neighbours v at token t and column n: through `bytes` of
// LDS that the wave has to itself, so that rows are written in whole lines.
// (Chunks of 4 results are XORed with the token against bank conflicts.)
template <int MT, int NT, int BYTES, class Get, class Store>
__device__ __forceinline__ void gemm_out(float* lds, Get get, Store store) {
  constexpr int kCols = 16 * NT, kFit = BYTES / (16 * kCols * 4), kRound = kFit < MT ? kFit : MT;
  constexpr int kLanes = kCols / 8, kRows = 64 / kLanes, kMask = 4 * NT - 1;
  static_assert(kRound >= 1 && MT % kRound == 0 && (NT & (NT - 1)) == 0, "whole rounds");
  const int lane = threadIdx.x & 63, n16 = lane & 15, kb = lane >> 4;
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += kRound) {
#pragma unroll
    for (int m = 0; m < kRound; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<gemm_f32x4*>(lds + (m * 16 + n16) * kCols + (((4 * nt + kb) ^ (n16 & kMask)) << 2)) = get(m0 + m, nt);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll 2
    for (int r = lane / kLanes; r < 16 * kRound; r += kRows) {
      const int c = 2 * (lane % kLanes);
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const gemm_f32x4 q = *reinterpret_cast<const gemm_f32x4*>(lds + r * kCols + (((c + h) ^ (r & 15 & kMask)) << 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = q[i];
      }
      store(m0 * 16 + r, 4 * c, v);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace moeq4
