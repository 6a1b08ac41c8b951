// Products C[t, n] = sum_k A[t, k] B[n, k] on the matrix cores: of 16-bit
// numbers, the operands' rows along k or across, or of E4M3 codes with a scale
// per 128.  A step is 128 bytes of every row (64 or 128 elements).  Internal
// header.
//
//   gemm_tiles, gemm_tiles_scaled   many tokens: steps are copied into LDS
//   gemm_rows                       few tokens: B straight into the operands
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

// A step's sums of E4M3 codes, a's rows along the result's rows (4 kb + i),
// b's along its columns (lane % 16).
template <int KIND>
__device__ __forceinline__ gemm_f32x4 gemm_product(const GemmFrag& a, const GemmFrag& b) {
  gemm_f32x4 s = {0, 0, 0, 0};
  if constexpr (KIND == kGemmFp8) {
    const gemm_i32x8 x = {a.v[0][0], a.v[0][1], a.v[0][2], a.v[0][3], a.v[1][0], a.v[1][1], a.v[1][2], a.v[1][3]};
    const gemm_i32x8 y = {b.v[0][0], b.v[0][1], b.v[0][2], b.v[0][3], b.v[1][0], b.v[1][1], b.v[1][2], b.v[1][3]};
    s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, s, 0, 0, 0, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gemm_e4m3_bf16(a.v[j >> 1][2 * (j & 1)], a.v[j >> 1][2 * (j & 1) + 1]),
                                                  gemm_e4m3_bf16(b.v[j >> 1][2 * (j & 1)], b.v[j >> 1][2 * (j & 1) + 1]), s, 0, 0, 0);
  }
  return s;
}

// ---- many tokens ----

// MT x NT tiles of 16 x 16 results a wave, and WM x WN waves: kTok tokens x
// kRows rows of B.
template <int KIND_, int MT_, int NT_, int WM_, int WN_>
struct GemmShape {
  static constexpr int KIND = KIND_, MT = MT_, NT = NT_, WM = WM_, WN = WN_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, kTok = 16 * MT * WM, kRows = 16 * NT * WN;
  static constexpr int kScaleRows = (kRows + 127) / 128;
};

// The tiles of a launch: tok_tiles x row_tiles of them, each in `splits` parts
// of steps_per steps.  A workgroup takes one after another.  Workgroups b, b +
// 8, ... share an XCD (and its L2): each XCD takes a contiguous run, which goes
// through 8 token tiles at a time, so the 32 tiles that it works on together
// read 8 + 4 tiles of the operands.
struct GemmTiles {
  int tok_tiles, row_tiles, splits, steps_per, steps;
};
struct GemmPlace {
  int tok, row, split, step0, count;
};
struct GemmQueue {
  int next, end, stride;
  __device__ __forceinline__ explicit GemmQueue(const GemmTiles& t) {
    const int all = t.tok_tiles * t.row_tiles * t.splits, per = all / 8, rest = all % 8, xcd = blockIdx.x & 7;
    const int first = xcd * per + min(xcd, rest);
    next = first + (int)(blockIdx.x >> 3);
    end = first + per + (xcd < rest ? 1 : 0);
    stride = ((int)gridDim.x - xcd + 7) / 8;
  }
  __device__ __forceinline__ bool any() const { return next < end; }
  __device__ __forceinline__ GemmPlace take(const GemmTiles& t) {
    const int tiles = t.tok_tiles * t.row_tiles;
    const int id = next % tiles, split = next / tiles;
    next += stride;
    const int group = id / (8 * t.row_tiles), in = id % (8 * t.row_tiles), first = group * 8, size = min(t.tok_tiles - first, 8);
    GemmPlace p;
    p.tok = first + in % size;
    p.row = in / size;
    p.split = split;
    p.step0 = split * t.steps_per;
    p.count = min(t.steps - p.step0, t.steps_per);
    return p;
  }
};

// This wave's LDS reads and all but its last LEFT copies are done, and so are
// the other waves'.
template <int LEFT>
__device__ __forceinline__ void gemm_meet() {
  static_assert(LEFT < 64, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (LEFT >> 4) << 14 | 0x70);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A value that the compiler does not know to be the same for every tile: what
// depends on it would be worked out ahead of the tiles, and held through their
// loops.
__device__ __forceinline__ int gemm_opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 16 bytes a lane from memory into 1 KB of LDS, without passing registers.
__device__ __forceinline__ void gemm_copy(const unsigned char* from, unsigned char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Where a tile's rows lie: row r of its tokens at tok + tok_off(r), of B at
// row_base(r) + row_off(r), rows past the operand's end at some row within;
// offsets have 32 bits.  scales (E4M3): this thread's row of scales, one a
// step: thread tid < kTok has the tile's token tid's, the next kScaleRows
// threads have those of each 128 of B's rows.

// Products of 16-bit numbers: runs the workgroup's tiles, source.set(place)
// before each and store(place, acc) behind it.
//
// A source says for each operand whether its memory has the sum's axis along
// its rows (as above; step s begins at byte source.k(s)) or across them
// (kTokT, kRowT): then chunk c of 8 of the tile's tokens lies at column
// tok_col(c), in bytes, of rows tok_ld apart, the step's 64 from tok_at(s) on;
// columns past the operand's end at some within.  source.left(s) is the number
// of bytes along the sum's axis from step s on, above 0; a multiple of 16
// where an operand has that axis along its rows.
//
// LDS holds BUFFERS steps of all rows, 128 bytes each.  Chunk c of row r lies at
// place c ^ (r / 2 % 8), so that the 16 rows that are read together fall in
// different banks (of 64).  Of an operand with the axis across, it holds the
// step's 64 rows of 128 bytes (64 tokens) one after another, then the next
// tokens'; 16 lanes read 4 rows of 32 bytes and get a column of them each
// (ds_read_b64_tr_b16); 32 lanes read rows k to k + 3 and k + 8 to k + 11, so
// chunk c of row k lies at place c ^ (k / 2 % 2 * 4 + k / 8 % 2 * 2).
//
// A wave's instructions go through half a step (its chunks 0 to 3 or 4 to 7) at
// a time, while the next half's operands are on their way into registers; so
// the waves have read a step when its second half begins, meet there, once a
// step, and that half carries the copies of the step BUFFERS on into the LDS
// that became free.  Four waves of 128 x 128 results each: their sums fill the
// accumulator registers, and they read two thirds of what eight of 128 x 64
// would.  The instruction is of 16 x 16 x 32: one of 32 x 32 x 16 reads and
// writes twice the sums for a product, and the card's power, which bounds large
// products, lets it do 1800 and not 2050 TFLOP/s (operands in registers).
//
// Two buffers are enough where a step's instructions take 2048 clocks.  Small
// tiles have more, since what is on its way must last a memory's latency, about
// 2000 clocks; there the steps go BUFFERS at a time, past the last one with
// zeros: the compiler must see what is on its way at each read, and where a
// loop ends in several places it waits for all of it.

// LDS buffers of a shape's 16-bit steps: as many as one workgroup a compute
// unit leaves room for.  A tile of 128 x 128 takes 0.47 us a step with four and
// 0.86 with two workgroups of two buffers, one of 256 x 256 is bound by its
// products with two.
template <class S>
__host__ __device__ constexpr int gemm_buffers() {
  return S::kTok == 256 ? 2 : S::kRows > 128 ? 3 : 4;
}

// Four 16-bit numbers of a column: the 16 lanes' 8 bytes each, 4 rows of 4 lanes.
__device__ __forceinline__ uint2 gemm_read_column(const unsigned char* lds) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)lds));
}

template <class S, class Source, class Store>
__device__ __forceinline__ void gemm_tiles(const GemmTiles& tiles, Source& source, Store store) {
  constexpr int BUFFERS = gemm_buffers<S>();
  constexpr bool kTokT = Source::kTokT, kRowT = Source::kRowT;
  constexpr int MT = S::MT, NT = S::NT, KIND = S::KIND, kPass = S::kThreads / 8;
  constexpr int kCb = S::kRows / kPass, kCt = S::kTok / kPass, kCopies = kCb + kCt;
  constexpr int kReadsX = kTokT ? 2 * MT : MT, kReadsW = kRowT ? 2 * NT : NT;
  constexpr int kReads = kReadsX + kReadsW, kMul = MT * NT;  // of half a step
  constexpr int kEarly = kMul * 7 / 8;  // instructions that the reads are spread over: the last have a latency's time
  static_assert(S::kRows % 64 == 0 && S::kTok % 64 == 0 && kPass == 32, "copies of whole passes");
  // each an object of its own: the compiler then knows that reads of one do not wait for copies into another
  constexpr int kRowBytes = S::kRows * kGemmStep, kTokBytes = S::kTok * kGemmStep;
  __shared__ __attribute__((aligned(1024))) unsigned char b0[kRowBytes], b1[kRowBytes], b2[BUFFERS > 2 ? kRowBytes : 1], b3[BUFFERS > 3 ? kRowBytes : 1];
  __shared__ __attribute__((aligned(1024))) unsigned char t0[kTokBytes], t1[kTokBytes], t2[BUFFERS > 2 ? kTokBytes : 1], t3[BUFFERS > 3 ? kTokBytes : 1];
  static_assert(BUFFERS >= 2 && BUFFERS <= 4, "as many of them are used");
  auto rows_of = [&](int i) __attribute__((always_inline)) { return i == 0 ? b0 : i == 1 ? b1 : i == 2 ? b2 : b3; };
  auto toks_of = [&](int i) __attribute__((always_inline)) { return i == 0 ? t0 : i == 1 ? t1 : i == 2 ? t2 : t3; };
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, kb = lane >> 4;
  const int wm = wave % S::WM, wn = wave / S::WM;
  const int chunk = ((tid & 7) ^ ((tid >> 4) & 7)) * 16;
  const int along = (n16 << 7) + ((kb ^ (n16 >> 1)) << 4);
  const int across = ((8 * kb + (lane >> 2 & 3)) << 7) + ((lane >> 3 & 1) << 6) + ((kb & 1) << 5) + ((lane & 3) << 3);
  // a wave's first tile, and its first four with the axis across: tiles are quarters of a row of 64 tokens
  const auto quarter = [&](int tile) __attribute__((always_inline)) { return tile / 4 * (64 * kGemmStep) + (across ^ (tile % 4 << 5)); };
  const int tok0 = wm * MT, row0 = wn * NT;
  const int tok_at = tok0 * 16 * kGemmStep + along, tok_q[4] = {quarter(tok0), quarter(tok0 + 1), quarter(tok0 + 2), quarter(tok0 + 3)};
  const int row_at = row0 * 16 * kGemmStep + along, row_q[4] = {quarter(row0), quarter(row0 + 1), quarter(row0 + 2), quarter(row0 + 3)};

  GemmQueue queue(tiles);
  GemmPlace at, now;
  // rows' offsets; of an operand with the axis across, two rows' offsets and then columns'
  uint32_t off_b[kRowT ? kCb / 2 + 2 : kCb], off_t[kTokT ? kCt / 2 + 2 : kCt], k = 0, b_row[2] = {}, t_row[2] = {};
  const unsigned char *b_from = nullptr, *t_from = nullptr;
  auto place = [&](int i) __attribute__((always_inline)) {
    const int s = at.step0 + min(i, at.count - 1), left = source.left(s);  // (past the end: of the same rows)
    if constexpr (!kTokT || !kRowT) k = source.k(s) + min(chunk, left - 16);
    const uint32_t last = (uint32_t)(left / 2 - 1);
    if constexpr (kTokT) {
      t_from = source.tok_at(s);
#pragma unroll
      for (int j = 0; j < 2; ++j) t_row[j] = left >= kGemmStep ? off_t[kCt / 2 + j] : min(off_t[kCt / 2 + j], last * (uint32_t)source.tok_ld());
    }
    if constexpr (kRowT) {
      b_from = source.row_at(s);
#pragma unroll
      for (int j = 0; j < 2; ++j) b_row[j] = left >= kGemmStep ? off_b[kCb / 2 + j] : min(off_b[kCb / 2 + j], last * (uint32_t)source.row_ld());
    }
  };
  auto copy = [&](int to, int c) __attribute__((always_inline)) {
    if (c < kCb) {
      unsigned char* lds = rows_of(to) + c * kPass * kGemmStep + wave * 1024;
      if constexpr (kRowT)
        gemm_copy(b_from + (off_b[c / 2] + b_row[c % 2]), lds);
      else
        gemm_copy(source.row_base(c * kPass + tid / 8) + (off_b[c] + k), lds);
    } else {
      c -= kCb;
      unsigned char* lds = toks_of(to) + c * kPass * kGemmStep + wave * 1024;
      if constexpr (kTokT)
        gemm_copy(t_from + (off_t[c / 2] + t_row[c % 2]), lds);
      else
        gemm_copy(source.tok + (off_t[c] + k), lds);
    }
  };
  auto start = [&]() __attribute__((always_inline)) {  // the next tile and its first steps
    at = queue.take(tiles);
    source.set(at);
    const int mine = gemm_opaque(tid / 8), column = gemm_opaque((tid & 7) ^ (tid >> 4 & 1) << 2 ^ (tid >> 6 & 1) << 1);
    if constexpr (kRowT) {
#pragma unroll
      for (int c = 0; c < kCb / 2; ++c) off_b[c] = source.row_col(8 * c + column);
#pragma unroll
      for (int j = 0; j < 2; ++j) off_b[kCb / 2 + j] = (uint32_t)(mine + 32 * j) * (uint32_t)source.row_ld();
    } else {
#pragma unroll
      for (int c = 0; c < kCb; ++c) off_b[c] = source.row_off(c * kPass + mine);
    }
    if constexpr (kTokT) {
#pragma unroll
      for (int c = 0; c < kCt / 2; ++c) off_t[c] = source.tok_col(8 * c + column);
#pragma unroll
      for (int j = 0; j < 2; ++j) off_t[kCt / 2 + j] = (uint32_t)(mine + 32 * j) * (uint32_t)source.tok_ld();
    } else {
#pragma unroll
      for (int c = 0; c < kCt; ++c) off_t[c] = source.tok_off(c * kPass + mine);
    }
#pragma unroll
    for (int i = 0; i < BUFFERS; ++i) {
      place(i);
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(i, c);
    }
  };
  gemm_i32x4 w[2][NT], x[2][MT];  // of half h: chunk 4 h + kb of a row
  gemm_f32x4 acc[MT][NT];
  auto read_across = [&](gemm_i32x4& to, const unsigned char* lds, const int (&q)[4], int h, int j) __attribute__((always_inline)) {
    const int tile = j / 2, part = j % 2;  // (rows 8 kb + 4 part on of the half's 32)
    const uint2 v = gemm_read_column(lds + q[tile % 4] + (tile / 4 * 64 + h * 32 + part * 4) * kGemmStep);
    to[2 * part] = (int)v.x;
    to[2 * part + 1] = (int)v.y;
  };
  auto read = [&](int from, int h, int r) __attribute__((always_inline)) {
    const int q = r - kReadsW;
    if (r < kReadsW) {
      if constexpr (kRowT)
        read_across(w[h][r / 2], rows_of(from), row_q, h, r);
      else
        w[h][r] = *reinterpret_cast<const gemm_i32x4*>(rows_of(from) + (row_at ^ 64 * h) + r * 16 * kGemmStep);
    } else {
      if constexpr (kTokT)
        read_across(x[h][q / 2], toks_of(from), tok_q, h, q);
      else
        x[h][q] = *reinterpret_cast<const gemm_i32x4*>(toks_of(from) + (tok_at ^ 64 * h) + q * 16 * kGemmStep);
    }
  };
  auto multiply = [&](int h, int j, bool first) __attribute__((always_inline)) {
    const int mt = j / NT, nt = j % NT;
    const gemm_f32x4 c = first ? gemm_f32x4{} : acc[mt][nt];
    if constexpr (KIND == kGemmBf16)
      acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gemm_bf16x8, w[h][nt]), __builtin_bit_cast(gemm_bf16x8, x[h][mt]), c, 0, 0, 0);
    else
      acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(gemm_f16x8, w[h][nt]), __builtin_bit_cast(gemm_f16x8, x[h][mt]), c, 0, 0, 0);
  };
  // half a step, reading the next one, of buffer `from`; the copies into `to` with it (-1: none)
  auto pass = [&](int h, int from, int to, bool first = false) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kMul; ++q) {
#pragma unroll
      for (int j = q * kReads / kEarly; j < (q + 1) * kReads / kEarly && j < kReads; ++j) read(from, h ^ 1, j);
#pragma unroll
      for (int j = q * kCopies / kMul; to >= 0 && j < (q + 1) * kCopies / kMul; ++j) copy(to, j);
      multiply(h, q, first);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto keep = [&](gemm_i32x4& v, int bytes) __attribute__((always_inline)) {
    if constexpr (kTokT && kRowT) {  // an end anywhere
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = bytes >= 4 * i + 4 ? v[i] : bytes == 4 * i + 2 ? v[i] & 0xffff : 0;
    } else if (bytes <= 0) {
      v = gemm_i32x4{0, 0, 0, 0};
    }
  };
  auto cut = [&](int h, int i) __attribute__((always_inline)) {  // past the axis' end, or the last step: zeros
    const int left = i < now.count ? source.left(now.step0 + i) - h * 64 : 0;
    if (left < 64) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) keep(w[h][nt], left - 16 * kb);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) keep(x[h][mt], left - 16 * kb);
    }
  };

  if (!queue.any()) return;
  start();
  while (true) {
    now = at;
    gemm_meet<(BUFFERS - 1) * kCopies>();  // the first step is there
#pragma unroll
    for (int j = 0; j < kReads; ++j) read(0, 0, j);
    cut(0, 0);
    pass(0, 0, -1, true);
    cut(1, 0);
    constexpr int kOnWay = (BUFFERS - 2) * kCopies;  // copies of later steps than the next
    gemm_meet<kOnWay>();
    int i = 0;
    auto body = [&](int buf) __attribute__((always_inline)) {
      const int next = (buf + 1) % BUFFERS;
      place(i + BUFFERS);
      pass(1, next, buf);
      ++i;
      cut(0, i);
      pass(0, next, -1);
      cut(1, i);
      gemm_meet<kOnWay>();
    };
    if constexpr (BUFFERS == 2) {
      while (i + 1 < now.count) {
        body(0);
        if (i + 1 >= now.count) break;
        body(1);
      }
    } else {
      while (i + 1 < now.count) {
        body(0);
        body(1);
        body(2);
        if constexpr (BUFFERS > 3) body(3);
      }
      gemm_meet<0>();  // nothing is on its way into the next tile's LDS
    }
    // the last half step, from registers; the LDS is the next tile's
    const bool more = queue.any();
    if (more) start();
#pragma unroll
    for (int j = 0; j < kMul; ++j) multiply(1, j, false);
    store(now, acc);
    if (!more) break;
  }
}

// Products of E4M3 codes with a scale per step, 8 waves of 128 x 64 results
// (or 4 of fewer).  A step's sums come out of one instruction (or four of
// kGemmFp8Wide) into registers of their own and enter the accumulators by a
// multiply-add each, two instructions behind, so that these never wait; the
// accumulators have to lie among the vector registers for that.
//
// LDS holds two steps as above.  A wave reads a token tile two groups of
// matrix instructions ahead, the next step's too, and its rows of B within a
// step's last group, each behind its last use.  The waves meet twice a step:
// once when all have read B and the first half of their token tiles, whose LDS
// then takes the copies of the step after the next, and once when all have
// read the second half.  So copies have more than a step's time, and nobody
// waits for the last ones.  Steps go in pairs, for an odd number of them with
// one of zeros, since the compiler must see what is on its way at each read:
// where a loop ends in two places it waits for everything.
template <class S, class Source, class Store>
__device__ __forceinline__ void gemm_tiles_scaled(const GemmTiles& tiles, int kbytes, Source& source, Store store) {
  constexpr int MT = S::MT, NT = S::NT, KIND = S::KIND, kPass = S::kThreads / 8;
  constexpr int kCb = S::kRows / kPass, kCh = S::kTok / 2 / kPass;  // copies of B, of half the tokens
  constexpr int kHalf = S::kTok / 2 * kGemmStep;
  static_assert(S::kRows % kPass == 0 && S::kTok / 2 % kPass == 0 && S::kTok + S::kScaleRows <= S::kThreads, "copies of whole passes");
  static_assert(MT % 4 == 0, "a ring of four token tiles");
  __shared__ __attribute__((aligned(1024))) unsigned char b0[S::kRows * kGemmStep], b1[S::kRows * kGemmStep];
  __shared__ __attribute__((aligned(1024))) unsigned char lo0[kHalf], lo1[kHalf], hi0[kHalf], hi1[kHalf];
  __shared__ float scale0[S::kTok + 64], scale1[S::kTok + 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, kb = lane >> 4;
  const int wm = wave % S::WM, wn = wave / S::WM;
  const int chunk = ((tid & 7) ^ ((tid >> 4) & 7)) * 16;
  const int tok_at = (wm * MT * 8 + n16) * kGemmStep + ((kb ^ (n16 >> 1)) << 4);
  const int row_at = (wn * NT * 16 + n16) * kGemmStep + ((kb ^ (n16 >> 1)) << 4);

  GemmQueue queue(tiles);
  GemmPlace at;
  uint32_t off_b[kCb], off_t[2][kCh], k = 0;
  auto place = [&](int i) __attribute__((always_inline)) {
    // past the end: of the same rows, since a NaN times zero stays one
    k = min((at.step0 + min(i, at.count - 1)) * kGemmStep + chunk, kbytes - 16);
  };
  auto copy_lo = [&](int to, int c) __attribute__((always_inline)) {
    if (c < kCb)
      gemm_copy(source.row_base(c * kPass + tid / 8) + (off_b[c] + k), (to ? b1 : b0) + c * kPass * kGemmStep + wave * 1024);
    else
      gemm_copy(source.tok + (off_t[0][c - kCb] + k), (to ? lo1 : lo0) + (c - kCb) * kPass * kGemmStep + wave * 1024);
  };
  auto copy_scales = [&](int i, int to) __attribute__((always_inline)) {
    if (tid < S::kTok + S::kScaleRows)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(source.scales + at.step0 + min(i, at.count - 1)),
                                       (__attribute__((address_space(3))) void*)((to ? scale1 : scale0) + wave * 64), 4, 0, 0);
  };
  auto copy_hi = [&](int to, int c) __attribute__((always_inline)) {
    gemm_copy(source.tok + (off_t[1][c] + k), (to ? hi1 : hi0) + c * kPass * kGemmStep + wave * 1024);
  };
  auto copy_all = [&](int i) __attribute__((always_inline)) {
    place(i);
#pragma unroll
    for (int c = 0; c < kCb + kCh; ++c) copy_lo(i, c);
    copy_scales(i, i);
#pragma unroll
    for (int c = 0; c < kCh; ++c) copy_hi(i, c);
  };
  GemmFrag x[4], w[NT];
  float f[4], w_scale = 0.0f, w_next = 0.0f;
  gemm_f32x4 acc[MT][NT], sum[4];
  auto read = [&](const unsigned char* lds, int at, int more) __attribute__((always_inline)) {
    GemmFrag r;  // (chunk kb + 4 lies at the place with bit 2 flipped)
    r.v[0] = *reinterpret_cast<const gemm_i32x4*>(lds + at + more);
    r.v[1] = *reinterpret_cast<const gemm_i32x4*>(lds + (at ^ 64) + more);
    return r;
  };
  auto read_x = [&](int from, int mt) __attribute__((always_inline)) {
    const unsigned char* half = mt < MT / 2 ? (from ? lo1 : lo0) : (from ? hi1 : hi0);
    x[mt % 4] = read(half, tok_at, mt % (MT / 2) * 16 * kGemmStep);
    if (mt == 0) w_next = (from ? scale1 : scale0)[S::kTok + wn * NT * 16 / 128];
    f[mt % 4] = (from ? scale1 : scale0)[(wm * MT + mt) * 16 + n16];
  };
  auto read_w = [&](int from, int nt) __attribute__((always_inline)) { w[nt] = read(from ? b1 : b0, row_at, nt * 16 * kGemmStep); };
  auto cut = [&](int i) __attribute__((always_inline)) {  // past the rows' end, or the last step: one operand's zeros
    const int left = i < at.count ? kbytes - (at.step0 + i) * kGemmStep : 0;
    if (left < kGemmStep) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (kb * 16 + 64 * j >= left) w[nt].v[j] = gemm_i32x4{0, 0, 0, 0};
    }
  };
  auto body = [&](int buf, int i) __attribute__((always_inline)) {
    constexpr int kLo = kCb + kCh, kLoPer = (kLo + MT / 2 - 1) / (MT / 2), kHiPer = (kCh + 1) / 2;
    float fs[4];  // the factors of the sums that are still to be added
    w_scale = w_next;
    auto add = [&](int j) __attribute__((always_inline)) {
      gemm_f32x4& a = acc[j / NT][j % NT];
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = __builtin_fmaf(sum[j % 4][e], fs[j % 4], a[e]);
      asm volatile("" : "+v"(a));  // stays here: sunk below, each sum would hold registers of its own
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt == MT / 2 - 2) {  // B and the first half have been read; the second half is there
        gemm_meet<kCb + 2 * kCh>();
        place(i + 2);
      }
      if (mt + 2 < MT) read_x(buf, mt + 2);
      if (mt == MT - 2) {  // the second half has been read; the next step's B and first half are there
        gemm_meet<kCb + 2 * kCh>();
        copy_scales(i + 2, buf);
      }
      if (mt == MT - 1) {
        read_x(buf ^ 1, 0);
        read_x(buf ^ 1, 1);
      }
      __builtin_amdgcn_sched_barrier(0);  // reads first: they are a group's time ahead of their use
      if (mt >= MT / 2 - 2 && mt < MT - 2) {
#pragma unroll
        for (int c = (mt - (MT / 2 - 2)) * kLoPer; c < (mt - (MT / 2 - 2) + 1) * kLoPer && c < kLo; ++c) copy_lo(buf, c);
      }
      if (mt >= MT - 2) {
#pragma unroll
        for (int c = (mt - (MT - 2)) * kHiPer; c < (mt - (MT - 2) + 1) * kHiPer && c < kCh; ++c) copy_hi(buf, c);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int j = mt * NT + nt;
        sum[j % 4] = gemm_product<KIND>(w[nt], x[mt % 4]);
        fs[j % 4] = f[mt % 4] * w_scale;
        if (mt == MT - 1) read_w(buf ^ 1, nt);
        if (j >= 2) add(j - 2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    add(MT * NT - 2);
    add(MT * NT - 1);
    cut(i + 1);
  };

  while (queue.any()) {
    at = queue.take(tiles);
    source.set(at);
#pragma unroll
    for (int c = 0; c < kCb; ++c) off_b[c] = source.row_off(c * kPass + tid / 8);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const int r = c * kPass + tid / 8;
        off_t[h][c] = source.tok_off(r / (8 * MT) * (16 * MT) + h * (8 * MT) + r % (8 * MT));
      }
    copy_all(0);
    gemm_meet<0>();
    copy_all(1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        acc[mt][nt] = gemm_f32x4{0, 0, 0, 0};
        asm volatile("" : "+v"(acc[mt][nt]));  // hides the zeros, which the compiler would carry along in registers of their own
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) read_w(0, nt);
    cut(0);
    read_x(0, 0);
    read_x(0, 1);
    int i = 0;
    do {
      body(0, i);
      body(1, i + 1);
      i += 2;
    } while (i < at.count);
    gemm_meet<0>();  // no copy is on its way, and no read, when the next tile's begin
    store(at, acc);
  }
}

// ---- few tokens ----

// J groups of 8 rows of B against G groups of 8 tokens, rows read once.  A
// load of 16 bytes a lane takes 8 whole lines of 128 bytes, one a row: 16 rows
// of 64 bytes each, what an operand of 16 rows would take, are read at 3.8 and
// not 5.5 TB/s (6144 rows of 6144 bytes, the loads alone).  So an operand's row
// m is row m / 2 of the group, of whose line it holds the chunks 2 kb + m % 2,
// and tokens likewise: results (m, t) with m % 2 = t % 2 are the sums over one
// half of the chunks each, the others mean nothing.

// A product of 16 bytes a lane: one instruction of 16-bit numbers onto acc, two
// of E4M3 codes made bf16, whose sums times f go onto acc.
template <int KIND>
__device__ __forceinline__ void gemm_chunk(gemm_i32x4 w, gemm_i32x4 x, float f, gemm_f32x4& acc) {
  if constexpr (KIND == kGemmFp8Wide) {
    gemm_f32x4 s = {0, 0, 0, 0};
    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gemm_e4m3_bf16(w[0], w[1]), gemm_e4m3_bf16(x[0], x[1]), s, 0, 0, 0);
    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gemm_e4m3_bf16(w[2], w[3]), gemm_e4m3_bf16(x[2], x[3]), s, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(s[i], f, acc[i]);
  } else if constexpr (KIND == kGemmBf16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gemm_bf16x8, w), __builtin_bit_cast(gemm_bf16x8, x), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(gemm_f16x8, w), __builtin_bit_cast(gemm_f16x8, x), acc, 0, 0, 0);
  }
}

// This lane's row of 8, token of 8 and chunk in the above.
__device__ __forceinline__ int gemm_rows_index() { return (threadIdx.x & 15) >> 1; }
__device__ __forceinline__ int gemm_rows_chunk() { return 2 * ((threadIdx.x & 63) >> 4) + (threadIdx.x & 1); }

// Steps first, first + stride, ... below `steps` of the lane's rows and tokens
// into acc; U steps' loads are on their way together.
template <int KIND, int J, int G, int U>
__device__ __forceinline__ void gemm_rows(const unsigned char* const (&row)[J], const unsigned char* const (&tok)[G], int kbytes,
                                          int first, int stride, int steps, const float* sw, const float* const (&sx)[G],
                                          gemm_f32x4 (&acc)[J][G]) {
  const int at = gemm_rows_chunk() * 16;
  for (int s = first; s < steps; s += U * stride) {
    gemm_i32x4 w[U][J], x[U][G];
    float f[U][G];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = s + u * stride;
      if (step < steps) {
        const int k = min(step * kGemmStep + at, kbytes - 16);
#pragma unroll
        for (int j = 0; j < J; ++j) w[u][j] = __builtin_nontemporal_load(reinterpret_cast<const gemm_i32x4*>(row[j] + k));
#pragma unroll
        for (int g = 0; g < G; ++g) x[u][g] = *reinterpret_cast<const gemm_i32x4*>(tok[g] + k);
        if constexpr (gemm_scaled(KIND)) {
#pragma unroll
          for (int g = 0; g < G; ++g) f[u][g] = sx[g][step];
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all are on their way before the first is waited for
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = s + u * stride;
      if (step >= steps) break;
      if (step * kGemmStep + at >= kbytes) {  // past the rows' end: zeros
#pragma unroll
        for (int j = 0; j < J; ++j) w[u][j] = gemm_i32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) x[u][g] = gemm_i32x4{0, 0, 0, 0};
      }
      float ws = 1.0f;
      if constexpr (gemm_scaled(KIND)) ws = sw[step];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < J; ++j) gemm_chunk<KIND>(w[u][j], x[u][g], gemm_scaled(KIND) ? f[u][g] * ws : 1.0f, acc[j][g]);
    }
  }
}

// The two halves' sums, and those of the workgroup's waves in their order:
// behind it lds[0][j][g][lane] is the result of row 2 (lane / 16) + lane % 2
// of group j and token lane % 16 / 2 of group g.
template <int J, int G, int WAVES>
__device__ __forceinline__ void gemm_join_waves(float (&lds)[WAVES][J][G][64], const gemm_f32x4 (&acc)[J][G]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, odd = lane & 1;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // of its four rows, two rows' halves: a lane keeps the row that is its own and gives the other's
      const float low = odd ? acc[j][g][1] : acc[j][g][0], high = odd ? acc[j][g][3] : acc[j][g][2];
      const float mine = odd ? high : low, given = odd ? low : high;
      lds[wave][j][g][lane] = mine + __shfl_xor(given, 1);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < J * G * 64; i += 64 * WAVES) {
    float* at = &lds[0][0][0][0] + i;
    float v = at[0];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) v += at[k * J * G * 64];
    at[0] = v;  // (read by this thread alone so far)
  }
  __syncthreads();
}

// ---- results ----

// Eight neighbours' sums over the parts of a split K, added in their order; four
// parts' loads are on their way together (15 parts of 16 x 1104: one by one 6.1 us).
__device__ __forceinline__ void gemm_join8(const float* part, size_t stride, int splits, float (&s)[8]) {
  norm_load8(part, 8, s);
  for (int p = 1; p < splits; p += 4) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) norm_load8(part + (size_t)min(p + u, splits - 1) * stride, 8, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p + u < splits) s[j] += v[u][j];
  }
}

// A lane's sums go straight to memory, four neighbours of a token's results at
// a time: of a 16 x 16 tile those from 4 (lane / 16) on of token lane % 16.

// Results in vector registers from here on, and no sooner: of all tiles at
// once they would not fit beside the accumulator registers.
__device__ __forceinline__ gemm_f32x4 gemm_here(gemm_f32x4 v) {
  asm volatile("" : "+v"(v));
  return v;
}

template <class T>
__device__ __forceinline__ uint2 gemm_pack4(gemm_f32x4 v) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]});
}

// Fours of two tiles as 16-bit numbers, made eight neighbours of a lane, so that
// lanes write 16 bytes and a token's four lanes 64: of 32 each, the writes'
// number and not their bytes bound the stores (5 us of a tile).  Rows of 16
// lanes (a0 a1 a2 a3) and (b0 b1 b2 b3) are swapped to (a0 a2 b0 b2) and (a1 a3
// b1 b3): eight from 8 (lane / 16) on of a's 16 and then b's.
__device__ __forceinline__ uint4 gemm_eight16(uint2 a, uint2 b) {
  const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false), y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
  const auto u = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false), v = __builtin_amdgcn_permlane16_swap(y[0], y[1], false, false);
  return make_uint4(u[0], v[0], u[1], v[1]);
}

// The first `left` of eight 16-bit neighbours, or of four fp32, at any element's place.
__device__ __forceinline__ void gemm_put16(void* p, int left, uint4 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef u32x4 u32x4_any __attribute__((aligned(2)));
  if (left >= 8) {
    *reinterpret_cast<u32x4_any*>(p) = u32x4{v.x, v.y, v.z, v.w};
  } else {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) static_cast<uint16_t*>(p)[i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
  }
}
// Past the caches, where a token's four lanes write whole 64 bytes.
__device__ __forceinline__ void gemm_put32_past(float* p, gemm_f32x4 v) { __builtin_nontemporal_store(v, reinterpret_cast<gemm_f32x4*>(p)); }
__device__ __forceinline__ void gemm_put32(float* p, int left, gemm_f32x4 v) {
  typedef gemm_f32x4 f32x4_any __attribute__((aligned(4)));
  if (left >= 4) {
    *reinterpret_cast<f32x4_any*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) p[i] = v[i];
  }
}

}  // namespace moeq4
