// Modified scores and key intervals of the biased attention calls.
//
// A query at position pos sees the keys lo <= j < hi of its sequence,
//   lo = max(key_start[row], pos - window + 1, 0),  hi = max(pos + 1, prefix),
// with scores s' = cap tanh(s / cap) - slope |pos - j|.  Everything is kept in
// base-2 units (times log2 e), as in the plain kernels.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

// Interval of a query at position pos of a sequence of ctx tokens; lo == hi: it sees
// nothing and its output is zero.
__device__ __forceinline__ void key_interval(const AttnParams& p, int row, int pos, int ctx,
                                             int bidir, int* lo, int* hi) {
  int h = max(pos + 1, min(bidir, ctx));
  int l = 0;
  if (p.key_start) l = max(l, __ldg(p.key_start + row));
  if (p.window > 0) l = max(l, pos - p.window + 1);
  *hi = h;
  *lo = min(l, h);
}

// Keys of a decode row, its sequence's last token: the query's position is hi - 1.  A
// context beyond the block table or the caller's bound is clamped and flagged.
struct RowKeys {
  int lo, hi;
};
__device__ __forceinline__ RowKeys mods_row_keys(const AttnParams& p, int row, bool report) {
  const int cap = min(p.max_blocks_per_seq * kBlockSize, p.max_context);
  int ctx = __ldg(p.context_lens + row);
  if (ctx < 0 || ctx > cap) {
    if (report) flag_error(p.errors, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : cap;
  }
  RowKeys r;
  key_interval(p, row, ctx - 1, ctx, 0, &r.lo, &r.hi);
  return r;
}

// First key of a row's partitions: lo rounded down to a whole block.
__device__ __forceinline__ int first_block_key(int lo) { return lo & ~(kBlockSize - 1); }

// Partitions of a row with interval [lo, hi).
__device__ __forceinline__ int mods_parts(const AttnParams& p, int lo, int hi) {
  return hi > lo ? (hi - first_block_key(lo) + p.partition - 1) / p.partition : 0;
}

// tanh(x) for |x| <= kTanhPoly as x + x^3 q(x^2), q of degree 2: its coefficients
// minimise the largest relative error there (iteratively reweighted least
// squares on Chebyshev points); with fp32 rounding 7e-7 relative.
constexpr float kTanhPoly = 0.5f;
constexpr float kTanh3 = -0.333281606f, kTanh5 = 0.132053599f, kTanh7 = -0.044750642f;
__device__ __forceinline__ float tanh_poly(float x) {
  const float x2 = x * x;
  const float q = fmaf(x2, fmaf(x2, kTanh7, kTanh5), kTanh3);
  return fmaf(x2 * x, q, x);
}

// tanh(x) = 1 - 2 / (e^2x + 1) on the MUFU (exponential and reciprocal, absolute
// error about 2^-23), the polynomial where that difference would cancel.  Both
// are good to 1e-6 relative, so the capped score is for any cap.  (The one-
// instruction tanh.approx is good to 2^-11 only: a capped score of 50 would be
// off by 0.024, its weight by 2 %.)
__device__ __forceinline__ float cap_tanh(float x) {
  const float e = fast_exp2(x * (2.0f * kLog2e));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
  return fabsf(x) <= kTanhPoly ? tanh_poly(x) : fmaf(-2.0f, r, 1.0f);
}

// Two E4M3 terms of each of the pair x (0 <= x <= 448, a softmax weight times a power
// of two): codes *hi of x rounded to four significant bits (on the bits of the fp32
// number: three of the mantissa stay), codes *lo of what that leaves.  Two
// conversions a pair, instead of the four that converting hi back from its codes
// would take.  hi + lo is good to 2^-8 of x; below E4M3's normal range, x < 2^-6, to
// 1.5 * 2^-10.
__device__ __forceinline__ void split_e4m3(float2 x, uint32_t* hi, uint32_t* lo) {
  const float hx = __uint_as_float((__float_as_uint(x.x) + 0x80000u) & 0xfff00000u);
  const float hy = __uint_as_float((__float_as_uint(x.y) + 0x80000u) & 0xfff00000u);
  *hi = __nv_cvt_float2_to_fp8x2(make_float2(hx, hy), __NV_SATFINITE, __NV_E4M3);
  *lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x - hx, x.y - hy), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace pkv
