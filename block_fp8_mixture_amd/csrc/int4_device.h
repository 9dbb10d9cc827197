// Device helpers of 4-bit integer weights w = s (q - z) as BF16 matrix
// operands.
//
// A code q becomes the BF16 value 16 + q by putting its four bits at the top
// of a mantissa of exponent 4 (0x4180 | q << 3): one shift and one and-or for two
// codes, exact. A group's sum then is s (sum a (16 + q) - (16 + z) sum a), with
// sum a from the matrix cores too (an operand of ones); 16 rather than a larger
// offset keeps the part that cancels within a few times the part that stays.
#pragma once

#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(uint4 a, uint4 b, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                 acc, 0, 0, 0);
}

// Eight codes (one word) as 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 int4_operand(uint32_t c) {
  constexpr uint32_t kMask = 0x00780078u, kOne = 0x41804180u;
  return uint4{(c << 3 & kMask) | kOne, (c >> 1 & kMask) | kOne, (c >> 5 & kMask) | kOne,
               (c >> 9 & kMask) | kOne};
}
// Eight BF16 values in that order.
__device__ __forceinline__ uint4 int4_order(uint4 x) {
  return uint4{__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
               __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

__device__ __forceinline__ float int4_scale(uint32_t bits, int f16) {
  const float h = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  return f16 ? h : bf16_to_f32(bits);
}

// exp(-g): v_exp_f32 of the product with log2(e), and what the product's rounding
// and the constant leave out as a factor 1 + d ln 2 (expf's code is three times as
// long, of which short launches feel the fetching).
__device__ __forceinline__ float exp_neg(float g) {
  constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;  // log2(e)
  const float t = -g * kHi;
  const float d = __builtin_fmaf(-g, kHi, -t) - g * kLo;
  const float e = __builtin_amdgcn_exp2f(t), r = __builtin_fmaf(e, d * 0.693147180559945f, e);
  return e > 0.0f && e < __builtin_inff() ? r : e;  // (0 and infinity times d may be NaN)
}

// SiLU(gate) * up in fp32; a NaN passes the clamps.
__device__ __forceinline__ float int4_gated(int act, float g, float u, float lim) {
  if (act == 1) g = g > lim ? lim : g;
  float s = g / (1.0f + exp_neg(g));
  if (act == 2) s = s > lim ? lim : s;
  if (act != 0) u = fabsf(u) > lim ? __builtin_copysignf(lim, u) : u;
  return s * u;
}

// First row and live rows of expert e (no counts: all rows are one expert's).
__device__ __forceinline__ int int4_seg_start(const Int4GemmArgs& p, int e) {
  return !p.counts ? 0 : p.seg_cap > 0 ? e * p.seg_cap : p.offsets[e];
}
__device__ __forceinline__ int int4_rows(const Int4GemmArgs& p, int e) {
  if (!p.counts) return p.row_cap;
  const int s0 = int4_seg_start(p, e);
  const int s1 = p.seg_cap > 0 ? s0 + p.seg_cap : p.offsets[e + 1];
  return segment_rows(s0, s1, p.counts[e], p.row_cap);
}
// Row of A behind row r, -1 if there is none (the entry's own sign decides:
// divided first, -1 .. -(a_row_div - 1) would be row 0).
__device__ __forceinline__ int int4_source(const Int4GemmArgs& p, int r) {
  const int v = p.a_row_map ? p.a_row_map[r] : r;
  const int src = p.a_row_map ? v / p.a_row_div : r;
  return v >= 0 && src < p.a_rows ? src : -1;
}

}  // namespace moe
