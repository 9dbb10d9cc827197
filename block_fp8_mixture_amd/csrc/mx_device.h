// Device helpers of MXFP4 (OCP Microscaling v1.0: E2M1 elements sharing one
// E8M0 scale per 32 consecutive columns) for the quantizers and the kernels
// that take 4-bit activations.
//
// Quantization of a block with largest magnitude amax (the conversion of the
// format's specification): the scale is the power of two floor(log2(amax)) -
// 2, the 2 being the exponent of E2M1's largest power of two, so amax / scale
// lies in [4, 8) and magnitudes past 6 saturate. On the float's bits: with e
// the biased exponent of amax, the byte is max(e - 2, 0). Blocks below
// 2^-124 (subnormal amax among them) share byte 0 = 2^-127, and an all-zero
// block has it too. A block that holds an infinity or a NaN (e = 255) gets
// byte 255, the format's NaN, and zero codes: E2M1 has neither, and the byte
// makes every value of the block NaN wherever it is read. Elements round to
// nearest, ties to the even code (v_cvt_scalef32_pk_fp4_*, checked against
// the grid for scale bytes 0..254, also at the ties): with one mantissa bit a
// value in [1, 6] times the scale is off by a fifth of itself at most (2.5
// becomes 2, 5 becomes 4), a saturated one by less than a quarter.
#pragma once

#include "device_common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// A block's scale byte from the float bits of its amax.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(byte - 127) as a float; byte 255 has none (its codes are zeroed).
__device__ __forceinline__ float mx_scale_float(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Larger of two magnitudes' bits, per 16-bit half (BF16 magnitudes order as
// their bits, and NaN above infinity, so no NaN is lost in a maximum).
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t bf16x2_abs(uint32_t w) { return w & 0x7FFF7FFFu; }
// The larger half of packed BF16 magnitudes, as float bits.
__device__ __forceinline__ uint32_t bf16x2_amax_bits(uint32_t m) {
  const uint32_t lo = m << 16, hi = m & 0xFFFF0000u;
  return lo > hi ? lo : hi;
}

// Eight codes (4 bytes, the first value in the lowest nibble) of four packed
// BF16 pairs, or of eight floats, under scale s.
__device__ __forceinline__ uint32_t mx_codes_bf16(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float s) {
  uint32_t v = 0;
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16x2_t, a), s, 0);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16x2_t, b), s, 1);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16x2_t, c), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16x2_t, d), s, 3);
}
__device__ __forceinline__ uint32_t mx_codes_f32(const float* x, float s) {
  uint32_t v = 0;
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[0], x[1], s, 0);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[2], x[3], s, 1);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[4], x[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, x[6], x[7], s, 3);
}

// Larger of the values of the four lanes of an aligned quad, in each of them.
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, false);  // [1,0,3,2]
  v = o > v ? o : v;
  o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, false);  // [2,3,0,1]
  return o > v ? o : v;
}

// Quantizes a block whose 32 values four neighbouring lanes hold, 8 each;
// every lane gets its 8 codes and the block's byte. BF16 values as loaded:
__device__ __forceinline__ uint32_t mx_quantize8_bf16(uint4 raw, uint32_t* byte) {
  const uint32_t m = pk_max_u16(pk_max_u16(bf16x2_abs(raw.x), bf16x2_abs(raw.y)),
                                pk_max_u16(bf16x2_abs(raw.z), bf16x2_abs(raw.w)));
  const uint32_t b = mx_scale_byte(quad_max_u32(bf16x2_amax_bits(m)));
  *byte = b;
  const uint32_t codes = mx_codes_bf16(raw.x, raw.y, raw.z, raw.w, mx_scale_float(b));
  return b == 255u ? 0u : codes;
}
// Floats:
__device__ __forceinline__ uint32_t mx_quantize8_f32(const float* x, uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  const uint32_t b = mx_scale_byte(quad_max_u32(m));
  *byte = b;
  const uint32_t codes = mx_codes_f32(x, mx_scale_float(b));
  return b == 255u ? 0u : codes;
}

}  // namespace moe
