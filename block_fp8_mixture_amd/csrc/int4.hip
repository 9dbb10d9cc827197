// 4-bit integer weights with a scale and optionally a zero point per group of
// 32, 64 or 128 columns of a row: quantization and the way back.
//
//   w = s (q - z), q in 0 .. 15; without zero points z = 8.
//   symmetric:   s = T(fl32(amax / 7)),                 q = rne(w / s) + 8
//   zero points: s = T(fl32(fl32(hi - lo) / 15)), z = rne(-lo / s), q = rne(w / s) + z
// with lo = min(least, 0), hi = max(largest, 0), T the scales' type (BF16 or
// FP16), z and q clamped to 0 .. 15, the quotients exact before their rounding
// (round half to even).
//
// A thread holds 8 consecutive columns, G / 8 neighbouring lanes a group.
#include <hip/hip_fp16.h>

#include <type_traits>

#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"
#include "quant_device.h"

namespace moe {
namespace {

constexpr int kI4Threads = 256;

__device__ __forceinline__ float scale16_to_f32(uint32_t bits, int f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(bits))) : bf16_to_f32(bits);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

// A lane's 8 values: their bits as they stand, or two to a word, and as floats.
template <int TYPE>
struct Weights8 {
  static constexpr bool kF32 = TYPE == kElemF32;
  static constexpr int kWords = kF32 ? 8 : 4;
  // Words of one value or a pair of values, unsigned and signed.
  using Word = std::conditional_t<kF32, uint32_t, u16x2>;
  using SignedWord = std::conditional_t<kF32, int32_t, i16x2>;
  uint32_t raw[kWords];

  __device__ __forceinline__ void load(const void* w, int64_t chunk) {
    const u32x4* p = reinterpret_cast<const u32x4*>(w) + chunk * (kWords / 4);
#pragma unroll
    for (int h = 0; h < kWords / 4; ++h) {
      const u32x4 v = p[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[4 * h + i] = v[i];
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (kF32) return __uint_as_float(raw[i]);
    const uint32_t u = raw[i / 2];
    if constexpr (TYPE == kElemBf16) return __uint_as_float(i & 1 ? u & 0xFFFF0000u : u << 16);
    return scale16_to_f32(u >> (16 * (i & 1)) & 0xFFFFu, 1);
  }
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false);
}

// Largest of the group's words as T's components, in every of its lanes: neighbours,
// pairs, then half rows and rows of 16 lanes mirrored.
template <typename T, int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto op = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b)));
  };
  v = op(v, dpp<0xB1>(v));
  v = op(v, dpp<0x4E>(v));
  if constexpr (LANES > 4) v = op(v, dpp<0x141>(v));
  if constexpr (LANES > 8) v = op(v, dpp<0x140>(v));
  return v;
}

// The largest of the group's values, as a float's bits and 0 if all are negative,
// after `flip` turned their signs or MASK took them away. Floats that are not negative
// order as their bits do, infinity and NaN last; negative ones are negative integers.
template <int TYPE, int LANES, typename T, uint32_t MASK>
__device__ __forceinline__ uint32_t group_top(const Weights8<TYPE>& x, uint32_t flip) {
  T m = __builtin_bit_cast(T, (x.raw[0] ^ flip) & MASK);
#pragma unroll
  for (int i = 1; i < Weights8<TYPE>::kWords; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(T, (x.raw[i] ^ flip) & MASK));
  const uint32_t v = group_max<T, LANES>(__builtin_bit_cast(uint32_t, m));
  if constexpr (TYPE == kElemF32) {
    return static_cast<int32_t>(v) < 0 ? 0 : v;
  } else {
    int32_t top = static_cast<int16_t>(v & 0xFFFFu);
    const int32_t other = static_cast<int32_t>(v) >> 16;
    top = top > other ? top : other;
    top = top > 0 ? top : 0;
    return TYPE == kElemBf16 ? static_cast<uint32_t>(top) << 16
                             : __float_as_uint(scale16_to_f32(static_cast<uint32_t>(top), 1));
  }
}

// rne(w / s), |w / s| below 2^20, from inv, 1 / s within a step.
// 16-bit weights: w and s have at most 11 significant bits, so a quotient of at least
// a quarter that is not half way between two integers is 2^-13 or more from there, and
// one refinement gives half ways exactly (the quotient's error before it is r / s, r
// exact; after it below half a step of a value that a float holds): rint is right.
// FP32 weights: n = rint(w inv) is next to it at most, and off only where the remainder
// w - n s, which one FMA gives exactly, says so.
template <bool F32>
__device__ __forceinline__ float rne_quotient(float w, float s, float inv) {
  const float q = w * inv;
  if constexpr (!F32) return rintf(__builtin_fmaf(__builtin_fmaf(-q, s, w), inv, q));
  const float n = rintf(q), rem = __builtin_fmaf(-n, s, w), twice = 2.0f * fabsf(rem);
  const bool odd = static_cast<int>(n) & 1;
  return twice > s || (twice == s && odd) ? n + __builtin_copysignf(1.0f, rem) : n;
}

// fl32(x / D), x not negative, D a small odd integer: x times the rounded reciprocal is
// within a step of the quotient, its remainder is exact where nothing underflows, and
// one more FMA then rounds the quotient correctly (Markstein).
template <int D>
__device__ __forceinline__ float over(float x) {
  if (__any(x < 0x1p-100f)) return x / static_cast<float>(D);
  constexpr float kInv = 1.0f / static_cast<float>(D);
  const float q = x * kInv;
  return __builtin_fmaf(__builtin_fmaf(-q, static_cast<float>(D), x), kInv, q);
}

// Bound by memory: 32768 x 7168 BF16 in groups of 128 without zero points 123 us, in
// groups of 32 with zero points 125 (4.7 TB/s, as a copy), FP32 in groups of 64 223;
// right behind another kernel's writes 154 to 160. Extrema of 16-bit values two to a word
// and rounding without a remainder's test per value: with neither, 165 and 203 us.
template <int TYPE, int G, bool ZEROS>
__global__ __launch_bounds__(kI4Threads) void int4_quant_kernel(const void* __restrict__ w, int64_t chunks,
                                                                int scale_f16, uint32_t* __restrict__ codes,
                                                                uint16_t* __restrict__ scales,
                                                                uint8_t* __restrict__ zeros) {
  constexpr int kLanes = G / 8;
  constexpr bool kF32 = TYPE == kElemF32;
  constexpr uint32_t kSign = kF32 ? 0x80000000u : 0x80008000u;
  using W = Weights8<TYPE>;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kI4Threads;
  auto quantize = [&](const W& x, int64_t c) __attribute__((always_inline)) {
    uint32_t top, lo = 0;
    float span;
    if constexpr (ZEROS) {
      const uint32_t hi = group_top<TYPE, kLanes, typename W::SignedWord, ~0u>(x, 0u);
      lo = group_top<TYPE, kLanes, typename W::SignedWord, ~0u>(x, kSign);
      top = max(lo, hi);
      span = over<15>(__uint_as_float(hi) + __uint_as_float(lo));
    } else {
      top = group_top<TYPE, kLanes, typename W::Word, ~kSign>(x, 0u);
      span = over<7>(__uint_as_float(top));
    }
    uint32_t bits = scale_f16 ? __half_as_ushort(__float2half_rn(span)) : f32_to_bf16(span);
    float s = scale16_to_f32(bits, scale_f16);
    const bool dead = top >= 0x7F800000u || !(s < __uint_as_float(0x7F800000u));
    const bool live = !dead && s > 0.0f;
    if (dead) bits = scale_f16 ? 0x7E00u : 0x7FC0u;  // NaN
    // Scales below 2^-64 and their weights are taken 2^64 times as large, so
    // that the reciprocal is finite.
    const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
    s = live ? s * up : 1.0f;
    const float inv = __builtin_amdgcn_rcpf(s);  // within a step; neither it nor s is subnormal
    float z = 8.0f;
    if constexpr (ZEROS) z = live ? fminf(rne_quotient<kF32>(__uint_as_float(lo) * up, s, inv), 15.0f) : 0.0f;
    // Four codes add up in a float's 16 bits.
    float sum[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = __builtin_amdgcn_fmed3f(rne_quotient<kF32>(x.value(4 * h + i) * up, s, inv) + z, 0.0f, 15.0f);
      sum[h] = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(q[3], 16.0f, q[2]), 16.0f, q[1]), 16.0f, q[0]);
    }
    const uint32_t rest = ZEROS ? 0u : 0x88888888u;
    codes[c] = live ? static_cast<uint32_t>(sum[0]) | static_cast<uint32_t>(sum[1]) << 16 : rest;
    if ((threadIdx.x & (kLanes - 1)) == 0) {
      scales[c / kLanes] = static_cast<uint16_t>(bits);
      if constexpr (ZEROS) zeros[c / kLanes] = static_cast<uint8_t>(z);
    }
  };
  // Whole groups of lanes take each step together: chunks is a multiple of kLanes.
  // Two steps' loads are issued before either is used.
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kI4Threads + threadIdx.x; c < chunks; c += 2 * stride) {
    const bool two = c + stride < chunks;
    W a, b;
    a.load(w, c);
    b.load(w, two ? c + stride : c);
    quantize(a, c);
    if (two) quantize(b, c + stride);
  }
}

// 8 columns per thread and step, so that a wave stores 1 KiB without gaps (with 16
// a thread, two stores of every other 16 bytes, 32768 x 7168 took 163 to 168 us), and
// four steps' loads issued before any is used: 124 to 128 us, 4.7 TB/s. A scale has at most 11 significant
// bits and q - z at most 9: the product is exact in float, and rounded once.
__global__ __launch_bounds__(kI4Threads) void int4_dequant_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint16_t* __restrict__ scales,
                                                                  const uint8_t* __restrict__ zeros,
                                                                  int scale_f16, int group_shift,
                                                                  int64_t chunks, uint4* __restrict__ out) {
  constexpr int kSteps = 4;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kI4Threads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kI4Threads + threadIdx.x; i < chunks; i += kSteps * stride) {
    uint32_t c[kSteps], s[kSteps], z[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int64_t at = i + k * stride < chunks ? i + k * stride : i;
      c[k] = codes[at];
      s[k] = scales[at >> group_shift];
      z[k] = zeros ? zeros[at >> group_shift] : 8u;
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (i + k * stride >= chunks) break;
      const float f = scale16_to_f32(s[k], scale_f16), off = static_cast<float>(z[k]);
      const uint32_t even = c[k] & 0x0F0F0F0Fu, odd = c[k] >> 4 & 0x0F0F0F0Fu;
      v4f lo, hi;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lo[2 * h] = (static_cast<float>(even >> (8 * h) & 0xFFu) - off) * f;
        lo[2 * h + 1] = (static_cast<float>(odd >> (8 * h) & 0xFFu) - off) * f;
        hi[2 * h] = (static_cast<float>(even >> (8 * h + 16) & 0xFFu) - off) * f;
        hi[2 * h + 1] = (static_cast<float>(odd >> (8 * h + 16) & 0xFFu) - off) * f;
      }
      const uint2 a = pack_bf16x4(lo), b = pack_bf16x4(hi);
      out[i + k * stride] = uint4{a.x, a.y, b.x, b.y};
    }
  }
}

// Workgroups of a grid-stride pass over `chunks` threads' worth of work.
dim3 stride_grid(int64_t chunks) {
  const int64_t need = (chunks + kI4Threads - 1) / kI4Threads;
  const int64_t cap = static_cast<int64_t>(device_cu_count()) * 16;
  return dim3(static_cast<unsigned>(need < cap ? need : cap));
}

template <int TYPE, int G>
hipError_t quant_group(const Int4QuantArgs& p, hipStream_t stream) {
  const int64_t chunks = p.rows * (p.cols / 8);
  if (p.zeros)
    hipLaunchKernelGGL((int4_quant_kernel<TYPE, G, true>), stride_grid(chunks), dim3(kI4Threads), 0, stream,
                       p.w, chunks, p.scale_f16, reinterpret_cast<uint32_t*>(p.codes), p.scales, p.zeros);
  else
    hipLaunchKernelGGL((int4_quant_kernel<TYPE, G, false>), stride_grid(chunks), dim3(kI4Threads), 0, stream,
                       p.w, chunks, p.scale_f16, reinterpret_cast<uint32_t*>(p.codes), p.scales, p.zeros);
  return hipGetLastError();
}

template <int TYPE>
hipError_t quant_type(const Int4QuantArgs& p, hipStream_t stream) {
  switch (p.group) {
    case 32: return quant_group<TYPE, 32>(p, stream);
    case 64: return quant_group<TYPE, 64>(p, stream);
    default: return quant_group<TYPE, 128>(p, stream);
  }
}

}  // namespace

hipError_t launch_int4_quant(const Int4QuantArgs& p, hipStream_t stream) {
  switch (p.type) {
    case kElemF32: return quant_type<kElemF32>(p, stream);
    case kElemBf16: return quant_type<kElemBf16>(p, stream);
    default: return quant_type<kElemF16>(p, stream);
  }
}

hipError_t launch_int4_dequant(const uint8_t* codes, const uint16_t* scales, int scale_f16,
                               const uint8_t* zeros, int64_t rows, int cols, int group, uint16_t* out,
                               hipStream_t stream) {
  const int64_t chunks = rows * (cols / 8);
  const int shift = group == 32 ? 2 : group == 64 ? 3 : 4;
  hipLaunchKernelGGL(int4_dequant_kernel, stride_grid(chunks), dim3(kI4Threads), 0, stream,
                     reinterpret_cast<const uint32_t*>(codes), scales, zeros, scale_f16, shift, chunks,
                     reinterpret_cast<uint4*>(out));
  return hipGetLastError();
}

}  // namespace moe
