// 4-bit integer weights with a scale and optionally a zero point per group of
// 32, 64 or 128 columns of a row: quantization and the way back.
//
//   w = s (q - z), q in 0 .. 15; without zero points z = 8.
//   symmetric:   s = T(fl32(amax / 7)),                 q = rne(w / s) + 8
//   zero points: s = T(fl32(fl32(hi - lo) / 15)), z = rne(-lo / s), q = rne(w / s) + z
// with lo = min(least, 0), hi = max(largest, 0), T the scales' type (BF16 or
// FP16), z and q clamped to 0 .. 15, the quotients exact before their rounding
// (round half to even): a product w * fl32(1 / s) rounded to an integer, then
// put right by the remainder w - n s, which one FMA gives exactly.
//
// A thread holds 8 consecutive columns, G / 8 neighbouring lanes a group.
#include <hip/hip_fp16.h>

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

template <int TYPE>
__device__ __forceinline__ Vals8 load8(const void* w, int64_t chunk) {
  if constexpr (TYPE == kElemF32) {
    const float4* p = reinterpret_cast<const float4*>(w) + 2 * chunk;
    const float4 a = p[0], b = p[1];
    return Vals8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  } else {
    const uint4 raw = reinterpret_cast<const uint4*>(w)[chunk];
    if constexpr (TYPE == kElemBf16) return unpack_bf16x8(raw);
    Vals8 r;
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = scale16_to_f32(u[i / 2] >> (16 * (i & 1)) & 0xFFFFu, 1);
    return r;
  }
}

// rne(w / s) for |w / s| below 2^20 and s normal.
__device__ __forceinline__ float quotient_rne(float w, float s, float inv) {
  float n = rintf(w * inv);
  const float rem = __builtin_fmaf(-n, s, w), twice = 2.0f * fabsf(rem);
  const bool odd = static_cast<int>(n) & 1;
  if (twice > s || (twice == s && odd)) n += __builtin_copysignf(1.0f, rem);
  return n;
}

template <int TYPE, int G, bool ZEROS>
__global__ __launch_bounds__(kI4Threads) void int4_quant_kernel(const void* __restrict__ w, int64_t chunks,
                                                                int scale_f16, uint32_t* __restrict__ codes,
                                                                uint16_t* __restrict__ scales,
                                                                uint8_t* __restrict__ zeros) {
  constexpr int kLanes = G / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kI4Threads;
  // Whole groups of lanes take each step together: chunks is a multiple of kLanes.
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kI4Threads + threadIdx.x; c < chunks; c += stride) {
    const Vals8 x = load8<TYPE>(w, c);
    float lo = 0.0f, hi = 0.0f;
    uint32_t top = 0;  // largest magnitude's bits: a NaN or an infinity shows in them
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x.v[i]);
      hi = fmaxf(hi, x.v[i]);
      const uint32_t b = __float_as_uint(x.v[i]) & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
      if constexpr (ZEROS) {
        lo = fminf(lo, __shfl_xor(lo, d, 64));
        hi = fmaxf(hi, __shfl_xor(hi, d, 64));
      }
      const uint32_t o = __shfl_xor(top, d, 64);
      top = o > top ? o : top;
    }
    const float span = ZEROS ? (hi - lo) / 15.0f : __uint_as_float(top) / 7.0f;
    uint32_t bits = scale_f16 ? __half_as_ushort(__float2half_rn(span)) : f32_to_bf16(span);
    float s = scale16_to_f32(bits, scale_f16);
    const bool dead = top >= 0x7F800000u || !(s < __uint_as_float(0x7F800000u));
    const bool live = !dead && s > 0.0f;
    if (dead) bits = scale_f16 ? 0x7E00u : 0x7FC0u;  // NaN
    // Scales below 2^-64 and their weights are taken 2^64 times as large, so
    // that the reciprocal is finite.
    const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
    s *= up;
    const float inv = 1.0f / (live ? s : 1.0f);
    float z = ZEROS ? 0.0f : 8.0f;
    if (ZEROS && live) z = fminf(quotient_rne(-lo * up, s, inv), 15.0f);
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = live ? quotient_rne(x.v[i] * up, s, inv) : 0.0f;
      const float q = fminf(fmaxf(n + z, 0.0f), 15.0f);
      out |= static_cast<uint32_t>(q) << (4 * i);
    }
    codes[c] = out;
    if ((threadIdx.x & (kLanes - 1)) == 0) {
      scales[c / kLanes] = static_cast<uint16_t>(bits);
      if constexpr (ZEROS) zeros[c / kLanes] = static_cast<uint8_t>(z);
    }
  }
}

// 16 columns per thread: 8 bytes of codes, 32 of output. A scale has at most 11
// significant bits and q - z at most 9: the product is exact in float, and
// rounded once.
__global__ __launch_bounds__(kI4Threads) void int4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint16_t* __restrict__ scales,
                                                                  const uint8_t* __restrict__ zeros,
                                                                  int scale_f16, int group_shift,
                                                                  int64_t chunks, uint16_t* __restrict__ out) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kI4Threads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kI4Threads + threadIdx.x; i < chunks; i += stride) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + 8 * i);
    const int64_t g = i >> group_shift;
    const float s = scale16_to_f32(scales[g], scale_f16);
    const int z = zeros ? zeros[g] : 8;
    uint4 o[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = (j < 2 ? c.x : c.y) >> (16 * (j & 1));
      v4f v;
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = static_cast<float>(static_cast<int>(u >> (4 * h) & 15u) - z) * s;
      const uint2 b = pack_bf16x4(v);
      uint32_t* to = reinterpret_cast<uint32_t*>(o) + 2 * j;
      to[0] = b.x;
      to[1] = b.y;
    }
    reinterpret_cast<uint4*>(out)[2 * i] = o[0];
    reinterpret_cast<uint4*>(out)[2 * i + 1] = o[1];
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
  const int64_t chunks = rows * (cols / 16);
  const int shift = group == 32 ? 1 : group == 64 ? 2 : 3;
  hipLaunchKernelGGL(int4_dequant_kernel, stride_grid(chunks), dim3(kI4Threads), 0, stream, codes, scales,
                     zeros, scale_f16, shift, chunks, out);
  return hipGetLastError();
}

}  // namespace moe
