// RMS norm with the residual's addition and the layer's activation
// quantization: per live token t, with h = bf16(x + residual) (x itself
// without a residual),
//   y = bf16( fl32( h / sqrt(mean(h^2) + eps) * weight ) ),
// the middle in 64 bits, and the codes and scales of y as moe_act_quant makes
// them (but for NaN, which FP8 codes keep here). The norm is of the stored sum and the
// codes are of the stored y, so the fused pass gives what the three passes in a row
// give where y is finite; in 64 bits the order of the row's sum does not reach y's
// rounding.
//
// A workgroup owns a row. A thread holds 8-column vectors in registers, so the
// row is read once; 16 neighbouring lanes hold a 128-column group, as in the
// quantization kernels. Bound by memory: 4096 x 7168 with residual, BF16 output and
// FP8 codes 54 us (4.9 TB/s); one row of 4096 3.5 us, a launch and two trips to memory.
#include <type_traits>

#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"
#include "quant_device.h"

namespace moe {
namespace {

constexpr int kNoFmt = -1;

// Eight floats to BF16 as four packed words (NaN stays NaN).
__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
  const uint2 a = pack_bf16x4(v4f{v[0], v[1], v[2], v[3]});
  const uint2 b = pack_bf16x4(v4f{v[4], v[5], v[6], v[7]});
  return uint4{a.x, a.y, b.x, b.y};
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <int FMT, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void rmsnorm_kernel(NormArgs p) {
  constexpr int kWaves = THREADS / 64;
  __shared__ double s_sum[kWaves];
  const int64_t row = flat_block();
  if (row >= clamp_live(p.t_live_dev, p.t_cap)) return;
  const int tid = threadIdx.x, vecs = p.hidden / 8;
  const uint16_t* x = p.x + row * p.ld;
  const int64_t base = row * p.hidden;

  uint4 h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * THREADS;
    h[i] = v < vecs ? *reinterpret_cast<const uint4*>(x + 8 * v) : uint4{0, 0, 0, 0};
  }
  if (p.residual) {
    uint4 r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * THREADS;
      r[i] = v < vecs ? *reinterpret_cast<const uint4*>(p.residual + base + 8 * v) : uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vals8 a = unpack_bf16x8(h[i]);
      const Vals8 b = unpack_bf16x8(r[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] += b.v[j];
      h[i] = pack_bf16x8(a.v);
      const int v = tid + i * THREADS;
      if (v < vecs) *reinterpret_cast<uint4*>(p.residual_out + base + 8 * v) = h[i];
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Vals8 a = unpack_bf16x8(h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(a.v[j]), static_cast<double>(a.v[j]), sum);
  }
  sum = wave_sum(sum);
  if (kWaves > 1) {
    if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += s_sum[w];
  }
  const double rstd = 1.0 / sqrt(sum / p.hidden + p.eps);

#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * THREADS;
    if (v >= vecs) break;  // whole 16-lane groups: vecs is a multiple of 16
    Vals8 g;
    if (p.weight_f32) {
      const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(p.weight) + 8 * v);
      const float4 a = w[0], b = w[1];
      g = Vals8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    } else {
      g = unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.weight) + 8 * v));
    }
    Vals8 a = unpack_bf16x8(h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a.v[j] = static_cast<float>(static_cast<double>(a.v[j]) * rstd * static_cast<double>(g.v[j]));
    const uint4 y = pack_bf16x8(a.v);
    if (p.y) *reinterpret_cast<uint4*>(p.y + base + 8 * v) = y;
    if constexpr (FMT == kMxfp4) {
      uint32_t byte;
      const uint32_t codes = mx_quantize8_bf16(y, &byte);
      *reinterpret_cast<uint32_t*>(p.xq + (base + 8 * v) / 2) = codes;
      if ((tid & 3) == 0) static_cast<uint8_t*>(p.xs)[(base + 8 * v) / kMxBlock] = static_cast<uint8_t>(byte);
    } else if constexpr (FMT != kNoFmt) {
      float s;
      const uint2 codes = quantize8<FMT, true>(unpack_bf16x8(y), &s, p.rounding);
      *reinterpret_cast<uint2*>(p.xq + base + 8 * v) = codes;
      if ((tid & 15) == 0) store_scale(p.xs, FMT, static_cast<int64_t>(v / 16) * p.t_cap + row, s);
    }
  }
}

template <int FMT, int THREADS, int NV>
hipError_t norm_launch(const NormArgs& p, hipStream_t stream) {
  hipLaunchKernelGGL((rmsnorm_kernel<FMT, THREADS, NV>), flat_grid(p.t_cap), dim3(THREADS), 0, stream, p);
  return hipGetLastError();
}

template <int FMT>
hipError_t norm_fmt(const NormArgs& p, hipStream_t stream) {
  const int vecs = p.hidden / 8;
  if (vecs <= 64) return norm_launch<FMT, 64, 1>(p, stream);
  if (vecs <= 256) return norm_launch<FMT, 256, 1>(p, stream);
  if (vecs <= 512) return norm_launch<FMT, 256, 2>(p, stream);
  if (vecs <= 768) return norm_launch<FMT, 256, 3>(p, stream);
  if (vecs <= 1024) return norm_launch<FMT, 256, 4>(p, stream);
  if (vecs <= 2048) return norm_launch<FMT, 1024, 2>(p, stream);
  return norm_launch<FMT, 1024, 4>(p, stream);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& p, hipStream_t stream) {
  if (!p.xq) return norm_fmt<kNoFmt>(p, stream);
  switch (p.fmt) {
    case kFp32: return norm_fmt<kFp32>(p, stream);
    case kFp32Pow2: return norm_fmt<kFp32Pow2>(p, stream);
    case kMxfp4: return norm_fmt<kMxfp4>(p, stream);
    default: return norm_fmt<kUe8m0>(p, stream);
  }
}

}  // namespace moe
