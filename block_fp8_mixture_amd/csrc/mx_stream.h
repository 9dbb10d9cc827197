// Operands of v_mfma_scale_f32_16x16x128_f8f6f4 straight from row-major MXFP4
// tensors in global memory or LDS, for kernels that stream weights.
//
// K order. An operand lane (row l % 16, group g = l / 16) holds 32 consecutive
// K values of an instruction's 128, any 32 as long as both operands agree. Of
// 256 values two instructions j = 0, 1 give lane group g the blocks 2 g + j:
// the first load then touches all of a row's 128-byte line, so the memory is
// asked for whole lines (with blocks g and 4 + g, for two halves of each).
#pragma once

#include "device_common.h"
#include "gemm_device.h"

namespace moe {

// One 128-wide instruction; J: which byte of the scale words.
template <int J>
__device__ __forceinline__ v4f mfma_l4(uint4 w, uint32_t ws, uint4 x, uint32_t xs, v4f acc) {
  const v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z),
                 static_cast<int>(w.w), 0, 0, 0, 0};
  const v8i b = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z),
                 static_cast<int>(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, J, static_cast<int>(ws), J,
                                                          static_cast<int>(xs));
}

// A lane's part of 256 K values of a row: the codes of its blocks 2 g and
// 2 g + 1 and their scale bytes (bytes 0 and 1). Of a row's last 128 values
// (`half`) the lane has block g alone: the second load repeats it, and the
// tokens' second codes are zeros. No branch, so that loads stay together.
struct L4Frag {
  uint4 c[2];
  uint32_t s;
};
struct L4Lane {
  uint32_t c0, c1, s;        // byte offsets of a chunk's two loads and of its scales
  uint32_t shift, scale_mask;
  uint32_t second;           // mask of the second codes
};
__device__ __forceinline__ L4Lane l4_lane(int g, bool half) {
  L4Lane l;
  l.c0 = half ? 16 * g : 32 * g;
  l.c1 = half ? 16 * g : 32 * g + 16;
  l.s = half ? g & 2 : 2 * g;
  l.shift = half ? 8 * (g & 1) : 0;
  l.scale_mask = half ? 0xFFu : 0xFFFFu;
  l.second = half ? 0u : ~0u;
  return l;
}
// `codes` and `scales` are uniform, `row` and `srow` the lane's row in them.
__device__ __forceinline__ void l4_load(L4Frag& f, const uint8_t* codes, uint32_t row, const uint8_t* scales,
                                        uint32_t srow, int chunk, const L4Lane& l) {
  const uint8_t* c = codes + chunk * 128;
  f.c[0] = *reinterpret_cast<const uint4*>(c + (row + l.c0));
  f.c[1] = *reinterpret_cast<const uint4*>(c + (row + l.c1));
  f.s = *reinterpret_cast<const uint16_t*>(scales + chunk * 8 + (srow + l.s));
}
__device__ __forceinline__ uint32_t l4_scales(const L4Frag& f, const L4Lane& l) {
  return (f.s >> l.shift) & l.scale_mask;
}

// Chunks of 256 K values that share `s` of `shares` takes.
__device__ __forceinline__ int l4_split(int chunks, int s, int shares) {
  return static_cast<unsigned>(chunks * s) / static_cast<unsigned>(shares);
}

}  // namespace moe
