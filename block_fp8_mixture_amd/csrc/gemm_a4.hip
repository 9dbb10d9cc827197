// Grouped GEMM with MXFP4 activations and MXFP4 weights.
//
// For every expert e and live row r of its segment
//   C[r, n] = bf16( sum_k a(ar, k) * w(e, n, k) ),  ar the row's source,
// with a and w the values of MXFP4 tensors (E2M1 codes, one E8M0 byte per 32
// consecutive K). gfx950's v_mfma_scale_f32_16x16x128_f8f6f4 takes both
// operands as E2M1 and both scales as bytes, and accumulates in fp32, so the
// product needs no arithmetic outside the matrix cores but the final
// rounding. Operand layout (both operands alike, measured on the chip): lane
// l holds row l % 16 and the 32 K values [32 g, 32 g + 32) of the
// instruction's 128, g = l / 16, in 16 bytes, the even value in the low
// nibble, with that block's byte as its scale; the result's lane l holds
// token l % 16 and weight rows 4 (l / 16) + v.
#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kA4Threads = 256;
constexpr int kA4Waves = kA4Threads / 64;
constexpr int kA4TileM = 64;  // token rows of a wave task, four 16-row tiles
constexpr int kA4Tiles = kA4TileM / 16;
constexpr int kA4TileN = 32;  // weight rows of a wave task, two 16-row tiles

__device__ __forceinline__ int a4_seg_start(const W4Args& p, int e) {
  return p.seg_cap > 0 ? e * p.seg_cap : p.offsets[e];
}
__device__ __forceinline__ int a4_rows(const W4Args& p, int e) {
  const int s0 = a4_seg_start(p, e);
  const int s1 = p.seg_cap > 0 ? s0 + p.seg_cap : p.offsets[e + 1];
  return segment_rows(s0, s1, p.counts[e], p.row_cap);
}

// Exclusive prefix over the experts of ceil(rows / M), into s_pref[0..E]; all
// threads of the workgroup call it.
template <int M>
__device__ void a4_prefix(const W4Args& p, int* s_pref, int* s_wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.num_experts;
  constexpr int kPer = (kMaxExperts + kA4Threads - 1) / kA4Threads;
  int tiles[kPer], run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    const int rows = e < E ? a4_rows(p, e) : 0;
    tiles[i] = (rows + M - 1) / M;
    run += tiles[i];
  }
  int incl = run;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) s_wsum[wave] = incl;
  __syncthreads();
  int base = incl - run;
  for (int w = 0; w < wave; ++w) base += s_wsum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < E) s_pref[e] = base;
    base += tiles[i];
  }
  if (tid == kA4Threads - 1) s_pref[E] = base;
  __syncthreads();
}

// The expert whose units hold unit u (s_pref ascending, s_pref[0] = 0).
__device__ __forceinline__ int a4_expert_of(const int* s_pref, int E, int u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pref[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The K range of a share, in 128-wide steps.
__device__ __forceinline__ int a4_split(int kb, int s, int shares) { return kb * s / shares; }

__device__ __forceinline__ v4f mfma_a4(uint4 w, uint32_t ws, uint4 x, uint32_t xs, v4f acc) {
  const v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z),
                 static_cast<int>(w.w), 0, 0, 0, 0};
  const v8i b = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z),
                 static_cast<int>(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, 0, static_cast<int>(ws), 0,
                                                          static_cast<int>(xs));
}

// A wave task is (expert, 64 token rows, 32 weight rows, a share of K); the
// operands go from global memory straight into the MFMA registers. The S
// waves of a K split add their partial sums in LDS in wave order, so the
// result does not depend on which finishes first.
__global__ __launch_bounds__(kA4Threads, 2) void gemm_a4_kernel(W4Args p) {
  __shared__ int s_pref[kMaxExperts + 1];
  __shared__ int s_wsum[kA4Waves];
  __shared__ __attribute__((aligned(16))) float s_red[kA4Waves][64 * 4 * 2 * kA4Tiles];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int E = p.num_experts, N = p.n, K = p.k, KB = K / kGroup;
  a4_prefix<kA4TileM>(p, s_pref, s_wsum);
  const int nt = N / kA4TileN;
  const int tasks = s_pref[E] * nt;
  if (tasks == 0) return;
  int S = 1;
  while (S < kA4Waves && tasks * S * 2 <= static_cast<int>(gridDim.x) * kA4Waves && S * 2 <= KB) S *= 2;
  const int per_wg = kA4Waves / S;
  const int units = (tasks + per_wg - 1) / per_wg;
  const int share = wave & (S - 1);

  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int t = unit * per_wg + wave / S;
    const bool live = t < tasks;
    v4f acc[2][kA4Tiles] = {};
    int rows_here = 0, row0 = 0, n0 = 0, mt = 0;
    if (live) {
      const int tm = t / nt;
      n0 = (t - tm * nt) * kA4TileN;
      const int e = a4_expert_of(s_pref, E, tm);
      const int m0 = (tm - s_pref[e]) * kA4TileM;
      rows_here = min(kA4TileM, a4_rows(p, e) - m0);
      row0 = a4_seg_start(p, e) + m0;
      mt = (rows_here + 15) >> 4;
      const int64_t wrow = static_cast<int64_t>(e) * N + n0 + r16;
      const uint8_t* wp = p.w + wrow * (K / 2) + 16 * g;
      const uint8_t* wsp = p.w_scales + wrow * (K / kMxBlock);
      // Source rows; a row past the tile's end or without a source reads row
      // 0, and its results are dropped or zeroed.
      const uint8_t* xp[kA4Tiles];
      const uint8_t* xsp[kA4Tiles];
      bool has[kA4Tiles];
#pragma unroll
      for (int m = 0; m < kA4Tiles; ++m) {
        const int j = 16 * m + r16;
        int src = -1;
        if (j < rows_here) {
          const int r = row0 + j;
          src = p.a_row_map ? p.a_row_map[r] / p.a_row_div : r;
          if (static_cast<unsigned>(src) >= static_cast<unsigned>(p.a_rows)) src = -1;
        }
        has[m] = src >= 0;
        const int64_t s0 = src < 0 ? 0 : src;
        xp[m] = p.a + s0 * (K / 2) + 16 * g;
        xsp[m] = static_cast<const uint8_t*>(p.a_scales) + s0 * (K / kMxBlock);
      }
      const int kb1 = a4_split(KB, share + 1, S);
      for (int kb = a4_split(KB, share, S); kb < kb1; ++kb) {
        uint4 w[2];
        uint32_t ws[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = *reinterpret_cast<const uint4*>(wp + static_cast<int64_t>(16 * i) * (K / 2) + kb * 64);
          ws[i] = *reinterpret_cast<const uint32_t*>(wsp + static_cast<int64_t>(16 * i) * (K / kMxBlock) + kb * 4) >> (8 * g);
        }
#pragma unroll
        for (int m = 0; m < kA4Tiles; ++m) {
          if (m < mt) {
            const uint4 x = *reinterpret_cast<const uint4*>(xp[m] + kb * 64);
            const uint32_t xs = *reinterpret_cast<const uint32_t*>(xsp[m] + kb * 4) >> (8 * g);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i][m] = mfma_a4(w[i], ws[i], x, xs, acc[i][m]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kA4Tiles; ++m)
        if (!has[m]) acc[0][m] = acc[1][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (S > 1) {
      v4f* mine = reinterpret_cast<v4f*>(s_red[wave]) + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < kA4Tiles; ++m)
          if (m < mt) mine[64 * (i * kA4Tiles + m)] = acc[i][m];
      __syncthreads();
      if (share == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int m = 0; m < kA4Tiles; ++m)
            if (m < mt)
              for (int w = wave + 1; w < wave + S; ++w)
                acc[i][m] += (reinterpret_cast<v4f*>(s_red[w]) + lane)[64 * (i * kA4Tiles + m)];
      }
      __syncthreads();  // the slots are free for the next unit
    }
    if (live && share == 0) {
#pragma unroll
      for (int m = 0; m < kA4Tiles; ++m) {
        if (16 * m + r16 < rows_here) {
          uint16_t* crow = p.c + static_cast<int64_t>(row0 + 16 * m + r16) * N + n0 + 4 * g;
#pragma unroll
          for (int i = 0; i < 2; ++i) *reinterpret_cast<uint2*>(crow + 16 * i) = pack_bf16x4(acc[i][m]);
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_grouped_gemm_a4(const W4Args& g, hipStream_t stream) {
  hipLaunchKernelGGL(gemm_a4_kernel, dim3(4 * device_cu_count()), dim3(kA4Threads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace moe
