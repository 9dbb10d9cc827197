// Products of BF16 rows with 4-bit integer weights (scale and zero point per
// group of columns), dense or per expert over its live rows:
//   C[r, n] = bf16( sum_g s[n, g] * sum_{j in g} a[r, j] (q[n, j] - z[n, g]) )
// or, gated, bf16(SiLU(C[r, n]) * C[r, n + N/2]) of the unrounded sums.
//
// v_mfma_f32_16x16x32_bf16 with the rows of A as its first operand (lane l
// holds row l % 16 and the K values 8 (l / 16) .. + 7) and weight rows as its
// second (alike); lane l of the result holds weight row l % 16 and rows of A
// 4 (l / 16) + v, so a lane needs one row's scales.
#include "int4_device.h"

namespace moe {
namespace {

constexpr int kI4Threads = 256;
constexpr int kI4Waves = kI4Threads / 64;

// The expert and the token tile of work unit u: units are the 16 MT-row tiles of
// the experts in order. False if there are fewer.
template <int TM>
__device__ __forceinline__ bool int4_unit(const Int4GemmArgs& p, int u, int* expert, int* row0, int* rows) {
  if (!p.counts) {
    *expert = 0;
    *row0 = u * TM;
    *rows = min(TM, p.row_cap - *row0);
    return *rows > 0;
  }
  // Each wave scans the experts 64 at a time.
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 64) {
    const int e = e0 + lane;
    const int c = e < p.num_experts ? int4_rows(p, e) : 0;
    const int tiles = (c + TM - 1) / TM;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const int all = __shfl(incl, 63, 64);
    if (u < before + all) {
      const uint64_t past = __ballot(before + incl > u);
      const int l = __builtin_ctzll(past);
      const int tile = u - before - (__shfl(incl, l, 64) - __shfl(tiles, l, 64));
      *expert = e0 + l;
      *row0 = tile * TM;
      *rows = min(TM, __shfl(c, l, 64) - *row0);
      return true;
    }
    before += all;
  }
  return false;
}

// R weight tiles of 16 rows (gated: tile 0 gate rows, tile 1 the up rows of the
// same columns), MT row tiles of A; the waves share K.
template <int G, int MT, bool GATED>
__global__ __launch_bounds__(kI4Threads) void int4_stream_kernel(Int4GemmArgs p) {
  constexpr int R = 2;
  __shared__ v4f s_sum[kI4Waves][R][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int out_n = GATED ? p.n / 2 : p.n;
  const int col_tiles = (out_n + (GATED ? 16 : 16 * R) - 1) / (GATED ? 16 : 16 * R);
  const int64_t task = flat_block();
  const int unit = static_cast<int>(task / col_tiles), tile = static_cast<int>(task % col_tiles);
  int expert, row0, rows;
  if (!int4_unit<16 * MT>(p, unit, &expert, &row0, &rows)) return;
  expert = __builtin_amdgcn_readfirstlane(expert);
  row0 = __builtin_amdgcn_readfirstlane(row0) + int4_seg_start(p, expert);
  rows = __builtin_amdgcn_readfirstlane(rows);
  const int K = p.k, groups = K / G;

  // Lanes past the last weight row take the last one's place.
  int wrow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = min((GATED ? tile : tile * R + r) * 16 + col, out_n - 1);
    wrow[r] = GATED && r ? c + out_n : c;
  }
  const uint8_t* w[R];
  const uint16_t* sc[R];
  const uint8_t* zr[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t at = static_cast<int64_t>(expert) * p.n + wrow[r];
    w[r] = p.w + at * (K / 2);
    sc[r] = p.scales + at * groups;
    zr[r] = p.zeros ? p.zeros + at * groups : nullptr;
  }
  const uint16_t* a[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = 16 * m + col;
    const int src = t < rows ? int4_source(p, row0 + t) : -1;
    a[m] = src < 0 ? nullptr : p.a + static_cast<int64_t>(src) * K;
  }

  const v4f zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  v4f total[R][MT], acc[R][MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] = zero4;
#pragma unroll
    for (int r = 0; r < R; ++r) total[r][m] = acc[r][m] = zero4;
  }

  const int blocks = (K + 127) / 128;
  const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (wave + 1) / kI4Waves);
  for (int b = static_cast<int>(static_cast<int64_t>(blocks) * wave / kI4Waves); b < b1; ++b) {
    uint4 c[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c[r] = uint4{0, 0, 0, 0};
      if (128 * b + 32 * g < K) c[r] = *reinterpret_cast<const uint4*>(w[r] + 64 * b + 16 * g);
      // Groups of fewer than 128 columns: word j of every lane within columns 32 j .. + 31.
      if constexpr (G < 128) c[r] = row_transpose(c[r]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = G < 128 ? 128 * b + 32 * j + 8 * g : 128 * b + 32 * g + 8 * j;
      uint4 x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        x[m] = uint4{0, 0, 0, 0};
        if (a[m] && k < K) x[m] = *reinterpret_cast<const uint4*>(a[m] + k);
        x[m] = int4_order(x[m]);
        sum[m] = mfma_bf16(x[m], ones, sum[m]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 q = int4_operand(j == 0 ? c[r].x : j == 1 ? c[r].y : j == 2 ? c[r].z : c[r].w);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = mfma_bf16(x[m], q, acc[r][m]);
      }
      if ((32 * (j + 1)) % G == 0) {
        const int at = min((128 * b + 32 * j) / G, groups - 1);  // past K: sums of zeros
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float s = int4_scale(sc[r][at], p.scale_f16);
          const float off = 16.0f + (zr[r] ? static_cast<float>(zr[r][at]) : 8.0f);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              total[r][m][v] = __builtin_fmaf(s, __builtin_fmaf(-off, sum[m][v], acc[r][m][v]), total[r][m][v]);
            acc[r][m] = zero4;
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[m] = zero4;
      }
    }
  }

#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) s_sum[wave][r][m][lane] = total[r][m];
  __syncthreads();
  // A wave finishes the tiles (r, m) of its number; gated, both of a pair.
  for (int i = wave; i < (GATED ? MT : R * MT); i += kI4Waves) {
    const int m = i % MT, r = i / MT;
    v4f v = s_sum[0][r][m][lane], u = zero4;
#pragma unroll
    for (int k = 1; k < kI4Waves; ++k) v += s_sum[k][r][m][lane];
    if constexpr (GATED) {
      u = s_sum[0][1][m][lane];
#pragma unroll
      for (int k = 1; k < kI4Waves; ++k) u += s_sum[k][1][m][lane];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = int4_gated(p.act, v[k], u[k], p.limit);
    }
    const int n = (GATED ? tile : tile * R + r) * 16 + col;
    const uint2 bits = pack_bf16x4(v);
    if (n < out_n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 16 * m + 4 * g + k;
        const uint32_t b = k < 2 ? bits.x : bits.y;
        if (t < rows)
          p.c[static_cast<int64_t>(row0 + t) * out_n + n] = static_cast<uint16_t>(k & 1 ? b >> 16 : b);
      }
    }
  }
}

template <int G, int MT, bool GATED>
hipError_t stream_launch(const Int4GemmArgs& p, hipStream_t stream) {
  constexpr int TM = 16 * MT;
  const int out_n = GATED ? p.n / 2 : p.n, cols = GATED ? 16 : 32;
  // Every tile but an expert's last is full.
  const int64_t used = p.num_experts < p.row_cap ? p.num_experts : p.row_cap;
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  const int64_t tasks = (out_n + cols - 1) / cols * units;
  hipLaunchKernelGGL((int4_stream_kernel<G, MT, GATED>), flat_grid(tasks), dim3(kI4Threads), 0, stream, p);
  return hipGetLastError();
}

template <int G, bool GATED>
hipError_t stream_rows(const Int4GemmArgs& p, hipStream_t stream) {
  if (p.max_rows_per_expert <= 16) return stream_launch<G, 1, GATED>(p, stream);
  if (p.max_rows_per_expert <= 32) return stream_launch<G, 2, GATED>(p, stream);
  return stream_launch<G, 4, GATED>(p, stream);
}

template <int G>
hipError_t stream_act(const Int4GemmArgs& p, hipStream_t stream) {
  return p.act >= 0 ? stream_rows<G, true>(p, stream) : stream_rows<G, false>(p, stream);
}

}  // namespace

hipError_t launch_gemm_int4(const Int4GemmArgs& p, hipStream_t stream) {
  switch (p.group) {
    case 32: return stream_act<32>(p, stream);
    case 64: return stream_act<64>(p, stream);
    default: return stream_act<128>(p, stream);
  }
}

}  // namespace moe
