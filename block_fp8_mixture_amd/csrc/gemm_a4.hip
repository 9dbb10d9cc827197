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
#include <type_traits>

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
constexpr int kA4Small = 64;  // experts with more rows go to the tiled kernel

__device__ __forceinline__ int a4_seg_start(const W4Args& p, int e) {
  return p.seg_cap > 0 ? e * p.seg_cap : p.offsets[e];
}
__device__ __forceinline__ int a4_rows(const W4Args& p, int e) {
  const int s0 = a4_seg_start(p, e);
  const int s1 = p.seg_cap > 0 ? s0 + p.seg_cap : p.offsets[e + 1];
  return segment_rows(s0, s1, p.counts[e], p.row_cap);
}

// Exclusive prefix over the experts of ceil(rows / M), into s_pref[0..E], for
// the experts of more than kA4Small rows or (not LARGE) at most `most`; all
// threads of the workgroup call it.
template <int M, bool LARGE>
__device__ void a4_prefix(const W4Args& p, int* s_pref, int* s_wsum, int most = INT32_MAX) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.num_experts;
  constexpr int kPer = (kMaxExperts + kA4Threads - 1) / kA4Threads;
  int tiles[kPer], run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    const int rows = e < E ? a4_rows(p, e) : 0;
    tiles[i] = (LARGE ? rows > kA4Small : rows <= most) ? (rows + M - 1) / M : 0;
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
template <bool SMALL_ONLY>
__global__ __launch_bounds__(kA4Threads, 2) void gemm_a4_kernel(W4Args p) {
  __shared__ int s_pref[kMaxExperts + 1];
  __shared__ int s_wsum[kA4Waves];
  __shared__ __attribute__((aligned(16))) float s_red[kA4Waves][64 * 4 * 2 * kA4Tiles];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int E = p.num_experts, N = p.n, K = p.k, KB = K / kGroup;
  a4_prefix<kA4TileM, false>(p, s_pref, s_wsum, SMALL_ONLY ? kA4Small : INT32_MAX);
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

// ---- large experts: TM x TN output tiles through LDS -----------------------
//
// Four waves, one per SIMD, as 2 (tokens) x 2 (weights): each owns a TM/2 x
// TN/2 piece, 32 x 32 MFMA tiles whose accumulators stay in registers for the
// whole K (both scales are applied in the matrix cores, so nothing rescales
// them). A stage is 128 K values of the tile's rows, 64 bytes each, fetched by
// direct-to-LDS loads three stages ahead into a ring of four; 16-byte chunk c
// of row r sits at slot c ^ ((r >> 2) & 3), so the 16 lanes one ds_read_b128
// cycle serves (16 rows, the same chunk) hit distinct banks.
//
// Stage s runs as two halves of one 64-wide K step each: half 0 issues the
// loads of stage s + 3 and reads half 1's fragments while its MFMAs run; then
// a wait for this wave's loads of stage s + 1 and the stage's only barrier;
// half 1 reads the next stage's first fragments under its own MFMAs. The
// slot that stage s + 3 goes to held stage s - 1, whose last reads returned
// before the barrier of stage s - 1.
//
// Scales: with K a multiple of 512 (WIDE) a row's 16 bytes of four stages are
// fetched at once into s_sc and held in registers for those stages; otherwise
// each stage brings its rows' 4 bytes.
constexpr int kA4TThreads = 256;

typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ v16f mfma_a4_32(uint4 w, uint4 x, v16f acc, uint32_t ws, uint32_t xs, std::false_type) {
  const v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
  const v8i b = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 0, static_cast<int>(ws), 0, static_cast<int>(xs));
}
__device__ __forceinline__ v16f mfma_a4_32(uint4 w, uint4 x, v16f acc, uint32_t ws, uint32_t xs, std::true_type) {
  const v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
  const v8i b = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 2, static_cast<int>(ws), 2, static_cast<int>(xs));
}

// Direct-to-LDS loads: lane l's bytes land at dst + l * 16 (4).
__device__ __forceinline__ void load_lds16(const uint8_t* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const uint8_t* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 4, 0, 0);
}

template <int TM, int TN, bool WIDE>
__global__ __launch_bounds__(kA4TThreads, 1) void gemm_a4_tiled_kernel(W4Args p) {
  constexpr int MI = TM / 64, NI = TN / 64;   // 32-row MFMA tiles of a wave: tokens, weights
  constexpr int ROWS = TM + TN;               // weight rows first
  constexpr int NL = ROWS / 64;               // code loads per wave and stage
  constexpr int NLW = TN / 64;                //   of them weights
  constexpr int SL = ROWS / 256;              // scale loads per wave (a group of stages, or a stage)
  constexpr int kStage = ROWS * 64;
  static_assert(ROWS % 256 == 0 || ROWS % 128 == 0, "");
  __shared__ __attribute__((aligned(1024))) uint8_t s_st0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s_st1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s_st2[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s_st3[kStage];
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc0[WIDE ? ROWS * 4 : ROWS];
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc1[WIDE ? 1 : ROWS];
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc2[WIDE ? 1 : ROWS];
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc3[WIDE ? 1 : ROWS];
  __shared__ int s_pref[kMaxExperts + 1];
  __shared__ int s_wsum[kA4Waves];
  __shared__ int s_src[TM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, h = lane >> 5;
  const int E = p.num_experts, N = p.n, K = p.k, KB = K / kGroup;
  const int ntn = (N + TN - 1) / TN;
  a4_prefix<TM, true>(p, s_pref, s_wsum);
  const int total = s_pref[E] * ntn;

  for (int t0 = blockIdx.x; t0 < total; t0 += gridDim.x) {
    const int tile = t0;
    // Row tiles of an expert fastest: neighbouring tiles share a weight slab.
    int e, mt, n0;
    {
      int lo = 0, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pref[mid] * ntn <= tile) lo = mid; else hi = mid - 1;
      }
      e = lo;
      const int local = tile - s_pref[e] * ntn;
      const int mtiles = s_pref[e + 1] - s_pref[e];
      n0 = (local / mtiles) * TN;
      mt = local % mtiles;
    }
    const int rows_here = min(TM, a4_rows(p, e) - mt * TM);
    const int row0 = a4_seg_start(p, e) + mt * TM;
    __syncthreads();  // the previous tile is done with s_src and the stages
    for (int i = tid; i < TM; i += kA4TThreads) {
      int src = -1;
      if (i < rows_here) {
        const int r = row0 + i;
        src = p.a_row_map ? p.a_row_map[r] / p.a_row_div : r;
        if (static_cast<unsigned>(src) >= static_cast<unsigned>(p.a_rows)) src = -1;
      }
      s_src[i] = src;
    }
    __syncthreads();

    // Load q of a stage (wave w's i-th: q = 4 i + w) fills rows 16 q .. 16 q +
    // 15; lane l lands in row 16 q + l / 4, slot l % 4. Rows without a source
    // and weight rows past N load a valid row, never used.
    const uint8_t* src[NL];
    const int chunk = (lane & 3) ^ (lane >> 4);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = 16 * (4 * i + wave) + (lane >> 2);
      if (i < NLW) {
        const int n = min(n0 + row, N - 1);
        src[i] = p.w + (static_cast<int64_t>(e) * N + n) * (K / 2) + chunk * 16;
      } else {
        const int a = max(s_src[row - TN], 0);
        src[i] = p.a + static_cast<int64_t>(a) * (K / 2) + chunk * 16;
      }
    }
    // Scale load i of wave w: rows 64 (4 i + w) .. + 63, a row per lane.
    const uint8_t* ssrc[SL];
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int row = 64 * (4 * i + wave) + lane;
      if (row < TN) {
        const int n = min(n0 + row, N - 1);
        ssrc[i] = p.w_scales + (static_cast<int64_t>(e) * N + n) * (K / kMxBlock);
      } else {
        const int a = max(s_src[min(row, ROWS - 1) - TN], 0);
        ssrc[i] = static_cast<const uint8_t*>(p.a_scales) + static_cast<int64_t>(a) * (K / kMxBlock);
      }
    }
    auto issue = [&](int s, uint8_t* st, uint32_t* sc) {
      const int kb = min(s, KB - 1);
#pragma unroll
      for (int i = 0; i < NL; ++i)
        load_lds16(src[i] + kb * 64, st + (4 * i + wave) * 1024);
      if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < SL; ++i)
          load_lds4(ssrc[i] + kb * 4, sc + (4 * i + wave) * 64);
      }
    };
    auto issue_scales = [&](int q) {  // WIDE: the four stages 4q .. 4q + 3
      const int kb = min(4 * q, KB - 4);
#pragma unroll
      for (int i = 0; i < SL; ++i)
        load_lds16(ssrc[i] + kb * 4, s_sc0 + (4 * i + wave) * 256);
    };
    constexpr int PER = NL + (WIDE ? 0 : SL);  // loads per wave and stage

    v16f acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j) acc[i][j] = v16f{};
    uint4 fw[2][NI], fx[2][MI];
    uint4 scw[NI], scx[MI];         // WIDE: the rows' bytes of four stages
    uint32_t cw[NI], cx[MI];        // this stage's, the lane's half in bytes 0 and 2
    const int wrow = wn * (TN / 2) + r32, xrow = TN + wm * (TM / 2) + r32;
    const int swz = (r32 >> 2) & 3;
    auto frags = [&](const uint8_t* st, auto kk_t) {
      constexpr int kk = decltype(kk_t)::value;
      const int off = ((2 * kk + h) ^ swz) << 4;
#pragma unroll
      for (int i = 0; i < NI; ++i) fw[kk][i] = *reinterpret_cast<const uint4*>(st + (wrow + 32 * i) * 64 + off);
#pragma unroll
      for (int j = 0; j < MI; ++j) fx[kk][j] = *reinterpret_cast<const uint4*>(st + (xrow + 32 * j) * 64 + off);
    };
    auto read_group_scales = [&]() {
#pragma unroll
      for (int i = 0; i < NI; ++i) scw[i] = *reinterpret_cast<const uint4*>(s_sc0 + (wrow + 32 * i) * 4);
#pragma unroll
      for (int j = 0; j < MI; ++j) scx[j] = *reinterpret_cast<const uint4*>(s_sc0 + (xrow + 32 * j) * 4);
    };
    auto stage_scales = [&](const uint32_t* sc, auto u_t) {
      constexpr int u = decltype(u_t)::value;
      auto pick = [](uint4 v) { return u == 0 ? v.x : (u == 1 ? v.y : (u == 2 ? v.z : v.w)); };
#pragma unroll
      for (int i = 0; i < NI; ++i) cw[i] = (WIDE ? pick(scw[i]) : sc[wrow + 32 * i]) >> (8 * h);
#pragma unroll
      for (int j = 0; j < MI; ++j) cx[j] = (WIDE ? pick(scx[j]) : sc[xrow + 32 * j]) >> (8 * h);
    };
    auto products = [&](auto kk_t) {
      constexpr int kk = decltype(kk_t)::value;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
          acc[i][j] = mfma_a4_32(fw[kk][i], fx[kk][j], acc[i][j], cw[i], cx[j], std::bool_constant<kk == 1>{});
    };
    const std::integral_constant<int, 0> k0;
    const std::integral_constant<int, 1> k1;
    // Past the last stage (K no multiple of 512) the tokens' codes are zeros.
    auto mask_tokens = [&](int s, auto kk_t) {
      if constexpr (!WIDE) {
        const uint32_t m = s < KB ? ~0u : 0u;
#pragma unroll
        for (int j = 0; j < MI; ++j) {
          uint4& x = fx[decltype(kk_t)::value][j];
          x = uint4{x.x & m, x.y & m, x.z & m, x.w & m};
        }
      }
    };
    // One stage: u = s % 4; cur and next its and the next stage's buffers,
    // fill the one stage s + 3 goes to. Within a half the reads of the next
    // one (and the direct-to-LDS loads) are spread between its MFMAs.
    auto stage = [&](int s, auto u_t, const uint8_t* cur, const uint8_t* next, uint8_t* fill,
                     const uint32_t* sc_next, uint32_t* sc_fill) {
      constexpr int u = decltype(u_t)::value;
      constexpr int M = MI * NI;
      issue(s + 3, fill, sc_fill);
      if constexpr (WIDE && u == 1) issue_scales(s / 4 + 1);
      frags(cur, k1);
      products(k0);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // MFMA
        if (i < MI + NI) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        if (i >= M - NL) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load
      }
      __builtin_amdgcn_sched_barrier(0);
      // The loads issued after those of stage s + 1: stages s + 2 and s + 3,
      // and the group's scales if issued with either.
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * PER + (WIDE && (u == 1 || u == 2) ? SL : 0)));
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      mask_tokens(s, k1);
      if constexpr (WIDE && u == 3) read_group_scales();
      frags(next, k0);
      products(k1);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < (WIDE && u == 3 ? 2 : 1) * (MI + NI)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      stage_scales(sc_next, std::integral_constant<int, (u + 1) & 3>{});
      mask_tokens(s + 1, k0);
    };
    if constexpr (WIDE) issue_scales(0);
    issue(0, s_st0, s_sc0);
    issue(1, s_st1, s_sc1);
    issue(2, s_st2, s_sc2);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * PER));
    lds_barrier();
    if constexpr (WIDE) read_group_scales();
    frags(s_st0, k0);
    stage_scales(s_sc0, k0);
    const std::integral_constant<int, 2> k2;
    const std::integral_constant<int, 3> k3;
    for (int s = 0; s < KB; s += 4) {
      stage(s, k0, s_st0, s_st1, s_st3, s_sc1, s_sc3);
      stage(s + 1, k1, s_st1, s_st2, s_st0, s_sc2, s_sc0);
      stage(s + 2, k2, s_st2, s_st3, s_st1, s_sc3, s_sc1);
      stage(s + 3, k3, s_st3, s_st0, s_st2, s_sc0, s_sc2);
    }
    __builtin_amdgcn_s_waitcnt(0);  // trailing loads have landed before a stage is reused
    __syncthreads();

    // Output: each wave turns its piece through a stage buffer of its own
    // (rows of TN/2 BF16, 16-byte chunk c of token row r at slot c ^ (r % 16))
    // and stores whole rows of the piece.
    {
      uint8_t* buf = wave == 0 ? s_st0 : (wave == 1 ? s_st1 : (wave == 2 ? s_st2 : s_st3));
      constexpr int kRowB = TN;  // TN/2 values x 2 bytes
      constexpr int kChunks = kRowB / 16;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j) {
          const int r = 32 * j + r32;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const v4f q = {acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
            const int c = 4 * i + v;
            *reinterpret_cast<uint2*>(buf + r * kRowB + ((c ^ (r & (kChunks - 1))) << 4) + 8 * h) = pack_bf16x4(q);
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      constexpr int kLanesRow = kChunks, kRowsPass = 64 / kLanesRow;
      const int c = lane % kLanesRow;
      const int n = n0 + wn * (TN / 2) + 8 * c;
#pragma unroll 4
      for (int q = 0; q < TM / 2 / kRowsPass; ++q) {
        const int r = q * kRowsPass + lane / kLanesRow;
        const int row = wm * (TM / 2) + r;
        uint4 v = *reinterpret_cast<const uint4*>(buf + r * kRowB + ((c ^ (r & (kChunks - 1))) << 4));
        if (row < rows_here && n < N) {
          if (s_src[row] < 0) v = uint4{0, 0, 0, 0};
          *reinterpret_cast<uint4*>(p.c + static_cast<int64_t>(row0 + row) * N + n) = v;
        }
      }
    }
  }
}

template <int TM, int TN>
hipError_t launch_a4_tiled(const W4Args& g, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(device_cu_count()));
  if (g.k % 512 == 0)
    hipLaunchKernelGGL((gemm_a4_tiled_kernel<TM, TN, true>), grid, dim3(kA4TThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((gemm_a4_tiled_kernel<TM, TN, false>), grid, dim3(kA4TThreads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm_a4(const W4Args& g, hipStream_t stream) {
  const bool large = g.max_rows_per_expert > kA4Small;
  const dim3 grid(static_cast<unsigned>(4 * device_cu_count()));
  if (!large) {
    hipLaunchKernelGGL(gemm_a4_kernel<false>, grid, dim3(kA4Threads), 0, stream, g);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(gemm_a4_kernel<true>, grid, dim3(kA4Threads), 0, stream, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_a4_tiled<256, 256>(g, stream);
}

}  // namespace moe
