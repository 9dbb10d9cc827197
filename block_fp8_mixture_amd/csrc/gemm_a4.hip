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
#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"
#include "mx_stream.h"

namespace moe {
namespace {

constexpr int kA4Threads = 256;
constexpr int kA4Waves = kA4Threads / 64;
constexpr int kA4TileM = 32;  // token rows of a wave task, two 16-row tiles
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

// Row of A behind row r, -1 if there is none. The entry's own sign decides:
// divided first, -1 .. -(a_row_div - 1) would be row 0.
__device__ __forceinline__ int a4_source(const W4Args& p, int r) {
  const int v = p.a_row_map ? p.a_row_map[r] : r;
  const int src = p.a_row_map ? v / p.a_row_div : r;
  return v >= 0 && src < p.a_rows ? src : -1;
}

// Exclusive prefix over the experts of units(e), into s_pref[0..E]; all
// threads of the workgroup call it.
template <typename Units>
__device__ void a4_prefix(int E, Units units, int* s_pref, int* s_wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kPer = (kMaxExperts + kA4Threads - 1) / kA4Threads;
  int tiles[kPer], run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    tiles[i] = e < E ? units(e) : 0;
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

// ---- few rows per expert: weights streamed into the matrix cores -----------

// A wave's operands: two 16-row tiles of weights and up to kA4Tiles of tokens.
struct A4Rows {
  const uint8_t* w[2];    // uniform: a tile's first row, its scales
  const uint8_t* ws[2];
  uint32_t wrow, wsrow;   // the lane's row in them
  uint32_t xrow[kA4Tiles], xsrow[kA4Tiles];  // and in A
};

// acc += the chunks [ch0, ch1) of 256 K values, MT token tiles. The operands
// of two chunks are loaded together; other waves' loads cover their products.
template <int MT>
__device__ __forceinline__ void a4_stream(const W4Args& p, A4Rows t, int g, int ch0, int ch1,
                                          v4f (&acc)[2][kA4Tiles]) {
  const int K = p.k;
  L4Frag w[2][2], x[2][MT];
  auto load = [&](int ch, int b) {
    const int c = min(ch, ch1 - 1);  // past the share: its last chunk, unused
    const L4Lane l = l4_lane(g, c * 256 + 128 >= K);
    // Opaque, so that the addresses stay a uniform base and a 32-bit offset (as
    // pointers of their own that step along K they take 60 registers more).
    asm volatile("" : "+v"(t.wrow), "+v"(t.wsrow));
#pragma unroll
    for (int m = 0; m < MT; ++m) asm volatile("" : "+v"(t.xrow[m]), "+v"(t.xsrow[m]));
#pragma unroll
    for (int m = 0; m < MT; ++m)
      l4_load(x[b][m], p.a, t.xrow[m], static_cast<const uint8_t*>(p.a_scales), t.xsrow[m], c, l);
#pragma unroll
    for (int i = 0; i < 2; ++i) l4_load(w[b][i], t.w[i], t.wrow, t.ws[i], t.wsrow, c, l);
  };
  auto products = [&](int ch, int b) {
    const L4Lane l = l4_lane(g, ch * 256 + 128 >= K);
    const uint32_t z = l.second;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t xs = l4_scales(x[b][m], l);
      const uint4 c1 = x[b][m].c[1];
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][m] = mfma_l4<0>(w[b][i].c[0], l4_scales(w[b][i], l), x[b][m].c[0], xs, acc[i][m]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[i][m] = mfma_l4<1>(w[b][i].c[1], l4_scales(w[b][i], l), uint4{c1.x & z, c1.y & z, c1.z & z, c1.w & z}, xs, acc[i][m]);
    }
  };
  for (int ch = ch0; ch < ch1; ch += 2) {
    load(ch, 0);
    load(ch + 1, 1);
    products(ch, 0);
    if (ch + 1 < ch1) products(ch + 1, 1);
  }
}

// A wave task is (expert, 32 token rows, 32 weight rows, a share of K); the
// operands go from global memory straight into the MFMA registers. The S
// waves of a K split add their partial sums in LDS in wave order, so the
// result does not depend on which finishes first. Bound by the weights: 8
// experts of 4 rows, N 4096, K 7168 (125 MB) 37.8 us from HBM (3.3 TB/s), 28
// to 29 where the last-level cache holds them from the call before (4.4 TB/s).
// There many waves with few registers (75) beat a pipeline of two chunks within
// a wave (182 registers, 32.4 us), and whole lines in K order half lines (36.1).
__global__ __launch_bounds__(kA4Threads, 2) void gemm_a4_kernel(W4Args p) {
  __shared__ int s_pref[kMaxExperts + 1];
  __shared__ int s_wsum[kA4Waves];
  __shared__ __attribute__((aligned(16))) float s_red[kA4Waves][64 * 4 * 2 * kA4Tiles];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int E = p.num_experts, N = p.n, K = p.k, chunks = (K + 255) / 256;
  a4_prefix(E, [&](int e) { return (a4_rows(p, e) + kA4TileM - 1) / kA4TileM; }, s_pref, s_wsum);
  const int nt = N / kA4TileN;
  const int tasks = __builtin_amdgcn_readfirstlane(s_pref[E]) * nt;
  if (tasks == 0) return;
  int S = 1;
  while (S < kA4Waves && tasks * S * 2 <= static_cast<int>(gridDim.x) * kA4Waves && S * 2 <= chunks) S *= 2;
  const int per_wg = kA4Waves / S;
  const int units = (tasks + per_wg - 1) / per_wg;
  const int share = wave & (S - 1);

  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int task = unit * per_wg + wave / S;
    const bool live = task < tasks;
    v4f acc[2][kA4Tiles] = {};
    int rows_here = 0, row0 = 0, n0 = 0, mt = 0;
    if (live) {
      // Row tiles of an expert run fastest: they share the weights.
      const int e = __builtin_amdgcn_readfirstlane(a4_expert_of(s_pref, E, task / nt));
      const int local = task - s_pref[e] * nt, mtiles = s_pref[e + 1] - s_pref[e];
      const int m0 = local % mtiles * kA4TileM;
      n0 = __builtin_amdgcn_readfirstlane(local / mtiles * kA4TileN);
      rows_here = __builtin_amdgcn_readfirstlane(min(kA4TileM, a4_rows(p, e) - m0));
      row0 = __builtin_amdgcn_readfirstlane(a4_seg_start(p, e) + m0);
      mt = (rows_here + 15) >> 4;
      const uint32_t pitch = K / 2, spitch = K / kMxBlock;
      A4Rows t;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = static_cast<int64_t>(e) * N + n0 + 16 * i;
        t.w[i] = p.w + row * pitch;
        t.ws[i] = p.w_scales + row * spitch;
      }
      t.wrow = r16 * pitch;
      t.wsrow = r16 * spitch;
      // Source rows; a row past the tile's end or without a source reads row
      // 0, and its results are dropped or zeroed.
      bool has[kA4Tiles];
#pragma unroll
      for (int m = 0; m < kA4Tiles; ++m) {
        const int j = 16 * m + r16;
        const int src = j < rows_here ? a4_source(p, row0 + j) : -1;
        has[m] = src >= 0;
        t.xrow[m] = static_cast<uint32_t>(max(src, 0)) * pitch;
        t.xsrow[m] = static_cast<uint32_t>(max(src, 0)) * spitch;
      }
      const int ch0 = __builtin_amdgcn_readfirstlane(chunks * share / S);
      const int ch1 = __builtin_amdgcn_readfirstlane(chunks * (share + 1) / S);
      if (mt == 1) a4_stream<1>(p, t, g, ch0, ch1, acc);
      else a4_stream<2>(p, t, g, ch0, ch1, acc);
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

// ---- more rows: TM x TN output tiles through LDS -----------------------
//
// Four waves, one per SIMD, as 2 (tokens) x 2 (weights): each owns every other
// 32 of the TM rows and half of the TN columns, 32 x 32 MFMA tiles whose
// accumulators stay in registers for the whole K (both scales are applied in the matrix cores, so nothing rescales
// them).
//
// A stage is 256 K values of the tile's rows: 128 bytes of each, one whole
// cache line per request (with half lines the same bytes took 1.2 times as
// long: the L2 answers requests, not bytes). Direct-to-LDS loads bring it into
// one of two buffers per operand; 16-byte chunk c of row r sits at slot c ^
// ((r >> 1) & 7), so the 16 lanes one ds_read_b128 cycle serves (16 rows, the
// same chunk) hit distinct banks. A stage runs as four quarters q of one
// 64-wide K step each, NI x MI MFMAs, under which the next fragments are read:
//   q = 0: the stage's remaining token fragments (held in registers from here
//          on) and the weights' of q = 1; barrier: the token buffer is free
//   q = 1: loads of the tokens of stage s + 2
//   q = 2: wait for this wave's loads of stage s + 1; barrier: they are there,
//          and the weight buffer is free
//   q = 3: the first fragments of stage s + 1; loads of the weights of s + 2
// (and in each the weights' fragments of the next quarter).
//
// The grid is persistent and the stream of stages goes on across tiles: the
// last two stages of a tile issue the next tile's first two, which land while
// its output is stored. Row sources of a tile are looked up two tiles ahead,
// during the output. A tile's stages are rounded up to an even number; K values past
// the end multiply zero codes.
//
// Scales: with K a multiple of 1024 (G = 4) a row's bytes of four stages are
// fetched at once, as two 16-byte loads of one line, with K a multiple of 512
// (G = 2) those of two stages, and held in registers two stages at a time;
// otherwise (G = 1) each stage brings its rows' bytes by two 4-byte loads.
//
// A tile of at most 64 rows (an expert's last, as a rule) takes stages that load
// those rows and multiply the first MFMA tile of each wave alone: 0.4 of a
// whole tile's time (32768 rows over 32 experts, K 7168, N 4096: 543 -> 529 us).
//
// Tiles of 64 rows take 128 columns, half the LDS, and two workgroups per CU:
// twice the stages in flight, and twice the tiles for the CUs where experts are
// few (64 x 256 tiles, one workgroup per CU, against them, the same inputs each time: 32
// experts of 16 rows, K 7168, N 4096 100 / 91 us, 256 experts of 2 rows, K 6144, N 512 89 / 79).
//
// Row tiles of an expert run fastest, so that neighbours share a weight slab.
constexpr int kA4TThreads = 256;
constexpr int kA4TileCols = 256;

typedef float v16f __attribute__((ext_vector_type(16)));

// One 64-wide K step: the first of its 128-wide block takes byte 0 of the
// scale words, the second byte 2.
template <bool SECOND>
__device__ __forceinline__ v16f mfma_a4_32(uint4 w, uint4 x, v16f acc, uint32_t ws, uint32_t xs) {
  const v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
  const v8i b = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
  if constexpr (SECOND)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 2, static_cast<int>(ws), 2, static_cast<int>(xs));
  else
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 0, static_cast<int>(ws), 0, static_cast<int>(xs));
}

// Direct-to-LDS loads: lane l's bytes land at dst + l * 16 (4).
__device__ __forceinline__ void load_lds16(const uint8_t* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const uint8_t* src, void* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 4, 0, 0);
}

constexpr int lp_or_one(int v) { return v > 0 ? v : 1; }

struct A4Tile {
  int e, n0, row0, rows;  // rows = 0: no tile
};

template <int TM, int TN, int G>
__global__ __launch_bounds__(kA4TThreads, 1) void gemm_a4_tiled_kernel(W4Args p) {
  constexpr int MI = TM / 64, NI = TN / 64;   // 32-row MFMA tiles of a wave: tokens, weights
  constexpr bool WIDE = G > 1;
  constexpr int U = G == 4 ? 4 : 2;           // stages per loop iteration
  constexpr int WL = TN / 32, XL = TM / 32;   // code loads per wave and stage
  constexpr int kScRows = 512;                // rows of scales: 256 for weights, 256 for tokens (all lanes load)
  static_assert(TN <= 256 && TM <= 256, "");
  static_assert(TM <= kA4TThreads, "one row source per thread");
  __shared__ __attribute__((aligned(1024))) uint8_t s_w0[TN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t s_w1[TN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t s_x0[TM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t s_x1[TM * 128];
  // The rows' 16 bytes of two stages (G = 4: and of the next two); G = 1: 4 and
  // 4 bytes of a stage, per buffer.
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc0[kScRows * (WIDE ? 2 * G : 2)];
  __shared__ __attribute__((aligned(1024))) uint32_t s_sc1[WIDE ? 1 : kScRows * 2];
  __shared__ int s_pref[kMaxExperts + 1];  // exclusive prefix of the row tiles over the experts
  __shared__ int s_row0[kMaxExperts];      // an expert's first row
  __shared__ int s_rows[kMaxExperts];      //   and its rows
  __shared__ int s_wsum[kA4Waves];
  __shared__ int s_src[3][TM];             // source rows of tile i at [i % 3]

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, h = lane >> 5;
  const int E = p.num_experts, N = p.n, K = p.k;
  const int P = (K + 255) / 256;  // stages with data
  const int P2 = (P + 1) & ~1;
  const int ntn = (N + TN - 1) / TN;
  for (int e = tid; e < E; e += kA4TThreads) {
    s_rows[e] = a4_rows(p, e);
    s_row0[e] = a4_seg_start(p, e);
  }
  __syncthreads();
  a4_prefix(E, [&](int e) { return (s_rows[e] + TM - 1) / TM; }, s_pref, s_wsum);
  const int total = s_pref[E] * ntn;

  auto locate = [&](int tile) {
    A4Tile t{0, 0, 0, 0};
    if (tile >= total) return t;
    int lo = 0, hi = E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] * ntn <= tile) lo = mid; else hi = mid - 1;
    }
    const int local = tile - s_pref[lo] * ntn, mtiles = s_pref[lo + 1] - s_pref[lo];
    const int m0 = (local % mtiles) * TM;
    t.e = __builtin_amdgcn_readfirstlane(lo);
    t.n0 = __builtin_amdgcn_readfirstlane((local / mtiles) * TN);
    t.row0 = __builtin_amdgcn_readfirstlane(s_row0[lo] + m0);
    t.rows = __builtin_amdgcn_readfirstlane(min(TM, s_rows[lo] - m0));
    return t;
  };
  // Source row of row `tid` of a tile, -1 if it has none.
  auto row_source = [&](const A4Tile& t) {
    return tid < t.rows ? a4_source(p, t.row0 + tid) : -1;
  };

  // Workgroups go round-robin over the 8 XCDs: neighbouring tiles, which share
  // operand rows, go to workgroups of one XCD and so to one L2. Within the XCD
  // they move on by one workgroup per round, so that a workgroup does not meet
  // the same (full or short) row tile of every expert.
  const unsigned grid = gridDim.x, xcds = grid % 8 == 0 ? 8 : 1, per_xcd = grid / xcds;
  auto tile_of = [&](unsigned round) {
    return static_cast<int>(round * grid + (blockIdx.x % xcds) * per_xcd + (blockIdx.x / xcds + round) % per_xcd);
  };
  unsigned round = 0;
  if (tile_of(0) >= total) return;
  A4Tile cur = locate(tile_of(0)), nxt = locate(tile_of(1));
  if (tid < TM) {
    s_src[0][tid] = row_source(cur);
    s_src[1][tid] = row_source(nxt);
  }
  __syncthreads();

  // Load q of an operand's stage (wave w's i-th: q = 4 i + w) fills rows 8 q
  // .. 8 q + 7; lane l lands in row 8 q + l / 8, slot l % 8. Scale load i of
  // wave w fills rows 64 (4 i + w) .. + 63, a row per lane. Rows without a
  // source and weight rows past N load a valid row, never used. Addresses are
  // a uniform base and a 32-bit offset per lane (an operand's bytes, or one
  // expert's, are below 2^32).
  const uint32_t pitch = K / 2, spitch = K / kMxBlock;
  const int chunk = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  const uint32_t wlane = (8 * wave + (lane >> 3)) * pitch + chunk * 16;
  // Sources of the current tile [0] and the next [1]; the loads choose by
  // uniform selects (a branch would let MFMAs be moved past it, out of their
  // quarter). After a workgroup's last tile they load rows that exist, unused.
  struct Sources {
    const uint8_t* w;   // the first weight row
    const uint8_t* ws;  //   and its scale bytes
    int blocks;         // 32-row blocks of weights below N
    uint32_t wsoff, xsoff;
    uint32_t xoff[XL];
  } src[2];
  auto set_sources = [&](Sources& o, const A4Tile& t, const int* rows) {
    const int64_t row = static_cast<int64_t>(t.e) * N + t.n0;
    o.w = p.w + row * pitch;
    o.ws = p.w_scales + row * spitch;
    o.blocks = min(TN, N - t.n0) / 32;
    o.wsoff = static_cast<uint32_t>(min(64 * wave + lane, min(TN, N - t.n0) - 1)) * spitch;
    o.xsoff = static_cast<uint32_t>(max(rows[min(64 * wave + lane, TM - 1)], 0)) * spitch;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      o.xoff[i] = static_cast<uint32_t>(max(rows[8 * (4 * i + wave) + (lane >> 3)], 0)) * pitch + chunk * 16;
  };
  // Byte offset of stage s of the current tile, or for s >= P2 of stage s - P2
  // of the next. With K an odd multiple of 128 the last stage's second half
  // lies past the row: its lanes load the first half again.
  auto stage_index = [&](int s) { return min(s < P2 ? s : s - P2, P - 1); };
  auto past_end = [&](int kb) -> uint32_t {
    if constexpr (WIDE) return 0u;
    return kb * 256 + 128 >= K && chunk >= 4 ? 64u : 0u;
  };
  auto issue_tokens = [&](int s, uint8_t* buf, auto n_t) {  // the tile's first 32 n_t rows
    const int kb = stage_index(s);
    const bool n = s >= P2;
    const uint8_t* base = p.a + kb * 128;
    const uint32_t back = past_end(kb);
#pragma unroll
    for (int i = 0; i < decltype(n_t)::value; ++i)
      load_lds16(base + ((n ? src[1].xoff[i] : src[0].xoff[i]) - back), buf + (4 * i + wave) * 1024);
  };
  auto issue_weights = [&](int s, uint8_t* buf) {
    const int kb = stage_index(s);
    const bool n = s >= P2;
    const uint8_t* base = (n ? src[1].w : src[0].w) + kb * 128;
    const int blocks = n ? src[1].blocks : src[0].blocks;
    const uint32_t back = past_end(kb);
#pragma unroll
    for (int i = 0; i < WL; ++i)
      load_lds16(base + static_cast<int64_t>(i < blocks ? i : 0) * 32 * pitch + (wlane - back), buf + (4 * i + wave) * 1024);
  };
  // The scales of stage s (G = 1), s and s + 1 (G = 2), s .. s + 3 (G = 4).
  auto issue_scales = [&](int s, uint32_t* sc) {
    const int kb = stage_index(s);
    const bool n = s >= P2;
    const uint8_t* wb = n ? src[1].ws : src[0].ws;
    const uint8_t* xb = static_cast<const uint8_t*>(p.a_scales);
    const uint32_t wo = n ? src[1].wsoff : src[0].wsoff, xo = n ? src[1].xsoff : src[0].xsoff;
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < G / 2; ++i) {
        load_lds16(wb + (kb * 8 + 16 * i) + wo, sc + kScRows * 4 * i + wave * 256);
        load_lds16(xb + (kb * 8 + 16 * i) + xo, sc + kScRows * 4 * i + 1024 + wave * 256);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = min(2 * kb + i, K / kGroup - 1) * 4;
        load_lds4(wb + b + wo, sc + kScRows * i + wave * 64);
        load_lds4(xb + b + xo, sc + kScRows * i + 256 + wave * 64);
      }
    }
  };
  constexpr int SCL = WIDE ? G : 4;  // its loads

  v16f acc[NI][MI];
  uint4 fw[2][NI];                // weight fragments of this quarter and the next
  uint4 fx[4][MI];                // token fragments of the stage's quarters
  uint4 scw[NI], scx[MI];         // scale bytes of two stages (not WIDE: of one, in x and y)
  uint32_t cw[NI], cx[MI];        // this quarter's, the lane's half in bytes 0 and 2
  int wrow = wn * (TN / 2) + r32, xrow = 32 * wm + r32;  // of the first MFMA tiles
  const int swz = (r32 >> 1) & 7;
  auto read_weights = [&](const uint8_t* buf, auto q_t) {
    constexpr int q = decltype(q_t)::value;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      fw[q & 1][i] = *reinterpret_cast<const uint4*>(buf + (wrow + 32 * i) * 128 + (((2 * q + h) ^ swz) << 4));
  };
  auto read_tokens = [&](const uint8_t* buf, auto q_t, auto mj_t) {
    constexpr int q = decltype(q_t)::value;
#pragma unroll
    for (int j = 0; j < decltype(mj_t)::value; ++j)
      fx[q][j] = *reinterpret_cast<const uint4*>(buf + (xrow + 64 * j) * 128 + (((2 * q + h) ^ swz) << 4));
  };
  auto read_pair_scales = [&](const uint32_t* sc) {  // WIDE
#pragma unroll
    for (int i = 0; i < NI; ++i) scw[i] = *reinterpret_cast<const uint4*>(sc + (wrow + 32 * i) * 4);
#pragma unroll
    for (int j = 0; j < MI; ++j) scx[j] = *reinterpret_cast<const uint4*>(sc + (256 + xrow + 64 * j) * 4);
  };
  auto read_stage_scales = [&](const uint32_t* sc) {  // not WIDE
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      scw[i].x = sc[wrow + 32 * i];
      scw[i].y = sc[kScRows + wrow + 32 * i];
    }
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      scx[j].x = sc[256 + xrow + 64 * j];
      scx[j].y = sc[kScRows + 256 + xrow + 64 * j];
    }
  };
  // The words of K block d (128 wide) of the held stages.
  auto block_scales = [&](auto d_t) {
    constexpr int d = decltype(d_t)::value;
    auto pick = [](uint4 v) { return d == 0 ? v.x : (d == 1 ? v.y : (d == 2 ? v.z : v.w)); };
#pragma unroll
    for (int i = 0; i < NI; ++i) cw[i] = pick(scw[i]) >> (8 * h);
#pragma unroll
    for (int j = 0; j < MI; ++j) cx[j] = pick(scx[j]) >> (8 * h);
  };
  auto products = [&](auto q_t, auto mj_t) {
    constexpr int q = decltype(q_t)::value;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < decltype(mj_t)::value; ++j)
        acc[i][j] = mfma_a4_32<(q & 1) == 1>(fw[q & 1][i], fx[q][j], acc[i][j], cw[i], cx[j]);
  };
  // K values past the end: zero codes.
  auto mask_tokens = [&](int s, auto q_t) {
    if constexpr (!WIDE) {
      constexpr int q = decltype(q_t)::value;
      const uint32_t m = s * 256 + q * 64 < K ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < MI; ++j) fx[q][j] = uint4{fx[q][j].x & m, fx[q][j].y & m, fx[q][j].z & m, fx[q][j].w & m};
    }
  };
  // Spreads LDS reads and then loads over a quarter's MFMAs.
  auto spread = [&](auto mj_t, auto reads_t, auto loads_t) {
    constexpr int M = NI * decltype(mj_t)::value;
    constexpr int reads = decltype(reads_t)::value, loads = decltype(loads_t)::value;
    // Twice the even rate, so that the last have arrived when the quarter ends
    // (evenly spread: 0.7 to 1.5 % more for 32768 rows of 7168 -> 4096).
    constexpr int rp = 2 * ((reads + M - 1) / M);  // reads per MFMA
    constexpr int lp = (loads + M - 1) / M;
    constexpr int l0 = M - (loads + lp - 1) / lp_or_one(lp);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                     // MFMA
      if (i * rp < reads) __builtin_amdgcn_sched_group_barrier(0x100, rp, 0);                // LDS reads
      if (loads > 0 && i >= l0) __builtin_amdgcn_sched_group_barrier(0x020, lp, 0);          // loads
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<int, 0> c0;
  const std::integral_constant<int, 1> c1;
  const std::integral_constant<int, 2> c2;
  const std::integral_constant<int, 3> c3;
  const std::integral_constant<int, MI> all;
  const std::integral_constant<int, XL> xl;
  const std::integral_constant<int, 2> xl_short;
  int buf = 0;  // s_src slot of the current tile

  // Stage s; V = s % U; mj: MFMA tiles of tokens that hold rows; xn: loads of
  // tokens for stage s + 2; its buffers w and x, and the next stage's.
  auto stage = [&](int s, auto v_t, auto mj, auto xn, uint8_t* w, uint8_t* x, const uint8_t* w_next, const uint8_t* x_next,
                   uint32_t* sc, const uint32_t* sc_next) {
    constexpr int V = decltype(v_t)::value, MJ = decltype(mj)::value, XN = decltype(xn)::value;
    // q = 0
    read_tokens(x, c1, mj);
    read_tokens(x, c2, mj);
    read_tokens(x, c3, mj);
    read_weights(w, c1);
    products(c0, mj);
    spread(mj, std::integral_constant<int, 3 * MJ + NI>{}, c0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // q = 1
    mask_tokens(s, c1);
    mask_tokens(s, c2);
    mask_tokens(s, c3);
    issue_tokens(s + 2, x, xn);
    read_weights(w, c2);
    products(c1, mj);
    spread(mj, std::integral_constant<int, NI>{}, xn);
    // q = 2
    block_scales(std::integral_constant<int, WIDE ? 2 * (V & 1) + 1 : 1>{});
    read_weights(w, c3);
    products(c2, mj);
    spread(mj, std::integral_constant<int, NI>{}, c0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(XN));  // all but the tokens of stage s + 2
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // q = 3. The scales of the next group or pair go where this one's last
    // were read two barriers ago at least.
    constexpr bool SCALES = !WIDE || V == U - 2;
    constexpr bool PAIR = WIDE && (V & 1) == 1;
    if constexpr (SCALES) issue_scales(s + 2, sc);
    issue_weights(s + 2, w);
    read_tokens(x_next, c0, all);
    read_weights(w_next, c0);
    if constexpr (PAIR) read_pair_scales(s_sc0 + (V == U - 1 ? 0 : kScRows * 4));
    products(c3, mj);
    spread(mj, std::integral_constant<int, (PAIR ? 2 : 1) * (MI + NI)>{},
           std::integral_constant<int, WL + (SCALES ? SCL : 0)>{});
    if constexpr (!WIDE) read_stage_scales(sc_next);
    block_scales(std::integral_constant<int, WIDE && (V & 1) == 0 ? 2 : 0>{});
    mask_tokens(s + 1 < P2 ? s + 1 : 0, c0);
  };
  set_sources(src[0], cur, s_src[0]);
  set_sources(src[1], nxt, s_src[1]);
  issue_scales(0, s_sc0);
  if constexpr (!WIDE) issue_scales(1, s_sc1);
  issue_tokens(0, s_x0, xl);
  issue_weights(0, s_w0);
  issue_tokens(1, s_x1, xl);
  issue_weights(1, s_w1);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(XL + WL));
  lds_barrier();
  if constexpr (WIDE) read_pair_scales(s_sc0);
  else read_stage_scales(s_sc0);
  read_tokens(s_x0, c0, all);
  read_weights(s_w0, c0);
  block_scales(c0);

  while (true) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j) acc[i][j] = v16f{};
    // U stages; the last two of them load xn2 rows' worth of tokens.
    auto stages = [&](int s, auto mj, auto xn, auto xn2) {
      // Keeps the LDS addresses of every buffer out of registers of their own.
      asm volatile("" : "+v"(wrow), "+v"(xrow));
      if constexpr (U == 4) {
        stage(s, c0, mj, xn, s_w0, s_x0, s_w1, s_x1, s_sc0, s_sc1);
        stage(s + 1, c1, mj, xn, s_w1, s_x1, s_w0, s_x0, s_sc1, s_sc0);
        stage(s + 2, c2, mj, xn2, s_w0, s_x0, s_w1, s_x1, s_sc0, s_sc1);
        stage(s + 3, c3, mj, xn2, s_w1, s_x1, s_w0, s_x0, s_sc1, s_sc0);
      } else {
        stage(s, c0, mj, xn2, s_w0, s_x0, s_w1, s_x1, s_sc0, s_sc1);
        stage(s + 1, c1, mj, xn2, s_w1, s_x1, s_w0, s_x0, s_sc1, s_sc0);
      }
    };
    if (MI > 1 && cur.rows <= 64) {
      int s = 0;
      for (; s + U < P2; s += U) stages(s, c1, xl_short, xl_short);
      stages(s, c1, xl_short, xl);
    } else {
      for (int s = 0; s < P2; s += U) stages(s, all, xl, xl);
    }

    // Output, and the row sources of the tile after the next. A lane holds
    // weight rows 8 v + 4 h .. + 3 (v = 0..3) of its token; the half waves swap
    // so that it has 8 consecutive ones of v = 2 u + h, and a row gets 32
    // contiguous bytes per store.
    const A4Tile after = locate(tile_of(round + 2));
    const int after_src = row_source(after);
    const int* from = s_src[buf];
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      if (64 * j >= cur.rows) break;
      const int row = 64 * j + 32 * wm + r32;
      const bool live = row < cur.rows;
      const uint32_t keep = from[row] < 0 ? 0u : ~0u;
      uint16_t* crow = p.c + static_cast<int64_t>(cur.row0 + row) * N + cur.n0 + wn * (TN / 2) + 8 * h;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const v16f& a = acc[i][j];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint2 e = pack_bf16x4(v4f{a[8 * u], a[8 * u + 1], a[8 * u + 2], a[8 * u + 3]});
          const uint2 o = pack_bf16x4(v4f{a[8 * u + 4], a[8 * u + 5], a[8 * u + 6], a[8 * u + 7]});
          const auto lo = __builtin_amdgcn_permlane32_swap(e.x, o.x, false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(e.y, o.y, false, false);
          const uint4 q = {lo[0] & keep, hi[0] & keep, lo[1] & keep, hi[1] & keep};
          if (live && cur.n0 + wn * (TN / 2) + 32 * i < N) *reinterpret_cast<uint4*>(crow + 32 * i + 16 * u) = q;
        }
      }
    }
    if (tid < TM) s_src[buf == 0 ? 2 : buf - 1][tid] = after_src;
    if (tile_of(++round) >= total) break;
    lds_barrier();  // the sources are written
    cur = nxt;
    nxt = after;
    src[0] = src[1];
    set_sources(src[1], nxt, s_src[buf == 0 ? 2 : buf - 1]);
    buf = buf == 2 ? 0 : buf + 1;
  }
  __builtin_amdgcn_s_waitcnt(0);  // no load may land after the workgroup's end
}

template <int TM, int TN>
hipError_t launch_a4_tiled(const W4Args& g, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(device_cu_count() * (TN < 256 ? 2 : 1)));
  if (g.k % 1024 == 0)
    hipLaunchKernelGGL((gemm_a4_tiled_kernel<TM, TN, 4>), grid, dim3(kA4TThreads), 0, stream, g);
  else if (g.k % 512 == 0)
    hipLaunchKernelGGL((gemm_a4_tiled_kernel<TM, TN, 2>), grid, dim3(kA4TThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((gemm_a4_tiled_kernel<TM, TN, 1>), grid, dim3(kA4TThreads), 0, stream, g);
  return hipGetLastError();
}

// Expected time of an expert's row tiles of tm rows, a whole tile's time being
// `full` and one of at most 64 rows' kA4ShortCost, when routing spreads rows at
// random (a Poisson count of that mean, near enough normal).
constexpr double kA4ShortCost = 0.4;
double expected_cost(double mean, int tm, double full) {
  const double step = tm > 64 ? kA4ShortCost : full;  // of the first rows, then of more than 64
  if (mean > 16.0 * tm) return (mean / tm - 0.5) * full + step + (full - step) * (1.0 - 64.0 / tm);
  const double sd = sqrt(mean) * 1.4142135623730951;
  auto more = [&](double rows) { return rows == 0.0 ? 1.0 : 0.5 * erfc((rows - mean) / sd); };
  double t = 0.0;
  for (double at = 0.0; at < mean + 4.0 * sd; at += tm) {
    t += step * more(at);
    if (tm > 64) t += (full - step) * more(at + 64.0);
  }
  return t;
}

}  // namespace

hipError_t launch_grouped_gemm_a4(const W4Args& g, hipStream_t stream) {
  const int cus = device_cu_count();
  const int rows = g.max_rows > 0 ? g.max_rows : g.row_cap;
  const int live = rows < g.num_experts ? rows : g.num_experts;  // experts with rows, at most
  const int64_t cols = (g.n + kA4TileCols - 1) / kA4TileCols;
  double mean = static_cast<double>(rows) / live;
  if (mean > g.max_rows_per_expert) mean = g.max_rows_per_expert;
  // Few weights: streamed, once per 32 rows, at 3.5 to 5 TB/s and some us around
  // them; a round of tiles through LDS takes 1.3 us per 256 K values instead,
  // whatever it holds. The two meet, for any K, at about 160 pieces of 256 weight
  // rows x 32 token rows. Streamed / tiled, us, weights from HBM: N 4096, K 7168,
  // experts x rows 1x1 11/20, 2x4 12/33, 8x4 38/38, 12x4 54/44, 16x4 72/49, 8x32
  // 55/41, 8x64 94/47, 4x100 82/38, 1x1000 156/56; N 7168, K 2048 4x16 14/13, 8x16
  // 23/16; N 1024, K 2048 32x4 13/13, 64x4 20/17; N 512, K 6144 32x2 16/30, 64x2
  // 33/34, 128x2 61/45. Of these the rule loses 8x32, whose pieces hold two row
  // tiles, and 1 us or less of the others.
  if (live * cols * static_cast<int64_t>(ceil(mean / kA4TileM)) * 8 < 5 * cus) {
    hipLaunchKernelGGL(gemm_a4_kernel, dim3(static_cast<unsigned>(4 * cus)), dim3(kA4Threads), 0, stream, g);
    return hipGetLastError();
  }
  // The tile height with the least expected time; whole tiles of 64, 128, 192
  // and 256 rows take 0.39, 0.7, 0.8 and 1. Measured, us: a layer of 64, 512
  // and 1024 tokens over 128 experts of 2048 -> 768, top 8, at 64 / 128: 83/90,
  // 101/105, 137/125; 32 experts of 40, 64 and 80 rows, K 7168, N 4096: 99/105,
  // 107/109, 152/115; of 150, 300, 520 and 1040 rows at 128 / 192 / 256:
  // 172/125/135, 242/201/207, 379/303/318 and 672/572/550; K 2048, N 7168:
  // 90/78/83, 139/118/121, 225/188/186 and 404/350/333.
  constexpr int kHeights[4] = {64, 128, 192, 256};
  constexpr double kCost[4] = {0.39, 0.7, 0.8, 1.0};
  int best = 0;
  double least = 1e300;
  for (int i = 0; i < 4; ++i) {
    const double t = expected_cost(mean, kHeights[i], kCost[i]);
    if (t < least) {
      least = t;
      best = i;
    }
  }
  switch (best) {
    case 0: return launch_a4_tiled<64, 128>(g, stream);
    case 1: return launch_a4_tiled<128, kA4TileCols>(g, stream);
    case 2: return launch_a4_tiled<192, kA4TileCols>(g, stream);
    default: return launch_a4_tiled<256, kA4TileCols>(g, stream);
  }
}

}  // namespace moe
