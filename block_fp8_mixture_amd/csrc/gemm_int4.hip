// Products of BF16 rows with 4-bit integer weights (scale and zero point per
// group of columns), dense or per expert over its live rows:
//   C[r, n] = bf16( sum_g s[n, g] * sum_{j in g} a[r, j] (q[n, j] - z[n, g]) )
// or, gated, bf16(SiLU(C[r, n]) * C[r, n + N/2]) of the unrounded sums.
//
// v_mfma_f32_16x16x32_bf16 with the rows of A as its first operand (lane l
// holds row l % 16 and the K values 8 (l / 16) .. + 7) and weight rows as its
// second (alike); lane l of the result holds weight row l % 16 and rows of A
// 4 (l / 16) + v, so a lane needs one row's scales.
#include <utility>

#include "int4_device.h"

namespace moe {
namespace {

// f(integral_constant 0), .., f(integral_constant N - 1).
template <typename F, int... I>
__device__ __forceinline__ void static_for_seq(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_seq(f, std::make_integer_sequence<int, N>{});
}

// The expert and the row tile of work unit u, units being the TM-row tiles, in
// order, of the experts that have rows and `many` more than p.few (or not). Every
// wave scans the counts, 256 experts at a time; *total: the units of them all, if
// asked for.
struct Int4Unit {
  int expert, row0, rows;  // first row and rows of the tile
};
__device__ __forceinline__ int int4_tiles(const Int4GemmArgs& p, int e, int tm, bool many) {
  const int c = e < p.num_experts ? min(p.counts[e], p.row_cap) : 0;
  return c > 0 && (c > p.few) == many ? (c + tm - 1) / tm : 0;
}
template <int TM, bool MANY>
__device__ __forceinline__ int64_t int4_units(const Int4GemmArgs& p) {
  if (!p.counts) return (p.row_cap + TM - 1) / TM;
  const int lane = threadIdx.x & 63;
  int64_t units = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 256) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += int4_tiles(p, e0 + 64 * i + lane, TM, MANY);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d, 64);
    units += c;
  }
  return units;
}
template <int TM, bool MANY>
__device__ __forceinline__ bool int4_unit(const Int4GemmArgs& p, int64_t u, Int4Unit* t) {
  if (!p.counts) {
    if (u * TM >= p.row_cap) return false;
    t->expert = 0;
    t->row0 = static_cast<int>(u) * TM;
    t->rows = min(TM, p.row_cap - t->row0);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 256) {
    int tiles[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) tiles[i] = int4_tiles(p, e0 + 64 * i + lane, TM, MANY);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int incl = tiles[i];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d, 64);
        if (lane >= d) incl += v;
      }
      const int all = __builtin_amdgcn_readlane(incl, 63);
      if (u < before + all) {
        const int l = __builtin_ctzll(__ballot(before + incl > u));
        const int first = __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles[i], l);
        const int e = e0 + 64 * i + l, at = static_cast<int>(u - before - first) * TM;
        t->expert = e;
        t->row0 = int4_seg_start(p, e) + at;
        t->rows = min(TM, int4_rows(p, e) - at);
        return t->rows > 0;
      }
      before += all;
    }
  }
  return false;
}

// ---- few rows per expert: weights streamed, exact -------------------------------
//
// A wave streams 16 R weight rows over its share of K straight into operands of
// 16x16x32 MFMAs, D blocks of 128 K values ahead (their loads, in order, hide
// each other's latency); the rows of A of a block pass through LDS of the wave's
// own, which turns whole-line loads into operands and needs no barrier. The waves
// of a workgroup share K and add up their sums at the end.
//
// Groups of fewer than 128 columns: a lane's 16 bytes are 32 columns of one
// group, but an instruction's 32 K values have to be of one group in every lane,
// so the wave's four rows of lanes swap words (row_transpose), and their scales
// likewise: row g loads group g's, and all get every group's.

// XL: row tiles of four rows of A. R: weight tiles of 16 rows (gated: the second
// half up rows of the first half's columns). W: waves.
template <int G, int XL, int R, int D, int W, bool GATED>
__device__ __forceinline__ void int4_stream_tile(const Int4GemmArgs& p, uint8_t* lds, const Int4Unit& t,
                                                 int tile) {
  constexpr int MT = (XL + 3) / 4, NC = GATED ? R / 2 : R;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int K = p.k, out_n = GATED ? p.n / 2 : p.n, groups = K / G;
  const int blocks = (K + 127) / 128;
  const int b0 = static_cast<int>(static_cast<unsigned>(blocks * wave) / W);
  const int b1 = static_cast<int>(static_cast<unsigned>(blocks * (wave + 1)) / W);
  uint8_t* const s_x = lds + wave * (MT * 4096);

  // Weight rows past the last take its place.
  const uint8_t* wb = p.w + static_cast<int64_t>(t.expert) * p.n * (K / 2);
  const uint16_t* sb = p.scales + static_cast<int64_t>(t.expert) * p.n * groups;
  const uint8_t* zb = p.zeros ? p.zeros + static_cast<int64_t>(t.expert) * p.n * groups : nullptr;
  uint32_t wo[R], so[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = min(16 * (NC * tile + r % NC) + col, out_n - 1) + (GATED && r >= NC ? out_n : 0);
    wo[r] = static_cast<uint32_t>(c) * static_cast<uint32_t>(K / 2);
    so[r] = static_cast<uint32_t>(c) * static_cast<uint32_t>(groups);
  }
  // Rows of A: load i covers rows 4 i .. + 3, 256 bytes of each. Rows without a
  // source load one that exists; their output is zero.
  const int live = (t.rows + 3) >> 2;
  uint32_t ao[XL];  // in units of 64 bytes, of which a row is a multiple
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = 4 * i + g;
    ao[i] = 0;
    if (r < t.rows) ao[i] = static_cast<uint32_t>(max(int4_source(p, t.row0 + r), 0)) * static_cast<uint32_t>(K / 32);
  }

  // Past K loads are of the row's start, and the scale is zero.
  u32x4 w[D][R], x[D][XL];
  uint32_t sc[D][R], zr[D][R];
  auto load = [&](auto d, int b) __attribute__((always_inline)) {
    const int k = 128 * min(b, b1 - 1);
    const uint32_t wk = k + 32 * g < K ? k / 2 + 16 * g : 0;
    const uint8_t* xa = reinterpret_cast<const uint8_t*>(p.a) + (k + 8 * col < K ? 2 * k + 16 * col : 0);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i < live) x[d][i] = *reinterpret_cast<const u32x4*>(xa + (static_cast<uint64_t>(ao[i]) << 6));
    const int gr = min((G < 128 ? k + 32 * g : k) / G, groups - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[d][r] = *reinterpret_cast<const u32x4*>(wb + (wo[r] + wk));
      sc[d][r] = sb[so[r] + gr];
      if (zb) zr[d][r] = zb[so[r] + gr];
    }
  };

  const v4f zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  v4f total[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) total[r][m] = zero4;

  auto block = [&](auto d, int b) __attribute__((always_inline)) {
    // Row 4 i + g, chunk col in slot col ^ row % 16: reads of a chunk of 16 rows
    // meet no bank twice.
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i < live)
        *reinterpret_cast<uint4*>(s_x + 1024 * i + 256 * g + ((col ^ ((4 * i + g) & 15)) << 4)) =
            int4_order(__builtin_bit_cast(uint4, x[d][i]));
    uint4 q[R];
    float s[R][4], off[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      q[r] = __builtin_bit_cast(uint4, w[d][r]);
      const float sv = G == 128 || 128 * b + 32 * g < K ? int4_scale(sc[d][r], p.scale_f16) : 0.0f;
      if constexpr (G == 128) {
        s[r][3] = sv;
        off[r][3] = 16.0f + (zb ? static_cast<float>(zr[d][r]) : 8.0f);
      } else {
        q[r] = row_transpose(q[r]);
        const uint32_t v = __float_as_uint(sv);
        const uint4 a = row_transpose(uint4{v, v, v, v});
        s[r][0] = __uint_as_float(a.x);
        s[r][1] = __uint_as_float(a.y);
        s[r][2] = __uint_as_float(a.z);
        s[r][3] = __uint_as_float(a.w);
        if (zb) {
          const uint32_t o = __float_as_uint(16.0f + static_cast<float>(zr[d][r]));
          const uint4 z = row_transpose(uint4{o, o, o, o});
          off[r][0] = __uint_as_float(z.x);
          off[r][1] = __uint_as_float(z.y);
          off[r][2] = __uint_as_float(z.z);
          off[r][3] = __uint_as_float(z.w);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) off[r][j] = 24.0f;
        }
      }
    }
    // (the loads' registers are free)
    load(d, b + D);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (MT > 1 && 4 * m >= live) break;
      v4f acc[R], sum = zero4;
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = zero4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = G == 128 ? 4 * g + j : 4 * j + g;
        const uint4 f = *reinterpret_cast<const uint4*>(s_x + 4096 * m + 256 * col + ((c ^ col) << 4));
        sum = mfma_bf16(f, ones, sum);
#pragma unroll
        for (int r = 0; r < R; ++r)
          acc[r] = mfma_bf16(f, int4_operand(j == 0 ? q[r].x : j == 1 ? q[r].y : j == 2 ? q[r].z : q[r].w), acc[r]);
        if ((32 * (j + 1)) % G == 0) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              total[r][m][v] = __builtin_fmaf(s[r][j], __builtin_fmaf(-off[r][j], sum[v], acc[r][v]), total[r][m][v]);
            acc[r] = zero4;
          }
          sum = zero4;
        }
      }
    }
  };
  if (b0 < b1) {
    static_for<D>([&](auto d) __attribute__((always_inline)) { load(d, b0 + d); });
    for (int b = b0; b < b1; b += D)
      static_for<D>([&](auto d) __attribute__((always_inline)) {
        if (b + d < b1) block(d, b + d);
      });
  }

  v4f* const s_sum = reinterpret_cast<v4f*>(lds);  // [W][R][MT][64]
  __syncthreads();                                 // the rows of A are read
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (MT == 1 || 4 * m < live) s_sum[((wave * R + r) * MT + m) * 64 + lane] = total[r][m];
  __syncthreads();
  // A wave finishes the tiles (c, m) of its number; gated, both of a pair.
  for (int i = wave; i < NC * MT; i += W) {
    const int m = i % MT, c = i / MT;
    if (MT > 1 && 4 * m >= live) continue;
    v4f v = zero4, u = zero4;
#pragma unroll
    for (int k = 0; k < W; ++k) v += s_sum[((k * R + c) * MT + m) * 64 + lane];
    if constexpr (GATED) {
#pragma unroll
      for (int k = 0; k < W; ++k) u += s_sum[((k * R + NC + c) * MT + m) * 64 + lane];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = int4_gated(p.act, v[k], u[k], p.limit);
    }
    const int n = 16 * (NC * tile + c) + col;
    const uint2 bits = pack_bf16x4(v);
    if (n < out_n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 16 * m + 4 * g + k;
        const uint32_t o = k < 2 ? bits.x : bits.y;
        if (r < t.rows)
          p.c[static_cast<int64_t>(t.row0 + r) * out_n + n] =
              int4_source(p, t.row0 + r) < 0 ? 0 : static_cast<uint16_t>(k & 1 ? o >> 16 : o);
      }
    }
  }
}

// XL: of the launch's largest tiles; a tile with fewer rows takes a smaller form.
// Workgroups stay and take tiles in turn: how many there are only the device knows.
template <int G, int XL, int R, int D, int W, bool GATED>
__global__ __launch_bounds__(64 * W, 1) void int4_stream_kernel(Int4GemmArgs p) {
  constexpr int MT = (XL + 3) / 4;
  constexpr int kX = W * MT * 4096, kSum = W * R * MT * 1024;
  __shared__ __attribute__((aligned(256))) uint8_t lds[kX > kSum ? kX : kSum];
  const int out_n = GATED ? p.n / 2 : p.n, cols = GATED ? 8 * R : 16 * R;
  const unsigned col_tiles = static_cast<unsigned>(out_n + cols - 1) / cols;
  const int64_t total = int4_units<4 * XL, false>(p) * col_tiles;
  for (int64_t task = blockIdx.x; task < total; task += gridDim.x) {
    int64_t u;
    int tile;
    if (task < INT32_MAX) {  // (a 64-bit division is long)
      u = static_cast<unsigned>(task) / col_tiles;
      tile = static_cast<unsigned>(task) % col_tiles;
    } else {
      u = task / col_tiles;
      tile = static_cast<int>(task % col_tiles);
    }
    Int4Unit t;
    if (!int4_unit<4 * XL, false>(p, u, &t)) continue;
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (XL > 4 && t.rows <= 4)
      int4_stream_tile<G, 1, R, 4, W, GATED>(p, lds, t, tile);
    else if (XL > 4 && t.rows <= 16)
      int4_stream_tile<G, 4, R, 3, W, GATED>(p, lds, t, tile);
    else
      int4_stream_tile<G, XL, R, D, W, GATED>(p, lds, t, tile);
    __syncthreads();  // the sums are read
  }
}

// ---- many rows per expert: tiles of BF16 rows through LDS ---------------------
//
// Here the matrix cores bound the product, and a sum per group outside them
// would cost as many instructions as they have to spare. So the weights enter
// them as the BF16 values bf16(s (q - z)) that moe_int4_dequant gives, made in
// registers as they are needed: each rounding is 2^-9 of its weight, over K
// weights a random error of about what the output's own rounding is.
//
// A code becomes a float by v_cvt_pk_f32_fp8: the E4M3 byte 0 .. 15 stands for
// q 2^-9. fma(q 2^-9, 2^9 s, -s z) is exact, two at a time rounded to BF16: 19
// instructions for 8 codes, against four 32x32x16 MFMAs of 32 cycles each that
// use them.
//
// A workgroup of four waves owns 32 TT rows of A and 128 NT weight rows, a wave
// all of the rows and 32 NT of the weight rows, whose codes it loads straight
// into registers (a tile of few rows of A and many weight rows moves the least:
// a weight is a quarter of an activation). The rows of A pass through LDS, two
// buffers of 128 K values. K order: the lanes of half h hold the 128 K values
// from 128 h of 256, so that a lane needs few scales and a row's 128-byte lines
// are loaded whole.

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kTlThreads = 256;

__device__ __forceinline__ v16f mfma_bf16_32(uint4 a, uint4 b, v16f acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                 acc, 0, 0, 0);
}

// The eight weights of a word, s9 = 2^9 s, sz = -s z, in four steps that go between
// MFMAs.
struct Int4Unpack {
  uint32_t even, odd;
  v2f e0, e1, o0, o1;
  uint4 f;
};
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), bf16x2));
}
template <int STEP>
__device__ __forceinline__ void int4_unpack(Int4Unpack& u, uint32_t c, float s9, float sz) {
  auto w = [&](float q) { return __builtin_fmaf(q, s9, sz); };
  if constexpr (STEP == 0) {
    u.even = c & 0x0F0F0F0Fu;
    u.odd = c >> 4 & 0x0F0F0F0Fu;
    u.e0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.even), false);
    u.o0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.odd), false);
  } else if constexpr (STEP == 1) {
    u.e1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.even), true);
    u.o1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(u.odd), true);
    u.e0[0] = w(u.e0[0]);
    u.o0[0] = w(u.o0[0]);
    u.e0[1] = w(u.e0[1]);
  } else if constexpr (STEP == 2) {
    u.o0[1] = w(u.o0[1]);
    u.f.x = pack_bf16x2(u.e0[0], u.o0[0]);
    u.e1[0] = w(u.e1[0]);
    u.o1[0] = w(u.o1[0]);
    u.f.y = pack_bf16x2(u.e0[1], u.o0[1]);
  } else {
    u.e1[1] = w(u.e1[1]);
    u.o1[1] = w(u.o1[1]);
    u.f.z = pack_bf16x2(u.e1[0], u.o1[0]);
    u.f.w = pack_bf16x2(u.e1[1], u.o1[1]);
  }
}

// Tile of this workgroup: workgroups go round-robin over the 8 XCDs; an XCD
// takes consecutive tiles, an expert's row tiles of one column tile first, so
// that its L2 serves their weights and the rows' next column tiles.
template <int TM>
__device__ __forceinline__ bool int4_tile(const Int4GemmArgs& p, int col_tiles, Int4Unit* t, int* tile) {
  const int64_t units = int4_units<TM, true>(p), total = units * col_tiles, per = (total + 7) / 8;
  const int64_t id = flat_block(), at = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || at >= total) return false;
  // Tiles in order of expert, then column tile, then row tile.
  if (!p.counts) {
    *tile = static_cast<int>(at / units);
    return int4_unit<TM, true>(p, at % units, t);
  }
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 64) {
    const int tiles = int4_tiles(p, e0 + lane, TM, true);
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const int all = __builtin_amdgcn_readlane(incl, 63);
    if (at < (before + all) * col_tiles) {
      const int l = __builtin_ctzll(__ballot((before + incl) * col_tiles > at));
      const int mine = __builtin_amdgcn_readlane(tiles, l), e = e0 + l;
      const int local = static_cast<int>(at - (before + __builtin_amdgcn_readlane(incl, l) - mine) * col_tiles);
      *tile = local / mine;
      t->expert = e;
      t->row0 = int4_seg_start(p, e) + local % mine * TM;
      t->rows = min(TM, int4_rows(p, e) - local % mine * TM);
      return t->rows > 0;
    }
    before += all;
  }
  return false;
}

template <int G, int TT, int NT, bool GATED>
__global__ __launch_bounds__(kTlThreads, 1) void int4_tiled_kernel(Int4GemmArgs p) {
  constexpr int TM = 32 * TT;               // rows of A
  constexpr int NC = GATED ? NT / 2 : NT;   // 32-column tiles of the output per wave
  constexpr int AL = TM * 16 / kTlThreads;  // 16-byte loads of A per thread and step
  constexpr int WL = 2 * NT;                // and of codes
  constexpr int NS = 128 / G;               // scales of a lane and weight row per 256 K values
  constexpr int kABytes = TM * 256, kWBytes = NT * 2048;  // of a step; codes: of one wave
  __shared__ __attribute__((aligned(256))) uint8_t s_buf[2 * kABytes + 8 * kWBytes];
  __shared__ uint8_t s_some[TM];
  uint8_t* const s_a = s_buf;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const s_w = s_buf + 2 * kABytes + wave * (2 * kWBytes);
  const int r32 = lane & 31, h = lane >> 5;
  const int K = p.k, out_n = GATED ? p.n / 2 : p.n, groups = K / G;
  Int4Unit t;
  int tile;
  if (!int4_tile<TM>(p, (out_n + 128 * NC - 1) / (128 * NC), &t, &tile)) return;
  const int expert = __builtin_amdgcn_readfirstlane(t.expert), rows = __builtin_amdgcn_readfirstlane(t.rows);
  const int row0 = __builtin_amdgcn_readfirstlane(t.row0);
  const int n0 = __builtin_amdgcn_readfirstlane(tile) * 128 * NC + wave * 32 * NC;
  const int blocks = (K + 255) / 256;

  // Rows of A: thread tid loads chunk tid % 16 of row tid / 16 + 16 i. Rows
  // without a source load one that exists; their output is zero.
  const uint16_t* a[AL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int r = (tid >> 4) + 16 * i;
    const int src = r < rows ? int4_source(p, row0 + r) : -1;
    a[i] = p.a + static_cast<int64_t>(max(src, 0)) * K;
    if ((tid & 15) == 0) s_some[r] = src >= 0;
  }
  const int chunk = tid & 15;
  const int ak = 128 * (chunk >> 3) + 8 * (chunk & 7);  // its first K value of 256, in the first step
  u32x4 ra[AL];
  auto at_a = [&](int b, int step) {  // (past K: the row's start)
    const int k = 256 * min(b, blocks - 1) + 64 * step + ak;
    return k < K ? k : 0;
  };
  auto load_a = [&](int at, int i) { ra[i] = *reinterpret_cast<const u32x4*>(a[i] + at); };
  const int put = (tid >> 4) * 256 + ((chunk ^ ((tid >> 4) & 15)) << 4);
  auto store_a = [&](int step, int i) {
    *reinterpret_cast<u32x4*>(s_a + step * kABytes + put + 4096 * i) = ra[i];
  };
  // Fragments of A's rows of block q: K values 8 q .. of both halves' 64.
  const int get = r32 * 256;
  auto read_a = [&](u32x4& x, int step, int q, int m) {
    const int at = get + (((8 * h + q) ^ (r32 & 15)) << 4);
    x = *reinterpret_cast<const u32x4*>(s_a + step * kABytes + at + 8192 * m);
  };

  // Codes go through LDS too, each wave its own: four neighbouring lanes load 64
  // bytes of a row, 16 rows a load (a lane with a row of its own, as the operand
  // has it, asks for 64 lines). Chunk 2 h' + i' of a row's step, the 32 K values
  // 128 h' + 64 step + 32 i', is in slot chunk ^ (row / 4 % 4): 16 rows' reads
  // of a chunk meet no bank twice. Weight rows past the last take its place.
  const uint8_t* wb = p.w + static_cast<int64_t>(expert) * p.n * (K / 2);
  auto weight_row = [&](int n, int r) {
    return static_cast<uint32_t>(min(n0 + 32 * (n % NC) + r, out_n - 1) + (GATED && n >= NC ? out_n : 0));
  };
  uint32_t wo[WL];
#pragma unroll
  for (int k = 0; k < WL; ++k) wo[k] = weight_row(k >> 1, 16 * (k & 1) + (lane >> 2)) * static_cast<uint32_t>(K / 2);
  const int wchunk = (lane & 3) ^ (lane >> 4);
  u32x4 rw[WL];
  auto at_w = [&](int b, int step) {  // (past K: the row's start)
    const uint32_t at = 128 * min(b, blocks - 1) + 32 * step + 64 * (wchunk >> 1) + 16 * (wchunk & 1);
    return 2 * at < static_cast<uint32_t>(K) ? at : 0u;
  };
  auto load_w = [&](uint32_t at, int k) { rw[k] = *reinterpret_cast<const u32x4*>(wb + (wo[k] + at)); };
  auto store_w = [&](int step, int k) {
    *reinterpret_cast<u32x4*>(s_w + step * kWBytes + 1024 * k + 16 * lane) = rw[k];
  };
  u32x4 w[2][NT];  // by the chunk's parity
  auto read_w = [&](u32x4& to, int step, int ii, int n) {
    const int at = r32 * 64 + (((2 * h + ii) ^ (r32 >> 2 & 3)) << 4);
    to = *reinterpret_cast<const u32x4*>(s_w + step * kWBytes + 2048 * n + at);
  };

  // A lane's scale in use, and the next as stored. Columns past K have the scale
  // zero: A's row is read from its start there. Selects go by masks: branches
  // would cut the MFMAs' schedule. Without zero points the loads read bytes of
  // the scales, unused.
  const uint16_t* sb = p.scales + static_cast<int64_t>(expert) * p.n * groups;
  const uint8_t* zb = p.zeros ? p.zeros + static_cast<int64_t>(expert) * p.n * groups
                              : reinterpret_cast<const uint8_t*>(sb);
  uint32_t so[NT], sc[NT], zr[NT];
  float s9[NT], sz[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) so[n] = weight_row(n, r32) * static_cast<uint32_t>(groups);
  uint32_t is_f16 = p.scale_f16 ? ~0u : 0u, has_z = p.zeros ? ~0u : 0u;
  asm volatile("" : "+v"(is_f16), "+v"(has_z));
  auto load_s = [&](int n, int k) {
    const uint32_t at = so[n] + min((k + 128 * h) / G, groups - 1);
    sc[n] = sb[at];
    zr[n] = zb[at];
  };
  auto use_s = [&](int n, int k) {
    const uint32_t half = __float_as_uint(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(sc[n]))));
    const uint32_t bits = (half & is_f16) | (sc[n] << 16 & ~is_f16);
    const uint32_t keep = static_cast<uint32_t>((k + 128 * h - K) >> 31);
    const float s = __uint_as_float(bits & keep);
    s9[n] = s * 512.0f;
    sz[n] = -s * static_cast<float>((zr[n] & has_z) | (8u & ~has_z));
  };

  v16f acc[NT][TT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < TT; ++m) acc[n][m] = v16f{};

  int aa = at_a(0, 0);
  uint32_t aw = at_w(0, 0);
#pragma unroll
  for (int i = 0; i < AL; ++i) load_a(aa, i);
#pragma unroll
  for (int k = 0; k < WL; ++k) load_w(aw, k);
#pragma unroll
  for (int n = 0; n < NT; ++n) load_s(n, 0);
  aa = at_a(0, 1);
  aw = at_w(0, 1);
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    store_a(0, i);
    load_a(aa, i);
  }
#pragma unroll
  for (int k = 0; k < WL; ++k) {
    store_w(0, k);
    load_w(aw, k);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    use_s(n, 0);
    load_s(n, NS > 1 ? G : 256);
  }
  lds_barrier();
  u32x4 x[2][TT];
#pragma unroll
  for (int m = 0; m < TT; ++m) read_a(x[0][m], 0, 0, m);
#pragma unroll
  for (int n = 0; n < NT; ++n) read_w(w[0][n], 0, 0, n);
  Int4Unpack u[2];  // the weights in use and the next tile's
  static_for<4>([&](auto k) __attribute__((always_inline)) { int4_unpack<k>(u[0], w[0][0][0], s9[0], sz[0]); });
  for (int b = 0; b < blocks; ++b) {
    // 16 blocks of 8 K values per half, 8 a step: the MFMAs of a weight tile go
    // between the instructions that make the next tile's weights, so that neither
    // waits for the other. The loads and LDS writes are spread over the blocks
    // (in bursts the waves wait for each other's, with the matrix cores idle): a
    // register is written to the next step's buffer and loaded for the step after
    // it (past the end: the last ones again, unused).
    static_for<16>([&](auto block) __attribute__((always_inline)) {
      constexpr int step = block / 8, q = block % 8, i = block / 4, j = block % 4;
      if constexpr (q == 0) {
        aa = at_a(b + 1, step);
        aw = at_w(b + 1, step);
      }
      if constexpr (q == 7) lds_barrier();
      // Slot k: an MFMA and what goes beside it, in this order.
      static_for<NT * TT>([&](auto k) __attribute__((always_inline)) {
        constexpr int n = k / TT, m = k % TT, slot = block * NT + n;
        acc[n][m] = mfma_bf16_32(u[slot & 1].f, __builtin_bit_cast(uint4, x[q & 1][m]), acc[n][m]);
        // The rows' fragments of the next block, and the next chunk of codes.
        if constexpr (k < TT) read_a(x[(q + 1) & 1][k], q == 7 ? step ^ 1 : step, (q + 1) & 7, k);
        if constexpr (j == 3 && k >= TT && k < TT + NT)
          read_w(w[(i + 1) & 1][k - TT], q < 4 ? step : step ^ 1, (i + 1) & 1, k - TT);
        // Pieces of A and of the codes, in the last block none: it reads the next
        // step's, past a barrier.
        constexpr int kPieces = AL + WL, kHalf = NT * TT / 2;
        constexpr int p0 = q * kPieces / 7, p1 = q < 7 ? (q + 1) * kPieces / 7 : p0;
        constexpr int piece = p0 + (k - kHalf) / 2;
        if constexpr (k >= kHalf && piece < p1) {
          if constexpr ((k - kHalf) % 2 == 0) {
            if constexpr (piece < AL) store_a(step ^ 1, piece);
            else store_w(step ^ 1, piece - AL);
          } else {
            if constexpr (piece < AL) load_a(aa, piece);
            else load_w(aw, piece - AL);
          }
        }
        // The last of a scale's weights were made in the slot before: the next
        // scale, and the load of the one after it.
        if constexpr (m == 0 && j == 3 && (i + 1) % (4 / NS) == 0) {
          constexpr int to = (i + 1) / (4 / NS), after = to + 1;
          use_s(n, 256 * (b + to / NS) + G * (to % NS));
          load_s(n, 256 * (b + after / NS) + G * (after % NS));
        }
        constexpr int nn = (n + 1) % NT, ni = n + 1 < NT ? i : (i + (j == 3)) & 3, nj = n + 1 < NT ? j : (j + 1) & 3;
        static_for<4 / TT>([&](auto l) __attribute__((always_inline)) {
          int4_unpack<4 / TT * m + l>(u[(slot + 1) & 1], w[ni & 1][nn][nj], s9[nn], sz[nn]);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }

  // Output, through LDS so that a row's columns leave in whole lines. A lane
  // holds weight rows 8 v + 4 h .. + 3 (v = 0 .. 3) of its row of A; a wave's
  // rows of 32 NC columns lie in chunks of 8 columns, chunk c in slot c ^ row % 16
  // (NC = 2: of half as long rows, c ^ row / 2 % 8).
  constexpr int kRow = 64 * NC, kChunks = 4 * NC;
  static_assert(4 * TM * kRow <= 2 * kABytes + 8 * kWBytes && (NC == 4 || NC == 2), "");
  lds_barrier();  // other waves still read A's rows
  uint8_t* const s_c = s_buf + wave * (TM * kRow);
  auto slot = [&](int c, int row) { return (c ^ (NC == 4 ? row & 15 : row >> 1 & 7)) << 4; };
#pragma unroll
  for (int m = 0; m < TT; ++m) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        v4f o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[k] = acc[n][m][4 * v + k];
          if constexpr (GATED) o[k] = int4_gated(p.act, o[k], acc[n + NC][m][4 * v + k], p.limit);
        }
        *reinterpret_cast<uint2*>(s_c + (32 * m + r32) * kRow + slot(4 * n + v, r32) + 8 * h) = pack_bf16x4(o);
      }
    }
  }
  const int c = lane % kChunks, col = n0 + 8 * c;
  for (int r = lane / kChunks; r < rows; r += 64 / kChunks) {
    uint4 bits = *reinterpret_cast<const uint4*>(s_c + r * kRow + slot(c, r));
    if (!s_some[r]) bits = uint4{0, 0, 0, 0};
    uint16_t* to = p.c + static_cast<int64_t>(row0 + r) * out_n + col;
    if (p.vector_out) {
      if (col < out_n) *reinterpret_cast<uint4*>(to) = bits;
    } else {
      const uint32_t u[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < out_n) to[k] = static_cast<uint16_t>(u[k / 2] >> (16 * (k & 1)));
    }
  }
}

template <int G, int XL, int R, int D, int W, bool GATED>
hipError_t stream_launch(const Int4GemmArgs& p, hipStream_t stream) {
  constexpr int TM = 4 * XL;
  const int out_n = GATED ? p.n / 2 : p.n, cols = GATED ? 8 * R : 16 * R;
  // Every tile but an expert's last is full.
  const int64_t used = p.num_experts < p.row_cap ? p.num_experts : p.row_cap;
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  const int64_t tasks = (out_n + cols - 1) / cols * units, cap = 2 * static_cast<int64_t>(device_cu_count());
  hipLaunchKernelGGL((int4_stream_kernel<G, XL, R, D, W, GATED>), dim3(static_cast<unsigned>(tasks < cap ? tasks : cap)),
                     dim3(64 * W), 0, stream, p);
  return hipGetLastError();
}

template <int G, bool GATED>
hipError_t stream_rows(const Int4GemmArgs& p, int bound, hipStream_t stream) {
  if (bound <= 4) return stream_launch<G, 1, 2, 4, 8, GATED>(p, stream);
  if (bound <= 16) return stream_launch<G, 4, 2, 3, 8, GATED>(p, stream);
  if (bound <= 32) return stream_launch<G, 8, 4, 2, 4, GATED>(p, stream);
  return stream_launch<G, 16, 4, 1, 4, GATED>(p, stream);
}

template <int G, int TT, int NT, bool GATED>
hipError_t tiled_launch(const Int4GemmArgs& p, hipStream_t stream) {
  constexpr int TM = 32 * TT, NC = GATED ? NT / 2 : NT;
  const int out_n = GATED ? p.n / 2 : p.n;
  const int64_t used = p.num_experts < p.row_cap / (p.few + 1) ? p.num_experts : p.row_cap / (p.few + 1);
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  // A multiple of 8: every XCD's share rounded up.
  const int64_t tasks = (units * ((out_n + 128 * NC - 1) / (128 * NC)) + 7) / 8 * 8;
  hipLaunchKernelGGL((int4_tiled_kernel<G, TT, NT, GATED>), flat_grid(tasks), dim3(kTlThreads), 0, stream, p);
  return hipGetLastError();
}

template <int G, bool GATED>
hipError_t gemm_launch(Int4GemmArgs p, hipStream_t stream) {
  const int out_n = GATED ? p.n / 2 : p.n;
  p.vector_out = out_n % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
  if (p.max_rows_per_expert <= kInt4FewRows) {
    p.few = INT32_MAX;  // whatever the counts say
    return stream_rows<G, GATED>(p, p.max_rows_per_expert, stream);
  }
  p.few = kInt4FewRows;
  if (p.counts) {
    const hipError_t e = stream_rows<G, GATED>(p, kInt4FewRows, stream);
    if (e != hipSuccess) return e;
  }
  return tiled_launch<G, 4, 4, GATED>(p, stream);
}

template <int G>
hipError_t gemm_act(const Int4GemmArgs& p, hipStream_t stream) {
  return p.act >= 0 ? gemm_launch<G, true>(p, stream) : gemm_launch<G, false>(p, stream);
}

}  // namespace

hipError_t launch_gemm_int4(const Int4GemmArgs& p, hipStream_t stream) {
  switch (p.group) {
    case 32: return gemm_act<32>(p, stream);
    case 64: return gemm_act<64>(p, stream);
    default: return gemm_act<128>(p, stream);
  }
}

}  // namespace moe
