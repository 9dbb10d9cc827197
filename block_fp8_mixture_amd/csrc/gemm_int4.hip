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
    const int tiles = c <= p.few ? (c + TM - 1) / TM : 0;
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

// f(integral_constant 0), .., f(integral_constant N - 1).
template <typename F, int... I>
__device__ __forceinline__ void static_for_seq(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_seq(f, std::make_integer_sequence<int, N>{});
}

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
struct Int4Tile {
  int expert, row0, rows, col_tile;
};
template <int TM>
__device__ __forceinline__ bool int4_tile(const Int4GemmArgs& p, int col_tiles, Int4Tile* t) {
  const int lane = threadIdx.x & 63;
  int64_t units = 0;
  if (!p.counts) {
    units = (p.row_cap + TM - 1) / TM;
  } else {
    for (int e0 = 0; e0 < p.num_experts; e0 += 64) {
      const int e = e0 + lane;
      int c = e < p.num_experts ? int4_rows(p, e) : 0;
      c = c > p.few ? (c + TM - 1) / TM : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d, 64);
      units += c;
    }
  }
  const int64_t total = units * col_tiles, per = (total + 7) / 8;
  const int64_t id = flat_block(), at = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || at >= total) return false;
  if (!p.counts) {
    t->expert = 0;
    t->row0 = static_cast<int>(at % units) * TM;
    t->rows = min(TM, p.row_cap - t->row0);
    t->col_tile = static_cast<int>(at / units);
    return true;
  }
  int64_t before = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 64) {
    const int e = e0 + lane;
    const int c = e < p.num_experts ? int4_rows(p, e) : 0;
    const int tiles = c > p.few ? (c + TM - 1) / TM : 0;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const int all = __shfl(incl, 63, 64);
    if (at < (before + all) * col_tiles) {
      const int l = __builtin_ctzll(__ballot((before + incl) * col_tiles > at));
      const int mine = __shfl(tiles, l, 64), rows = __shfl(c, l, 64);
      const int local = static_cast<int>(at - (before + __shfl(incl, l, 64) - mine) * col_tiles);
      t->expert = e0 + l;
      t->row0 = local % mine * TM;
      t->rows = min(TM, rows - t->row0);
      t->col_tile = local / mine;
      return true;
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
  Int4Tile t;
  if (!int4_tile<TM>(p, (out_n + 128 * NC - 1) / (128 * NC), &t)) return;
  const int expert = __builtin_amdgcn_readfirstlane(t.expert), rows = __builtin_amdgcn_readfirstlane(t.rows);
  const int row0 = __builtin_amdgcn_readfirstlane(t.row0) + int4_seg_start(p, expert);
  const int n0 = __builtin_amdgcn_readfirstlane(t.col_tile) * 128 * NC + wave * 32 * NC;
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
    if (p.max_rows_per_expert <= 16) return stream_launch<G, 1, GATED>(p, stream);
    if (p.max_rows_per_expert <= 32) return stream_launch<G, 2, GATED>(p, stream);
    return stream_launch<G, 4, GATED>(p, stream);
  }
  p.few = kInt4FewRows;
  if (p.counts) {
    const hipError_t e = stream_launch<G, 4, GATED>(p, stream);
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
