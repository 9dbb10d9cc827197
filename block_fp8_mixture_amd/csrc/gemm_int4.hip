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

// The eight weights of a word: s9 = 2^9 s, sz = -s z.
__device__ __forceinline__ uint4 int4_weights(uint32_t c, float s9, float sz) {
  const uint32_t even = c & 0x0F0F0F0Fu, odd = c >> 4 & 0x0F0F0F0Fu;
  const v2f e0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(even), false);
  const v2f e1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(even), true);
  const v2f o0 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(odd), false);
  const v2f o1 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(odd), true);
  auto w = [&](float q) { return __builtin_fmaf(q, s9, sz); };
  const uint2 a = pack_bf16x4(v4f{w(e0[0]), w(o0[0]), w(e0[1]), w(o0[1])});
  const uint2 b = pack_bf16x4(v4f{w(e1[0]), w(o1[0]), w(e1[1]), w(o1[1])});
  return uint4{a.x, a.y, b.x, b.y};
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
  constexpr int NS = 128 / G;               // scales of a lane and weight row per 256 K values
  __shared__ __attribute__((aligned(256))) uint8_t s_a[2][TM * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const int K = p.k, out_n = GATED ? p.n / 2 : p.n, groups = K / G;
  Int4Tile t;
  if (!int4_tile<TM>(p, (out_n + 128 * NC - 1) / (128 * NC), &t)) return;
  const int expert = __builtin_amdgcn_readfirstlane(t.expert), rows = __builtin_amdgcn_readfirstlane(t.rows);
  const int row0 = __builtin_amdgcn_readfirstlane(t.row0) + int4_seg_start(p, expert);
  const int n0 = __builtin_amdgcn_readfirstlane(t.col_tile) * 128 * NC + wave * 32 * NC;

  // Rows of A: thread tid loads chunk tid % 16 of row tid / 16 + 16 i. Rows
  // without a source load one that exists; their output is not this product's.
  const uint16_t* a[AL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int r = (tid >> 4) + 16 * i;
    const int src = r < rows ? int4_source(p, row0 + r) : -1;
    a[i] = p.a + static_cast<int64_t>(max(src, 0)) * K;
  }
  const int chunk = tid & 15;
  const int ak = 128 * (chunk >> 3) + 8 * (chunk & 7);  // its first K value of 256, in the first step
  u32x4 ra0[AL], ra1[AL];  // of the first and the second step
  auto load_a = [&](u32x4 (&ra)[AL], int b, int step) {  // (past K: the row's start)
    const int k = 256 * b + 64 * step + ak;
    const int at = k < K ? k : 0;
#pragma unroll
    for (int i = 0; i < AL; ++i) ra[i] = *reinterpret_cast<const u32x4*>(a[i] + at);
  };
  const int put = (tid >> 4) * 256 + ((chunk ^ ((tid >> 4) & 15)) << 4);
  auto store_a = [&](const u32x4 (&ra)[AL], int step) {
#pragma unroll
    for (int i = 0; i < AL; ++i) *reinterpret_cast<u32x4*>(&s_a[step][put + 4096 * i]) = ra[i];
  };

  // Weights: rows past the last take its place.
  const uint8_t* wb = p.w + static_cast<int64_t>(expert) * p.n * (K / 2);
  const uint16_t* sb = p.scales + static_cast<int64_t>(expert) * p.n * groups;
  // (without zero points the loads read bytes of the scales, unused)
  const uint8_t* zb = p.zeros ? p.zeros + static_cast<int64_t>(expert) * p.n * groups
                              : reinterpret_cast<const uint8_t*>(sb);
  uint32_t wo[NT], so[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = min(n0 + 32 * (n % NC) + r32, out_n - 1) + (GATED && n >= NC ? out_n : 0);
    wo[n] = static_cast<uint32_t>(c) * static_cast<uint32_t>(K / 2);
    so[n] = static_cast<uint32_t>(c) * static_cast<uint32_t>(groups);
  }
  const int blocks = (K + 255) / 256;
  uint4 w[NT][4];
  auto load_w = [&](int b, int n, int i) {  // (past K: the row's start)
    const uint32_t at = 128 * min(b, blocks - 1) + 64 * h + 16 * i;
    w[n][i] = *reinterpret_cast<const uint4*>(wb + (wo[n] + (2 * at < static_cast<uint32_t>(K) ? at : 0u)));
  };
  // A lane's scale in use, and the next as stored. Columns past K have the scale
  // zero: A's row is read from its start there. Selects go by masks: branches
  // would cut the MFMAs' schedule.
  uint32_t sc[NT], zr[NT];
  float s9[NT], sz[NT];
  uint32_t is_f16 = p.scale_f16 ? ~0u : 0u, has_z = p.zeros ? ~0u : 0u;
  asm volatile("" : "+v"(is_f16), "+v"(has_z));
  auto load_s = [&](int n, int k) {
    const int at = min((k + 128 * h) / G, groups - 1);
    sc[n] = sb[so[n] + at];
    zr[n] = zb[so[n] + at];
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

  load_a(ra0, 0, 0);
  load_a(ra1, 0, 1);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    load_s(n, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_w(0, n, i);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    use_s(n, 0);
    load_s(n, NS > 1 ? G : 256);
  }
  store_a(ra0, 0);
  lds_barrier();
  const int get = r32 * 256;
  // Row fragments of block (step, q): K values 8 q .. of both halves' 64.
  auto read_x = [&](uint4 (&x)[TT], int step, int q) {
    const int at = get + (((8 * h + q) ^ (r32 & 15)) << 4);
#pragma unroll
    for (int m = 0; m < TT; ++m) x[m] = *reinterpret_cast<const uint4*>(&s_a[step][at + 8192 * m]);
  };
  auto weights = [&](int n, int i, int j) {
    const uint32_t c = j == 0 ? w[n][i].x : j == 1 ? w[n][i].y : j == 2 ? w[n][i].z : w[n][i].w;
    return int4_weights(c, s9[n], sz[n]);
  };
  uint4 x[2][TT];
  read_x(x[0], 0, 0);
  uint4 f = weights(0, 0, 0);
  for (int b = 0; b < blocks; ++b) {
    // 16 blocks of 8 K values per half: the MFMAs of a weight tile go between
    // the instructions that make the next tile's weights, so that neither waits
    // for the other.
    static_for<16>([&](auto block) __attribute__((always_inline)) {
        constexpr int step = block / 8, q = block % 8, i = block / 4, j = block % 4;
        // The rows of the step after the next (past the end: the last block's
        // again, unused). The next step's are written three blocks before its
        // first and read in this step's last block, past a barrier.
        if constexpr (block == 0) load_a(ra0, min(b + 1, blocks - 1), 0);
        if constexpr (block == 8) load_a(ra1, min(b + 1, blocks - 1), 1);
        if constexpr (block == 5) store_a(ra1, 1);
        if constexpr (block == 13) store_a(ra0, 0);
        if (q == 7) lds_barrier();
        read_x(x[(q + 1) & 1], q == 7 ? step ^ 1 : step, (q + 1) & 7);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // The last of a scale's weights were made in the slot before: the next
          // scale, q' of block b', and the load of the one after it.
          if constexpr (j == 3 && (i + 1) % (4 / NS) == 0) {
            constexpr int to = (i + 1) / (4 / NS), after = to + 1;
            use_s(n, 256 * (b + to / NS) + G * (to % NS));
            load_s(n, 256 * (b + after / NS) + G * (after % NS));
          }
          const uint4 next = n + 1 < NT ? weights(n + 1, i, j) : weights(0, (i + (j == 3)) & 3, (j + 1) & 3);
#pragma unroll
          for (int m = 0; m < TT; ++m) acc[n][m] = mfma_bf16_32(f, x[q & 1][m], acc[n][m]);
          f = next;
        }
        // (word 3 of chunk i is in use until the block's third slot)
        if (j == 3) {
#pragma unroll
          for (int n = 0; n < NT; ++n) load_w(b + 1, n, i);
        }
#pragma unroll
        for (int k = 0; k < NT * TT; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                             // MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, q == 0 || j == 3 ? 6 : 5, 0);      // VALU
          if (k < TT) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                 // LDS read
          if (q == 5 && k < AL) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);       // LDS write
          if (q == 0 || j == 3) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);       // load
        }
        __builtin_amdgcn_sched_barrier(0);
    });
  }

  // A lane holds weight rows 8 v + 4 h .. + 3 (v = 0 .. 3) of its row of A.
#pragma unroll
  for (int m = 0; m < TT; ++m) {
    const int r = 32 * m + r32;
    if (r >= rows) continue;
    const bool some = int4_source(p, row0 + r) >= 0;
    uint16_t* c = p.c + static_cast<int64_t>(row0 + r) * out_n;
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
        uint2 bits = pack_bf16x4(o);
        if (!some) bits = uint2{0, 0};
        const int col = n0 + 32 * n + 8 * v + 4 * h;
        if (p.vector_out) {
          if (col < out_n) *reinterpret_cast<uint2*>(c + col) = bits;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (col + k < out_n) c[col + k] = static_cast<uint16_t>((k < 2 ? bits.x : bits.y) >> (16 * (k & 1)));
        }
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
  p.vector_out = out_n % 4 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 7) == 0;
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
