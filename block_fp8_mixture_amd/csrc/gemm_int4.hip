// Products of BF16 rows with 4-bit integer weights (scale and zero point per
// group of columns), dense or per expert over its live rows:
//   C[r, n] = bf16( sum_g s[n, g] * sum_{j in g} a[r, j] (q[n, j] - z[n, g]) )
// or, gated, bf16(SiLU(C[r, n]) * C[r, n + N/2]) of the unrounded sums.
//
// v_mfma_f32_16x16x32_bf16 with the rows of A as its first operand (lane l
// holds row l % 16 and the K values 8 (l / 16) .. + 7) and weight rows as its
// second (alike); lane l of the result holds weight row l % 16 and rows of A
// 4 (l / 16) + v, so a lane needs one row's scales.
#include <cmath>
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

// Inclusive sum over the lanes up to each.
__device__ __forceinline__ int wave_scan(int v) {
  auto add = [&](int u) { v = static_cast<int>(static_cast<unsigned>(v) + static_cast<unsigned>(u)); };
  add(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));  // row_shr 1, 2, 4, 8
  add(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true));  // lane 15 of the row before
  add(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, true));  // lane 31
  return v;
}

// Units of work are the TM-row tiles, in order, of the experts with more than
// p.rows_over rows and not more than p.rows_to. Every wave scans the counts. (Counts
// whose sum overflows are no align's: they wrap, and may find nothing.)
struct Int4Unit {
  int expert, row0, rows;  // first row and rows of the tile; no rows: not a segment
  int tiles, first;        // units of the expert, and its first one's number
};
constexpr int kScan = 8;  // experts of a lane at once: their loads wait for one another's only
__device__ __forceinline__ int int4_tiles(const Int4GemmArgs& p, int e, int tm) {
  const int c = e < p.num_experts ? min(p.counts[e], p.seg_cap > 0 ? p.seg_cap : p.row_cap) : 0;
  return c > p.rows_over && c <= p.rows_to ? (c + tm - 1) / tm : 0;
}
// Unit u; false past the last. *more: whether there may be one `step` on.
template <int TM>
__device__ __forceinline__ bool int4_find(const Int4GemmArgs& p, int u, int step, Int4Unit* t, bool* more) {
  if (!p.counts) {
    t->tiles = (p.row_cap + TM - 1) / TM;
    t->first = t->expert = 0;
    t->row0 = u * TM;
    t->rows = min(TM, p.row_cap - u * TM);
    *more = u + step < t->tiles;
    return u < t->tiles;
  }
  const int lane = threadIdx.x & 63;
  unsigned before = 0;
  const unsigned want = static_cast<unsigned>(u);
  for (int e0 = 0; e0 < p.num_experts; e0 += 64 * kScan) {
    int tiles[kScan], found = -1;
#pragma unroll
    for (int i = 0; i < kScan; ++i) tiles[i] = int4_tiles(p, e0 + 64 * i + lane, TM);
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      if (e0 + 64 * i >= p.num_experts) break;
      const unsigned incl = static_cast<unsigned>(wave_scan(tiles[i]));
      const unsigned all = static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(incl), 63));
      const uint64_t lanes = __ballot(want - before < incl);
      if (want - before < all && lanes != 0) {
        const int l = __builtin_ctzll(lanes);
        t->tiles = __builtin_amdgcn_readlane(tiles[i], l);
        t->first = static_cast<int>(before + static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(incl), l)) -
                                    static_cast<unsigned>(t->tiles));
        found = e0 + 64 * i + l;
      }
      before += all;
    }
    if (found >= 0) {
      if (want - static_cast<unsigned>(t->first) >= static_cast<unsigned>(t->tiles)) return false;
      const int at = (u - t->first) * TM;
      t->expert = found;
      t->row0 = int4_seg_start(p, found) + at;
      t->rows = min(TM, int4_rows(p, found) - at);
      *more = want + step < before || e0 + 64 * kScan < p.num_experts;
      return true;
    }
  }
  return false;
}
// Their number.
template <int TM>
__device__ __forceinline__ int int4_units(const Int4GemmArgs& p) {
  if (!p.counts) return (p.row_cap + TM - 1) / TM;
  const int lane = threadIdx.x & 63;
  int units = 0;
  for (int e0 = 0; e0 < p.num_experts; e0 += 64 * kScan) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < kScan; ++i) c += int4_tiles(p, e0 + 64 * i + lane, TM);
    units += __builtin_amdgcn_readlane(wave_scan(c), 63);
  }
  return units;
}

// ---- few rows per expert: weights streamed, exact -------------------------------
//
// A wave streams 16 R weight rows over its share of K into operands of 16x16x32
// MFMAs, blocks of 128 K values, the next asked for while one is computed. Both
// operands pass through LDS of the wave's own, without a barrier: a load takes 64
// or 256 consecutive bytes of a row, four lanes to a line (with a lane per row, as
// the operands have it, the address path handles a line per lane, and 1 token of
// 4096 -> 4096 took 10 us with the weights in L2). The waves of a workgroup share K and
// add up their sums at the end: many waves of few blocks rather than few waves
// with many loads in flight, because a launch of a few microseconds also feels
// how long its code takes to arrive.
//
// Bound by latency up to some 20 MB of weights (a launch, the first loads, LDS, the
// sums), beyond by the weights' bytes; captured, with cold weights: 1 row 7168 -> 4096
// gated 9 us, 16 rows 2048 -> 7168 8 us, 1 token's 8 experts 4096 -> 1024 12.5 us, 64
// tokens' 256 experts 6144 -> 512 (417 MB) 71 us, 5.9 TB/s (a copy of 1 GiB 5.15).
//
// Groups of fewer than 128 columns: an instruction's 32 K values have to be of one
// group in every lane, so a lane reads word g of each 16 bytes of a row, else
// 16 bytes of its own.

// XL: row tiles of four rows of A. R: weight tiles of 16 rows (gated: the second
// half up rows of the first half's columns; a single tile 8 rows of each). W: waves.
template <int G, int XL, int R, int W, bool GATED>
__device__ __forceinline__ void int4_stream_tile(const Int4GemmArgs& p, uint8_t* lds, const Int4Unit& t) {
  constexpr int MT = (XL + 3) / 4;
  constexpr int NC = GATED && R > 1 ? R / 2 : R;      // tiles that hold the output's columns
  constexpr int C = GATED ? 8 * R : 16 * R;           // these
  constexpr int D = XL > 1 ? 1 : 2;                   // blocks ahead
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int K = p.k, out_n = GATED ? p.n / 2 : p.n, groups = K / G;
  const int blocks = (K + 127) / 128;
  const int b0 = static_cast<int>(static_cast<unsigned>(blocks * wave) / W);
  const int b1 = static_cast<int>(static_cast<unsigned>(blocks * (wave + 1)) / W);
  uint8_t* const s_x = lds + wave * ((XL + R) * 1024);
  uint8_t* const s_w = s_x + XL * 1024;

  // Lane l loads chunk l % 4 (of 16 bytes) of row l / 4 of a tile's block, into
  // slot l % 4: chunk c of row r is in slot c ^ r / 4 % 4, so that reads of a chunk
  // of 16 rows meet no bank twice; and the scale of group l % 4 of it. Weight rows
  // past the last take its place.
  const uint8_t* wb = p.w + static_cast<int64_t>(t.expert) * p.n * (K / 2);
  const uint16_t* sb = p.scales + static_cast<int64_t>(t.expert) * p.n * groups;
  const uint8_t* zb = p.zeros ? p.zeros + static_cast<int64_t>(t.expert) * p.n * groups : nullptr;
  const int n0 = static_cast<int>(blockIdx.x) * C, sub = lane & 3, chunk = sub ^ g;
  uint32_t wo[R], so[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int w = lane >> 2;
    const bool up = GATED && (R > 1 ? r >= NC : w >= 8);
    const int c = min(n0 + 16 * (r % NC) + (GATED && R == 1 ? w & 7 : w), out_n - 1) + (up ? out_n : 0);
    wo[r] = static_cast<uint32_t>(c) * static_cast<uint32_t>(K / 2);
    so[r] = static_cast<uint32_t>(c) * static_cast<uint32_t>(groups);
  }
  // Rows of A: load i covers rows 4 i .. + 3, 256 bytes of each. Rows without a
  // source load one that exists; their output is zero.
  const int live = (t.rows + 3) >> 2;
  uint32_t ao[XL];  // in units of 64 bytes, of which a row is a multiple

  // Past K loads are of the row's start, and the scale is zero.
  struct Loaded {
    u32x4 w[R], x[XL];
    uint32_t sc[R], zr[R];
  };
  auto load_w = [&](Loaded& l, int b) __attribute__((always_inline)) {
    const int k = 128 * min(b, b1 - 1);
    const uint32_t wk = k + 32 * chunk < K ? k / 2 + 16 * chunk : 0;
    const int gr = min(k / G + sub, groups - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l.w[r] = *reinterpret_cast<const u32x4*>(wb + (wo[r] + wk));
      l.sc[r] = sb[so[r] + gr];
      if (zb) l.zr[r] = zb[so[r] + gr];
    }
  };
  auto load_x = [&](Loaded& l, int b) __attribute__((always_inline)) {
    const int k = 128 * min(b, b1 - 1);
    const uint8_t* xa = reinterpret_cast<const uint8_t*>(p.a) + (k + 8 * col < K ? 2 * k + 16 * col : 0);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i < live) l.x[i] = *reinterpret_cast<const u32x4*>(xa + (static_cast<uint64_t>(ao[i]) << 6));
  };

  const v4f zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  v4f total[R][MT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) total[r][m] = zero4;

  // Row r's chunk c of 16 bytes is in slot c ^ r % 16: reads of a chunk of 16 rows
  // meet no bank twice. A lane writes chunk col of rows 4 i + g, and reads row
  // col's chunks 4 g + j (groups of fewer columns: 4 j + g). With four rows at most
  // all lanes read those.
  const int row = XL == 1 ? col & 3 : col;
  uint32_t put = 256 * g + ((col ^ g) << 4);
  uint32_t get = 256 * row + (((G == 128 ? 4 * g : g) ^ row) << 4);
  const uint32_t wget = 64 * col + (((G == 128 ? g : 0) ^ (col >> 2)) << 4) + (G == 128 ? 0 : 4 * g);
  auto block = [&](Loaded& l, int b) __attribute__((always_inline)) {
    // Opaque: the addresses of every row would be kept in registers.
    asm volatile("" : "+v"(put), "+v"(get));
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i < live)
        *reinterpret_cast<uint4*>(s_x + (put ^ ((i & 3) << 6)) + 1024 * i) = int4_order(__builtin_bit_cast(uint4, l.x[i]));
    uint4 q[R];
    float s[R][4], off[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) *reinterpret_cast<u32x4*>(s_w + 1024 * r + 16 * lane) = l.w[r];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (G == 128) {
        q[r] = *reinterpret_cast<const uint4*>(s_w + 1024 * r + wget);
      } else {
        q[r].x = *reinterpret_cast<const uint32_t*>(s_w + 1024 * r + wget);
        q[r].y = *reinterpret_cast<const uint32_t*>(s_w + 1024 * r + (wget ^ 16));
        q[r].z = *reinterpret_cast<const uint32_t*>(s_w + 1024 * r + (wget ^ 32));
        q[r].w = *reinterpret_cast<const uint32_t*>(s_w + 1024 * r + (wget ^ 48));
      }
      // Row col's scales and zero points, from the lanes that loaded them.
      const float sv = 128 * b + G * sub < K ? int4_scale(l.sc[r], p.scale_f16) : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((32 * (j + 1)) % G != 0) continue;
        const int from = 4 * (4 * col + 32 * j / G);
        s[r][j] = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(sv)));
        off[r][j] = 16.0f + (zb ? static_cast<float>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(l.zr[r]))) : 8.0f);
      }
    }
    // (the loads' registers are free)
    load_w(l, b + D);
    load_x(l, b + D);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (MT > 1 && 4 * m >= live) break;
      v4f acc[R], sum = zero4;
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = zero4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 f = *reinterpret_cast<const uint4*>(s_x + (get ^ (j << (G == 128 ? 4 : 6))) + 4096 * m);
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
      // (the next row tile's fragments read ahead would not fit the registers)
      if constexpr (MT > 1) __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The weights ahead of what looks up the rows of A.
  Loaded l0, l1;
  if (b0 < b1) {
    load_w(l0, b0);
    if constexpr (D > 1) load_w(l1, b0 + 1);
  }
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = 4 * i + g;
    ao[i] = 0;
    if (r < t.rows) ao[i] = static_cast<uint32_t>(max(int4_source(p, t.row0 + r), 0)) * static_cast<uint32_t>(K / 32);
  }
  if (b0 < b1) {
    load_x(l0, b0);
    if constexpr (D > 1) load_x(l1, b0 + 1);
  }
  for (int b = b0; b < b1; b += D) {
    block(l0, b);
    if constexpr (D > 1) {
      if (b + 1 < b1) block(l1, b + 1);
    }
  }

  float* const s_sum = reinterpret_cast<float*>(lds);  // [W][R][MT][64 lanes][4]
  constexpr int kWave = R * MT * 256;
  __syncthreads();  // the rows of A are read
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (MT == 1 || 4 * m < live) *reinterpret_cast<v4f*>(s_sum + wave * kWave + ((r * MT + m) * 64 + lane) * 4) = total[r][m];
  __syncthreads();
  for (int i = tid; i < t.rows * C; i += 64 * W) {
    const int r = i / C, c = i % C;
    const float* from = s_sum + (((c / 16) * MT + r / 16) * 64 + c % 16 + 16 * (r % 16 / 4)) * 4 + r % 4;
    float v = 0.0f, u = 0.0f;
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      v += from[w * kWave];
      if constexpr (GATED) u += from[w * kWave + (R > 1 ? NC * MT * 256 : 32)];  // (32: eight lanes on)
    }
    if constexpr (GATED) v = int4_gated(p.act, v, u, p.limit);
    if (int4_source(p, t.row0 + r) < 0) v = 0.0f;
    if (n0 + c < out_n)
      p.c[static_cast<int64_t>(t.row0 + r) * out_n + n0 + c] = static_cast<uint16_t>(pack_bf16x4(v4f{v, v, v, v}).x);
  }
}

// A workgroup takes units of a column tile in turn: how many there are only the
// device knows.
template <int G, int XL, int R, int W, bool GATED>
__global__ __launch_bounds__(64 * W, XL == 8 ? 1 : 4) void int4_stream_kernel(Int4GemmArgs p) {
  constexpr int MT = (XL + 3) / 4;
  constexpr int kX = W * (XL + R) * 1024, kSum = W * R * MT * 1024;
  __shared__ __attribute__((aligned(256))) uint8_t lds[kX > kSum ? kX : kSum];
  bool more = true;
  for (int u = blockIdx.y; more; u += gridDim.y) {
    Int4Unit t;
    if (!int4_find<4 * XL>(p, u, gridDim.y, &t, &more)) break;
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows > 0) int4_stream_tile<G, XL, R, W, GATED>(p, lds, t);
    __syncthreads();  // the sums are read
  }
}

// ---- many rows per expert: tiles of BF16 rows through LDS ---------------------
//
// The weights enter the matrix cores as the integers q - z, which BF16 holds exactly
// (-255 .. 15). A group's sum starts from zero and is scaled into a total in fp32, so
// what a row gets does not depend on how many other rows its expert has, but for the
// order of a sum. (Weights rounded to BF16 before the product need no second set of
// accumulators: 32 x 32 tiles of 16 registers in a wave's 64 or 128 rows; their error of
// 2^-9 each made the output's 0.0022 of its root mean square, gated 0.0027, where its
// own rounding is 0.0017.)
//
// A SIMD has two waves: one alone issues an instruction of the vector unit every 4
// cycles at most, so that those beside an MFMA of 32 cycles soon show (with registers
// alone, 15.0 ns an MFMA; with 6 FMAs beside each 22 in one wave, 17.7 in two). Beside
// an MFMA there are here 3.5 for the weights (4.75 with zero points), 2 for the scale in
// groups of 128, 8 in groups of 32, and one or two for addresses.
//
// A workgroup of eight waves owns 32 TT rows of A and 256 weight rows (gated: 128
// columns, of a wave's 32 rows 16 gates and their 16 ups), a wave all of the rows and 32
// of the weight rows. Both pass through LDS in steps of 128 K values, two buffers, the
// rows of A shared, the codes a wave's own; the loads of the step after next are in
// registers meanwhile. A step's K values are taken 32 at a time, of them 16 h + 8 t ..
// + 7 by the lanes of half h in the t-th MFMA. The loop ends with the last group: no K
// value past it is multiplied. A tile of at most half its rows has a loop of its own.
//
// Bound by the power that MFMAs, conversions and LDS reads take together (1.6 to 1.75
// GHz, matrix cores busy 0.56): 2048 rows, K 7168, N 8192 in groups of 128 take 245
// us, in groups of 32 with zero points 290, 4096 rows to 16384 columns 905 us (1.06 PF;
// a BF16 product of the same sizes by the library 178 to 193 and 650 to 685 us).

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kTlWaves = 8, kTlThreads = 64 * kTlWaves;

__device__ __forceinline__ v16f mfma_bf16_32(u32x4 a, uint4 b, v16f acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                 acc, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), bf16x2));
}
// The eight integers q - z of a word as BF16, in four steps that go between MFMAs.
// ZEROS: the E4M3 byte 0 .. 15 stands for q 2^-9, and fma(q 2^-9, 2^9, -z) is exact: 19
// instructions. Otherwise z is 8, and v_cvt_off_f32_i4 makes (q - 8) / 16 of the four
// bits q ^ 8 in a byte's lower half: 14, and the totals are a sixteenth.
struct Int4Unpack {
  uint32_t even, odd;
  v2f e0, e1, o0, o1;
  uint4 f;
};
template <int I>
__device__ __forceinline__ float int4_off(uint32_t c) {
  return __builtin_amdgcn_cvt_off_f32_i4(static_cast<int>(I == 1 ? c >> 8 & 0xFFu : c >> (8 * I)));
}
template <bool ZEROS, int STEP>
__device__ __forceinline__ void int4_unpack(Int4Unpack& u, uint32_t c, float z) {
  if constexpr (ZEROS) {
    auto w = [&](float q) { return __builtin_fmaf(q, 512.0f, -z); };
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
  } else {
    if constexpr (STEP == 0) {
      u.even = c ^ 0x88888888u;
      u.odd = __builtin_amdgcn_alignbit(u.even, u.even, 4);  // (a shift would be one with those of the bytes)
      u.e0[0] = int4_off<0>(u.even);
      u.o0[0] = int4_off<0>(u.odd);
    } else if constexpr (STEP == 1) {
      u.e0[1] = int4_off<1>(u.even);
      u.o0[1] = int4_off<1>(u.odd);
      u.f.x = pack_bf16x2(u.e0[0], u.o0[0]);
    } else if constexpr (STEP == 2) {
      u.e1[0] = int4_off<2>(u.even);
      u.o1[0] = int4_off<2>(u.odd);
      u.f.y = pack_bf16x2(u.e0[1], u.o0[1]);
      u.e1[1] = int4_off<3>(u.even);
    } else {
      u.o1[1] = int4_off<3>(u.odd);
      u.f.z = pack_bf16x2(u.e1[0], u.o1[0]);
      u.f.w = pack_bf16x2(u.e1[1], u.o1[1]);
    }
  }
}

// Tile of this workgroup: workgroups go round-robin over the 8 XCDs; an XCD
// takes consecutive tiles, an expert's row tiles of one column tile first, so
// that its L2 serves their weights and the rows' next column tiles.
template <int TM>
__device__ __forceinline__ bool int4_tile(const Int4GemmArgs& p, int col_tiles, Int4Unit* t, int* tile) {
  const int64_t total = static_cast<int64_t>(int4_units<TM>(p)) * col_tiles, per = (total + 7) / 8;
  const int64_t id = flat_block(), at = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || at >= total) return false;
  // Unit at / col_tiles is one of the expert's; its tiles go column by column.
  int u = 0, local = 0;
  if (at < INT32_MAX) {  // (a 64-bit division is long)
    u = static_cast<int>(static_cast<unsigned>(at) / static_cast<unsigned>(col_tiles));
    local = static_cast<int>(at) - u * col_tiles;
  } else {
    u = static_cast<int>(at / col_tiles);
    local = static_cast<int>(at % col_tiles);
  }
  bool more;
  if (!int4_find<TM>(p, u, 1, t, &more)) return false;
  const int64_t mine = static_cast<int64_t>(u - t->first) * col_tiles + local;
  int row;
  if (mine < INT32_MAX) {
    row = static_cast<int>(static_cast<unsigned>(mine) % static_cast<unsigned>(t->tiles));
    *tile = static_cast<int>(static_cast<unsigned>(mine) / static_cast<unsigned>(t->tiles));
  } else {
    row = static_cast<int>(mine % t->tiles);
    *tile = static_cast<int>(mine / t->tiles);
  }
  // From unit u's rows to row tile `row`.
  const int rows = p.counts ? int4_rows(p, t->expert) : p.row_cap;
  t->row0 += (row - (u - t->first)) * TM;
  t->rows = min(TM, rows - row * TM);
  return t->rows > 0;
}

template <int G, int TT, bool GATED, bool ZEROS>
__global__ __launch_bounds__(kTlThreads, 2) void int4_tiled_kernel(Int4GemmArgs p) {
  constexpr int TM = 32 * TT;               // rows of A
  constexpr int WC = GATED ? 16 : 32;       // columns of the output per wave
  constexpr int TN = kTlWaves * WC;
  constexpr int NG = 128 / G;               // groups of a step
  constexpr int kABytes = TM * 256, kWBytes = 2048;  // of a step; codes: of one wave
  __shared__ __attribute__((aligned(256))) uint8_t s_buf[2 * kABytes + 2 * kTlWaves * kWBytes];
  __shared__ uint8_t s_some[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const s_a = s_buf;
  uint8_t* const s_w = s_buf + 2 * kABytes + wave * (2 * kWBytes);
  const int r32 = lane & 31, h = lane >> 5;
  const int K = p.k, out_n = GATED ? p.n / 2 : p.n, groups = K / G;
  Int4Unit t;
  int tile;
  if (!int4_tile<TM>(p, (out_n + TN - 1) / TN, &t, &tile)) return;
  const int expert = __builtin_amdgcn_readfirstlane(t.expert), rows = __builtin_amdgcn_readfirstlane(t.rows);
  const int row0 = __builtin_amdgcn_readfirstlane(t.row0);
  const int n0 = __builtin_amdgcn_readfirstlane(tile) * TN;
  const int steps = (K + 127) / 128;

  // Rows of A: thread tid loads chunk tid % 16 (of 8 K values) of row tid / 16 + 32 i
  // into slot chunk ^ row % 16: reads of a chunk of 16 rows meet no bank twice. Rows without a source load one that exists; their
  // output is zero. Past K loads are of the row's start, unused.
  int src[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int r = (tid >> 4) + 32 * i;
    src[i] = r < rows ? int4_source(p, row0 + r) : -1;
  }
  const int chunk = tid & 15;
  const int put = (tid >> 4) * 256 + ((chunk ^ ((tid >> 4) & 15)) << 4);
  // Codes: four neighbouring lanes load 64 bytes of a row, 16 rows a load. Chunk c (of
  // 32 K values) of a row is in slot c ^ (row / 4 % 4): 16 rows' reads of a chunk meet
  // no bank twice. Weight rows past the last take its place.
  const uint8_t* wb = p.w + static_cast<int64_t>(expert) * p.n * (K / 2);
  auto weight_row = [&](int r) {
    const int col = min(n0 + WC * wave + (GATED ? r & 15 : r), out_n - 1);
    return static_cast<uint32_t>(GATED && r >= 16 ? col + out_n : col);
  };
  uint32_t wo[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) wo[k] = weight_row(16 * k + (lane >> 2)) * static_cast<uint32_t>(K / 2);
  const int wchunk = (lane & 3) ^ (lane >> 4);
  const uint16_t* sb = p.scales + static_cast<int64_t>(expert) * p.n * groups;
  const uint8_t* zb = ZEROS ? p.zeros + static_cast<int64_t>(expert) * p.n * groups : nullptr;
  const uint32_t so = weight_row(r32) * static_cast<uint32_t>(groups);
  const uint16_t* a[TT];
  u32x4 ra[TT], rw[2];
  int ka = 0;
  uint32_t kw = 0;
  auto at = [&](int step) __attribute__((always_inline)) {
    const int k = 128 * min(step, steps - 1);
    ka = k + 8 * chunk < K ? k + 8 * chunk : 0;
    kw = k + 32 * wchunk < K ? k / 2 + 16 * wchunk : 0;
  };
  // Pieces of a step: TT of the rows, two of the codes.
  auto load = [&](int i) __attribute__((always_inline)) {
    if (i < TT) ra[i] = *reinterpret_cast<const u32x4*>(a[i] + ka);
    else rw[i - TT] = *reinterpret_cast<const u32x4*>(wb + (wo[i - TT] + kw));
  };
  auto store = [&](int buf, int i) __attribute__((always_inline)) {
    if (i < TT) *reinterpret_cast<u32x4*>(s_a + buf * kABytes + put + 8192 * i) = ra[i];
    else *reinterpret_cast<u32x4*>(s_w + buf * kWBytes + 1024 * (i - TT) + 16 * lane) = rw[i - TT];
  };
  // Scales and zero points as stored, of a whole step's groups at once: the address path
  // handles a line for every weight row, however few of its bytes are asked for (a load
  // per group: 300 rows 7168 -> 4096 gated in groups of 32 with zero points 136 us).
  struct Scales {
    uint32_t s[(NG + 1) / 2], z;
  };
  const int whole = K / 128;
  uint32_t is_f16 = p.scale_f16 ? ~0u : 0u;  // (branches would cut the MFMAs' schedule)
  asm volatile("" : "+v"(is_f16));
  auto load_s = [&](Scales& to, int step) __attribute__((always_inline)) {
    const uint32_t g = so + min(step, whole - 1) * NG;
    if constexpr (NG == 1) {
      to.s[0] = sb[g];
      if constexpr (ZEROS) to.z = zb[g];
    } else {
      __builtin_memcpy(to.s, sb + g, 2 * NG);
      if constexpr (ZEROS) __builtin_memcpy(&to.z, zb + g, NG);
    }
  };
  auto scale_of = [&](uint32_t bits) __attribute__((always_inline)) {
    const uint32_t half = __float_as_uint(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits))));
    return __uint_as_float((half & is_f16) | (bits << 16 & ~is_f16));
  };
  auto scale = [&](const Scales& r, int i) __attribute__((always_inline)) { return scale_of(r.s[i / 2] >> (16 * (i & 1))); };
  auto zero = [&](const Scales& r, int i) __attribute__((always_inline)) {
    return ZEROS ? static_cast<float>(r.z >> (8 * i) & 0xFFu) : 0.0f;
  };
  // K values 16 j .. of a step lie in chunks 4 (j / 2) + 2 h + j % 2: the slot's bits of j
  // are one exclusive or with the first one's.
  const uint32_t fa = r32 * 256 + (((2 * h) ^ (r32 & 15)) << 4), fw = r32 * 64 + ((r32 >> 2 & 3) << 4) + 8 * h;
  auto codes = [&](int buf, int c) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint2*>(s_w + ((fw + buf * kWBytes) ^ (c << 4)));
  };
  auto fragment = [&](int buf, int j, int m) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(s_a + ((fa + buf * kABytes) ^ ((4 * (j >> 1) + (j & 1)) << 4)) + 8192 * m);
  };

  constexpr int KS = G / 16;  // MFMAs of a group and row tile
  v16f total[TT], acc[TT];
#pragma unroll
  for (int m = 0; m < TT; ++m) total[m] = acc[m] = v16f{};
  auto add = [&](int m, float s) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < 16; ++v) total[m][v] = __builtin_fmaf(s, acc[m][v], total[m][v]);
  };

  // The weights ahead of what waits for the rows' numbers.
  at(0);
#pragma unroll
  for (int i = TT; i < TT + 2; ++i) load(i);
  Scales now{}, next{};
  if (whole > 0) load_s(now, 0);
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    a[i] = p.a + static_cast<int64_t>(max(src[i], 0)) * K;
    if ((tid & 15) == 0) s_some[(tid >> 4) + 32 * i] = src[i] >= 0;
    load(i);
  }
  at(1);
#pragma unroll
  for (int i = 0; i < TT + 2; ++i) {
    store(0, i);
    load(i);
  }
  lds_barrier();
  // The first LT row tiles have rows.
  auto sums = [&](auto live_tiles) __attribute__((always_inline)) {
    constexpr int LT = live_tiles;
    float s_done = 0.0f, s_now = scale(now, 0), z = zero(now, 0);
    if (whole > 0) load_s(next, 1);
    u32x4 x[2][LT];
#pragma unroll
    for (int m = 0; m < LT; ++m) x[0][m] = fragment(0, 0, m);
    uint2 q[2] = {codes(0, 0), uint2{0, 0}};
    Int4Unpack u[2];
    static_for<4>([&](auto k) __attribute__((always_inline)) { int4_unpack<ZEROS, k>(u[0], q[0].x, z); });
    for (int step = 0; step < whole; ++step) {
      const int buf = step & 1;
      at(step + 2);  // (past the end: the last ones again, unused)
      static_for<8>([&](auto jj) __attribute__((always_inline)) {
        constexpr int j = jj;
        // The next step's rows are in the other buffer, and this one's read.
        if constexpr (j == 7) lds_barrier();
        static_for<LT>([&](auto mm) __attribute__((always_inline)) {
          constexpr int m = mm;
          // The group before this one is complete: its sums, scaled.
          if constexpr (j % KS == 0) {
            add(m, s_done);
            acc[m] = mfma_bf16_32(x[j & 1][m], u[j & 1].f, v16f{});
          } else {
            acc[m] = mfma_bf16_32(x[j & 1][m], u[j & 1].f, acc[m]);
          }
          x[(j + 1) & 1][m] = fragment(j == 7 ? buf ^ 1 : buf, (j + 1) & 7, m);
          if constexpr (j % 2 == 0 && m == 0) q[(j / 2 + 1) & 1] = codes(j == 6 ? buf ^ 1 : buf, (j / 2 + 1) & 3);
          // The scale of the next group, and the load of those two steps on.
          if constexpr ((j + 1) % KS == 0 && m == 0) {
            constexpr int g = (j + 1) / KS % NG;
            if constexpr (g == 0 && NG > 1) {
              now = next;
              // (copies, before the registers are loaded again: else the load would be
              // waited for, to be copied)
              for (uint32_t& w : now.s) asm volatile("" : "+v"(w));
              if constexpr (ZEROS) asm volatile("" : "+v"(now.z));
            }
            s_done = s_now;
            s_now = scale(NG > 1 ? now : next, g);
            z = zero(NG > 1 ? now : next, g);
            if constexpr (g == 0) load_s(next, step + 2);
          }
          constexpr int half = ((j + 1) / 2) & 1;
          static_for<4 / LT>([&](auto l) __attribute__((always_inline)) {
            int4_unpack<ZEROS, 4 / LT * m + l>(u[(j + 1) & 1], (j + 1) & 1 ? q[half].y : q[half].x, z);
          });
          // A piece of the next step's data, and its register's next load.
          constexpr int piece = j < LT ? j : j - LT + TT;
          if constexpr (piece < TT + 2 && m == (LT == 4 ? 1 : 0)) store(buf ^ 1, piece);
          if constexpr (piece < TT + 2 && m == (LT == 4 ? 2 : LT - 1)) load(piece);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    }
#pragma unroll
    for (int m = 0; m < LT; ++m) add(m, s_done);
    // The last groups, where they are not a whole step.
    if constexpr (NG > 1) {
      const int buf = whole & 1;
      for (int g = whole * NG; g < groups; ++g) {
        const float s = scale_of(sb[so + g]);
        if constexpr (ZEROS) z = static_cast<float>(zb[so + g]);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const int at_j = (g - whole * NG) * KS + j;
          const uint2 w = codes(buf, at_j >> 1);
          static_for<4>([&](auto k) __attribute__((always_inline)) { int4_unpack<ZEROS, k>(u[0], at_j & 1 ? w.y : w.x, z); });
#pragma unroll
          for (int m = 0; m < LT; ++m) acc[m] = mfma_bf16_32(fragment(buf, at_j, m), u[0].f, j == 0 ? v16f{} : acc[m]);
        }
#pragma unroll
        for (int m = 0; m < LT; ++m) add(m, s);
      }
    }
  };
  if (rows > 16 * TT)
    sums(std::integral_constant<int, TT>{});
  else
    sums(std::integral_constant<int, TT / 2>{});

  // Output, through LDS so that a row's columns leave in whole lines. A lane holds its
  // column's rows 8 v + 4 h + k of 32 (v, k = 0 .. 3). Gated: lanes 0 .. 15 and 32 ..
  // hold gates, the others ups of the same columns; of two rows, the first half gets
  // the first's gate and up, the second half the second's. Then neighbouring columns
  // exchange one of two rows, so that a lane writes two columns of one. Chunk c of 8
  // columns of a row is in slot c ^ 4 f, f telling apart the four rows of a write.
  constexpr int kRow = 2 * TN;
  static_assert(TM * kRow <= 2 * kABytes, "");
  uint8_t* const s_c = s_buf;
  lds_barrier();  // the rows are read
  auto write = [&](int row, int col, float v0, float v1) __attribute__((always_inline)) {
    // v0, v1: this column's values of rows row and row + 1 (gated: row + 2)
    const bool odd = lane & 1;
    const float other = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(odd ? v0 : v1), 0xB1, 0xF, 0xF, false));
    const uint32_t two = odd ? pack_bf16x2(other, v1) : pack_bf16x2(v0, other);
    const int r = row + (odd ? (GATED ? 2 : 1) : 0), f = (GATED ? r >> 1 & 1 : r & 1) | (GATED ? (r & 1) << 1 : r >> 1 & 2);
    const int at = 2 * (col & ~1);
    *reinterpret_cast<uint32_t*>(s_c + r * kRow + ((at >> 4 ^ (f << 2)) << 4) + (at & 15)) = two;
  };
#pragma unroll
  for (int m = 0; m < TT; ++m) {
    if (32 * m >= rows) break;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = ZEROS ? total[m][4 * v + k] : 16.0f * total[m][4 * v + k];
      const int row = 32 * m + 8 * v + 4 * h;
      if constexpr (GATED) {
        float g[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(o[2 * k]), __float_as_uint(o[2 * k + 1]), false, false);
          g[k] = int4_gated(p.act, __uint_as_float(both[0]), __uint_as_float(both[1]), p.limit);
        }
        write(row + (r32 >> 4), 16 * wave + (r32 & 15), g[0], g[1]);
      } else {
        write(row, 32 * wave + r32, o[0], o[1]);
        write(row + 2, 32 * wave + r32, o[2], o[3]);
      }
    }
  }
  lds_barrier();
  constexpr int kChunks = TN / 8;
  const int c = tid % kChunks, col = n0 + 8 * c;
#pragma unroll
  for (int i = 0; i < TM * kChunks / kTlThreads; ++i) {
    const int r = tid / kChunks + i * (kTlThreads / kChunks);
    const int f = (GATED ? r >> 1 & 1 : r & 1) | (GATED ? (r & 1) << 1 : r >> 1 & 2);
    uint4 bits = *reinterpret_cast<const uint4*>(s_c + r * kRow + ((c ^ (f << 2)) << 4));
    if (!s_some[r]) bits = uint4{0, 0, 0, 0};
    if (r >= rows) continue;
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

// Experts of more than `over` and at most `to` rows.
template <int G, int XL, int R, int W, bool GATED>
hipError_t stream_launch(Int4GemmArgs p, int over, int to, hipStream_t stream) {
  constexpr int TM = 4 * XL;
  p.rows_over = over;
  p.rows_to = to;
  const int out_n = GATED ? p.n / 2 : p.n, cols = GATED ? 8 * R : 16 * R;
  // Every tile but an expert's last is full.
  const int64_t fit = p.row_cap / (over + 1), used = p.num_experts < fit ? p.num_experts : fit;
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  if (units == 0) return hipSuccess;
  // About a workgroup of 16 waves, or two of 8, for a CU: more would wait for it
  // only to find that there is no unit for them.
  const int64_t tiles = (out_n + cols - 1) / cols, stay = (16 / W * device_cu_count() + tiles - 1) / tiles;
  const int64_t y = units < stay ? units : stay;
  hipLaunchKernelGGL((int4_stream_kernel<G, XL, R, W, GATED>), dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(y)),
                     dim3(64 * W), 0, stream, p);
  return hipGetLastError();
}

// Experts of at most `bound` rows (to: the largest count taken as such).
template <int G, bool GATED>
hipError_t stream_rows(const Int4GemmArgs& p, int bound, int to, hipStream_t stream) {
  const int out_n = GATED ? p.n / 2 : p.n;
  const bool narrow = !p.counts && (out_n + (GATED ? 15 : 31)) / (GATED ? 16 : 32) <= device_cu_count() / 2;
  if (bound <= 4)
    return narrow ? stream_launch<G, 1, 1, 16, GATED>(p, 0, to, stream) : stream_launch<G, 1, 2, 16, GATED>(p, 0, to, stream);
  int over = 0;
  if (bound <= 16 || p.counts) {
    const int t = bound <= 16 ? to : 16;
    const hipError_t e = narrow      ? stream_launch<G, 4, 1, 16, GATED>(p, 0, t, stream)
                         : p.counts ? stream_launch<G, 4, 2, 8, GATED>(p, 0, t, stream)
                                    : stream_launch<G, 4, 2, 16, GATED>(p, 0, t, stream);
    if (e != hipSuccess || bound <= 16) return e;
    over = 16;
  }
  return stream_launch<G, 8, 2, 8, GATED>(p, over, to, stream);
}

template <int G, int TT, bool GATED>
hipError_t tiled_launch(Int4GemmArgs p, hipStream_t stream) {
  constexpr int TM = 32 * TT, TN = kTlWaves * (GATED ? 16 : 32);
  p.rows_over = kInt4FewRows;
  p.rows_to = INT32_MAX;
  const int out_n = GATED ? p.n / 2 : p.n;
  const int64_t fit = p.row_cap / (kInt4FewRows + 1), used = p.num_experts < fit ? p.num_experts : fit;
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  // A multiple of 8: every XCD's share rounded up.
  const int64_t tasks = (units * ((out_n + TN - 1) / TN) + 7) / 8 * 8;
  if (p.zeros)
    hipLaunchKernelGGL((int4_tiled_kernel<G, TT, GATED, true>), flat_grid(tasks), dim3(kTlThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((int4_tiled_kernel<G, TT, GATED, false>), flat_grid(tasks), dim3(kTlThreads), 0, stream, p);
  return hipGetLastError();
}

// Expected time, us, of the forms that more than kInt4FewRows rows can take, by
// the tiles that there are for each CU (r). Tiled forms: a superstep of 256 K
// values takes 1.8 to 2.25 us a round of 64 x 256 tiles, 2.65 to 3.85 of 128 x 256
// ones (the more the fuller the chip, whose clock falls), and 6 or 7 us go around it;
// streamed tiles of 32 x 32 take 2.5 us and 0.2 for every 128 K values. Over several
// experts the last tiles are of fewer rows: a last round costs what it holds. Measured
// (streamed, 64 x 256, 128 x 256), us, for rows, K, N in groups of 128: 300, 6144, 1000:
// 26, 48, 73; 70, 4096, 4096: 18, 35, 51; 300, 2048, 7168: 58, 22, 30; 300, 7168, 4096
// gated: 70, 57, 87; 512, 4096, 4096: 79, 38, 53; 1024, 4096, 4096: 137, 42, 55; 1024,
// 2048, 7168: -, 43, 36; 2048, 4096, 4096: 261, 87, 70; 2048, 7168, 8192: -, 306, 251.
// Smaller groups and zero points take all three longer alike: groups of 32 with zero
// points by a third to a half.
struct Int4Costs {
  double stream, small, medium;
};
Int4Costs int4_costs(const Int4GemmArgs& p, int out_n, int gated) {
  const double cus = device_cu_count(), blocks = (p.k + 255) / 256;
  const double experts = p.counts ? (p.num_experts < p.row_cap ? p.num_experts : p.row_cap) : 1.0;
  const double mean = p.row_cap / experts;
  // Row tiles: of one expert known, of several half a tile more than they fill.
  auto units = [&](int tm) { return p.num_experts > 1 ? experts * (mean / tm + 0.5) : ceil(p.row_cap / static_cast<double>(tm)); };
  auto cols = [&](int c) { return ceil(out_n / static_cast<double>(gated ? c / 2 : c)); };
  auto fill = [](double r) { return r < 1.0 ? r : 1.0; };
  auto rounds = [&](double r) { return p.num_experts > 1 ? (r + 0.3 > 1.0 ? r + 0.3 : 1.0) : ceil(r); };
  const double rs = units(32) * cols(32) / cus, r2 = units(64) * cols(256) / cus;
  const double r4 = units(128) * cols(256) / cus;
  return {ceil(rs) * (2.5 + 0.4 * blocks), 6.0 + blocks * rounds(r2) * (1.8 + 0.45 * fill(r2)),
          7.0 + blocks * rounds(r4) * (2.65 + 1.2 * fill(r4))};
}

template <int G, bool GATED>
hipError_t gemm_launch(Int4GemmArgs p, hipStream_t stream) {
  const int out_n = GATED ? p.n / 2 : p.n;
  p.vector_out = out_n % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
  // (a count past the bound is computed all the same)
  if (p.max_rows_per_expert <= kInt4FewRows) return stream_rows<G, GATED>(p, p.max_rows_per_expert, INT32_MAX, stream);
  const Int4Costs t = int4_costs(p, out_n, GATED);
  if (t.stream <= t.small && t.stream <= t.medium)
    return stream_rows<G, GATED>(p, p.max_rows_per_expert, INT32_MAX, stream);
  if (p.counts) {
    const hipError_t e = stream_rows<G, GATED>(p, kInt4FewRows, kInt4FewRows, stream);
    if (e != hipSuccess) return e;
  }
  return t.small <= t.medium ? tiled_launch<G, 2, GATED>(p, stream) : tiled_launch<G, 4, GATED>(p, stream);
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
