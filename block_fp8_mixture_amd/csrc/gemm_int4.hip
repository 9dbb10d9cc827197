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
// sums), beyond by the weights' bytes: 1 row 7168 -> 4096 gated 9 us, 16 rows 2048 ->
// 7168 8 us, 1 token's 8 experts 4096 -> 1024 12.5 us, 64 tokens' 256 experts 6144 ->
// 512 (417 MB) 71 us, 5.9 TB/s (a copy of 1 GiB 5.15).
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
// A workgroup of four waves owns 32 TT rows of A and 128 NT weight rows (gated: 64
// NT columns), a wave all of the rows and 32 NT of the weight rows: a tile of few rows
// of A and many weight rows moves the least, a weight being a quarter of an activation.
// Both pass through LDS, the rows of A in buffers that the workgroup shares, a wave's
// codes in its own, two steps of 128 K values each. K order: the lanes of half h hold
// the 128 K values from 128 h of 256, so that a lane needs few scales and a row's
// 128-byte lines are loaded whole.
//
// Bound by the matrix cores at the clock they are left (1.7 GHz with all of them
// busy): 2048 rows, K 7168, N 8192 take 207 us, 4096 rows to 16384 columns 773 us (1.24
// PF; a BF16 product of the same sizes by the library 193 and 650 us).

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
        constexpr int kPieces = AL + WL, kMost = 2 * ((kPieces + 6) / 7);  // slots that a block's take
        constexpr int kHalf = NT * TT / 2 < NT * TT - kMost ? NT * TT / 2 : NT * TT - kMost;
        static_assert(kHalf >= 0, "a block's pieces fit its slots");
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
  // (of rows half or a quarter as long c ^ row / 2 % 8, c ^ row / 4 % 4).
  constexpr int kRow = 64 * NC, kChunks = 4 * NC;
  static_assert(4 * TM * kRow <= 2 * kABytes + 8 * kWBytes && (NC == 4 || NC == 2 || NC == 1), "");
  lds_barrier();  // other waves still read A's rows
  uint8_t* const s_c = s_buf + wave * (TM * kRow);
  auto slot = [&](int c, int row) { return (c ^ (NC == 4 ? row & 15 : NC == 2 ? row >> 1 & 7 : row >> 2 & 3)) << 4; };
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

template <int G, int TT, int NT, bool GATED>
hipError_t tiled_launch(Int4GemmArgs p, hipStream_t stream) {
  constexpr int TM = 32 * TT, NC = GATED ? NT / 2 : NT;
  p.rows_over = kInt4FewRows;
  p.rows_to = INT32_MAX;
  const int out_n = GATED ? p.n / 2 : p.n;
  const int64_t fit = p.row_cap / (kInt4FewRows + 1), used = p.num_experts < fit ? p.num_experts : fit;
  const int64_t units = p.counts ? p.row_cap / TM + used : (p.row_cap + TM - 1) / TM;
  // A multiple of 8: every XCD's share rounded up.
  const int64_t tasks = (units * ((out_n + 128 * NC - 1) / (128 * NC)) + 7) / 8 * 8;
  hipLaunchKernelGGL((int4_tiled_kernel<G, TT, NT, GATED>), flat_grid(tasks), dim3(kTlThreads), 0, stream, p);
  return hipGetLastError();
}

// Expected time, us, of the forms that more than kInt4FewRows rows can take, by
// the tiles that there are for each CU (r). Tiled forms: a superstep of 256 K
// values takes 2.4 us a round of 64 x 256 tiles, 3 to 4 of 128 x 256 ones and 4.7
// to 7.3 of 128 x 512 ones (the more the fuller the chip, whose clock falls), and
// some 5 us go around it; streamed tiles of 32 x 32 take 2.5 us and 0.2 for every
// 128 K values. Measured (streamed, 64 x 256, 128 x 256, 128 x 512), us, for rows,
// K, N: 300, 6144, 1000: 30, 57, 70, 125; 70, 4096, 4096: 15, 38, 46, 79; 300,
// 2048, 7168: 56, 24, 30, 49; 300, 7168, 4096 gated: 68, 65, 83, 144; 512, 4096,
// 4096: -, 42, 51, 84; 1024, 4096, 4096: 134, 51, 54, 86; 1024, 2048, 7168: -, 41,
// 36, 52; 2048, 4096, 4096: -, 85, 70, 92; 2048, 7168, 8192: -, 276, 226, 207.
struct Int4Costs {
  double stream, small, medium, large;
};
Int4Costs int4_costs(const Int4GemmArgs& p, int out_n, int gated) {
  const double cus = device_cu_count(), blocks = (p.k + 255) / 256;
  const double experts = p.counts ? (p.num_experts < p.row_cap ? p.num_experts : p.row_cap) : 1.0;
  const double mean = p.row_cap / experts;
  // Row tiles: of one expert known, of several half a tile more than they fill.
  auto units = [&](int tm) { return p.num_experts > 1 ? experts * (mean / tm + 0.5) : ceil(p.row_cap / static_cast<double>(tm)); };
  auto cols = [&](int c) { return ceil(out_n / static_cast<double>(gated ? c / 2 : c)); };
  auto fill = [](double r) { return r < 1.0 ? r : 1.0; };
  const double rs = units(32) * cols(32) / cus, r2 = units(64) * cols(256) / cus;
  const double r4 = units(128) * cols(256) / cus, r8 = units(128) * cols(512) / cus;
  return {ceil(rs) * (2.5 + 0.4 * blocks), 5.0 + blocks * 2.4 * ceil(r2),
          5.0 + blocks * ceil(r4) * (3.0 + fill(r4)), 5.0 + blocks * ceil(r8) * (4.7 + 2.6 * fill(r8))};
}

template <int G, bool GATED>
hipError_t gemm_launch(Int4GemmArgs p, hipStream_t stream) {
  const int out_n = GATED ? p.n / 2 : p.n;
  p.vector_out = out_n % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
  // (a count past the bound is computed all the same)
  if (p.max_rows_per_expert <= kInt4FewRows) return stream_rows<G, GATED>(p, p.max_rows_per_expert, INT32_MAX, stream);
  const Int4Costs t = int4_costs(p, out_n, GATED);
  if (t.stream <= t.small && t.stream <= t.medium && t.stream <= t.large)
    return stream_rows<G, GATED>(p, p.max_rows_per_expert, INT32_MAX, stream);
  if (p.counts) {
    const hipError_t e = stream_rows<G, GATED>(p, kInt4FewRows, kInt4FewRows, stream);
    if (e != hipSuccess) return e;
  }
  if (t.small <= t.medium && t.small <= t.large) return tiled_launch<G, 2, 2, GATED>(p, stream);
  if (t.medium <= t.large) return tiled_launch<G, 4, 2, GATED>(p, stream);
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
