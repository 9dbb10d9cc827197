// The expert layer with MXFP4 activations and weights for a few tokens (at
// most kL4MaxPairs routed pairs), in two launches:
//   1. per (expert in use, 32 columns of the FC2 input): the tokens' MXFP4
//      quantization, FC1's 32 gate and 32 up rows, SiLU(gate) * up and its
//      MXFP4 quantization (one block of 32 columns per token);
//   2. per 16 output columns: FC2 for every pair and the top-k sum.
// Nothing passes between the two but the quantized FC2 input, in the caller's
// workspace, so calls may overlap on different streams.
//
// Both read each weight of the experts in use once and are bound by that:
// the weights go from global memory straight into the operands of
// v_mfma_scale_f32_16x16x128_f8f6f4, every load of a wave's K share issued
// before the first is used, and the waves of a workgroup split K.
//
// Measured, captured: 288 experts of 4096 -> 512, top 8: 15.3 us at 1 token
// (27 MB of weights), 27.2 us at 4 (about 100 MB: 3.7 TB/s over both launches,
// where a large copy runs at 4.8). Alone FC1 takes 9.8 and 16.8 us, FC2 6.1 and
// 9.8. Of the 15 us of 1 token about 6 are the bytes; the rest is two launches'
// ramps, each a chain of ids, weights, quantization, products and a reduction
// over the waves. 32 experts of 7168 -> 2048: 47 us at
// 1 token (187 MB, 4.0 TB/s). FC1 is bound by its instructions where the
// weights are in cache, so its addresses are 32-bit offsets from uniform bases
// and its tokens are found with scalar operations: with 64-bit addresses, a
// division per lane and a loop over sets of 16 tokens (which spilled) the same
// calls took 17.1, 32.8 and 53.1 us.
//
// Routing. A pair's workgroups compare its expert with those of all pairs (one
// id per lane, one ballot): the lowest pair of an expert works for all of its
// tokens, the others' workgroups leave. No table is built.
#include "device_common.h"
#include "gemm_device.h"
#include "kernels.h"
#include "mx_device.h"
#include "mx_stream.h"
#include "quant_device.h"

namespace moe {
namespace {

constexpr int kL1Threads = 512;
constexpr int kL1Waves = kL1Threads / 64;
constexpr int kL2Threads = 1024;
constexpr int kL2Waves = kL2Threads / 64;

// The r-th set bit of m (64 if there are fewer).
__device__ __forceinline__ int nth_bit(uint64_t m, int r) {
  for (int i = 0; i < r && m; ++i) m &= m - 1;
  return m ? __builtin_ctzll(m) : 64;
}

// LDS of a workgroup's tokens: codes and scale bytes, rows padded so that 16
// rows' chunks fall on distinct banks.
__host__ __device__ constexpr int l4_code_stride(int hidden) { return hidden / 2 + 16; }
__host__ __device__ constexpr int l4_scale_stride(int hidden) { return hidden / kMxBlock + 4; }

size_t l4_token_bytes(int hidden, int t_cap) {
  return static_cast<size_t>(t_cap < 16 ? t_cap : 16) * (l4_code_stride(hidden) + l4_scale_stride(hidden));
}
// What FC1 has beside them: the shares' partial sums and the tokens' pairs.
constexpr size_t kL1Lds = kL1Waves * 4 * 64 * sizeof(v4f) + 16 * sizeof(uint64_t);

__global__ __launch_bounds__(kL1Threads, 4) void layer_a4_fc1_kernel(LayerA4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];  // the tokens
  __shared__ __attribute__((aligned(16))) v4f s_part[kL1Waves][4][64];
  __shared__ uint64_t s_pairs[16];  // the tokens' pairs with the expert
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int PQ = a.t_cap * a.topk;
  const int pair = blockIdx.y;
  // Which expert, and for which pairs.
  const int t_live = clamp_live(a.t_live_dev, a.t_cap);
  const int id = lane < PQ ? a.ids[lane] - a.expert_start : -1;
  const int e = __builtin_amdgcn_readlane(id, pair);
  const uint64_t mine = __ballot(lane < t_live * a.topk && id == e);
  if (static_cast<unsigned>(e) >= static_cast<unsigned>(a.num_experts) || mine == 0 ||
      __builtin_ctzll(mine) != pair)
    return;
  // Their tokens: a token may have the expert more than once, and its row is
  // computed once. Sixteen tokens per workgroup (a loop here costs spilled
  // registers).
  const uint64_t token_bits = ~uint64_t{0} >> (64 - a.topk);
  uint64_t left = mine;
  auto next_token = [&](int* t) {
    *t = static_cast<int>(static_cast<unsigned>(__builtin_ctzll(left)) * a.token_of >> 16);
    const uint64_t of = left & token_bits << (*t * a.topk);
    left ^= of;
    return of;  // its pairs with this expert
  };
  int t;
  for (unsigned i = 0; i < 16 * blockIdx.z && left; ++i) next_token(&t);
  if (left == 0) return;
  const uint64_t pass = left;
  int nt = 0;
  while (left && nt < 16) {
    next_token(&t);
    ++nt;
  }
  left = pass;

  const unsigned H = a.hidden, I = a.inter;
  const int col0 = blockIdx.x * 32;
  const int chunks = (H + 255) / 256;
  const int ch0 = l4_split(chunks, wave, kL1Waves), ch1 = l4_split(chunks, wave + 1, kL1Waves);
  // Row tiles: gate rows col0 .. +15, +16 .. +31, then the up rows.
  const int64_t first = static_cast<int64_t>(e) * 2 * I + col0;
  const uint8_t* wb[4];
  const uint8_t* sb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = first + (i >> 1) * I + (i & 1) * 16;
    wb[i] = a.w1 + row * (H / 2);
    sb[i] = a.w1_scales + row * (H / kMxBlock);
  }
  const uint32_t wrow = r16 * (H / 2), srow = r16 * (H / kMxBlock);
  const int XS = l4_code_stride(H), XB = l4_scale_stride(H);
  const int width = min(a.t_cap, 16);  // tokens of a workgroup, at most
  uint8_t* s_x = s_dyn;
  uint8_t* s_xs = s_dyn + width * XS;

  // The first two chunks' weights go out before anything waits. Chunks past
  // the share load its last one, unused.
  L4Frag w[2][4];
  auto load = [&](int ch, L4Frag (&f)[4]) {
    const int c = min(ch, max(ch1 - 1, 0));
    const L4Lane l = l4_lane(g, c * 256 + 128 >= H);
#pragma unroll
    for (int i = 0; i < 4; ++i) l4_load(f[i], wb[i], wrow, sb[i], srow, c, l);
  };
  // The tokens to LDS, 8 values per thread and step. The loads of the
  // first two tokens' first two steps go out ahead of the weights (loads
  // return in order).
  const int per = H / 8;
  auto row_of = [&](int t) { return a.x + static_cast<int64_t>(t) * H; };
  auto load_item = [&](const uint16_t* row, int c) {
    return *reinterpret_cast<const uint4*>(row + min(c, per - 1) * 8);
  };
  auto store_item = [&](int k, int c, uint4 raw) {
    uint32_t byte;
    const uint32_t codes = mx_quantize8_bf16(raw, &byte);
    if (c >= per) return;  // whole quads: per is a multiple of 16
    *reinterpret_cast<uint32_t*>(s_x + k * XS + c * 4) = codes;
    if ((c & 3) == 0) s_xs[k * XB + (c >> 2)] = static_cast<uint8_t>(byte);
  };
  int tok0;
  const uint64_t of0 = next_token(&tok0);
  int tok1 = tok0;
  const uint64_t of1 = nt > 1 ? next_token(&tok1) : 0;
  const uint16_t *row0 = row_of(tok0), *row1 = row_of(tok1);
  const uint4 raw00 = load_item(row0, tid), raw01 = load_item(row0, tid + kL1Threads);
  const uint4 raw10 = load_item(row1, tid), raw11 = load_item(row1, tid + kL1Threads);
  __builtin_amdgcn_sched_barrier(0);
  load(ch0, w[0]);
  load(ch0 + 1, w[1]);
  __builtin_amdgcn_sched_barrier(0);
  store_item(0, tid, raw00);
  if (per > kL1Threads) store_item(0, tid + kL1Threads, raw01);
  if (nt > 1) {
    store_item(1, tid, raw10);
    if (per > kL1Threads) store_item(1, tid + kL1Threads, raw11);
  }
  if (tid == 0) {
    s_pairs[0] = of0;
    s_pairs[1] = of1;
  }
  for (int k = per > 2 * kL1Threads ? 0 : 2; k < nt; ++k) {
    uint64_t of = 0;
    if (k >= 2) of = next_token(&t);
    const uint16_t* row = row_of(k == 0 ? tok0 : (k == 1 ? tok1 : t));
    for (int c = k < 2 ? tid + 2 * kL1Threads : tid; c - tid < per; c += 2 * kL1Threads) {
      const uint4 r0 = load_item(row, c), r1 = load_item(row, c + kL1Threads);
      store_item(k, c, r0);
      if (c - tid + kL1Threads < per) store_item(k, c + kL1Threads, r1);
    }
    if (tid == 0 && k >= 2) s_pairs[k] = of;
  }
  lds_barrier();  // (leaves the weights in flight)
  v4f acc[4] = {};
  // Columns past the tokens repeat the last.
  const uint32_t xrow = min(r16, nt - 1) * XS, xsrow = min(r16, nt - 1) * XB;
  auto products = [&](int ch, const L4Frag (&f)[4]) {
    const L4Lane l = l4_lane(g, ch * 256 + 128 >= H);
    L4Frag x;
    l4_load(x, s_x, xrow, s_xs, xsrow, ch, l);
    const uint32_t xs = l4_scales(x, l), m = l.second;
    const uint4 x1 = {x.c[1].x & m, x.c[1].y & m, x.c[1].z & m, x.c[1].w & m};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = mfma_l4<0>(f[i].c[0], l4_scales(f[i], l), x.c[0], xs, acc[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = mfma_l4<1>(f[i].c[1], l4_scales(f[i], l), x1, xs, acc[i]);
  };
  int ch = ch0;
  for (; ch + 2 < ch1; ch += 2) {
    products(ch, w[0]);
    load(ch + 2, w[0]);
    products(ch + 1, w[1]);
    load(ch + 3, w[1]);
  }
  if (ch < ch1) products(ch, w[0]);
  if (ch + 1 < ch1) products(ch + 1, w[1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) s_part[wave][i][lane] = acc[i];
  __syncthreads();
  // The shares add in wave order, a value quartet per thread.
  if (tid < 256) {
    v4f sum = s_part[0][tid >> 6][lane];
#pragma unroll
    for (int w = 1; w < kL1Waves; ++w) sum += s_part[w][tid >> 6][lane];
    s_part[0][tid >> 6][lane] = sum;
  }
  __syncthreads();
  // Thread (token, column): 32 lanes hold a token's 32 columns. Value
  // (column c, token k) of a tile pair lies in tile c / 16, lane 16 (c % 16 /
  // 4) + k, element c % 4.
  const int k = tid >> 5, c = tid & 31;
  if (k < nt) {
    const int src = 16 * ((c & 15) >> 2) + k;
    const uint2 b = pack_bf16x4(v4f{s_part[0][c >> 4][src][c & 3], s_part[0][2 + (c >> 4)][src][c & 3], 0.0f, 0.0f});  // C1 is BF16
    const float y = swiglu_any<true>(a.act, bf16_to_f32(b.x & 0xFFFFu), bf16_to_f32(b.x >> 16), a.act_limit, a.rounding);
    // The block's largest magnitude, over the 32 lanes that hold it (all or
    // none of them are here).
    uint32_t amax = quad_max_u32(__float_as_uint(y) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      const uint32_t o = __shfl_xor(static_cast<int>(amax), d, 64);
      amax = o > amax ? o : amax;
    }
    const uint32_t byte = mx_scale_byte(amax);
    // Lane c even packs columns c and c + 1; every eighth stores four bytes.
    const float y1 = __shfl_xor(y, 1, 64);
    uint32_t code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y, y1, mx_scale_float(byte), 0) & 0xFFu;
    if (byte == 255u) code = 0;
    code |= __shfl_xor(static_cast<int>(code), 2, 64) << 8;
    code |= __shfl_xor(static_cast<int>(code), 4, 64) << 16;
    for (uint64_t to = s_pairs[k]; to; to &= to - 1) {
      const int64_t at = static_cast<int64_t>(__builtin_ctzll(to)) * I + col0;
      if ((c & 7) == 0) *reinterpret_cast<uint32_t*>(a.hq + at / 2 + c / 2) = code;
      if (c == 0) a.hs[at / kMxBlock] = static_cast<uint8_t>(byte);
    }
  }
}

// A wave task is (expert in use, a share of K); the shares of a pair's row
// add in order before its BF16 rounding, then out[t] = sum over ascending k of
// w[t, k] * row, in fp32.
__global__ __launch_bounds__(kL2Threads, 4) void layer_a4_fc2_kernel(LayerA4Args a) {
  extern __shared__ __attribute__((aligned(16))) float s_slot[];  // [share][pair][16 columns]
  __shared__ float s_w[64];
  __shared__ int s_ok[64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int TK = a.topk, PQ = a.t_cap * TK;
  const int t_live = clamp_live(a.t_live_dev, a.t_cap);
  const int id = lane < PQ ? a.ids[lane] - a.expert_start : -1;
  const float tw = lane < PQ ? a.topk_w[lane] : 0.0f;
  const bool ok = lane < t_live * TK && static_cast<unsigned>(id) < static_cast<unsigned>(a.num_experts);
  // Pairs with this lane's expert: one ballot per bit of an expert id.
  uint64_t eq = __ballot(ok);
  for (int b = 31 - __builtin_clz(a.num_experts | 1); b >= 0; --b) {
    const bool bit = (id >> b) & 1;
    const uint64_t m = __ballot(ok && bit);
    eq &= bit ? m : ~m;
  }
  const uint64_t below = (uint64_t{1} << lane) - 1;
  const uint64_t leaders = __ballot(ok && (eq & below) == 0);
  const int n_lead = __popcll(leaders);
  if (wave == 0) {
    s_w[lane] = tw;
    s_ok[lane] = ok;
  }
  const int H = a.hidden, I = a.inter;
  const int n0 = blockIdx.x * 16;
  const int chunks = (I + 255) / 256;
  int S = 1;
  while (max(n_lead, 1) * S * 2 <= kL2Waves && S * 2 <= chunks) S *= 2;
  for (int task = wave; task < n_lead * S; task += kL2Waves) {
    const int share = task & (S - 1);
    const int lead = nth_bit(leaders, task / S);
    const int e = __builtin_amdgcn_readlane(id, lead);
    const uint64_t mine = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(eq), lead))) |
                          static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(eq >> 32), lead))) << 32;
    const int n_tok = __popcll(mine);
    const int64_t row = static_cast<int64_t>(e) * H + n0;
    const uint8_t* wb = a.w2 + row * (I / 2);
    const uint8_t* sb = a.w2_scales + row * (I / kMxBlock);
    const uint32_t wrow = r16 * (I / 2), srow = r16 * (I / kMxBlock);
    const int ch0 = l4_split(chunks, share, S), ch1 = l4_split(chunks, share + 1, S);
    for (int t0 = 0; t0 < n_tok; t0 += 16) {
      const int q = nth_bit(mine, t0 + min(r16, n_tok - t0 - 1));
      const uint32_t xrow = q * (I / 2), xsrow = q * (I / kMxBlock);
      v4f acc = {};
      // Two chunks' loads together (past the share: its last one, unused).
      for (int ch = ch0; ch < ch1; ch += 2) {
        const int c1 = min(ch + 1, ch1 - 1);
        const L4Lane l0 = l4_lane(g, ch * 256 + 128 >= I), l1 = l4_lane(g, c1 * 256 + 128 >= I);
        L4Frag w[2], x[2];
        l4_load(w[0], wb, wrow, sb, srow, ch, l0);
        l4_load(w[1], wb, wrow, sb, srow, c1, l1);
        l4_load(x[0], a.hq, xrow, a.hs, xsrow, ch, l0);
        l4_load(x[1], a.hq, xrow, a.hs, xsrow, c1, l1);
        auto products = [&](int u, const L4Lane& l) {
          const uint32_t ws = l4_scales(w[u], l), xs = l4_scales(x[u], l), m = l.second;
          const uint4 x1 = {x[u].c[1].x & m, x[u].c[1].y & m, x[u].c[1].z & m, x[u].c[1].w & m};
          acc = mfma_l4<0>(w[u].c[0], ws, x[u].c[0], xs, acc);
          acc = mfma_l4<1>(w[u].c[1], ws, x1, xs, acc);
        };
        products(0, l0);
        if (ch + 1 < ch1) products(1, l1);
      }
      if (t0 + r16 < n_tok)
        *reinterpret_cast<v4f*>(s_slot + (share * PQ + q) * 16 + 4 * g) = acc;
    }
  }
  __syncthreads();
  for (int i = tid; i < t_live * 8; i += kL2Threads) {
    const int t = i >> 3, c = (i & 7) * 2;
    float o0 = 0.0f, o1 = 0.0f;
    for (int k0 = 0; k0 < TK; k0 += 4) {  // four pairs' reads together
      float y0[4], y1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y0[j] = y1[j] = 0.0f;
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = t * TK + min(k0 + j, TK - 1);
          const float2 v = *reinterpret_cast<const float2*>(s_slot + (s * PQ + q) * 16 + c);
          y0[j] += v.x;
          y1[j] += v.y;
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = t * TK + min(k0 + j, TK - 1);
        if (k0 + j >= TK || !s_ok[q]) continue;
        const uint2 b = pack_bf16x4(v4f{y0[j], y1[j], 0.0f, 0.0f});
        o0 = fmaf(s_w[q], bf16_to_f32(b.x & 0xFFFFu), o0);
        o1 = fmaf(s_w[q], bf16_to_f32(b.x >> 16), o1);
      }
    }
    const uint2 b = pack_bf16x4(v4f{o0, o1, 0.0f, 0.0f});
    *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(t) * H + n0 + c) = b.x;
  }
}

}  // namespace

bool layer_a4_fits(int t_cap, int topk, int hidden) {
  const int64_t pairs = static_cast<int64_t>(t_cap) * topk;
  return pairs >= 1 && pairs <= kL4MaxPairs && l4_token_bytes(hidden, t_cap) + kL1Lds <= kLdsBytes;
}

hipError_t launch_layer_a4(const LayerA4Args& a, hipStream_t stream) {
  const int pairs = a.t_cap * a.topk;
  if (!layer_a4_fits(a.t_cap, a.topk, a.hidden)) return hipErrorInvalidValue;
  LayerA4Args p = a;
  p.token_of = 65536 / a.topk + 1;  // q * token_of >> 16 is q / topk for q < 64, topk <= 64
  hipLaunchKernelGGL(layer_a4_fc1_kernel,
                     dim3(static_cast<unsigned>(a.inter / 32), static_cast<unsigned>(pairs),
                          static_cast<unsigned>((a.t_cap + 15) / 16)),
                     dim3(kL1Threads), l4_token_bytes(a.hidden, a.t_cap), stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // The kernel's shares at their most, with one expert in use: 16 columns of
  // them per pair.
  const int chunks = (a.inter + 255) / 256;
  int shares = 1;
  while (shares * 2 <= kL2Waves && shares * 2 <= chunks) shares *= 2;
  const size_t lds = static_cast<size_t>(shares) * pairs * 16 * sizeof(float);
  hipLaunchKernelGGL(layer_a4_fc2_kernel, dim3(static_cast<unsigned>(a.hidden / 16)), dim3(kL2Threads), lds, stream, a);
  return hipGetLastError();
}

}  // namespace moe
