// Top-k routing from router logits: scores (softmax or sigmoid), an optional
// selection bias, expert groups, the top-k of each token in descending order
// and their weights.
//
// L lanes per token (16 or 64) hold the token's row in registers, expert
// v * L + lane in slot v. Experts are ordered by a key whose unsigned order is
// theirs, ties to the lower index: without a bias the logit's 32 bits, with one
// score + bias in 64 bits (two experts whose scores differ past 32 bits must
// not change places). High word 0 is an expert that is never picked (logit
// -inf or NaN, a group that lost). Each round takes the largest key over the
// lanes, high words first (v_max_u32 with a DPP operand: one instruction a
// step), low words only where high words are equal, then the lowest index that
// has it; lane r keeps the r-th expert. Its score is computed anew at the end
// (one per lane) rather than carried through the rounds. Scores are computed
// in 64 bits and rounded once, as weights.
//
// Bound by its instructions and, for few tokens, by one wave's latency: 4.6 us
// captured for 1 token of 288 experts, 11.5 us for 4096 tokens of 256 with a
// bias and 8 groups (4 MB, 1 us to read). Of those 11.5 the eight rounds take
// 3.2 (0.4 each, top 8 against top 1), the 64-bit exponentials and divisions
// 1.5, the groups 1.2. With 64-bit
// maxima in the rounds, a score carried through them and one lane per group
// the same calls took 5.5 and 13.9 us.
#include <hip/hip_fp16.h>

#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRtThreads = 256;
constexpr int kRtWaves = kRtThreads / 64;

// Float and double bits in an order that unsigned comparison follows.
__device__ __forceinline__ uint32_t ordered32(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 equals +0
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered64(double d) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(d + 0.0));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_ordered64(uint64_t k) {
  const uint64_t u = k >> 63 ? k ^ 0x8000000000000000ull : ~k;
  return __longlong_as_double(static_cast<long long>(u));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t old, uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(old), static_cast<int>(v),
                                                           CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float from_ordered32(uint32_t k) {
  return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint32_t lane32(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
  return static_cast<uint64_t>(lane32(static_cast<uint32_t>(v >> 32), lane)) << 32 |
         lane32(static_cast<uint32_t>(v), lane);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t max32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t min32(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Over a token's L lanes, the result in each: quad_perm [1,0,3,2], [2,3,0,1],
// row_half_mirror, row_mirror, then the rows of 16 (uniform for L = 64).
template <int L>
__device__ __forceinline__ uint32_t token_max32(uint32_t v) {
  v = max32(v, dpp32<0xB1>(0, v));
  v = max32(v, dpp32<0x4E>(0, v));
  v = max32(v, dpp32<0x141>(0, v));
  v = max32(v, dpp32<0x140>(0, v));
  if constexpr (L == 16) return v;
  return max32(max32(lane32(v, 0), lane32(v, 16)), max32(lane32(v, 32), lane32(v, 48)));
}
template <int L>
__device__ __forceinline__ double token_sum(double v) {
  auto step = [&](auto ctrl) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t o = static_cast<uint64_t>(dpp32<decltype(ctrl)::value>(0, static_cast<uint32_t>(u >> 32))) << 32 |
                       dpp32<decltype(ctrl)::value>(0, static_cast<uint32_t>(u));
    v += __longlong_as_double(static_cast<long long>(o));
  };
  step(std::integral_constant<int, 0xB1>());
  step(std::integral_constant<int, 0x4E>());
  step(std::integral_constant<int, 0x141>());
  step(std::integral_constant<int, 0x140>());
  if constexpr (L == 16) return v;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  auto row = [&](int r) { return __longlong_as_double(static_cast<long long>(lane64(u, 16 * r))); };
  return (row(0) + row(1)) + (row(2) + row(3));
}

__device__ __forceinline__ float load_logit(int type, const void* p, int64_t i) {
  if (type == kLogitF32) return static_cast<const float*>(p)[i];
  if (type == kLogitBf16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// Keys of a token in LDS, spread so that the groups' scans meet few banks.
__host__ __device__ constexpr int key_slot(int e) { return e + (e >> 5) * 8; }

// V: experts per lane. GROUPED: num_groups > 1.
template <int L, int V, bool BIAS, bool GROUPED>
__global__ __launch_bounds__(kRtThreads) void route_kernel(RouteArgs a) {
  constexpr int T = 64 / L;  // tokens per wave
  __shared__ uint64_t s_key[GROUPED ? kRtWaves * T : 1][GROUPED ? key_slot(V * L) : 1];
  const int lane = threadIdx.x & 63, sub = lane & (L - 1);
  const int t_live = clamp_live(a.t_live_dev, a.t_cap);
  const int slot = threadIdx.x / L;  // of the workgroup's tokens
  const int64_t t = flat_block() * (kRtWaves * T) + slot;
  if (t - lane / L >= t_live) return;  // the wave's first token
  const int E = t < t_live ? a.num_experts : 0;
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + sub;
    x[v] = e < E ? load_logit(a.logit_type, a.logits, t * a.ld + e) : -INFINITY;
  }
  uint32_t hi[V], lo[BIAS ? V : 1];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = x[v] == x[v] ? fminf(x[v], 3.40282346638528859812e38f) : -INFINITY;
    hi[v] = x[v] > -INFINITY ? ordered32(x[v]) : 0u;
  }
  // Scores of every expert where the order, a group's value or the softmax's
  // sum over all experts needs them; otherwise only the picked ones' below.
  const bool all_scores = BIAS || (GROUPED && a.group_top == 2) || (a.score == kSoftmax && !a.renormalize);
  double top = 0.0;
  if (a.score == kSoftmax) {
    uint32_t m = hi[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max32(m, hi[v]);
    m = token_max32<L>(m);
    top = m ? from_ordered32(m) : 0.0f;
  }
  // Up to the softmax's common factor 1 / sum, which `norm` brings in.
  auto raw_score = [&](float f) {
    if (a.score == kSoftmax) return exp(static_cast<double>(f) - top);
    return 1.0 / (1.0 + exp(-static_cast<double>(f)));
  };
  double norm = 1.0;
  [[maybe_unused]] double p[V];
  if (all_scores) {
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = raw_score(x[v]);
      sum += p[v];
    }
    if (a.score == kSoftmax) {
      sum = token_sum<L>(sum);
      norm = sum > 0.0 ? sum : 1.0;
      if constexpr (BIAS || GROUPED) {
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] /= norm;
      }
    }
  }
  if constexpr (BIAS) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      const double s = e < E && hi[v] ? p[v] + static_cast<double>(a.bias[e]) : -INFINITY;
      const uint64_t k = s > -INFINITY ? ordered64(s) : 0;  // a NaN bias never wins
      hi[v] = static_cast<uint32_t>(k >> 32);
      lo[v] = static_cast<uint32_t>(k);
    }
  }

  if constexpr (GROUPED) {
    const int G = a.num_groups, size = a.num_experts / G;
    const int shift = a.group_shift;  // 2^shift lanes per group
    uint64_t* keys = s_key[slot];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint64_t k;
      if constexpr (BIAS) k = static_cast<uint64_t>(hi[v]) << 32 | lo[v];
      else if (a.group_top == 2) k = hi[v] ? ordered64(p[v]) : 0;
      else k = hi[v];
      keys[key_slot(v * L + sub)] = k;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's own LDS writes, in order
    // The two largest of the lane's group: a share per lane, then joined.
    const int g = sub >> shift, part = sub & ((1 << shift) - 1);
    uint64_t b0 = 0, b1 = 0;
    if (g < G)
      for (int i = part; i < size; i += 1 << shift) {
        const uint64_t k = keys[key_slot(g * size + i)];
        b1 = max64(b1, min64(b0, k));
        b0 = max64(b0, k);
      }
    for (int d = 1; d < 1 << shift; d <<= 1) {
      const uint64_t c0 = __shfl_xor(static_cast<unsigned long long>(b0), d, 64);
      const uint64_t c1 = __shfl_xor(static_cast<unsigned long long>(b1), d, 64);
      b1 = max64(min64(b0, c0), max64(b1, c1));
      b0 = max64(b0, c0);
    }
    uint64_t value = b0;  // of group_top 1 without a bias: the logit's order
    if (a.group_top == 2 && b1 != 0) value = ordered64(from_ordered64(b0) + from_ordered64(b1));
    // A group is kept if fewer than top_groups are better (larger, or equal
    // with a lower index).
    int better = 0;
    for (int h = 0; h < G; ++h) {
      uint64_t o;
      if constexpr (L == 64) o = lane64(value, h << shift);
      else o = __shfl(static_cast<unsigned long long>(value), (lane & ~(L - 1)) + (h << shift), 64);
      better += o > value || (o == value && h < g);
    }
    const uint64_t kept = __ballot(g < G && better < a.top_groups) >> (lane & ~(L - 1));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int of = (v * L + sub) * a.group_of >> 20;
      if (!((kept >> (of << shift & 63)) & 1)) hi[v] = 0;
    }
  }

  // The picks, best first; lane r keeps the r-th.
  int my_id = -1;
  for (int r = 0; r < a.topk; ++r) {
    uint32_t best = hi[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max32(best, hi[v]);
    best = token_max32<L>(best);
    if (__ballot(best != 0) == 0) break;  // nothing left to pick
    // Ties: the largest low word, then the lowest index (as its complement, so
    // that 0 is none).
    uint32_t low = 0;
    if constexpr (BIAS) {
#pragma unroll
      for (int v = 0; v < V; ++v) low = max32(low, hi[v] == best ? lo[v] : 0u);
      low = token_max32<L>(low);
    }
    uint32_t first = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) {
      bool is = hi[v] == best;
      if constexpr (BIAS) is = is && lo[v] == low;
      first = is ? ~static_cast<uint32_t>(v * L + sub) : first;
    }
    const int e = static_cast<int>(~token_max32<L>(first));
#pragma unroll
    for (int v = 0; v < V; ++v) hi[v] = v * L + sub == e ? 0u : hi[v];
    if (sub == r && best != 0) my_id = e;
  }
  // The picked expert's logit, from the lane that holds it.
  const int from = (lane & ~(L - 1)) + (max(my_id, 0) & (L - 1));
  float mine = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float o = __shfl(x[v], from, 64);
    mine = max(my_id, 0) / L == v ? o : mine;
  }
  double w = my_id >= 0 ? raw_score(mine) / norm : 0.0;
  if (a.renormalize) {
    const double total = token_sum<L>(w);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (t < t_live && sub < a.topk) {
    const int64_t at = t * a.topk + sub;
    a.ids[at] = my_id;
    a.weights[at] = static_cast<float>(w * static_cast<double>(a.scale));
  }
}

template <int L, int V>
void route_bg(const RouteArgs& a, hipStream_t stream) {
  const int tokens = kRtThreads / L;  // of a workgroup
  const dim3 grid = flat_grid((static_cast<int64_t>(a.t_cap) + tokens - 1) / tokens);
  const bool grouped = a.num_groups > 1;
  if (a.bias && grouped)
    hipLaunchKernelGGL((route_kernel<L, V, true, true>), grid, dim3(kRtThreads), 0, stream, a);
  else if (a.bias)
    hipLaunchKernelGGL((route_kernel<L, V, true, false>), grid, dim3(kRtThreads), 0, stream, a);
  else if (grouped)
    hipLaunchKernelGGL((route_kernel<L, V, false, true>), grid, dim3(kRtThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((route_kernel<L, V, false, false>), grid, dim3(kRtThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, hipStream_t stream) {
  RouteArgs a = args;
  const int E = a.num_experts;
  // 16 lanes per token, four tokens per wave, need a quarter of the waves and
  // little more than one row of 64's instructions each; 64 lanes keep more
  // waves in flight. us captured, 16 / 64 lanes (softmax, top 2, 6 or 8):
  //   8 experts: 2.5 / 2.5 at 1 token, 2.9 / 3.8 at 4096, 6.8 / 24 at 65536
  //   64: 3.4 / 3.1, 3.8 / 4.8, 13 / 37;  128: 5.2 / 5.6 at 4096, 7.3 / 14 at 16384
  //   256: 6.7 / 6.7 at 4096, 7.6 / 9.9 at 8192, 32 / 57 at 65536; with a bias
  //   and groups by their two best 14.0 / 11.5 at 4096, 21 / 28 at 16384
  const bool narrow = (E <= 64 || (E <= 256 && a.t_cap >= 8192)) && a.topk <= 16 && a.num_groups <= 16;
  const int lanes = narrow ? 16 : 64;
  a.group_shift = 0;
  while (a.num_groups << (a.group_shift + 1) <= lanes) ++a.group_shift;
  a.group_of = (1 << 20) / (E / a.num_groups) + 1;  // e * group_of >> 20 is e / size for e < 1024, size <= 512
  if (narrow && E <= 16)
    route_bg<16, 1>(a, stream);
  else if (narrow && E <= 32)
    route_bg<16, 2>(a, stream);
  else if (narrow && E <= 64)
    route_bg<16, 4>(a, stream);
  else if (narrow && E <= 128)
    route_bg<16, 8>(a, stream);
  else if (narrow)
    route_bg<16, 16>(a, stream);
  else if (E <= 64)
    route_bg<64, 1>(a, stream);
  else if (E <= 128)
    route_bg<64, 2>(a, stream);
  else if (E <= 256)
    route_bg<64, 4>(a, stream);
  else if (E <= 512)
    route_bg<64, 8>(a, stream);
  else
    route_bg<64, 16>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
