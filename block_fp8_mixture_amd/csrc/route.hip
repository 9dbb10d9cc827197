// Top-k routing from router logits: scores (softmax or sigmoid), an optional
// selection bias, expert groups, the top-k of each token in descending order
// and their weights.
//
// One wave per token holds the token's row in registers (expert v * 64 +
// lane in slot v). Experts are ordered by a 64-bit key, larger first, ties to
// the lower index:
//  - without a bias by the logit itself: its float's order in the high word,
//    the complemented index in the low one;
//  - with a bias by score + bias in 64 bits (two experts whose scores differ
//    past 32 bits must not change places), the index apart.
// Key 0 is an expert that is never picked (logit -inf or NaN, a group that
// lost). Each round takes the wave's largest key; lane r keeps the r-th
// expert's score, and the weights form at the end. Scores are computed in 64
// bits and rounded once, as weights.
#include <hip/hip_fp16.h>

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
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  const uint32_t lo = dpp32<CTRL>(0, static_cast<uint32_t>(v));
  const uint32_t hi = dpp32<CTRL>(0, static_cast<uint32_t>(v >> 32));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The wave's largest key, in every lane (a uniform value).
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  v = max64(v, dpp64<0xB1>(v));   // quad_perm [1,0,3,2]
  v = max64(v, dpp64<0x4E>(v));   // quad_perm [2,3,0,1]
  v = max64(v, dpp64<0x141>(v));  // row_half_mirror
  v = max64(v, dpp64<0x140>(v));  // row_mirror
  return max64(max64(lane64(v, 0), lane64(v, 16)), max64(lane64(v, 32), lane64(v, 48)));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (TYPE == kLogitF32) return static_cast<const float*>(p)[i];
  else if constexpr (TYPE == kLogitBf16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

// V: experts per lane. GROUPED: num_groups > 1.
template <int TYPE, int V, bool BIAS, bool GROUPED>
__global__ __launch_bounds__(kRtThreads) void route_kernel(RouteArgs a) {
  __shared__ uint64_t s_key[GROUPED ? kRtWaves : 1][GROUPED ? V * 64 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kRtWaves + wave;
  if (t >= clamp_live(a.t_live_dev, a.t_cap)) return;
  const int E = a.num_experts;
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    x[v] = e < E ? load_logit<TYPE>(a.logits, t * a.ld + e) : -INFINITY;
    x[v] = x[v] == x[v] ? fminf(x[v], 3.40282346638528859812e38f) : -INFINITY;
  }
  // Scores of every expert where the order, a group's value or the softmax's
  // sum over all experts needs them; otherwise only the picked ones' below.
  const bool all_scores = BIAS || (GROUPED && a.group_top == 2) || (a.score == kSoftmax && !a.renormalize);
  double top = 0.0;
  if (a.score == kSoftmax) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = group_max<64>(m);
    top = m > -INFINITY ? m : 0.0;
  }
  // Up to the softmax's common factor 1 / sum, which `norm` brings in.
  auto raw_score = [&](float f) {
    if (a.score == kSoftmax) return exp(static_cast<double>(f) - top);
    return 1.0 / (1.0 + exp(-static_cast<double>(f)));
  };
  double norm = 1.0;
  double p[V];
  if (all_scores) {
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = raw_score(x[v]);
      sum += p[v];
    }
    if (a.score == kSoftmax) {
      sum = wave_sum(sum);
      norm = sum > 0.0 ? sum : 1.0;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] /= norm;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 0.0;
  }

  // Keys. Without a bias and in the grouped case by score, the group's value
  // takes the score's key and the pick the logit's.
  uint64_t key[V];
  auto logit_key = [&](int v) -> uint64_t {
    const int e = v * 64 + lane;
    return x[v] > -INFINITY ? static_cast<uint64_t>(ordered32(x[v])) << 32 | static_cast<uint32_t>(~e) : 0;
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (BIAS) {
      const int e = v * 64 + lane;
      const double s = e < E && x[v] > -INFINITY ? p[v] + static_cast<double>(a.bias[e]) : -INFINITY;
      key[v] = s > -INFINITY ? ordered64(s) : 0;  // a NaN bias never wins
    } else {
      key[v] = logit_key(v);
    }
  }

  if constexpr (GROUPED) {
    const int G = a.num_groups, size = E / G;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint64_t k = key[v];
      if (!BIAS && a.group_top == 2) k = k ? ordered64(p[v]) : 0;
      s_key[wave][v * 64 + lane] = k;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's own LDS writes, in order
    // Lane g: the two largest of group g (other lanes: nothing).
    uint64_t b0 = 0, b1 = 0;
    if (lane < G)
      for (int i = 0; i < size; ++i) {
        const uint64_t k = s_key[wave][lane * size + i];
        if (k > b0) {
          b1 = b0;
          b0 = k;
        } else if (k > b1) {
          b1 = k;
        }
      }
    uint64_t value;
    if (a.group_top == 2) {
      value = b0 == 0 ? 0 : (b1 == 0 ? b0 : ordered64(from_ordered64(b0) + from_ordered64(b1)));
    } else {
      value = BIAS ? b0 : b0 >> 32;  // by the logit alone: the index is no part of a group's value
    }
    // A group is kept if fewer than top_groups are better (larger, or equal
    // with a lower index).
    int better = 0;
    for (int h = 0; h < G; ++h) {
      const uint64_t o = lane64(value, h);
      better += o > value || (o == value && h < lane);
    }
    const uint64_t kept = __ballot(lane < G && better < a.top_groups);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      if (e < E && !((kept >> (e / size)) & 1)) key[v] = 0;
    }
  }

  // The picks, best first; lane r keeps the r-th.
  int my_id = -1;
  double my_p = 0.0;
  for (int r = 0; r < a.topk; ++r) {
    uint64_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max64(best, key[v]);
    best = wave_max64(best);
    if (best == 0) break;  // nothing left to pick
    int e;
    if constexpr (BIAS) {
      // The lowest index that has this key: slots ascend, then lanes.
      e = -1;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint64_t m = __ballot(key[v] == best);
        if (e < 0 && m) e = v * 64 + __builtin_ctzll(m);
      }
    } else {
      e = static_cast<int>(~static_cast<uint32_t>(best));
    }
    e = __builtin_amdgcn_readfirstlane(e);
    double pv = 0.0;
    float xv = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if ((e >> 6) == v) {
        pv = p[v];
        xv = x[v];
        if ((e & 63) == lane) key[v] = 0;
      }
    }
    const uint64_t pb = lane64(static_cast<uint64_t>(__double_as_longlong(pv)), e & 63);
    const float xb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(xv), e & 63));
    if (lane == r) {
      my_id = e;
      my_p = __longlong_as_double(static_cast<long long>(pb));
      if (!all_scores) my_p = xb;  // the logit for now
    }
  }
  if (!all_scores) my_p = my_id >= 0 ? raw_score(static_cast<float>(my_p)) : 0.0;
  double w = my_p;
  if (a.renormalize) {
    const double total = wave_sum(my_p);
    w = total > 0.0 ? my_p / total : 0.0;
  }
  if (lane < a.topk) {
    const int64_t at = static_cast<int64_t>(t) * a.topk + lane;
    a.ids[at] = my_id;
    a.weights[at] = static_cast<float>(w * static_cast<double>(a.scale));
  }
}

template <int TYPE, int V>
void route_bg(const RouteArgs& a, dim3 grid, hipStream_t stream) {
  const bool grouped = a.num_groups > 1;
  if (a.bias && grouped)
    hipLaunchKernelGGL((route_kernel<TYPE, V, true, true>), grid, dim3(kRtThreads), 0, stream, a);
  else if (a.bias)
    hipLaunchKernelGGL((route_kernel<TYPE, V, true, false>), grid, dim3(kRtThreads), 0, stream, a);
  else if (grouped)
    hipLaunchKernelGGL((route_kernel<TYPE, V, false, true>), grid, dim3(kRtThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((route_kernel<TYPE, V, false, false>), grid, dim3(kRtThreads), 0, stream, a);
}

template <int TYPE>
void route_v(const RouteArgs& a, dim3 grid, hipStream_t stream) {
  if (a.num_experts <= 64)
    route_bg<TYPE, 1>(a, grid, stream);
  else if (a.num_experts <= 128)
    route_bg<TYPE, 2>(a, grid, stream);
  else if (a.num_experts <= 256)
    route_bg<TYPE, 4>(a, grid, stream);
  else if (a.num_experts <= 512)
    route_bg<TYPE, 8>(a, grid, stream);
  else
    route_bg<TYPE, 16>(a, grid, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.t_cap) + kRtWaves - 1) / kRtWaves));
  if (a.logit_type == kLogitF32)
    route_v<kLogitF32>(a, grid, stream);
  else if (a.logit_type == kLogitBf16)
    route_v<kLogitBf16>(a, grid, stream);
  else
    route_v<kLogitF16>(a, grid, stream);
  return hipGetLastError();
}

}  // namespace moe
