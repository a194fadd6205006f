// MoE router: the topk largest logits of every token and their softmax
// weights, and the gradient of those weights with respect to the logits.
//
//   chosen e_0, e_1, ..: logits descending, equal logits by ascending id
//   normalise: w_k = exp(z[e_k] - z[e_0]) / sum over the chosen
//   else:      w_k = exp(z[e_k] - z[e_0]) / sum over all experts
//   dz[e] = q_e ([e = e_k] dw_k - sum_j w_j dw_j), q the softmax that made w
//
// One wave per token, experts spread over its lanes, V per lane. All sums
// are float32.
#include "device.h"
#include "train.h"

namespace vcoll {
namespace {

using namespace dev;

constexpr uint32_t kOrderMasked = 0x007FFFFFu;   // order of -inf

// Unsigned integers in the order of the floats: zeros equal, NaN above all.
__device__ __forceinline__ uint32_t order_of(float z) {
  if (z != z) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

template <int D, int V>
__device__ __forceinline__ void load_logits(const void* row, int experts, int lane, float* z) {
  using S = Storage<D>;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    z[v] = e < experts ? S::widen1(static_cast<const typename S::elem*>(row)[e]) : -INFINITY;
  }
}

template <int D, int V>
__global__ __launch_bounds__(kBlock) void route_kernel(const RouteArgs a) {
  const int lane = threadIdx.x % 64;
  const int i = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock / 64) + threadIdx.x / 64;
  if (t >= a.tokens) return;
  using E = typename Storage<D>::elem;
  float z[V];
  load_logits<D, V>(static_cast<const E*>(a.logits[i]) + t * a.experts, a.experts, lane, z);
  uint32_t order[V];
#pragma unroll
  for (int v = 0; v < V; ++v) order[v] = order_of(z[v]);
  int id = -1;
  float chosen = -INFINITY;
  for (int k = 0; k < a.topk; ++k) {
    uint64_t best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t key = (static_cast<uint64_t>(order[v]) << 32) | (0xFFFFFFFFu - (lane + 64 * v));
      best = key > best ? key : best;
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
      const uint64_t other = __shfl_xor(best, m);
      best = other > best ? other : best;
    }
    if ((best >> 32) <= kOrderMasked) break;
    const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    float ze = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e / 64 == v) ze = z[v];
      if (e == lane + 64 * v) order[v] = 0;
    }
    ze = __shfl(ze, e % 64);
    if (lane == k) {
      id = e;
      chosen = ze;
    }
  }
  const float peak = __shfl(chosen, 0);
  const float mine = id >= 0 ? expf(chosen - peak) : 0.0f;
  float total = mine;
  if (!a.normalise) {
    total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) total += lane + 64 * v < a.experts ? expf(z[v] - peak) : 0.0f;
  }
  total = wave_sum(total);
  if (lane < a.topk) {
    a.ids[i][t * a.topk + lane] = id;
    a.weights[i][t * a.topk + lane] = id >= 0 ? mine / total : 0.0f;
  }
}

template <int D, int V>
__global__ __launch_bounds__(kBlock) void route_backward_kernel(const RouteBackwardArgs a) {
  const int lane = threadIdx.x % 64;
  const int i = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock / 64) + threadIdx.x / 64;
  if (t >= a.tokens) return;
  using S = Storage<D>;
  using E = typename S::elem;
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < a.topk) {
    id = a.ids[i][t * a.topk + lane];
    if (id < 0 || id >= a.experts) id = -1;
    if (id >= 0) {
      w = a.weights[i][t * a.topk + lane];
      dw = a.d_weights[i][t * a.topk + lane];
    }
  }
  const float mean = wave_sum(w * dw);
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  const float term = a.normalise ? w * (dw - mean) : dw;
  for (int k = 0; k < a.topk; ++k) {
    const int e = __shfl(id, k);
    const float x = __shfl(term, k);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == lane + 64 * v) d[v] += x;
  }
  if (!a.normalise) {
    float z[V];
    load_logits<D, V>(static_cast<const E*>(a.logits[i]) + t * a.experts, a.experts, lane, z);
    float peak = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) peak = fmaxf(peak, z[v]);
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) peak = fmaxf(peak, __shfl_xor(peak, m));
    float total = 0.0f;
    const bool empty = peak == -INFINITY;           // every expert masked: no weight, no gradient
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = empty || lane + 64 * v >= a.experts ? 0.0f : expf(z[v] - peak);
      total += z[v];
    }
    total = wave_sum(total);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = empty ? 0.0f : z[v] / total * (d[v] - mean);
  }
  E* out = static_cast<E*>(a.d_logits[i]) + t * a.experts;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 64 * v < a.experts) out[lane + 64 * v] = S::narrow1(d[v]);
}

template <int D, class F>
hipError_t by_width(int experts, F&& run) {
  if (experts <= 64) return run(std::integral_constant<int, 1>{});
  if (experts <= 128) return run(std::integral_constant<int, 2>{});
  if (experts <= 256) return run(std::integral_constant<int, 4>{});
  if (experts <= 512) return run(std::integral_constant<int, 8>{});
  return run(std::integral_constant<int, kMaxExperts / 64>{});
}

dim3 token_grid(int64_t tokens, int ranks) {
  return dim3(static_cast<unsigned>((tokens + kBlock / 64 - 1) / (kBlock / 64)), ranks);
}

template <int D>
hipError_t launch_route_dt(const RouteArgs& a, hipStream_t stream) {
  return by_width<D>(a.experts, [&](auto v) {
    return launch(route_kernel<D, decltype(v)::value>, token_grid(a.tokens, a.ranks), a, stream);
  });
}

template <int D>
hipError_t launch_route_backward_dt(const RouteBackwardArgs& a, hipStream_t stream) {
  return by_width<D>(a.experts, [&](auto v) {
    return launch(route_backward_kernel<D, decltype(v)::value>, token_grid(a.tokens, a.ranks), a, stream);
  });
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, vcoll_dtype dtype, hipStream_t stream) {
  return dtype == VCOLL_F32 ? launch_route_dt<VCOLL_F32>(a, stream) : launch_route_dt<VCOLL_BF16>(a, stream);
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, vcoll_dtype dtype, hipStream_t stream) {
  return dtype == VCOLL_F32 ? launch_route_backward_dt<VCOLL_F32>(a, stream)
                            : launch_route_backward_dt<VCOLL_BF16>(a, stream);
}

}  // namespace vcoll
