// MoE router: the topk largest logits of every token and their softmax
// weights, and the gradient of those weights with respect to the logits.
//
//   chosen e_0, e_1, ..: logits descending, equal logits by ascending id
//   normalise: w_k = exp(z[e_k] - z[e_0]) / sum over the chosen
//   else:      w_k = exp(z[e_k] - z[e_0]) / sum over all experts
//   dz[e] = q_e ([e = e_k] dw_k - sum_j w_j dw_j), q the softmax that made w
//
// L lanes share a token, V logits each. All sums are float32.
#include "device.h"
#include "train.h"

namespace vcoll {
namespace {

using namespace dev;

// ----------------------------------------------------------------------------
// lanes of one token: rotations inside rows of 16 lanes, shuffles beyond

template <int N>
__device__ __forceinline__ float other(float x) {
  if constexpr (N >= 16) return __shfl_xor(x, N);
  else return __uint_as_float(rotate16<N>(__float_as_uint(x)));
}

template <int N>
__device__ __forceinline__ double other(double x) {
  if constexpr (N >= 16) {
    return __shfl_xor(x, N);
  } else {
    const uint64_t u = __double_as_longlong(x);
    const uint64_t r = (static_cast<uint64_t>(rotate16<N>(static_cast<uint32_t>(u >> 32))) << 32) |
                       rotate16<N>(static_cast<uint32_t>(u));
    return __longlong_as_double(r);
  }
}

// Reductions whose result is the same in all L lanes (of a sum too: the pairs
// that two lanes add differ in order only).
template <int L, class T, class F>
__device__ __forceinline__ T across(T x, F&& join) {
  if constexpr (L > 32) x = join(x, other<32>(x));
  if constexpr (L > 16) x = join(x, other<16>(x));
  x = join(x, other<8>(x));
  x = join(x, other<4>(x));
  x = join(x, other<2>(x));
  return join(x, other<1>(x));
}

template <int L>
__device__ __forceinline__ float sum_across(float x) {
  return across<L>(x, [](float a, float b) { return a + b; });
}

// exp(x) for x <= 0 as 2^(x log2 e): off by the rounding of the product,
// |x| 2^-24 relative, which x, a difference of float32 logits, is off by too.
// Results below 2^-126 are 0.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896f); }

// ----------------------------------------------------------------------------
// logits: lane l of a token holds elements l * VE + j of every run of L * VE
// (16-byte loads), or elements l + L * v

template <int D, int L, int V, bool VEC>
__device__ __forceinline__ int expert_at(int lane, int v) {
  constexpr int VE = Storage<D>::kVE;
  if constexpr (VEC) return (v / VE * L + lane) * VE + v % VE;
  else return lane + L * v;
}

template <int D, int L, int V, bool VEC>
__device__ __forceinline__ void load_logits(const void* row, int experts, int lane, bool live, float* z) {
  using S = Storage<D>;
  using E = typename S::elem;
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < V; v += S::kVE) {
      const int e = expert_at<D, L, V, VEC>(lane, v);
      if (live && e < experts) {
        S::widen(__builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(static_cast<const E*>(row) + e)), z + v);
      } else {
#pragma unroll
        for (int c = 0; c < S::kVE; ++c) z[v + c] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_at<D, L, V, VEC>(lane, v);
      z[v] = live && e < experts ? S::widen1(static_cast<const E*>(row)[e]) : -INFINITY;
    }
  }
}

template <int D, int L, int V, bool VEC>
__device__ __forceinline__ void store_logits(void* row, int experts, int lane, const float* d) {
  using S = Storage<D>;
  using E = typename S::elem;
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < V; v += S::kVE) {
      const int e = expert_at<D, L, V, VEC>(lane, v);
      if (e < experts)
        __builtin_nontemporal_store(S::narrow(d + v), reinterpret_cast<u32x4_any*>(static_cast<E*>(row) + e));
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_at<D, L, V, VEC>(lane, v);
      if (e < experts) static_cast<E*>(row)[e] = S::narrow1(d[v]);
    }
  }
}

// ----------------------------------------------------------------------------
// selection keys
//
// A logit and its expert make one double in [1, 2): 32 fraction bits in the
// order of the floats (zeros equal, NaN above all), then 10 bits that fall
// with the expert's id. No two experts share a key, and the larger of two
// keys is one instruction. An expert that cannot be chosen has a key below 1.

__device__ __forceinline__ double key_of(float z, int e) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  uint32_t order = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  if (z != z) order = 0xFFFFFFFFu;
  const uint32_t high = z == -INFINITY ? 0 : 0x3FF00000u | (order >> 12);
  const uint32_t low = (order << 20) | (static_cast<uint32_t>(kMaxExperts - 1 - e) << 10);
  return __longlong_as_double((static_cast<uint64_t>(high) << 32) | low);
}

__device__ __forceinline__ int key_expert(double key) {
  return kMaxExperts - 1 - static_cast<int>((__double_as_longlong(key) >> 10) & (kMaxExperts - 1));
}

__device__ __forceinline__ float key_logit(double key) {
  const uint32_t order = static_cast<uint32_t>(__double_as_longlong(key) >> 20);
  return __uint_as_float((order & 0x80000000u) ? order ^ 0x80000000u : ~order);
}

// Comparators of Batcher's odd-even merge sort of N (a power of two) keys.
template <int N>
struct Network {
  int a[N * 4 + 1] = {}, b[N * 4 + 1] = {};
  int size = 0;
  constexpr Network() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k; ++i)
            if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[size] = i + j;
              b[size] = i + j + k;
              ++size;
            }
  }
};

template <int V>
__device__ __forceinline__ void sort_descending(double* key) {
  static_for<0, Network<V>().size>([&](auto c) {
    constexpr int i = Network<V>().a[decltype(c)::value], j = Network<V>().b[decltype(c)::value];
    const double x = key[i], y = key[j];
    key[i] = __builtin_fmax(x, y);
    key[j] = __builtin_fmin(x, y);
  });
}

// Every lane sorts its V keys once; a round takes the largest head over the
// token's lanes and moves that lane's list up. W: how much of its list a lane
// can need (topk <= W, or W = V).
template <int D, int L, int V, int W, bool VEC>
__global__ __launch_bounds__(kBlock) void route_kernel(const RouteArgs a) {
  using E = typename Storage<D>::elem;
  const int lane = threadIdx.x % L;
  const int i = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock / L) + threadIdx.x / L;
  const bool live = t < a.tokens;
  float z[V];
  load_logits<D, L, V, VEC>(static_cast<const E*>(a.logits[i]) + t * a.experts, a.experts, lane, live, z);
  double key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = key_of(z[v], expert_at<D, L, V, VEC>(lane, v));
  sort_descending<V>(key);
  double chosen = 0.0, first = 0.0;
  for (int k = 0; k < a.topk; ++k) {
    const double best = across<L>(key[0], [](double x, double y) { return __builtin_fmax(x, y); });
    if (k == 0) first = best;
    if (lane == k) chosen = best;
    const bool mine = key[0] == best;
#pragma unroll
    for (int w = 0; w + 1 < W; ++w) {
      const double here = key[w], next = key[w + 1];
      key[w] = mine ? next : here;
    }
    key[W - 1] = mine ? 0.0 : key[W - 1];
  }
  const bool taken = chosen >= 1.0;
  const float peak = key_logit(first);
  const float mine = taken ? exp_of(key_logit(chosen) - peak) : 0.0f;
  float total = mine;
  if (!a.normalise) {
    total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      total += expert_at<D, L, V, VEC>(lane, v) < a.experts ? exp_of(z[v] - peak) : 0.0f;
  }
  total = sum_across<L>(total);
  if (live && lane < a.topk) {
    a.ids[i][t * a.topk + lane] = taken ? key_expert(chosen) : -1;
    a.weights[i][t * a.topk + lane] = taken ? mine / total : 0.0f;
  }
}

// The topk gradient terms reach their experts' lanes through a float row in LDS.
template <int D, int L, int V, bool VEC>
__global__ __launch_bounds__(kBlock) void route_backward_kernel(const RouteBackwardArgs a) {
  using E = typename Storage<D>::elem;
  __shared__ float row[kBlock / L][L * V];
  const int lane = threadIdx.x % L, token = threadIdx.x / L;
  const int i = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock / L) + token;
  const bool live = t < a.tokens;
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (live && lane < a.topk) {
    id = a.ids[i][t * a.topk + lane];
    if (id < 0 || id >= a.experts) id = -1;
    if (id >= 0) {
      w = a.weights[i][t * a.topk + lane];
      dw = a.d_weights[i][t * a.topk + lane];
    }
  }
  float z[V];
  if (!a.normalise)
    load_logits<D, L, V, VEC>(static_cast<const E*>(a.logits[i]) + t * a.experts, a.experts, lane, live, z);
#pragma unroll
  for (int v = 0; v < V; ++v) row[token][lane + L * v] = 0.0f;
  const float mean = sum_across<L>(w * dw);
  __syncthreads();
  if (id >= 0) row[token][id] = a.normalise ? w * (dw - mean) : dw;
  __syncthreads();
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = row[token][expert_at<D, L, V, VEC>(lane, v)];
  if (!a.normalise) {
    float peak = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) peak = fmaxf(peak, z[v]);
    peak = across<L>(peak, [](float x, float y) { return fmaxf(x, y); });
    const bool empty = peak == -INFINITY;           // every expert masked: no weight, no gradient
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[v] = empty ? 0.0f : exp_of(z[v] - peak);
      total += z[v];
    }
    const float scale = empty ? 0.0f : 1.0f / sum_across<L>(total);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = z[v] * scale * (d[v] - mean);
  }
  if (live) store_logits<D, L, V, VEC>(static_cast<E*>(a.d_logits[i]) + t * a.experts, a.experts, lane, d);
}

// ----------------------------------------------------------------------------
// launch: 16 lanes per token where they hold its logits and its chosen
// experts, else the whole wave

template <class F>
hipError_t by_shape(int experts, int topk, F&& run) {
  using std::integral_constant;
  if (topk <= 16 && experts <= 64) return run(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (topk <= 16 && experts <= 128) return run(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (topk <= 16 && experts <= 256) return run(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  if (experts <= 64) return run(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (experts <= 256) return run(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  if (experts <= 512) return run(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return run(integral_constant<int, 64>{}, integral_constant<int, kMaxExperts / 64>{});
}

template <int L>
dim3 token_grid(int64_t tokens, int ranks) {
  constexpr int per = kBlock / L;
  return dim3(static_cast<unsigned>((tokens + per - 1) / per), ranks);
}

template <int D>
hipError_t launch_route_dt(const RouteArgs& a, hipStream_t stream) {
  return by_shape(a.experts, a.topk, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value, VE = Storage<D>::kVE;
    const dim3 grid = token_grid<L>(a.tokens, a.ranks);
    if constexpr (V % VE == 0) {
      if (a.experts % VE == 0) {
        if constexpr (V > 8)
          if (a.topk <= 8) return launch(route_kernel<D, L, V, 8, true>, grid, a, stream);
        return launch(route_kernel<D, L, V, V, true>, grid, a, stream);
      }
    }
    return launch(route_kernel<D, L, V, V, false>, grid, a, stream);
  });
}

template <int D>
hipError_t launch_route_backward_dt(const RouteBackwardArgs& a, hipStream_t stream) {
  return by_shape(a.experts, a.topk, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value, VE = Storage<D>::kVE;
    const dim3 grid = token_grid<L>(a.tokens, a.ranks);
    if constexpr (V % VE == 0)
      if (a.experts % VE == 0) return launch(route_backward_kernel<D, L, V, true>, grid, a, stream);
    return launch(route_backward_kernel<D, L, V, false>, grid, a, stream);
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
