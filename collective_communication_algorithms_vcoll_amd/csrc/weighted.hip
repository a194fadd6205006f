// Weighted MoE combine and its gradient.
//
//   out[t]          = sum_k w[t, k] * expert_out[slot(t, k)]
//   d_expert[slot]  = w[t, k] * d_out[t]
//   d_weights[t, k] = <d_out[t], expert_out[slot(t, k)]>
//
// One workgroup per token: the token's row stays in registers while the rows
// of its slots stream past, so every byte moves once. Sums are float32, over
// k in slot order; one rounding per stored element. A slot outside the expert
// buffers contributes nothing.
#include "device.h"
#include "train.h"

namespace vcoll {
namespace {

using namespace dev;

constexpr int kRowsInFlight = 8;   // slots whose loads are issued together

template <int D>
__global__ __launch_bounds__(kBlock) void weighted_kernel(const WeightedArgs a) {
  using S = Storage<D>;
  using E = typename S::elem;
  constexpr int VE = S::kVE;
  const int tid = threadIdx.x;
  const int i = blockIdx.y;
  const int64_t t = blockIdx.x;
  const int32_t* slot = a.slots[i] + 2 * t * a.topk;
  const float* weight = a.weights[i] ? a.weights[i] + t * a.topk : nullptr;
  E* out = static_cast<E*>(a.out[i]) + t * a.hidden;
  auto source = [&](int k) -> const E* {
    const int j = slot[2 * k], r = slot[2 * k + 1];
    if (j < 0 || j >= a.p || r < 0 || r >= a.expert_rows[j]) return nullptr;
    return static_cast<const E*>(a.expert_out[j]) + r * a.hidden;
  };
  const int64_t nvec = a.vec ? a.hidden / VE : 0;
  for (int64_t x = tid; x < nvec; x += kBlock) {
    float sum[VE] = {};
    for (int k0 = 0; k0 < a.topk; k0 += kRowsInFlight) {
      u32x4 row[kRowsInFlight];
      float w[kRowsInFlight];
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) {
        const E* src = k0 + q < a.topk ? source(k0 + q) : nullptr;
        w[q] = src && weight ? weight[k0 + q] : 1.0f;
        row[q] = src ? ld16(src, x * 16) : u32x4{0, 0, 0, 0};
        if (!src) w[q] = 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) {
        float f[VE];
        S::widen(row[q], f);
#pragma unroll
        for (int c = 0; c < VE; ++c) sum[c] += w[q] * f[c];
      }
    }
    st16(out, x * 16, S::narrow(sum));
  }
  for (int64_t x = nvec * VE + tid; x < a.hidden; x += kBlock) {
    float sum = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
      const E* src = source(k);
      if (src) sum += (weight ? weight[k] : 1.0f) * S::widen1(src[x]);
    }
    out[x] = S::narrow1(sum);
  }
}

template <int D>
__global__ __launch_bounds__(kBlock) void weighted_backward_kernel(const WeightedBackwardArgs a) {
  using S = Storage<D>;
  using E = typename S::elem;
  constexpr int VE = S::kVE;
  __shared__ float part[kBlock / 64][kRowsInFlight];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const int i = blockIdx.y;
  const int64_t t = blockIdx.x;
  const int32_t* slot = a.slots[i] + 2 * t * a.topk;
  const float* weight = a.weights[i] + t * a.topk;
  const E* dy = static_cast<const E*>(a.d_out[i]) + t * a.hidden;
  const int64_t nvec = a.vec ? a.hidden / VE : 0;
  for (int k0 = 0; k0 < a.topk; k0 += kRowsInFlight) {
    const E* src[kRowsInFlight];
    E* dst[kRowsInFlight];
    float w[kRowsInFlight], dot[kRowsInFlight];
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) {
      src[q] = nullptr;
      dst[q] = nullptr;
      w[q] = dot[q] = 0.0f;
      if (k0 + q < a.topk) {
        const int j = slot[2 * (k0 + q)], r = slot[2 * (k0 + q) + 1];
        if (j >= 0 && j < a.p && r >= 0 && r < a.expert_rows[j]) {
          src[q] = static_cast<const E*>(a.expert_out[j]) + r * a.hidden;
          dst[q] = static_cast<E*>(a.d_expert_out[j]) + r * a.hidden;
          w[q] = weight[k0 + q];
        }
      }
    }
    for (int64_t x = tid; x < nvec; x += kBlock) {
      u32x4 row[kRowsInFlight];
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) row[q] = src[q] ? ld16(src[q], x * 16) : u32x4{0, 0, 0, 0};
      float g[VE];
      S::widen(*reinterpret_cast<const u32x4*>(dy + x * VE), g);
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) {
        if (!src[q]) continue;
        float f[VE], d[VE];
        S::widen(row[q], f);
#pragma unroll
        for (int c = 0; c < VE; ++c) {
          dot[q] += g[c] * f[c];
          d[c] = w[q] * g[c];
        }
        st16(dst[q], x * 16, S::narrow(d));
      }
    }
    for (int64_t x = nvec * VE + tid; x < a.hidden; x += kBlock) {
      const float g = S::widen1(dy[x]);
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q)
        if (src[q]) {
          dot[q] += g * S::widen1(src[q][x]);
          dst[q][x] = S::narrow1(w[q] * g);
        }
    }
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) {
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) dot[q] += __shfl_xor(dot[q], m);
      if (lane == 0) part[wave][q] = dot[q];
    }
    __syncthreads();
    if (tid < kRowsInFlight && k0 + tid < a.topk) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < kBlock / 64; ++v) sum += part[v][tid];
      a.d_weights[i][t * a.topk + k0 + tid] = sum;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_weighted(const WeightedArgs& a, vcoll_dtype dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.tokens), a.ranks);
  if (dtype == VCOLL_F32) return launch(weighted_kernel<VCOLL_F32>, grid, a, stream);
  return launch(weighted_kernel<VCOLL_BF16>, grid, a, stream);
}

hipError_t launch_weighted_backward(const WeightedBackwardArgs& a, vcoll_dtype dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.tokens), a.ranks);
  if (dtype == VCOLL_F32) return launch(weighted_backward_kernel<VCOLL_F32>, grid, a, stream);
  return launch(weighted_backward_kernel<VCOLL_BF16>, grid, a, stream);
}

}  // namespace vcoll
