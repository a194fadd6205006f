// AdamW over many tensors in one launch per kAdamwTensors of them.
//
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
//   x = (1 - lr wd) x - lr / bc1 * m / (sqrt(v) / sqrt(bc2) + eps)
//
// in float32, each operation rounded, no fused multiply-add. x is the float32
// parameter, or the float32 master copy of a bfloat16 one, which is stored
// beside it rounded to nearest.
//
// 8-bit states: m as E4M3 codes, v as unsigned codes with 5 exponent and 3
// fraction bits (v has no sign and twice the exponent range of m), one
// power-of-two scale per 128 elements: the smallest that keeps the group's
// largest value at or below the format's (448, 1.875). Codes are rounded up
// with probability equal to the fraction lost. A moving average needs that:
// one step changes v by 0.1 %, far below half a code step (3-6 %), so
// rounding to nearest would leave every v where it is.
#include "device.h"
#include "train.h"

namespace vcoll {
namespace {

using namespace dev;

constexpr int kPer = 8;                            // elements per thread
constexpr int kGroupLanes = kAdamwGroup / kPer;    // lanes that share a scale
static_assert(kAdamwTile == kPer * kBlock, "one tile per workgroup");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

__device__ __forceinline__ void load8(const float* p, float* f) {
  Storage<VCOLL_F32>::widen(*reinterpret_cast<const u32x4_any*>(p), f);
  Storage<VCOLL_F32>::widen(*reinterpret_cast<const u32x4_any*>(p + 4), f + 4);
}
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
  Storage<VCOLL_BF16>::widen(*reinterpret_cast<const u32x4_any*>(p), f);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<u32x4_any*>(p) = Storage<VCOLL_F32>::narrow(f);
  *reinterpret_cast<u32x4_any*>(p + 4) = Storage<VCOLL_F32>::narrow(f + 4);
}
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
  *reinterpret_cast<u32x4_any*>(p) = Storage<VCOLL_BF16>::narrow(f);
}
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(uint16_t x) { return Storage<VCOLL_BF16>::widen1(x); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }
__device__ __forceinline__ void store1(uint16_t* p, float f) { *p = Storage<VCOLL_BF16>::narrow1(f); }

// The first `live` of 8 elements at p; zeros beyond.
template <class T>
__device__ __forceinline__ void load_some(const T* p, int live, float* f) {
  if (live == kPer) {
    load8(p, f);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) f[c] = c < live ? widen1(p[c]) : 0.0f;
  }
}
template <class T>
__device__ __forceinline__ void store_some(T* p, int live, const float* f) {
  if (live == kPer) {
    store8(p, f);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (c < live) store1(p + c, f[c]);
  }
}
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int live) {
  if (live == kPer) return *reinterpret_cast<const u32x2_any*>(p);
  u32x2 w = {0, 0};
#pragma unroll
  for (int c = 0; c < kPer; ++c)
    if (c < live) w[c / 4] |= static_cast<uint32_t>(p[c]) << (8 * (c % 4));
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int live, u32x2 w) {
  if (live == kPer) {
    *reinterpret_cast<u32x2_any*>(p) = w;
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (c < live) p[c] = static_cast<uint8_t>(w[c / 4] >> (8 * (c % 4)));
  }
}

// --- the two 8-bit formats ---------------------------------------------------

// m: sign, 4 exponent bits with bias 7, 3 fraction bits; 0x7F is NaN.
__device__ __forceinline__ float decode_m(uint32_t code) {
  const uint32_t a = code & 0x7Fu;
  float f = a < 8 ? static_cast<float>(a) * 0x1p-9f : __uint_as_float((a << 20) + ((127u - 7u) << 23));
  if (a == 0x7Fu) f = __uint_as_float(0x7FC00000u);
  return (code & 0x80u) ? -f : f;
}
// v: 5 exponent bits with bias 31, 3 fraction bits.
__device__ __forceinline__ float decode_v(uint32_t code) {
  return code < 8 ? static_cast<float>(code) * 0x1p-33f : __uint_as_float((code << 20) + ((127u - 31u) << 23));
}

// Both encoders add 20 random bits below the last kept fraction bit and cut:
// on the float's own bits, where a carry moves on to the next binade as it
// should, or below the smallest normal on the value in units of 2^-20 of the
// format's smallest step.
__device__ __forceinline__ uint32_t encode_m(float y, uint32_t r) {
  const float a = fabsf(y);
  if (!(a <= 3.402823466e38f)) return 0x7Fu;
  const uint32_t code = a < 0x1p-6f ? (static_cast<uint32_t>(a * 0x1p29f) + r) >> 20
                                    : ((__float_as_uint(a) + r) >> 20) - ((127u - 7u) << 3);
  return code | (y < 0.0f ? 0x80u : 0u);
}
__device__ __forceinline__ uint32_t encode_v(float y, uint32_t r) {
  if (!(y <= 1.875f)) return 0xFFu;                 // infinite or NaN: the largest code
  return y < 0x1p-30f ? (static_cast<uint32_t>(y * 0x1p53f) + r) >> 20
                      : ((__float_as_uint(y) + r) >> 20) - ((127u - 31u) << 3);
}

// Exponent k of the smallest 2^k with amax <= top * 2^k, top = 1.fraction *
// 2^(above - 127): 0 for an empty group, within [-126, 126].
__device__ __forceinline__ int scale_exponent(float amax, uint32_t fraction, int above) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 0;
  const int k = static_cast<int>(u >> 23) - above + ((u & 0x7FFFFFu) > fraction ? 1 : 0);
  return k < -126 ? -126 : (k > 126 ? 126 : k);
}
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// Largest finite |x| over the 8 elements of the 16 lanes of a group.
__device__ __forceinline__ float group_max(const float* x) {
  float m = 0.0f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float a = fabsf(x[c]);
    m = a <= 3.402823466e38f ? fmaxf(m, a) : m;
  }
#pragma unroll
  for (int d = kGroupLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kGroupLanes));
  return m;
}

// P: storage of the parameter (float: no master copy), G: of the gradient.
template <class P, class G, int BITS>
__global__ __launch_bounds__(kBlock) void adamw_kernel(const AdamwArgs a) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.t[mid].tile_start <= static_cast<int>(blockIdx.x)) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor& T = a.t[lo];
  const int64_t e0 = static_cast<int64_t>(blockIdx.x - T.tile_start) * kAdamwTile + threadIdx.x * kPer;
  const int64_t left = T.n - e0;
  const int live = left >= kPer ? kPer : (left > 0 ? static_cast<int>(left) : 0);
  constexpr bool kMaster = !std::is_same<P, float>::value;
  float* const x_at = (kMaster ? T.master : static_cast<float*>(T.param)) + e0;

  float g[kPer], m[kPer], v[kPer], x[kPer];
  load_some(static_cast<const G*>(T.grad) + e0, live, g);
  load_some(x_at, live, x);
  if constexpr (BITS == 32) {
    load_some(static_cast<const float*>(T.exp_avg) + e0, live, m);
    load_some(static_cast<const float*>(T.exp_avg_sq) + e0, live, v);
  } else {
    const u32x2 cm = load_codes(static_cast<const uint8_t*>(T.exp_avg) + e0, live);
    const u32x2 cv = load_codes(static_cast<const uint8_t*>(T.exp_avg_sq) + e0, live);
    const float sm = live ? T.exp_avg_scale[e0 / kAdamwGroup] : 1.0f;
    const float sv = live ? T.exp_avg_sq_scale[e0 / kAdamwGroup] : 1.0f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      m[c] = decode_m((cm[c / 4] >> (8 * (c % 4))) & 0xFFu) * sm;
      v[c] = decode_v((cv[c / 4] >> (8 * (c % 4))) & 0xFFu) * sv;
    }
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float gc = g[c] * a.grad_scale;
    m[c] = m[c] * a.beta1 + gc * a.one_minus_beta1;
    v[c] = v[c] * a.beta2 + (gc * gc) * a.one_minus_beta2;
    const float move = m[c] / (sqrtf(v[c]) * a.root_bc2 + a.eps);
    x[c] = x[c] * a.decay - move * a.step_size;
  }
  store_some(x_at, live, x);
  if constexpr (kMaster) store_some(static_cast<P*>(T.param) + e0, live, x);
  if constexpr (BITS == 32) {
    store_some(static_cast<float*>(T.exp_avg) + e0, live, m);
    store_some(static_cast<float*>(T.exp_avg_sq) + e0, live, v);
  } else {
    if (live < kPer) {                              // a short group's scale is that of its own elements
#pragma unroll
      for (int c = 0; c < kPer; ++c)
        if (c >= live) m[c] = v[c] = 0.0f;
    }
    const int km = scale_exponent(group_max(m), 0x600000u, 135);
    const int kv = scale_exponent(group_max(v), 0x700000u, 127);
    const float im = power_of_two(-km), iv = power_of_two(-kv);
    u32x2 cm = {0, 0}, cv = {0, 0};
    const uint32_t high = T.key + mix32(static_cast<uint32_t>(static_cast<uint64_t>(e0) >> 32));
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const uint32_t h = mix32(static_cast<uint32_t>(e0 + c) + high);
      cm[c / 4] |= encode_m(m[c] * im, (h >> 16) << 4) << (8 * (c % 4));
      cv[c / 4] |= encode_v(v[c] * iv, (h & 0xFFFFu) << 4) << (8 * (c % 4));
    }
    if (live) {
      store_codes(static_cast<uint8_t*>(T.exp_avg) + e0, live, cm);
      store_codes(static_cast<uint8_t*>(T.exp_avg_sq) + e0, live, cv);
      if (e0 % kAdamwGroup == 0) {
        T.exp_avg_scale[e0 / kAdamwGroup] = power_of_two(km);
        T.exp_avg_sq_scale[e0 / kAdamwGroup] = power_of_two(kv);
      }
    }
  }
}

// The float32 values of 8-bit states: 8 elements per thread.
__global__ __launch_bounds__(kBlock) void unpack_kernel(const UnpackArgs a) {
  const int64_t e0 = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * kPer;
  if (e0 >= a.n) return;
  const int live = a.n - e0 >= kPer ? kPer : static_cast<int>(a.n - e0);
  const u32x2 cm = load_codes(a.exp_avg + e0, live);
  const u32x2 cv = load_codes(a.exp_avg_sq + e0, live);
  const float sm = a.exp_avg_scale[e0 / kAdamwGroup], sv = a.exp_avg_sq_scale[e0 / kAdamwGroup];
  float m[kPer], v[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    m[c] = decode_m((cm[c / 4] >> (8 * (c % 4))) & 0xFFu) * sm;
    v[c] = decode_v((cv[c / 4] >> (8 * (c % 4))) & 0xFFu) * sv;
  }
  store_some(a.exp_avg_out + e0, live, m);
  store_some(a.exp_avg_sq_out + e0, live, v);
}

template <class P, class G>
hipError_t launch_adamw_bits(const AdamwArgs& a, int32_t tiles, int bits, hipStream_t stream) {
  if (bits == 32) return launch(adamw_kernel<P, G, 32>, dim3(tiles), a, stream);
  return launch(adamw_kernel<P, G, 8>, dim3(tiles), a, stream);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int32_t tiles, vcoll_dtype param, vcoll_dtype grad, int state_bits,
                        hipStream_t stream) {
  if (param == VCOLL_F32) {
    if (grad == VCOLL_F32) return launch_adamw_bits<float, float>(a, tiles, state_bits, stream);
    return launch_adamw_bits<float, uint16_t>(a, tiles, state_bits, stream);
  }
  if (grad == VCOLL_F32) return launch_adamw_bits<uint16_t, float>(a, tiles, state_bits, stream);
  return launch_adamw_bits<uint16_t, uint16_t>(a, tiles, state_bits, stream);
}

hipError_t launch_unpack(const UnpackArgs& a, hipStream_t stream) {
  const int64_t tiles = (a.n + kAdamwTile - 1) / kAdamwTile;
  return launch(unpack_kernel, dim3(static_cast<unsigned>(tiles)), a, stream);
}

}  // namespace vcoll
