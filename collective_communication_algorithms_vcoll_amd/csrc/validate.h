// Argument checks shared by the C entry points, and the translation of HIP
// launch errors. Host code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"
#include "vcoll.h"

namespace vcoll {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// text of the calling thread's last HIP error, for vcoll_last_hip_error
inline thread_local const char* g_last_hip_error = "";

inline vcoll_status from_hip(hipError_t e) {
  if (e == hipSuccess) return VCOLL_OK;
  g_last_hip_error = hipGetErrorString(e);
  return VCOLL_ERR_HIP;
}

inline int64_t elem_bytes(vcoll_dtype d) { return d == VCOLL_F32 ? 4 : (d == VCOLL_BF16 ? 2 : 1); }

inline bool valid_dtype(int d) { return d == VCOLL_F32 || d == VCOLL_BF16; }

// the all-to-all only moves rows, so it also takes raw bytes
inline bool valid_a2a_dtype(int d) { return valid_dtype(d) || d == VCOLL_U8; }

inline bool valid_p(int p) { return p >= 1 && p <= kMaxRanks; }

// rows x topk within int32 (the row indices of the MoE maps), tested by
// division so that the product is only formed once it is known to fit
inline bool pairs_fit(int64_t rows, int topk) { return topk >= 1 && rows >= 0 && rows <= INT32_MAX / topk; }

// Element counts up to 2^48: far beyond any buffer, and small enough that
// every byte offset (count x 4 bytes x up to 128 ranks) fits in int64.
constexpr int64_t kMaxCount = int64_t(1) << 48;

inline bool valid_count(int64_t n) { return n >= 0 && n <= kMaxCount; }

// A buffer of `rows` rows of `row_bytes` bytes stays within 2^56 bytes.
inline bool fits(int64_t rows, int64_t row_bytes) {
  return row_bytes <= 0 || rows <= (int64_t(1) << 56) / row_bytes;
}

inline bool all_set(int p, const void* const* ptrs) {
  if (!ptrs) return false;
  for (int r = 0; r < p; ++r)
    if (!ptrs[r]) return false;
  return true;
}

inline bool all_aligned(int p, const void* const* ptrs) {
  for (int r = 0; r < p; ++r)
    if (!aligned16(ptrs[r])) return false;
  return true;
}

}  // namespace vcoll
