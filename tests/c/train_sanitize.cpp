// Host half of the training-step operators (train_api.cpp) with recording
// stubs in place of the kernel launchers: every rank, pair and tensor is
// described by exactly one launch, and the launches fit their limits.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "train.h"

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) {                                                      \
      std::printf("line %d: %s\n", __LINE__, #c);                    \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

static int g_launches = 0;
static std::vector<const void*> g_seen;          // first buffer of every rank or tensor, in launch order
static int64_t g_tiles = 0;

namespace vcoll {
hipError_t launch_route(const RouteArgs& a, vcoll_dtype, hipStream_t) {
  ++g_launches;
  CHECK(a.ranks >= 1 && a.ranks <= kTokenRanks);
  for (int i = 0; i < a.ranks; ++i) g_seen.push_back(a.logits[i]);
  return hipSuccess;
}
hipError_t launch_route_backward(const RouteBackwardArgs& a, vcoll_dtype, hipStream_t) {
  ++g_launches;
  for (int i = 0; i < a.ranks; ++i) g_seen.push_back(a.d_logits[i]);
  return hipSuccess;
}
hipError_t launch_sort(const SortArgs& a, hipStream_t) {
  ++g_launches;
  CHECK(a.blocks >= 1 && a.blocks <= 256 && a.tile >= 1 && a.tile % 1024 == 0);
  CHECK(static_cast<int64_t>(a.blocks) * a.tile >= a.pairs);
  CHECK(a.pairs == 0 || static_cast<int64_t>(a.blocks - 1) * a.tile < a.pairs);
  CHECK(static_cast<uint64_t>(a.blocks) * static_cast<uint64_t>(a.tile) <= UINT32_MAX);
  return hipSuccess;
}
hipError_t launch_weighted(const WeightedArgs& a, vcoll_dtype, hipStream_t) {
  ++g_launches;
  for (int i = 0; i < a.ranks; ++i) g_seen.push_back(a.out[i]);
  return hipSuccess;
}
hipError_t launch_weighted_backward(const WeightedBackwardArgs& a, vcoll_dtype, hipStream_t) {
  ++g_launches;
  for (int i = 0; i < a.ranks; ++i) g_seen.push_back(a.d_out[i]);
  return hipSuccess;
}
hipError_t launch_adamw(const AdamwArgs& a, int32_t tiles, vcoll_dtype, vcoll_dtype, int, hipStream_t) {
  ++g_launches;
  CHECK(a.count >= 1 && a.count <= kAdamwTensors);
  int64_t at = 0;
  for (int k = 0; k < a.count; ++k) {
    CHECK(a.tile_start[k] == at && a.t[k].n > 0);
    CHECK(a.t[k].shift >= 0 && a.t[k].shift < 32);
    at += (a.t[k].n + a.t[k].shift + kAdamwTile - 1) / kAdamwTile;
    g_seen.push_back(a.t[k].param);
  }
  for (int k = a.count; k < kAdamwTensors; ++k) CHECK(a.tile_start[k] == INT32_MAX);
  CHECK(at == tiles);
  g_tiles += tiles;
  return hipSuccess;
}
hipError_t launch_unpack(const UnpackArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
}  // namespace vcoll

// distinct 16-byte aligned addresses that are never dereferenced
static std::vector<void*> fake(int n) {
  std::vector<void*> v(n);
  for (int i = 0; i < n; ++i) v[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(0x100000 + 0x1000 * i));
  return v;
}

template <class T>
static T* const* as(const std::vector<void*>& v) { return reinterpret_cast<T* const*>(v.data()); }

int main() {
  for (int p : {1, 2, 31, 32, 33, 72, 128}) {
    const std::vector<void*> f = fake(p);
    const void* const* in = const_cast<const void* const*>(f.data());
    const std::vector<int64_t> rows(p, 5);
    const int launches = (p + 31) / 32;
    auto seen = [&](int want) {
      CHECK(g_launches == want && static_cast<int>(g_seen.size()) == p);
      for (int i = 0; i < p; ++i) CHECK(g_seen[i] == f[i]);
      g_launches = 0;
      g_seen.clear();
    };
    CHECK(vcoll_moe_route(p, 3, 8, 2, VCOLL_F32, 1, in, as<int32_t>(f), as<float>(f), nullptr) == VCOLL_OK);
    seen(launches);
    CHECK(vcoll_moe_route_backward(p, 3, 8, 2, VCOLL_BF16, 1, nullptr, as<const int32_t>(f), as<const float>(f),
                                   as<const float>(f), f.data(), nullptr) == VCOLL_OK);
    seen(launches);
    CHECK(vcoll_moe_combine_weighted(p, 3, 2, 7, VCOLL_F32, in, rows.data(), as<const int32_t>(f), nullptr, f.data(),
                                     nullptr) == VCOLL_OK);
    seen(launches);
    CHECK(vcoll_moe_combine_weighted_backward(p, 3, 2, 7, VCOLL_F32, in, in, rows.data(), as<const int32_t>(f),
                                              as<const float>(f), f.data(), as<float>(f), nullptr) == VCOLL_OK);
    seen(launches);
    for (int64_t tokens : {int64_t(0), int64_t(1), int64_t(129), int64_t(4096), int64_t(INT32_MAX) / p}) {
      int64_t bytes = -1;
      CHECK(vcoll_moe_sort_workspace(p, tokens, 1, 8, &bytes) == VCOLL_OK && bytes >= 0);
      CHECK(vcoll_moe_sort(p, tokens, 1, 8, as<const int32_t>(f), as<int32_t>(f), as<int32_t>(f)[0], f[0], bytes,
                           nullptr) == VCOLL_OK);
      CHECK(g_launches == 1);
      g_launches = 0;
      if (bytes > 0) {
        CHECK(vcoll_moe_sort(p, tokens, 1, 8, as<const int32_t>(f), as<int32_t>(f), as<int32_t>(f)[0], f[0], bytes - 1,
                             nullptr) == VCOLL_ERR_BUFFER_TOO_SMALL);
        CHECK(g_launches == 0);
      }
    }
  }
  const vcoll_adamw_hyper hyper = {1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, 0, 0};
  for (int count : {1, 47, 48, 49, 200}) {
    const std::vector<void*> f = fake(count);
    std::vector<vcoll_adamw_tensor> t(count);
    int64_t tiles = 0;
    int live = 0;
    for (int k = 0; k < count; ++k) {
      t[k] = {k % 5 == 4 ? 0 : 1 + 777 * k, f[k], f[k], nullptr, f[k], f[k], nullptr, nullptr};
      tiles += (t[k].n + vcoll::kAdamwTile - 1) / vcoll::kAdamwTile;
      live += t[k].n > 0;
    }
    g_tiles = 0;
    CHECK(vcoll_adamw(count, t.data(), VCOLL_F32, VCOLL_BF16, 32, &hyper, nullptr) == VCOLL_OK);
    CHECK(g_launches == (live + 47) / 48 && static_cast<int>(g_seen.size()) == live && g_tiles == tiles);
    g_launches = 0;
    g_seen.clear();
  }
  std::printf("OK\n");
  return 0;
}
