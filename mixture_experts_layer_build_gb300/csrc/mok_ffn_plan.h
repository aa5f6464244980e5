// mok_ffn_plan.h -- the feed-forward block's host-side arithmetic (plain C++, no CUDA types, so host tests can drive it).
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define MOK_PLAN_FN __host__ __device__
#else
#define MOK_PLAN_FN
#endif

namespace mok {

constexpr int64_t kFfnMaxTokens = (int64_t{1} << 31) - 257;  // row indices of padded tiles stay within 31 bits

// Limit of the wait for a tile of k_blocks K blocks, where that of other waits is `base`: 2 us more for every block, which
// takes 0.2 to 0.45.  (K blocks of a weight gradient are 64 tokens: 2 s alone cover 284 million tokens at 0.45.)
MOK_PLAN_FN constexpr uint64_t tile_wait_ns(uint64_t base, int64_t k_blocks) {
  return base + static_cast<uint64_t>(k_blocks) * 2000u;
}

}  // namespace mok
