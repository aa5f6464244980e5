// mok_philox.cuh -- the counter-based draws of dropout: Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011), one call per 8 values.
#pragma once
#include <cstdint>

#include "mok.h"

namespace mok {

struct DropArgs {
  const uint64_t* rng;  // {seed, offset} on the device; nullptr: nothing is dropped
  uint32_t below;       // (threshold << 16) - 1 of a draw in the upper half of a word: kept when above it
  float scale;          // 65536 / (65536 - threshold), 0 when everything is dropped
};

// Host: false when p is not in [0, 1] or the state's address is unusable.  d == nullptr: no dropout.  The
// threshold is 0 .. 65536; at 0 nothing is drawn, at 65536 `below` is the largest word, which no draw
// is above.
inline bool make_drop(const mok_dropout* d, DropArgs* out) {
  *out = DropArgs{nullptr, 0u, 1.0f};
  if (!d) return true;
  if (!(d->p >= 0.0f && d->p <= 1.0f) || !d->rng || (reinterpret_cast<uintptr_t>(d->rng) & 7u)) return false;
  const uint32_t t = static_cast<uint32_t>(static_cast<double>(d->p) * 65536.0 + 0.5);
  if (t == 0) return true;
  out->rng = d->rng;
  out->below = static_cast<uint32_t>((static_cast<uint64_t>(t) << 16) - 1u);
  out->scale = t >= 65536u ? 0.0f : static_cast<float>(65536.0 / (65536.0 - t));
  return true;
}

#ifdef __CUDACC__
// The generator's state, the same in every lane and known to be: the round keys are then kept in uniform
// registers.  All lanes of the warp load it.
struct DropState {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ void load(const DropArgs& d) {
    uint2 k = make_uint2(0, 0), o = make_uint2(0, 0);
    if (d.rng) {
      k = *reinterpret_cast<const uint2*>(d.rng);
      o = *reinterpret_cast<const uint2*>(d.rng + 1);
    }
    k0 = __shfl_sync(0xffffffffu, k.x, 0), k1 = __shfl_sync(0xffffffffu, k.y, 0);
    o0 = __shfl_sync(0xffffffffu, o.x, 0), o1 = __shfl_sync(0xffffffffu, o.y, 0);
  }
};

// The eight 16-bit draws of 8-value group `group`, two per word (low half first).  Each round
// multiplies two counter words by fixed odd constants and mixes the halves of the products with the
// other two words and the round key (the key plus the round number times fixed increments).
__device__ __forceinline__ void philox8(const DropState& s, uint64_t group, uint32_t (&w)[4]) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32), c2 = s.o0, c3 = s.o1;
#pragma unroll
  for (uint32_t i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ (s.k0 + i * 0x9E3779B9u);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ (s.k1 + i * 0xBB67AE85u);
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// Zeroes the dropped values of a group with draws w, 8 fp32 as bit patterns (a select: what a dropped
// value holds does not matter); the caller scales by d.scale.
__device__ __forceinline__ void drop_bits(uint32_t (&v)[8], const DropArgs& d, const uint32_t (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (w[j] << 16) > d.below ? v[2 * j] : 0u;
    v[2 * j + 1] = w[j] > d.below ? v[2 * j + 1] : 0u;
  }
}
#endif

}  // namespace mok
