// mok_philox.cuh -- the counter-based draws of dropout: Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011), one call per 8 values.
#pragma once
#include <cstdint>

#include "mok.h"

namespace mok {

struct DropArgs {
  const uint64_t* rng;  // {seed, offset} on the device; nullptr: no dropout
  uint32_t thr;         // a value is dropped when its 16-bit draw is below thr (0 .. 65536)
  float scale;          // 65536 / (65536 - thr), 0 when everything is dropped
};

// Host: false when p is not in [0, 1] or the state's address is unusable.  d == nullptr: no dropout.
inline bool make_drop(const mok_dropout* d, DropArgs* out) {
  *out = DropArgs{nullptr, 0u, 1.0f};
  if (!d) return true;
  if (!(d->p >= 0.0f && d->p <= 1.0f) || !d->rng || (reinterpret_cast<uintptr_t>(d->rng) & 7u)) return false;
  out->rng = d->rng;
  out->thr = static_cast<uint32_t>(static_cast<double>(d->p) * 65536.0 + 0.5);
  out->scale = out->thr >= 65536u ? 0.0f : static_cast<float>(65536.0 / (65536.0 - out->thr));
  return true;
}

#ifdef __CUDACC__
// The eight 16-bit draws of 8-value group `group`, two per word (low half first).  Each round
// multiplies two counter words by fixed odd constants and mixes the halves of the products with the
// other two words and the round key (the key plus the round number times fixed increments).
__device__ __forceinline__ uint4 philox8(uint64_t seed, uint64_t offset, uint64_t group) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// v[j] = kept ? v[j] * scale : 0 for the 8 values of group `group` (a select: what a dropped value
// holds does not matter).
__device__ __forceinline__ void drop8(float (&v)[8], const DropArgs& d, uint64_t seed, uint64_t offset,
                                      uint64_t group) {
  const uint4 r = philox8(seed, offset, group);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (w[j] & 0xFFFFu) >= d.thr ? v[2 * j] * d.scale : 0.0f;
    v[2 * j + 1] = (w[j] >> 16) >= d.thr ? v[2 * j + 1] * d.scale : 0.0f;
  }
}
#endif

}  // namespace mok
