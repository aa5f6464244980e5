// mok_route.cuh -- what the calls on routed rows share.
#pragma once
#include "mok_internal.cuh"

namespace mok {

// The sizes of a schedule with or without the layer's staging; MOK_OK when its tables are there.
mok_status routed_sizes(const mok_schedule* s, Sizes* z);

// Whether two ranges of device memory have no byte in common (null: nothing there).
inline bool apart(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !a || !b || na <= 0 || nb <= 0 || x + static_cast<uintptr_t>(na) <= y || y + static_cast<uintptr_t>(nb) <= x;
}

// Whether n bytes at `out` spare every table of a schedule that a call on routed rows reads.
bool apart_from_tables(const mok_schedule& s, const Sizes& z, const void* out, int64_t n);

}  // namespace mok
