// mok_route.cuh -- what the calls on routed rows share.
#pragma once
#include "mok_internal.cuh"

namespace mok {

// The sizes of a schedule with or without the layer's staging; MOK_OK when its tables are there.
mok_status routed_sizes(const mok_schedule* s, Sizes* z);

}  // namespace mok
