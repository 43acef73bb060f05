// Host checks shared by the 8-bit cache's entry points.
#pragma once

#include "common.cuh"

namespace sv {

// SPEC_OK when the descriptor's heads, head_dim, pages and page_size are ones
// the 8-bit cache takes.
spec_status_t check_kv8(const spec_kv8_desc *c);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace sv
