// What the kernels of spec_verify_attn_kv8 share: the parameters of a call.
#pragma once

#include "attn_common.cuh"
#include "kv8.cuh"

namespace sv {

// One call: the shape and arrays of AttnParams (kc: the cache's tiles; vc
// unused), the cache's scales.
struct Kv8Params {
    AttnParams a;
    const float *scales;     // [n_pages][Hkv][2]
};

}  // namespace sv
