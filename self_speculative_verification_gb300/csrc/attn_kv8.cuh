// What the kernels of spec_verify_attn_kv8 share: the parameters of a call,
// and the tensor-core path's workspace and launch.
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

// The tensor-core path (bf16 rows): rows per unit, bytes of workspace, and a
// call, whose workspace begins at Q.a.part_o.
int kv8_tc_rows(const AttnParams &P);
bool kv8_tc_supported(const AttnParams &P);
size_t kv8_tc_workspace_bytes(const AttnParams &P);
spec_status_t launch_attn_kv8_tc(const Kv8Params &Q, cudaStream_t s);

}  // namespace sv
