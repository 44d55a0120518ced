// Parameter blocks and launch entry points of the operators on drafted tokens.
#pragma once

#include "kvc_params.h"

namespace kvc {

// The accepted path's rows into the cache (kvc_append_path).
struct PathParams {
    void* cache;
    float* scales;              // INT8 cache: row scales; else null
    const void* k_new;          // [B, T, Hkv, D]
    const void* v_new;
    const int32_t* pos;         // [B]
    const int32_t* path;        // [B, P]
    const int32_t* n_path;      // [B] or null
    const int32_t* table;
    uint32_t* err;
    long long layer_off, kv_off;
    long long sc_layer_off, sc_kv_off;
    int B, Hkv, T, P;
    int layout, window, sinks, capacity;
    int bs, num_blocks, maxb;
    int rope;
    unsigned long long theta[kMaxHalfDim];
};

cudaError_t launch_append_path(int dtype, int head_dim, const PathParams& p, cudaStream_t stream);

}  // namespace kvc
