// Parameter blocks and launch entry points of the operators on caches read or
// kept in part: block bounds, block selection, the plan of a selected decode,
// block weights, eviction.
#pragma once

#include "kvc_params.h"

namespace kvc {

// Bounds of blocks (kvc_block_bounds): codes [layers][num_blocks][Hkv][2][D]
// (largest, smallest), then their steps [layers][num_blocks][Hkv].
struct BoundsParams {
    const void* cache;
    const float* scales;        // INT8 cache: row scales; else null
    int8_t* codes;              // this layer's
    float* steps;               // this layer's
    const int32_t* pos;         // [B]
    const int32_t* n_tok;       // [B] or null
    const int32_t* table;
    uint32_t* err;
    long long layer_off;        // elements to this layer's K half
    long long sc_layer_off;     // scales to this layer's K half
    int B, Hkv, bs, num_blocks, maxb, n_new, slots;
    int heads, parts;           // kv heads of a warp; warps of a block
};

// Selection (kvc_select_blocks).
struct SelectParams {
    const int8_t* codes;        // this layer's bounds
    const float* steps;
    const void* q;              // [B, Hq, D]
    const int32_t* pos;         // [B]
    const int32_t* table;
    const uint32_t* valid;      // may be null
    uint32_t* err;
    uint32_t* keys;             // [B][Hkv][key_stride]: 0 no candidate, 0xffffffff always in, else the ordered score
    int32_t* blocks;            // [B][Hkv][k]
    int B, Hq, Hkv, G, bs, num_blocks, maxb;
    int k, first, recent;
    int key_stride;             // maxb in whole fours
    int rope;
    unsigned long long theta[kMaxHalfDim];
};

// The lists of a selected decode (kvc_decode_attention_selected).
struct SelectPlanParams {
    const int32_t* blocks;      // [B][Hkv][k] logical
    const int32_t* pos;
    const int32_t* table;
    const uint32_t* valid;      // may be null
    uint32_t* err;
    int32_t* list;              // [Hkv][B][k] physical, attended ones first
    int32_t* rows;              // [Hkv][B]
    int B, Hkv, bs, num_blocks, maxb, k;
};

// Weights of blocks (kvc_decode_attention_weighed).
struct WeighParams {
    const float* scores;        // [B][Hq][stride]: base-2 scores by position
    const float2* ml;           // [B][Hq]: (M, 1 / L)
    const int32_t* pos;
    const int32_t* table;
    const uint32_t* valid;      // may be null
    float* weights;             // [B][maxb]
    long long stride;
    float decay;
    int B, Hq, bs, num_blocks, maxb;
    int per;                    // blocks of a CTA
};

// Eviction (kvc_block_evict).
struct EvictParams {
    float* weights;             // [B][maxb]
    const int32_t* pos;
    int32_t* table;
    uint32_t* valid;            // may be null
    int32_t* refcount;
    int32_t* free_list;
    int32_t* free_count;
    uint32_t* err;
    uint32_t* ticket;           // zero between calls
    uint32_t* back;             // [ceil(num_blocks / 32)] blocks given back (zero between calls)
    int B, bs, num_blocks, maxb, keep, first, recent;
};

cudaError_t launch_block_bounds(int dtype, int head_dim, const BoundsParams& p, cudaStream_t stream);
cudaError_t launch_select(int dtype, int head_dim, const SelectParams& p, cudaStream_t stream);
cudaError_t launch_select_plan(const SelectPlanParams& p, cudaStream_t stream);
cudaError_t launch_weigh(const WeighParams& p, cudaStream_t stream);
cudaError_t launch_block_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace kvc
