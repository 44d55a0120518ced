// Parameter blocks and launch entry points of the shared-prefix decode
// (kvc_decode_attention_shared).
#pragma once

#include "kvc_params.h"

namespace kvc {

// Q tiles of 128 rows of one column: head_dim 256 leaves tensor memory for one.
__host__ __device__ constexpr int shared_q_tiles(int D) { return D == 256 ? 1 : 2; }
constexpr int kSharedCtas = 152;                // one prefix CTA per SM
// Fewest units of a share: each leaves partials to the combine.  (2, 4 and 8 measured
// the same: 64 sequences in groups of 8 with 2048 tokens, six readers with 1008.)
constexpr int kSharedMinTiles = 2;

struct SharedGroup {
    long long units0;     // units of the groups before
    long long rows0;      // partial rows of the groups before
    int kt, mt;           // tiles of a column; columns of a kv head
    int n, off, leader;   // members, their place in the member list, the first that shares
    int rows;             // shared rows (whole blocks)
    long long hu;         // units of a kv head
};

struct SharedHead {
    long long units;      // of all columns
    int ngroups, shares;
};

struct SharedParams {
    const void* q;
    const int32_t* pos;
    const int32_t* group;           // [B]
    const int32_t* table;           // [B, maxb]
    const uint32_t* valid;          // may be null
    uint32_t* err;
    // workspace
    uint32_t* ticket;               // zero between calls
    SharedHead* head;
    SharedGroup* groups;            // [B / 2]
    int4* seq;                      // [B]: place of its group in the member list (-1: none), rank, members, common blocks
    int2* seq_group;                // [B]: index in groups (-1: none), rank
    int32_t* members;               // [B]: the grouped sequences by group id, then by index
    int32_t* gmin;                  // [B]: scratch of the plan
    int32_t* start;                 // [B]: position the sequence's own keys begin at
    float2* part_ml;                // partial rows (m, l) ...
    float* part_o;                  // ... and o
    long long alt_rows;             // rows from a column's partials to those of its second warpgroup
    int B, Hq, Hkv, G, bs, num_blocks, maxb, layer;
    int tq, mq;                     // members of a Q tile, of a column
    int full_units;                 // units a tile of a full column: its Q tiles
    int ctas;
    int rope;
    float scale2;                   // softmax scale * log2(e)
    unsigned long long theta[kMaxHalfDim];
};

// What the combine takes from the decode of the sequences' own keys.
struct SharedDecode {
    const float2* part_ml;
    const float* part_o;
    const int32_t* seq_rows;
    uint32_t* counters;
    uint32_t* refs;
    void* out;
    long long num_blocks;
    int nsplit, max_items, ncounters;
};

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t stream);
cudaError_t launch_shared_prefix(int head_dim, const SharedParams& p, const CUtensorMap& map, cudaStream_t stream);
cudaError_t launch_shared_combine(int head_dim, const SharedParams& p, const SharedDecode& dp, cudaStream_t stream);

}  // namespace kvc
