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

constexpr int kTreeMax = 64;                    // tokens of a draft: one tile of keys
constexpr int kTreeCtas = 152;                  // one CTA per SM
// Fewest units (a tile of 64 keys for a tile of 128 rows) of a share: each leaves partials to the combine.
constexpr int kTreeMinTiles = 2;
// Q tiles of 128 rows of one column: head_dim 256 leaves tensor memory for one.
__host__ __device__ constexpr int tree_q_tiles(int D) { return D == 256 ? 1 : 2; }

// Whether shares first .. last of a column can be joined.  tree_kernel stores the two as it
// walks the columns; where one of its waits gave up, they are whatever the workspace held.
__host__ __device__ constexpr bool tree_shares_held(int first, int last, int ctas) {
    return first >= 0 && first <= last && last < ctas;
}

// Attention of a tree of drafted tokens (kvc_tree_attention).  A column is
// (sequence, kv head, up to mq tokens); its keys are tiles of 64: the cached rows
// (slots, or positions of a paged sequence), then the draft itself.
struct TreeParams {
    const void* q;              // [B, T, Hq, D]
    const void* k_new;          // [B, T, Hkv, D]
    const int32_t* pos;         // [B]: tokens in the cache (below 0: idle)
    const int32_t* parent;      // [B, T]
    const int32_t* table;
    const uint32_t* valid;      // may be null
    void* out;                  // [B, T, Hq, D]
    void* stage;                // BAKED: the draft's rotated keys [B, T, Hkv, D]
    uint32_t* err;
    float2* part_ml;            // [slots][rows]: slot = share + column
    float* part_o;
    int2* col_shares;           // [columns]: the first and the last share of each
    int B, T, Hq, Hkv, G, layer;
    int inv_g;                  // 65536 / G, rounded up
    int layout, window, sinks, capacity, bs, num_blocks, maxb;
    int tq, mq, ncol;           // tokens of a Q tile, of a column; columns of a (sequence, kv head)
    int col_units;              // units a tile of all columns of a kv head
    int last_units;             // units a tile of the last column: its Q tiles
    int rows;                   // partial rows of a slot
    int box, grouped;           // cached rows of a copy; whether the map counts groups of 8 rows
    int ctas;
    int comb_rows;              // rows of a combine CTA
    int rope;
    float scale2;               // softmax scale * log2(e)
    unsigned long long theta[kMaxHalfDim];
};

// One copy brings rows of K and V, every column block, in the order that the products
// take: [8 rows][K|V][column block][8 x 128 bytes].
//  cache   the layer's rows; where kv heads and blocks begin at multiples of 8 rows
//          (grouped) {64 columns, row of 8, column block, K|V, group of 8 rows}, boxes of a
//          block or of 64 rows; else {64 columns, row, column block, K|V}, boxes of 8 rows.
//  k, v    the draft's rows {64 columns, token, column block, kv head}, boxes of 8 tokens.
struct TreeMaps {
    CUtensorMap cache, k, v;
};

cudaError_t launch_tree(int head_dim, const TreeParams& p, const TreeMaps& maps, cudaStream_t stream);
cudaError_t launch_tree_stage(int head_dim, const TreeParams& p, cudaStream_t stream);
cudaError_t launch_append_path(int dtype, int head_dim, const PathParams& p, cudaStream_t stream);

}  // namespace kvc
