/*
 * kvc.h - C ABI of the decode-step KV-cache attention library (libkvc.so).
 *
 * One new query per sequence attends over a fixed-capacity KV cache kept in
 * one of three layouts, and the new token's K/V is appended to that cache;
 * a chunk of new tokens can be prefilled the same way (kvc_prefill), and the
 * cache can hold bf16, fp32 or per-row INT8 rows.
 * The operations follow these pages (cited by title and section):
 *
 *   [ring]   "Why sliding-window attention decodes with a ring KV cache"
 *            (2kiu.com/news/4318096)
 *   [share]  "Shared state, isolated problems: KV cache and batching"
 *            (pwwt.cn/news/6215824)
 *   [sink]   "Attention sinks and StreamingLLM" (openeuler.csdn.net)
 *   [primer] "KV cache primer" (pwwt.cn/news/5010196)
 *   [pool]   "KV cache paging" (cloudlnk.cn/blog/kv-cache-paging)
 *
 * Conventions shared by every entry point
 *   - Every buffer argument is a DEVICE pointer owned by the caller (cache,
 *     queries, outputs, tables, workspace); the library allocates no device
 *     memory.  `stream` is a cudaStream_t (NULL = the legacy default stream);
 *     every call except kvc_get_error only enqueues work on it and returns.
 *   - State the library keeps across calls (host side, thread-safe):
 *     (1) the TMA tensor maps of the last 8 bf16 / INT8 caches it decoded,
 *     keyed by (cache address, layers, rows per K half, head_dim, dtype,
 *     device): a cache freed and a different one allocated at the same
 *     address with the same shape reuses the maps, which are still correct,
 *     since they depend on nothing else;  (2) kvc_pager objects, which the
 *     caller creates and destroys;  (3) the fixed device scratch of
 *     kvc_decode_attention_noalloc (see there).  Everything else a call
 *     needs lives in the caller's workspace.
 *   - Return value: KVC_OK (0) or a negative KVC_ERR_* code.  On a negative
 *     code nothing was launched.  Errors that only the device can see (a
 *     block id out of range, an append into an unmapped block, a bad
 *     position) set bits in the workspace's error word; the kernel skips the
 *     offending access and carries on.  kvc_get_error() reads and clears them.
 *   - Element types: the cache, q, out, k_new and v_new share one element
 *     type (kvc_desc.dtype), except that an INT8 cache (KVC_I8) takes and
 *     returns bf16 q, out, k_new and v_new.  All arithmetic is fp32.
 *   - Alignment: cache, q, out, k_new, v_new and workspace must be 16-byte
 *     aligned (KVC_ERR_ALIGN otherwise).
 */
#ifndef KVC_H
#define KVC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KVC_API __attribute__((visibility("default")))
#else
#define KVC_API
#endif

/* Cache layouts.
 *  RING       [ring] 3.2-3.3, 5.1: W slots per (sequence, kv head); token p
 *             goes to slot p mod W.  Token t attends t-W+1 .. t ([ring] 2.2,
 *             6), itself included.
 *  SINK_RING  [sink] cache-set equation: S pinned sink slots, then a W-slot
 *             ring.  Token p goes to slot p (p < S) or S + ((p - S) mod W).
 *             Token t attends {0 .. S-1} U {t-W+1 .. t}.
 *  PAGED      [share] 3.1-3.2, [pool] "kernel forgets absent blocks": a pool
 *             of fixed-size blocks; block_table[b][p / block_size] names the
 *             physical block of token p (-1 = not mapped); a per-block valid
 *             bit drops non-resident blocks.  Token t attends every p <= t
 *             whose block is mapped and valid. */
typedef enum { KVC_LAYOUT_RING = 0, KVC_LAYOUT_SINK_RING = 1, KVC_LAYOUT_PAGED = 2 } kvc_layout;

/* RoPE handling (rotate-half pairs (i, i + D/2), theta_i = base^(-2i/D)).
 *  NONE          no rotation.
 *  BAKED         [primer] 4.5, [pool] "RoPE baked into K rows": K is rotated
 *                at its absolute position when appended; q is rotated at t.
 *  READ_INCACHE  [sink] "RoPE cache position shifting": K is stored raw and
 *                rotated when read, at its index in the compacted cache
 *                (sinks 0..S-1; window token p at p - max(0, t - C + 1),
 *                C = S + W); q at min(t, C - 1).  RING and SINK_RING only. */
typedef enum { KVC_ROPE_NONE = 0, KVC_ROPE_BAKED = 1, KVC_ROPE_READ_INCACHE = 2 } kvc_rope;

/* Cache element types.
 *  KVC_F32, KVC_BF16  rows stored as fp32 / bf16 (round to nearest even).
 *  KVC_I8             [primer] 5.1 (quantised cache: INT8 halves the bytes):
 *                     each stored row (one token's K or V of one kv head)
 *                     keeps int8 codes and one fp32 scale s = max|x| / 127,
 *                     codes rint(x / s) clamped to +-127 (IEEE fp32 quotient,
 *                     ties to even), read back as code * s; a zero row has
 *                     s = 0.  With baked RoPE the rotated key is quantised;
 *                     with READ_INCACHE the raw key is, and the decode
 *                     rotates code * s at the in-cache position.  q, out,
 *                     k_new and v_new are bf16.  Requires head_dim 128 or
 *                     256, and rows per K (or V) half of a layer (batch *
 *                     kv_heads * capacity, or num_blocks * kv_heads *
 *                     block_size) a multiple of 4.
 *                     Not accepted by the pool pager (kvc_pagein_issue). */
typedef enum { KVC_F32 = 0, KVC_BF16 = 1, KVC_I8 = 2 } kvc_dtype;

/* Cache geometry.  Cache memory layout ([primer] 3.1, K at index 0, V at 1):
 *   RING / SINK_RING: [layers, 2, batch, kv_heads, capacity, head_dim],
 *                     capacity = sinks + window;
 *   PAGED:            [layers, 2, num_blocks, kv_heads, block_size, head_dim].
 * KVC_I8: that array holds the int8 codes and is followed directly by the
 * fp32 row scales, [layers, 2, batch, kv_heads, capacity] (or [layers, 2,
 * num_blocks, kv_heads, block_size]); kvc_cache_bytes counts both.
 * q_heads must be a multiple of kv_heads; q head h reads kv head
 * h / (q_heads / kv_heads) ([share] 2.2 and 4.1, grouped-query attention).
 * Launch-grid limits (else KVC_ERR_DESC): batch <= 65535, P = q_heads / g4
 * <= 65535 and batch * P < 2^31, where g4 is the largest of 4, 2, 1 that
 * divides q_heads / kv_heads (q heads are processed in groups of g4). */
typedef struct kvc_desc {
    int32_t layout;             /* kvc_layout */
    int32_t rope;               /* kvc_rope */
    int32_t dtype;              /* kvc_dtype (cache element type) */
    int32_t layers;
    int32_t batch;              /* sequences (rows of block_table for PAGED) */
    int32_t q_heads;
    int32_t kv_heads;
    int32_t head_dim;           /* 64, 128 or 256 */
    int32_t window;             /* RING / SINK_RING: W */
    int32_t sinks;              /* SINK_RING: S >= 1; RING: 0 */
    int32_t block_size;         /* PAGED */
    int32_t num_blocks;         /* PAGED: physical blocks in the pool */
    int32_t max_blocks_per_seq; /* PAGED: columns of block_table */
    int32_t num_splits;         /* 0 = library choice; else KV splits per (sequence, kv head)
                                   for RING / SINK_RING, work items for PAGED */
    float rope_base;            /* e.g. 10000 */
    float softmax_scale;        /* 0 => 1 / sqrt(head_dim) */
} kvc_desc;

/* Host-detected status codes (nothing launched). */
#define KVC_OK 0
#define KVC_ERR_NULL (-1)        /* a required pointer is NULL */
#define KVC_ERR_DESC (-2)        /* inconsistent descriptor */
#define KVC_ERR_UNSUPPORTED (-3) /* combination not built (e.g. PAGED + READ_INCACHE) */
#define KVC_ERR_ALIGN (-4)       /* pointer not 16-byte aligned */
#define KVC_ERR_WORKSPACE (-5)   /* workspace smaller than kvc_workspace_bytes() */
#define KVC_ERR_ARG (-6)         /* argument out of range (layer, n_new, n) */
#define KVC_ERR_CUDA (-7)        /* a CUDA runtime call or launch failed */
#define KVC_ERR_TOO_LARGE (-8)   /* kvc_decode_attention_noalloc: the call needs more than
                                    KVC_NOALLOC_SCRATCH_BYTES of scratch */

/* Device-detected error bits, returned by kvc_get_error(). */
#define KVC_DEV_BAD_BLOCK 0x1u       /* block_table entry >= num_blocks (access skipped) */
#define KVC_DEV_UNMAPPED_APPEND 0x2u /* append into a logical block whose entry is -1 */
#define KVC_DEV_BAD_POSITION 0x4u    /* decode position < 0, or beyond the block table */
#define KVC_DEV_TIMEOUT 0x8u         /* a bounded wait inside a kernel gave up */
#define KVC_DEV_BAD_ENTRY 0x10u      /* kvc_block_table_write / kvc_valid_write entry out of range */
#define KVC_DEV_INTERNAL 0x20u       /* an index computed inside a kernel failed its bounds check
                                        (access skipped); a library bug, please report */
#define KVC_DEV_NO_FREE_BLOCK 0x40u  /* kvc_block_prepare: the free list ran out (that sequence skipped) */

/* Bytes of the cache tensor described by `d` (0 if `d` is invalid). */
KVC_API size_t kvc_cache_bytes(const kvc_desc* d);

/* Bytes of workspace that kvc_append / kvc_decode_attention /
 * kvc_block_table_write / kvc_valid_write need for `d` (0 if `d` is invalid).
 * The workspace holds the device error word, split-K partial results and
 * per-(sequence, kv head) completion counters, and for PAGED caches the
 * step's plan (attended rows and an attended-block directory per sequence,
 * the number of sequences reading each physical block) and the block
 * manager's scratch.  It must be zero-filled once before first use
 * (kvc_workspace_init); every call leaves it ready for the next one.  Calls
 * that share a workspace must not overlap on the GPU. */
KVC_API size_t kvc_workspace_bytes(const kvc_desc* d);

/* Zero-fill `workspace` (cudaMemsetAsync on `stream`). */
KVC_API int kvc_workspace_init(const kvc_desc* d, void* workspace, size_t workspace_bytes, void* stream);

/* Append n_new tokens per sequence to layer `layer` of the cache
 * ([ring] 3.3 and 5.1, [primer] 4.4: write in place, no allocation).
 *   k_new, v_new  [batch, n_new, kv_heads, head_dim], pre-RoPE.
 *   pos           [batch] int32: position of token 0 of each sequence; token
 *                 i is at pos[b] + i.  Tokens at negative positions are
 *                 skipped (left padding).
 *   block_table   PAGED: [batch, max_blocks_per_seq] int32; else NULL.
 * BAKED rotates K at its absolute position (the angle p * theta_i reduced
 * exactly as a 64-bit fixed-point fraction of a turn, its sine and cosine
 * and the rotation in fp32, stored rounded to nearest-even); V is never
 * rotated ([pool]).  For
 * RING / SINK_RING the cache ends as if the tokens were appended one at a
 * time in order: a token that a later token of the same call overwrites is
 * not written.  Ring appends must come in position order, one call per step,
 * before the attention call that reads them.  PAGED: an unmapped target
 * block sets KVC_DEV_UNMAPPED_APPEND; a block shared by several sequences
 * must be copied first by the caller (copy-on-write, [share] 3.2). */
KVC_API int kvc_append(const kvc_desc* d, void* cache, int32_t layer,
                       const void* k_new, const void* v_new, int32_t n_new,
                       const int32_t* pos, const int32_t* block_table,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Rotary positions of kvc_append_qk (host memory): pairs of the first `dim`
 * values of a head, pair i rotated by position * f_i.
 *  pairs      HALF: (i, i + dim / 2); INTERLEAVED: (2 i, 2 i + 1).
 *  dim        rotated values of a head: even, 0 .. head_dim (0: no rotation).
 *  scaling    NONE    f_i = base^(-2 i / dim);
 *             LINEAR  f_i / factor;
 *             YARN    f_i / factor * r_i + f_i (1 - r_i): r_i rises from 0 to 1
 *                     over the pairs between floor(pair_of(fast)) and
 *                     ceil(pair_of(slow)), clamped to 0 .. dim - 1, where
 *                     pair_of(n) = dim ln(original_len / (2 pi n)) / (2 ln base)
 *                     makes n turns within original_len positions;
 *             BANDS   f_i / factor * (1 - r_i) + f_i r_i: r_i rises from 0 to 1
 *                     as the turns original_len f_i / (2 pi) go from slow to fast.
 *  magnitude  factor on the rotated values; 0: 1, and for YARN with factor > 1
 *             0.1 ln(factor) + 1.
 * kvc_rotary_init checks the fields (KVC_ERR_ARG), and fills in magnitude (if
 * it is 0), turns (the frequencies as 2^64ths of a turn, so that position *
 * f_i is reduced exactly), ready and filled.  Zero the struct before its fields
 * are set, and call kvc_rotary_init again after a change of any of them: a
 * magnitude that the call before filled in, and that is still there, counts as
 * 0 and is worked out anew. */
typedef enum { KVC_PAIRS_HALF = 0, KVC_PAIRS_INTERLEAVED = 1 } kvc_pairs;
typedef enum { KVC_SCALING_NONE = 0, KVC_SCALING_LINEAR = 1, KVC_SCALING_YARN = 2, KVC_SCALING_BANDS = 3 }
    kvc_scaling;
typedef struct kvc_rotary {
    int32_t pairs;              /* kvc_pairs */
    int32_t dim;
    int32_t scaling;            /* kvc_scaling */
    int32_t original_len;       /* YARN, BANDS: positions the frequencies were made for */
    float base;                 /* > 1, e.g. 10000 */
    float factor;               /* > 0 (not NONE) */
    float fast;                 /* YARN, BANDS: turns, fast > slow > 0 */
    float slow;
    float magnitude;
    int32_t ready;              /* set by kvc_rotary_init */
    uint64_t turns[128];
    float filled;               /* set by kvc_rotary_init: the magnitude it filled in, 0: the caller's own */
} kvc_rotary;
KVC_API int kvc_rotary_init(kvc_rotary* rotary);

/* Norms and rotation of kvc_append_qk (host memory).  A weight pointer is
 * device memory, [head_dim] in the element type of q, 16-byte aligned; NULL:
 * that side is not normed. */
typedef struct kvc_qk {
    const kvc_rotary* rotary;   /* NULL: no rotation */
    const void* q_weight;
    const void* k_weight;
    float eps;                  /* >= 0; with 0 a zero row becomes NaN */
    float weight_offset;        /* added to every weight (1 for weights stored as w - 1) */
} kvc_qk;

/* The step between a layer's projection and its attention, in one pass: for
 * each token, every q and k head is normed, x / sqrt(mean(x^2) + eps) *
 * (weight + weight_offset), and rotated; q goes to q_out, k and v are
 * appended to layer `layer` of the cache as kvc_append appends them.  The
 * attention that follows uses the same descriptor, whose rope is NONE: the
 * rotation is done here.  The keys go to the cache alone, for decode steps;
 * kvc_prefill takes a chunk's rows itself and appends them.  (READ_INCACHE
 * caches take the norms alone, no rotation, else KVC_ERR_UNSUPPORTED; BAKED
 * caches are refused the same way, their decode would rotate q again.)
 *   q             [batch, n_new, q_heads, head_dim], k_new and v_new
 *                 [batch, n_new, kv_heads, head_dim]: token i of sequence b
 *                 starts at (b n_new + i) * stride elements, its heads dense.
 *                 A stride of 0 means dense; others are at least a token's
 *                 elements and multiples of 16 bytes, so that the three may
 *                 lie side by side in one projection's output.
 *   pos           [batch] int32: position of token 0 of each sequence.
 *   n_tok         [batch] int32 or NULL: tokens 0 .. n_tok[b] - 1 of sequence
 *                 b are real, those behind them padding (NULL: all n_new).
 *   q_out         [batch, n_new, q_heads, head_dim] dense; may be q itself
 *                 when q is dense, otherwise it overlaps no input.
 * Padding tokens and tokens at negative positions may hold anything; their
 * q_out rows stay as they were.  Device errors as in kvc_append (the token's q_out
 * is written all the same).  All arithmetic is fp32 and every stored value is
 * rounded once.  All pointers are 16-byte aligned but pos, n_tok and
 * block_table. */
KVC_API int kvc_append_qk(const kvc_desc* d, void* cache, int32_t layer, const void* q, const void* k_new,
                          const void* v_new, int32_t q_stride, int32_t k_stride, int32_t v_stride, int32_t n_new,
                          const int32_t* pos, const int32_t* n_tok, const int32_t* block_table,
                          const kvc_qk* qk, void* q_out, void* workspace, size_t workspace_bytes, void* stream);

/* Decode attention for one layer ([primer] 2.2 and 4.2, [sink] softmax
 * equations): out = softmax(q . K^T * scale) . V over the attended set of
 * each sequence, fp32 online softmax, split over the KV length into partial
 * results (m, l, o) in the workspace.  fp32 caches combine the partials in
 * the same kernel (the last CTA of a sequence); bf16 and INT8 caches launch
 * a separate combine kernel right behind the attention kernel (programmatic
 * dependent launch).  PAGED batches run a planning kernel before the
 * attention kernel (per sequence: attended rows, attended-block directory,
 * the readers of each block); a single paged sequence on a bf16 or INT8
 * cache is planned inside the attention kernel.
 *   q       [batch, q_heads, head_dim], pre-RoPE.
 *   pos     [batch] int32: position t of the token being decoded (already
 *           appended, so t attends to itself; [ring] 4.3).
 *   block_table, valid_bits  PAGED only (else NULL): block_table as in
 *           kvc_append; valid_bits [ceil(num_blocks / 32)] uint32, bit
 *           (k & 31) of word k / 32 set when physical block k is resident.
 *           valid_bits NULL = every block resident.
 *   out     [batch, q_heads, head_dim], same element type as q.
 * An empty attended set (a fully masked PAGED sequence) gives zeros. */
KVC_API int kvc_decode_attention(const kvc_desc* d, const void* cache, int32_t layer,
                                 const void* q, const int32_t* pos,
                                 const int32_t* block_table, const uint32_t* valid_bits,
                                 void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Score modifiers (host memory; slopes and start are device memory).  With
 * x = q . k * scale for a query of head h at position t and a key at p,
 *     s = x                                   softcap = 0
 *     s = softcap * tanh(x / softcap)         softcap > 0
 *     s = s - slopes[h] * (t - p)             slopes not NULL
 * and keys below the query's start are not attended (sinks among them): the
 * document it belongs to begins there.  A value below 0 counts as 0.
 * A softcap is 0 or KVC_SOFTCAP_MIN .. KVC_SOFTCAP_MAX (else KVC_ERR_ARG); a
 * capped score is off by a few 2^-23 softcap.
 * Cached rows below every start of their sequence may hold anything; all other
 * rows up to the query's position hold finite values, as for kvc_prefill. */
#define KVC_SOFTCAP_MIN 0.0009765625f
#define KVC_SOFTCAP_MAX 1024.0f
typedef struct kvc_score {
    const float* slopes;        /* [q_heads] or NULL */
    const int32_t* start;       /* decode [batch], prefill [batch, T]; or NULL */
    float softcap;              /* 0: none */
} kvc_score;

/* kvc_decode_attention with modified scores.  RING, SINK_RING and PAGED
 * caches, every element type; rope NONE or BAKED (READ_INCACHE is refused with
 * KVC_ERR_UNSUPPORTED).  A token whose start lies above its position attends
 * nothing and gets zeros.  PAGED blocks wholly below the start are not read,
 * nor are most bf16 and INT8 window rows below it. */
KVC_API int kvc_decode_attention_scored(const kvc_desc* d, const void* cache, int32_t layer, const void* q,
                                        const int32_t* pos, const int32_t* block_table, const uint32_t* valid_bits,
                                        const kvc_score* score, void* out, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* kvc_decode_attention for a PAGED batch whose groups of sequences share a
 * prefix (kvc_block_share): the shared keys and values are read and scored once
 * for a whole group.  The results are kvc_decode_attention's, whatever the
 * groups are (to the rounding of another order of sums): the call itself finds
 * how many leading blocks the tables of a group's sequences have in common,
 * among those that lie wholly at positions <= t for each of them.  It pays where
 * many mapped tokens are shared: from about 150,000 (sequences x shared tokens,
 * 8 kv heads of 128; 64 sequences in groups of 8 with 2048 shared tokens of up to
 * 8192 each: 200 us against kvc_decode_attention's 179, 32 readers of 16384
 * tokens: 105 against 200).  Below that kvc_decode_attention, which takes a
 * shared block from the L2 cache, is faster.
 *   group      [batch] int32: sequences with the same value 0 .. batch - 1 form
 *              a group; below 0: alone.  batch or more sets KVC_DEV_BAD_ENTRY
 *              (the sequence counts as alone).  Members without a whole block in
 *              common with the group's first that has one (idle slots, another
 *              prompt) count as alone; the others share what they all have.
 *   workspace  kvc_shared_workspace_bytes(d) bytes (0 if `d` is refused), set
 *              up by kvc_workspace_init; it serves the other decode calls too.
 * bf16 caches, blocks whose size is a multiple of 8 and divides 64 or is a
 * multiple of 64, at most 128 q heads for each kv head, else
 * KVC_ERR_UNSUPPORTED; rope NONE or BAKED.  The shared part runs on the tcgen05
 * tensor cores, one CTA per SM that holds its tensor memory while it runs. */
KVC_API size_t kvc_shared_workspace_bytes(const kvc_desc* d);
KVC_API int kvc_decode_attention_shared(const kvc_desc* d, const void* cache, int32_t layer, const void* q,
                                        const int32_t* pos, const int32_t* group, const int32_t* block_table,
                                        const uint32_t* valid_bits, void* out, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Long caches read in part: every block of a PAGED cache keeps the ends of its
 * keys, channel by channel; a decode step asks them which blocks can hold large
 * scores, and attends those alone.  Every element type and rope NONE or BAKED
 * (the keys as the cache stores them); kvc_decode_attention_selected bf16 and
 * INT8 caches.  Tables of at most 2^30 blocks a sequence, here, in
 * kvc_decode_attention_weighed and in kvc_block_evict (else KVC_ERR_UNSUPPORTED).
 *
 * Bounds of the blocks, caller-owned memory of kvc_bounds_bytes(d) bytes (0 if
 * `d` is refused), 16-byte aligned: int8 codes [layers, num_blocks, kv_heads, 2,
 * head_dim], at index 0 the largest key value of each channel, at 1 the
 * smallest, then fp32 steps [layers, num_blocks, kv_heads]:
 *     step = max over channels of max(|largest|, |smallest|) / 127,
 *     codes ceil(largest / step) and floor(smallest / step), clamped to +-127
 * (IEEE fp32 quotients; a step of 0 has codes 0).  A code * step lies outside of
 * its keys, or inside by no more than the fp32 roundings of step and quotient:
 * 2^-23 of the block's largest |key| of that head, where that is 127 * 2^-126
 * or more (smaller keys have a step that is no normal number, or 0).
 *
 * kvc_block_bounds works them out for every logical block that holds one of the
 * positions pos[b] .. pos[b] + n - 1 (n = n_tok[b], cut to 0 .. n_new; NULL:
 * n_new), from the block's first row to position pos[b] + n - 1: call it after
 * the append of those tokens, and after a block was copied (kvc_block_prepare)
 * or brought in.  Positions below 0 are padding.  A block that several
 * sequences map is written by each of them: they have to reach the same row of
 * it, or its codes and step may come from different ones.  Keys are finite.
 * Device errors as in kvc_append.  Workspace: kvc_workspace_bytes(d). */
KVC_API size_t kvc_bounds_bytes(const kvc_desc* d);
KVC_API int kvc_block_bounds(const kvc_desc* d, const void* cache, int32_t layer, void* bounds, const int32_t* pos,
                             int32_t n_new, const int32_t* n_tok, const int32_t* block_table, void* workspace,
                             size_t workspace_bytes, void* stream);

/* The k blocks of each sequence and kv head that a query at pos[b] is to attend.
 * With the query of a q head as codes c = rint(q / s_q), s_q = max|q| / 127
 * (rotated first when BAKED), a block's score is
 *     max over the kv head's q heads of  u * (s_q * step),
 *     u = sum over channels of max(c * largest code, c * smallest code),
 * u a whole number, the products fp32.  Candidates are the blocks 0 .. pos[b] /
 * block_size that are mapped and resident.  The first `first` and the last
 * `recent` of these numbers (mapped or not) are always in, the others by score,
 * equal scores by the lowest number.
 *   q        [batch, q_heads, head_dim], pre-RoPE, 16-byte aligned, finite.
 *   k        1 .. 2^24; first >= 0, recent >= 1, first + recent <= k (else
 *            KVC_ERR_ARG).  At most 128 q heads for each kv head.
 *   blocks   [batch, kv_heads, k] int32, out: logical blocks, ascending, -1
 *            behind the last.
 *   workspace  kvc_select_workspace_bytes(d, k) bytes (0 if refused), set up by
 *            kvc_workspace_init; it serves the other decode calls too. */
KVC_API size_t kvc_select_workspace_bytes(const kvc_desc* d, int32_t k);
KVC_API int kvc_select_blocks(const kvc_desc* d, const void* bounds, int32_t layer, const void* q, const int32_t* pos,
                              int32_t k, int32_t first, int32_t recent, const int32_t* block_table,
                              const uint32_t* valid_bits, int32_t* blocks, void* workspace, size_t workspace_bytes,
                              void* stream);

/* kvc_decode_attention over listed blocks of a PAGED bf16 or INT8 cache: the
 * query of q head h attends the positions <= pos[b] of the blocks that
 * blocks[b][h / (q_heads / kv_heads)] lists.
 *   blocks   [batch, kv_heads, k] int32, ascending; negative entries are none.
 *            An entry past the table, or not above those before it (a block
 *            listed twice), sets KVC_DEV_BAD_ENTRY and is left out.  Blocks that
 *            are unmapped, not resident or past the position are not attended.
 *   workspace  kvc_select_workspace_bytes(d, k) bytes.
 * An empty list gives zeros. */
KVC_API int kvc_decode_attention_selected(const kvc_desc* d, const void* cache, int32_t layer, const void* q,
                                          const int32_t* pos, const int32_t* blocks, int32_t k,
                                          const int32_t* block_table, const uint32_t* valid_bits, void* out,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* kvc_decode_attention of a PAGED bf16 or INT8 cache that also adds up how much
 * weight each block receives: for every entry of weights [batch,
 * max_blocks_per_seq] fp32,
 *     weights = decay * weights + sum over q heads and over the block's attended
 *               positions of the softmax weight (0 for a block that is not
 *               attended),
 * in an order of sums that depends on nothing but the shapes.  decay 0 .. 1 (else
 * KVC_ERR_ARG); with 0 the old values are not read.  One array can take several
 * layers' calls, the decay given to the step's first.  The caller zeroes a
 * sequence's row when another sequence takes its place.
 *   workspace  kvc_weighed_workspace_bytes(d) bytes (0 if `d` is refused): the
 *              decode workspace, which it serves as too, and a score for every q
 *              head and position. */
KVC_API size_t kvc_weighed_workspace_bytes(const kvc_desc* d);
KVC_API int kvc_decode_attention_weighed(const kvc_desc* d, const void* cache, int32_t layer, const void* q,
                                         const int32_t* pos, const int32_t* block_table, const uint32_t* valid_bits,
                                         float decay, float* weights, void* out, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* Attention of a tree of drafted tokens over a cache, as speculative decoding
 * verifies it: token i of sequence b continues token parent[b][i] of the draft
 * (-1: the sequence's last cached token), stands at position pos0[b] + its depth
 * (0 for a token whose parent is -1) and attends what a token there attends of the
 * positions below pos0[b], read from the cache as it stands, the tokens above it
 * in the draft and itself.  Nothing is appended (kvc_append_path does that for
 * the path that is kept).
 *   q            [batch, T, q_heads, head_dim] bf16, pre-RoPE.
 *   k_new, v_new [batch, T, kv_heads, head_dim] bf16, pre-RoPE.
 *   T            1 .. KVC_TREE_MAX (else KVC_ERR_ARG).
 *   pos0         [batch] int32: tokens in the cache.  Below 0: idle, zeros.
 *   parent       [batch, T] int32: -1 .. i - 1.  Below -1: no token (padding; its
 *                rows may hold anything).  i or more sets KVC_DEV_BAD_ENTRY and
 *                counts as no token.  What continues no token is none either; it
 *                gets zeros.
 *   block_table, valid_bits  PAGED as in kvc_decode_attention.
 *   out          [batch, T, q_heads, head_dim] bf16.
 *   workspace    kvc_tree_workspace_bytes(d, T) bytes (0 if refused), set up by
 *                kvc_workspace_init; it serves the decode calls too.
 * bf16 caches, rope NONE or BAKED, at most 128 q heads for each kv head; window
 * layouts with T <= window, paged ones with blocks whose size is a multiple of 8
 * and divides 64 or is a multiple of 64 (else KVC_ERR_UNSUPPORTED).  Cached rows
 * below pos0[b] and the tokens' rows hold finite values.  PAGED positions past the
 * table's end set KVC_DEV_BAD_POSITION; the table's are attended.  It runs on
 * the tcgen05 tensor cores, one CTA per SM that holds its tensor memory while it
 * runs. */
#define KVC_TREE_MAX 64
KVC_API size_t kvc_tree_workspace_bytes(const kvc_desc* d, int32_t T);
KVC_API int kvc_tree_attention(const kvc_desc* d, const void* cache, int32_t layer, const void* q, const void* k_new,
                               const void* v_new, int32_t T, const int32_t* pos0, const int32_t* parent,
                               const int32_t* block_table, const uint32_t* valid_bits, void* out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The accepted path of a tree of drafted tokens, appended: token path[b][j] of
 * the draft goes to position pos0[b] + j, for j < n_path[b], as kvc_append of
 * those tokens would put it (any layout, element type and rope).
 *   k_new, v_new  [batch, T, kv_heads, head_dim], pre-RoPE, 16-byte aligned.
 *   path          [batch, P] int32, entries 0 .. T - 1; another among the first
 *                 n_path[b] sets KVC_DEV_BAD_ENTRY and its position is not
 *                 written.
 *   n_path        [batch] int32 (NULL: P for all); above P counts as P
 *                 (KVC_DEV_BAD_ENTRY), below 0 as 0.
 * Sequences with pos0[b] < 0 append nothing.  Other device errors as in
 * kvc_append: PAGED, every block that the path reaches is mapped, and private to
 * the sequence, before the call (kvc_block_prepare at pos0[b] and at the first
 * row of each further block; it readies one position's block a call).
 * Workspace: kvc_workspace_bytes(d). */
KVC_API int kvc_append_path(const kvc_desc* d, void* cache, int32_t layer, const void* k_new, const void* v_new,
                            int32_t T, const int32_t* pos0, const int32_t* path, int32_t P, const int32_t* n_path,
                            const int32_t* block_table, void* workspace, size_t workspace_bytes, void* stream);

/* One decode step: kvc_append of the token at pos[b] (n_new = 1), then
 * kvc_decode_attention at pos[b], with the same arguments and results as
 * that pair of calls.  For bf16 and INT8 caches, RING / SINK_RING and PAGED
 * with one sequence (planned inside the attention kernel), the append is
 * fused into the attention kernel (the CTA that reads the token's row writes
 * it, with RoPE baked when BAKED, to the cache and to its own copy of the
 * tile); on other PAGED caches the planning kernel writes the tokens before
 * the attention kernel reads; fp32 RING / SINK_RING caches make the two calls
 * in turn.
 *   k_new, v_new  [batch, kv_heads, head_dim], pre-RoPE, 16-byte aligned. */
KVC_API int kvc_decode_step(const kvc_desc* d, void* cache, int32_t layer, const void* q,
                            const void* k_new, const void* v_new, const int32_t* pos,
                            const int32_t* block_table, const uint32_t* valid_bits,
                            void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Chunked prefill ([pool] "the real cost of long context": prefill in chunks
 * of 128-256 tokens; [ring] 3.1 and 5.2: the window as a mask on the score
 * matrix).  For each sequence b, T consecutive tokens at positions
 * pos0[b] + i (i < T): token i gets the output the decode step at that
 * position would give after the chunk's earlier tokens were appended --
 * attention of its q over its attended set A(pos0[b] + i), keys before
 * pos0[b] read from the cache as it stands (the state after position
 * pos0[b] - 1), the chunk's keys from k_new / v_new -- and then the chunk is
 * appended to the cache as kvc_append(n_new = T) would.  Positions below 0
 * are left padding: zero output, nothing appended.  PAGED positions past the
 * block table's end set KVC_DEV_BAD_POSITION; the keys before the chunk are
 * then those of the table.
 *   q          [batch, T, q_heads, head_dim] bf16, pre-RoPE.
 *   k_new, v_new [batch, T, kv_heads, head_dim] bf16, pre-RoPE.
 *   pos0       [batch] int32.
 *   block_table, valid_bits  PAGED as in kvc_decode_attention; the chunk's
 *              blocks must be mapped (the append reports unmapped ones).
 *   out        [batch, T, q_heads, head_dim] bf16.
 *   workspace  kvc_prefill_workspace_bytes(d, T) bytes: the decode workspace
 *              followed by the chunk's staged rows.
 * READ_INCACHE: each token's window keys at distance t - p and its sinks at
 * min(t, C - 1) - p, as the decode step at t rotates them.
 * bf16 caches (head_dim 64, 128 or 256) and INT8 caches (128 or 256: cached
 * rows are read back as code * scale, the chunk's own rows as the cache will
 * read them back).  KVC_ERR_UNSUPPORTED: an fp32 cache; at head_dim 256 or on
 * an INT8 cache, a ring or sink+ring chunk longer than the window, paged
 * blocks whose size is not a multiple of 8 dividing 64, or a GQA group that
 * does not divide 128.  Calls on one workspace must not overlap on the
 * GPU.  The attention runs on the tcgen05 tensor cores: a CTA of the
 * warp-specialised kernel (one per SM) holds all 512 tensor-memory columns
 * of its SM while it runs (the kernel for chunks longer than the window: 256
 * columns, two CTAs per SM), so a kernel of another library that holds an
 * SM's tensor memory at the same time delays it.  A wait that does not end
 * within its bound sets KVC_DEV_TIMEOUT in the device error word and the
 * CTA returns, leaving that chunk's output undefined. */
KVC_API size_t kvc_prefill_workspace_bytes(const kvc_desc* d, int32_t T);
KVC_API int kvc_prefill(const kvc_desc* d, void* cache, int32_t layer, const void* q,
                        const void* k_new, const void* v_new, int32_t T, const int32_t* pos0,
                        const int32_t* block_table, const uint32_t* valid_bits,
                        void* out, void* workspace, size_t workspace_bytes, void* stream);

/* kvc_prefill with modified scores: start is [batch, T], one for each token
 * of the chunk, so that documents packed into a sequence attend only
 * themselves.  bf16 and INT8 caches, any GQA group of up to 128 heads, rope
 * NONE or BAKED; window layouts take chunks no longer than the window, paged
 * ones blocks whose size is a multiple of 8 dividing 64 (else
 * KVC_ERR_UNSUPPORTED).  With a softcap and no slopes, values beyond 2^57 in
 * magnitude may overflow the sums.  Workspace as for kvc_prefill. */
KVC_API int kvc_prefill_scored(const kvc_desc* d, void* cache, int32_t layer, const void* q,
                               const void* k_new, const void* v_new, int32_t T, const int32_t* pos0,
                               const int32_t* block_table, const uint32_t* valid_bits, const kvc_score* score,
                               void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Batched block-table update ([share] 3.1 block table, 5.1 block manager):
 * for each i < n, block_table[seq[i]][logical_block[i]] = physical_block[i];
 * -1 unmaps.  When valid_bits is not NULL, each mapped physical block gets its
 * valid bit set (the data is in place); unmapping does not touch valid bits,
 * since other sequences may still map that block.  Entries out of range set
 * KVC_DEV_BAD_ENTRY and are skipped.  Two entries naming the same
 * (seq, logical_block) in one call: which one lands is unspecified. */
KVC_API int kvc_block_table_write(const kvc_desc* d, int32_t* block_table, uint32_t* valid_bits,
                                  int32_t n, const int32_t* seq, const int32_t* logical_block,
                                  const int32_t* physical_block,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Batched residency update ([pool] "kernel forgets absent blocks"): for each
 * i < n, set (value[i] != 0) or clear the valid bit of physical block slot[i]. */
KVC_API int kvc_valid_write(const kvc_desc* d, uint32_t* valid_bits, int32_t n,
                            const int32_t* slot, const int32_t* value,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Block manager of a paged cache ([share] 3.1-3.2 block table and prefix
 * sharing, 5.1 block manager, 6.1 reclaim on sequence end).  State, all
 * caller-owned device memory: the block table and valid bits as above,
 * refcount int32 [num_blocks] (table references of each block), free_list
 * int32 [num_blocks] used as a stack (entries 0 .. *free_count - 1, top last)
 * and free_count (one int32).  Start: table -1, refcount 0, free_list any
 * permutation of the blocks, *free_count = num_blocks, valid bits 0.
 * Within one call sequences are served in ascending order, exactly as one
 * after the other, so the results are deterministic. */

/* Before appending each sequence's next token (pos[b]; < 0: none), once per
 * token for all layers: a token at a block's first row whose logical block
 * is unmapped gets a new block from the top of the free list; a block
 * referenced by more than one sequence (count > 1) is copied first: a new
 * block receives its rows 0 .. pos mod block_size - 1 of every layer, K and
 * V, every kv head, the sequence's entry points at it, the shared block's
 * count drops by one (copy-on-write, [share] 3.2).  New blocks get count 1
 * and their valid bit (valid_bits may be NULL).  Errors (device bits): an
 * unmapped block entered mid-block (KVC_DEV_UNMAPPED_APPEND), a position past
 * the table (KVC_DEV_BAD_POSITION), an exhausted free list
 * (KVC_DEV_NO_FREE_BLOCK); the sequence is skipped.  Requires layers * 2 *
 * kv_heads <= 65535 (the copy's launch grid), else KVC_ERR_UNSUPPORTED. */
KVC_API int kvc_block_prepare(const kvc_desc* d, void* cache, const int32_t* pos, int32_t* block_table,
                              uint32_t* valid_bits, int32_t* refcount, int32_t* free_list, int32_t* free_count,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Prefix sharing ([share] 3.2, 5.1 share_prefix): for each i < n, logical
 * blocks 0 .. nblocks[i] - 1 of sequence dst_seq[i] point at those of
 * src_seq[i]; each shared block's count rises by one.  The destination's
 * entries must be unmapped, else KVC_DEV_BAD_ENTRY and the entry is skipped. */
KVC_API int kvc_block_share(const kvc_desc* d, int32_t* block_table, int32_t* refcount, int32_t n,
                            const int32_t* src_seq, const int32_t* dst_seq, const int32_t* nblocks,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Sequences end ([share] 6.1): for each listed sequence every mapped block's
 * count drops by one and its entry is unmapped; blocks whose count reaches
 * zero return to the free list in ascending block id and lose their valid
 * bit.  A sequence listed twice is released twice (caller error). */
KVC_API int kvc_block_release(const kvc_desc* d, int32_t* block_table, uint32_t* valid_bits, int32_t* refcount,
                              int32_t* free_list, int32_t* free_count, int32_t n, const int32_t* seq,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Blocks given back by weight: of each sequence's mapped blocks 0 .. pos[b] /
 * block_size, those beyond `keep` go, the lightest (weights, as
 * kvc_decode_attention_weighed adds them up) first, equal ones by the lowest
 * number; the first `first` and the last `recent` of these numbers stay.  A block
 * that goes is unmapped, its count drops by one and its weight becomes 0; blocks
 * whose count reaches zero return to the free list in ascending block id and
 * lose their valid bit (valid_bits may be NULL).  Later positions attend what is
 * left.  A weight that is NaN counts as the heaviest.  Sequences with pos[b] < 0
 * stay as they are.
 *   weights  [batch, max_blocks_per_seq] fp32.
 *   keep     >= first + recent, first >= 0, recent >= 1 (else KVC_ERR_ARG). */
KVC_API int kvc_block_evict(const kvc_desc* d, float* weights, const int32_t* pos, int32_t keep, int32_t first,
                            int32_t recent, int32_t* block_table, uint32_t* valid_bits, int32_t* refcount,
                            int32_t* free_list, int32_t* free_count, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Paging of a fixed pool of block slots between host memory and the device
 * ([pool] "KV cache paging": a fixed pool of resident slots; blocks move on
 * demand; the copy engine moves them while attention runs; LRU residency;
 * blocks inside a sliding window stay resident).  A paged cache whose
 * num_blocks slots hold logical blocks of sequence `seq`; the block table maps
 * resident logical blocks to their slot, absent ones to -1 (valid bit off).
 * The host copy of the K/V is pinned memory laid out
 * [logical block][layer][K|V][kv head][row][head_dim] in the cache dtype. */
typedef struct kvc_pager kvc_pager;

/* Host object tracking num_slots slots; NULL if num_slots < 1. */
KVC_API kvc_pager* kvc_pager_create(int32_t num_slots);
KVC_API void kvc_pager_destroy(kvc_pager* pager);

/* Host only.  The blocks one step needs (need[0 .. n-1], logical block ids;
 * pinned[i] != 0 keeps block need[i] resident in later steps until a later
 * call lists it with pinned 0; pinned may be NULL).  Missing blocks take, in
 * list order, the lowest free slot, else the least recently used slot whose
 * block is neither needed now nor pinned (ties: lowest slot).  Outputs (host
 * arrays of n entries): the page-ins (in_block, in_slot; *n_in) and the
 * victims (out_block, out_slot; *n_out).  KVC_ERR_ARG, nothing changed, if the
 * needed and pinned blocks do not fit. */
KVC_API int kvc_pager_plan(kvc_pager* pager, int32_t n, const int32_t* need, const uint8_t* pinned,
                           int32_t* n_in, int32_t* in_block, int32_t* in_slot,
                           int32_t* n_out, int32_t* out_block, int32_t* out_slot);

/* Compute stream: the victims' table entries (sequence seq) become -1 and
 * their slots' valid bits clear.  Host arrays; asynchronous. */
KVC_API int kvc_pager_evict(const kvc_desc* d, int32_t seq, int32_t n, const int32_t* out_block,
                            const int32_t* out_slot, int32_t* block_table, uint32_t* valid_bits, void* stream);

/* Copy stream, after the compute stream's work enqueued so far: one 2-D copy
 * per block (every layer, K and V) from host_kv into its slot, then an event
 * kept by the pager.  Work enqueued on the compute stream after this call
 * overlaps the copies. */
KVC_API int kvc_pagein_issue(kvc_pager* pager, const kvc_desc* d, void* cache, const void* host_kv, int32_t n,
                             const int32_t* in_block, const int32_t* in_slot, void* copy_stream,
                             void* compute_stream);

/* Compute stream waits for the last issue's copies, then the blocks' table
 * entries point at their slots and the slots' valid bits are set. */
KVC_API int kvc_pagein_commit(kvc_pager* pager, const kvc_desc* d, int32_t seq, int32_t n, const int32_t* in_block,
                              const int32_t* in_slot, int32_t* block_table, uint32_t* valid_bits,
                              void* compute_stream);

/* Size of the library's own fixed scratch array used by
 * kvc_decode_attention_noalloc: 8 MiB of device memory, reserved on every GPU
 * that loads the library, from the first use until the process exits. */
#define KVC_NOALLOC_SCRATCH_BYTES (8u << 20)

/* kvc_decode_attention for callers that cannot allocate device memory.
 *
 * Same operation, arguments and results as kvc_decode_attention, except that
 * the caller passes no workspace: the split-K partial results, completion
 * counters and (PAGED) work plan live in a fixed scratch array inside the
 * library (KVC_NOALLOC_SCRATCH_BYTES).  It is meant for code that must not
 * call cudaMalloc once it is running - a serving loop whose device memory is
 * fixed when it starts, or a plugin inside a host framework that owns all
 * device memory and offers no way to allocate - and so has nowhere to put a
 * workspace.  The pages have no counterpart of this entry point.
 *
 *   - It allocates nothing: no cudaMalloc / cudaFree, no allocating library
 *     call.  Inputs and outputs are still the caller's device buffers.
 *   - The first call on a device (with that device current) looks up the
 *     scratch array's device address; make that first call before any stream
 *     capture.  The address is kept per device and context: after the
 *     device's context was destroyed and created again (cudaDeviceReset),
 *     the next call looks it up again, so make that call outside capture
 *     too.  Later calls only enqueue work on `stream`.
 *   - Every call on a device shares the one scratch array and finds it as the
 *     previous call left it; the call clears the parts that must start at
 *     zero (error word, completion counters) on `stream` before its kernels.
 *     Calls that overlap on the GPU (different streams, no ordering between
 *     them) race on the scratch and give wrong results: order them.
 *   - A problem whose workspace (kvc_workspace_bytes) exceeds
 *     KVC_NOALLOC_SCRATCH_BYTES is rejected with KVC_ERR_TOO_LARGE before
 *     anything is launched.
 *   - Device-detected errors are not reported: the kernels still skip bad
 *     accesses, but there is no workspace for kvc_get_error to read. */
KVC_API int kvc_decode_attention_noalloc(const kvc_desc* d, const void* cache, int32_t layer,
                                         const void* q, const int32_t* pos,
                                         const int32_t* block_table, const uint32_t* valid_bits,
                                         void* out, void* stream);

/* Wait for `stream`, then return the workspace's device error bits
 * (KVC_DEV_*, 0 = none) and clear them.  Negative KVC_ERR_* on failure. */
KVC_API int kvc_get_error(void* workspace, void* stream);

/* Static description of a status code or device error bit. */
KVC_API const char* kvc_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* KVC_H */
