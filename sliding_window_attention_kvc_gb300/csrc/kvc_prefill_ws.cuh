// Chunked prefill attention on the tcgen05 tensor cores, warp-specialised
// ([pool] chunked prefill of 128-256 tokens; [ring] 3.1 and 5.2, the window as
// a mask on the score matrix; [sink] "RoPE cache position shifting").
//
// One CTA per SM: NQ tiles of 128 (token, q head) rows of one kv head of one
// sequence (NQ = 2 for head_dim 64 and 128, 1 for 256), one TMEM lane per row.
// Roles (warps):
//   0      producer: cuts the keys into 64-row tiles and loads each by TMA into
//          a ring of shared-memory stages ([column block][K|V][64 rows][128 B],
//          128-byte swizzle).  Ring and sink+ring caches are cut in slot space
//          (64 consecutive slots, one box), each slot holding the position it
//          had after position pos0 - 1; paged caches in blocks (the mapped and
//          valid blocks, packed 64 / bs to a tile); then the chunk's own rows
//          from the staged copy, 64 tokens to a tile.  It records each row's
//          position (-1: no key).
//   1 (3)  issue the tcgen05.mma (one thread of the warp):  S_i = Q_i K^T  into
//          one of two S buffers per Q tile, then O_i += P_i V; S of tile j + 1
//          is issued before P V of tile j, so the softmax of one tile overlaps
//          the products of the next.  Two issuing warps, one for each Q tile,
//          when one fix-up warp will do (bf16 rows without read-time RoPE).
//   2 (3)  fix-up: zero the V rows of absent keys (they may hold anything),
//          expand INT8 rows and, for read-time RoPE, rotate the raw K rows at
//          their positions.
//   4-7    softmax of Q tile 0 (one thread per row): masks (window, sinks,
//   (8-11)  causal), online softmax in base 2 with a lazy reference max (moved
//          only when a tile's max exceeds it by more than 8: probabilities stay
//          below 2^8), bf16 P into the S buffer it came from, O rescaled in TMEM
//          when the reference moved; at the end O / l to the output.
// Every wait is bounded (~1 s); a timeout sets KVC_DEV_TIMEOUT and every role
// stops; the CTA waits for its copies and products before freeing TMEM.
#pragma once

#include <atomic>
#include <type_traits>

#include "kvc_decode.cuh"
#include "kvc_tc.cuh"

namespace kvc {

namespace {

constexpr int kWsSoftmax0 = 4;              // first softmax warp
constexpr float kWsLazy = 8.f;

// Score modifiers a kernel is built for: a branch for each inside one kernel held the
// softmax to a schedule two to three times as long as the branch taken alone.
// kModFixed: capped scores alone, |s| <= cap2 <= kWsFixedCap in base 2: the reference
// is a constant and no maximum is sought.  It is the cap itself (weights <= 1, as with
// a sought maximum) while the smallest weight, 2^(-2 cap2), stays at or above 2^-100;
// with larger caps that smallest weight is kept there and the largest grows to 2^50:
// values up to 2^57 in magnitude still sum over 2^20 keys.  (8 rings of 4096, 256 tokens,
// cap 20: 259 us with the maximum, 232 us without.)
constexpr float kWsFixedCap = 75.f;
enum : int { kModPlain = 0, kModScore = 1, kModCap = 2, kModBias = 4, kModFixed = 8 };

enum : int { kTileSlot = 0, kTileSink = 1, kTileBlocks = 2, kTileStage = 3, kTileEnd = 4 };

template <int D>
struct WsShape {
    static constexpr int NQ = D == 256 ? 1 : 2;
    static constexpr int STAGES = D == 64 ? 4 : (D == 128 ? 4 : 2);
    static constexpr int CB = D / 64;                          // 64-column blocks of a row
    static constexpr int QBytes = kWsRows * D * 2;             // one Q tile
    static constexpr int KVBlock = 2 * kWsKeys * 128;          // one column block of K and V
    static constexpr int StageBytes = CB * KVBlock;            // K and V of 64 keys
    static constexpr int OffQ = 0;
    static constexpr int OffStage = OffQ + NQ * QBytes;
    static constexpr int OffP = OffStage + STAGES * StageBytes;   // (P lives in tensor memory)
    // INT8 caches: row scales of each stage's cache tile, [stage][K|V][68]:
    // copied from a row that is a multiple of 4 (whole 16-byte copies), the
    // tile's first row sc_off after it
    static constexpr int ScRows = kWsKeys + 4;
    static constexpr int OffScale = OffP;
    static constexpr int OffMeta = OffScale + STAGES * 2 * ScRows * 4;
    static constexpr int TmemCols = 512;
    static constexpr int SCol0 = NQ * D;                       // S buffers after the O tiles
    static_assert(NQ * D + NQ * 2 * kWsKeys <= TmemCols, "TMEM columns");
    // 4 control warps, then 4 softmax warps per Q tile (one thread per row)
    static constexpr int Threads = 32 * (kWsSoftmax0 + 4 * NQ);
};

// How the softmax masks a tile's keys: every key seen by every row of the
// CTA (no test), the chunk's own rows (key k at position kbase + k: a range
// test), or key by key from pos[].
enum : int { kMaskNone = 0, kMaskRange = 1, kMaskKeys = 2 };

struct alignas(16) WsStageMeta {
    int kind;
    int any_absent;          // some row has no key (its V is zeroed)
    int mask;                // kMaskNone / kMaskRange / kMaskKeys
    int kbase;               // kMaskRange: position of key 0
    int sc_off;              // INT8 cache tile: row 0's scale in the stage's scale area
    alignas(16) int pos[kWsKeys];   // position of each row, -1 = none
    alignas(16) float rel[kWsKeys]; // modified scores: position less pos0, for the distance bias
};

// the barriers follow the stages' records: whole 16-byte records keep them aligned
static_assert(sizeof(WsStageMeta) % 16 == 0, "stage records keep the barriers aligned");

struct WsBars {
    uint64_t full[4], ready[4], empty[4];
    uint64_t s_full[2][2], s_free[2][2], p_full[2], o_done[2], q_ready[2], fin[2];
    uint64_t fixb;           // INT8 with read-time RoPE: the fix-up threads, between expansion and rotation
    uint32_t tmem;
    int ntiles;              // set when the producer's end marker reaches the MMA thread
    int abort;
};

template <int D>
constexpr int ws_smem_bytes() {
    using S = WsShape<D>;
    return S::OffMeta + S::STAGES * (int)sizeof(WsStageMeta) + (int)sizeof(WsBars) + 1024;
}

// tile offsets inside a stage
__device__ __forceinline__ int ws_off(int r, int ch) {    // K row r, 16-byte chunk ch (of the row's D/8)
    return (ch >> 3) * (2 * kWsKeys * 128) + r * 128 + (((ch ^ r) & 7) << 4);
}

}  // namespace

// SCORE: scores with modifiers (p.score; no read-time RoPE): q is staged
// unscaled, the softmax warps apply scale, cap and bias to the scores; keys
// below every start of the CTA's tokens are absent, tiles of none but these
// are not loaded, and a GQA group need not divide 128 (rows past the last
// whole token stay empty).
template <int D, bool READ, bool Q8, int MOD>
__global__ void __launch_bounds__(WsShape<D>::Threads, 1)
    prefill_ws_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ PrefillMaps maps) {
    constexpr bool SCORE = MOD != kModPlain, CAP = (MOD & kModCap) != 0, BIAS = (MOD & kModBias) != 0,
                   FIXED = (MOD & kModFixed) != 0;
    static_assert(!FIXED || (CAP && !BIAS), "a fixed reference needs bounded scores");
    static_assert(!Q8 || D >= 128, "INT8 rows are whole 128-code boxes");
    static_assert(!(READ && SCORE), "modified scores: no read-time RoPE");
    using S = WsShape<D>;
    constexpr int NQ = S::NQ, NST = S::STAGES, CB = S::CB;
    // bf16 rows taken as they lie: an issuing warp for each Q tile, the second in the
    // place of a fix-up warp, which has little to do (plain ring, 128-token chunks: 135 ->
    // 122.5 us, paged 1.128 -> 1.123 ms; modified scores: 238 -> 232 and 198 -> 181 us)
    constexpr bool TWO = !READ && !Q8;
    extern __shared__ unsigned char ws_raw[];
    const uint32_t raw_u = smem_u32(ws_raw);
    unsigned char* sm = ws_raw + (((raw_u + 1023u) & ~1023u) - raw_u);
    const uint32_t sm_u = smem_u32(sm);
    WsStageMeta* meta = reinterpret_cast<WsStageMeta*>(sm + S::OffMeta);
    WsBars* bars = reinterpret_cast<WsBars*>(sm + S::OffMeta + NST * sizeof(WsStageMeta));
    volatile int* abort = &bars->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, b = blockIdx.z;
    const int G = p.G;
    const int tq = kWsRows / G;                      // tokens per Q tile
    const int i0 = blockIdx.x * tq * NQ;             // first token of the CTA
    const int pos0 = p.pos0[b];
    const int C = p.capacity;
    const bool paged = p.layout == kPaged;
    const int i_last = min(i0 + tq * NQ, p.T) - 1;   // last token of the CTA
    const int t_hi = pos0 + i_last;                  // its position
    const int t_lo = max(pos0 + i0, 0);
    const int t0 = pos0 - 1;                         // the cache holds positions <= t0
    // read-time RoPE: sink keys are scored with q at min(t, C - 1), so they form
    // tiles of their own, first (only cached sinks: chunk tokens below C need none)
    const int sink_tiles = READ && !paged && t0 >= 0 && t_hi >= 0 ? (min(p.sinks, t0 + 1) + kWsKeys - 1) / kWsKeys : 0;

    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->ready[s], TWO ? 1 : 2);
            mbar_init(&bars->empty[s], TWO ? NQ : 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int u = 0; u < 2; ++u) {
                mbar_init(&bars->s_full[i][u], 1);
                mbar_init(&bars->s_free[i][u], 4);
            }
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->q_ready[i], kWsRows);
        }
        mbar_init(&bars->fin[0], 1);
        mbar_init(&bars->fin[1], 1);
        mbar_init(&bars->fixb, 64);
        bars->ntiles = 0x7fffffff;
        bars->abort = 0;
        mbar_fence_init();
        if (p.layout == kPaged)
            tma_prefetch_desc(&maps.block);
        else
            tma_prefetch_desc(&maps.slot);
        tma_prefetch_desc(SCORE && maps.direct ? &maps.stage_k : &maps.stage);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)),
                     "r"(S::TmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    ws_fence_before();
    __syncthreads();
    ws_fence_after();
    const uint32_t tmem = bars->tmem;
    const long long unit = (long long)b * p.Hkv + h;
    // INT8 cache tiles: the codes of 128 columns (hh) of K or V (kv) land in the
    // stage's upper column blocks, 64 rows of 128 bytes, and are expanded in
    // place (see the fix-up role); their row scales go to the scale area
    auto code_at = [&](int s, int hh, int kv) -> unsigned char* {
        return sm + S::OffStage + s * S::StageBytes + (CB / 2 + hh) * S::KVBlock + kv * (kWsKeys * 128);
    };
    float* sc_area = reinterpret_cast<float*>(sm + S::OffScale);
    auto give_up = [&]() {
        if (!*abort) {
            bars->abort = 1;
            set_error(p.err, 0x8u /* KVC_DEV_TIMEOUT */);
        }
    };

    if (warp == 0) {
        // ============================ producer ==============================
        int idx = 0;
        bool ok = true;
        // SCORE: the lowest and highest start of the CTA's tokens
        int smin = 0, smax = 0;
        if constexpr (SCORE) {
            if (p.score.start && i_last >= i0) {
                smin = 0x7fffffff;
                for (int i = i0 + lane; i <= i_last; i += 32) {
                    const int v = max(0, p.score.start[(long long)b * p.T + i]);
                    smin = min(smin, v);
                    smax = max(smax, v);
                }
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) {
                    smin = min(smin, __shfl_xor_sync(0xffffffffu, smin, off));
                    smax = max(smax, __shfl_xor_sync(0xffffffffu, smax, off));
                }
            }
        }
        // next stage: wait until the MMA thread is done with its last tile
        auto acquire = [&]() -> int {
            const int s = idx % NST;
            if (idx >= NST && !ws_wait(&bars->empty[s], ((idx / NST) - 1) & 1, abort)) {
                if (lane == 0) give_up();
                ok = false;
            }
            return s;
        };
        auto unit_base = [&]() { return (long long)unit * C; };
        // window layouts: slot tiles.  Slot s holds the latest position <= t0
        // with that slot (p = s for sinks), or none.
        auto slot_pos = [&](int s, bool sinks_only, bool no_sinks) -> int {
            if (s >= C || t0 < 0) return -1;
            if (s < p.sinks) return (no_sinks || s > t0 || (SCORE && s < smin)) ? -1 : s;
            if (sinks_only || s > t0) return -1;
            const int q = t0 - (int)((unsigned)(t0 - s) % (unsigned)p.window);
            // window keys any token of the CTA can see
            return q >= t_lo - p.window + 1 && (!SCORE || q >= smin) ? q : -1;
        };
        auto issue_slot_tile = [&](int slot0, int kind) {
            const int s = acquire();
            if (!ok) return;
            int absent = 0, partial = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = lane + 32 * u;
                const int q = slot_pos(slot0 + r, kind == kTileSink, READ && kind == kTileSlot);
                meta[s].pos[r] = q;
                if constexpr (SCORE) {
                    meta[s].rel[r] = (float)(q - pos0);
                    partial |= q >= 0 && q < smax;
                }
                absent |= q < 0;
                // seen by every row of the CTA: a sink, or in the window of its
                // latest token (every key here is below the chunk's first position)
                partial |= q >= p.sinks && q <= t_hi - p.window;
            }
            absent = __any_sync(0xffffffffu, absent);
            partial = __any_sync(0xffffffffu, partial);
            __syncwarp();
            if (lane == 0) {
                meta[s].kind = kind;
                meta[s].any_absent = absent;
                meta[s].mask = (absent || partial) ? kMaskKeys : kMaskNone;
                unsigned char* dst = sm + S::OffStage + s * S::StageBytes;
                if constexpr (Q8) {
                    // codes by 128-column boxes; scales of the rows inside the half
                    // (a multiple of 4: whole 16-byte copies)
                    const long long urow = unit_base() + slot0, base4 = urow & ~3LL;
                    const int nsc = (int)min((long long)S::ScRows, p.half_rows - base4);   // a multiple of 4
                    meta[s].sc_off = (int)(urow - base4);
                    mbar_expect_tx(&bars->full[s], (uint32_t)(2 * (D / 128) * kWsKeys * 128 + 2 * nsc * 4));
#pragma unroll
                    for (int hh = 0; hh < D / 128; ++hh)
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv)
                            tma_load_4d(code_at(s, hh, kv), &maps.slot, 128 * hh, (int)urow, kv, p.layer, &bars->full[s]);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv)
                        bulk_load(sc_area + (s * 2 + kv) * S::ScRows, p.scales + p.sc_layer_off + kv * p.sc_kv_off + base4,
                                  (uint32_t)(nsc * 4), &bars->full[s]);
                } else if (maps.slot_whole) {
                    mbar_expect_tx(&bars->full[s], (uint32_t)S::StageBytes);
                    tma_load_5d(dst, &maps.slot, 0, (int)(unit_base() + slot0), 0, p.layer, 0, &bars->full[s]);
                } else {
                    mbar_expect_tx(&bars->full[s], (uint32_t)S::StageBytes);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
                        tma_load_4d(dst + cb * S::KVBlock, &maps.slot, cb * 64, (int)(unit_base() + slot0), 0, p.layer,
                                    &bars->full[s]);
                }
                mbar_arrive(&bars->full[s]);
            }
            ++idx;
        };
        // the chunk's own rows, tokens i_s .. i_s + 63
        auto issue_stage_tile = [&](int i_s) {
            if (SCORE && pos0 + min(i_s + kWsKeys - 1, i_last) < smin) return;   // no token sees this tile
            const int s = acquire();
            if (!ok) return;
            int absent = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = lane + 32 * u;
                const int i = i_s + r;
                const int q = (i <= i_last && pos0 + i >= 0 && (!SCORE || pos0 + i >= smin)) ? pos0 + i : -1;
                meta[s].pos[r] = q;
                if constexpr (SCORE) meta[s].rel[r] = (float)i;
                absent |= q < 0;
            }
            absent = __any_sync(0xffffffffu, absent);
            __syncwarp();
            if (lane == 0) {
                meta[s].kind = kTileStage;
                meta[s].any_absent = absent;
                meta[s].mask = kMaskRange;
                meta[s].kbase = pos0 + i_s;
                unsigned char* dst = sm + S::OffStage + s * S::StageBytes;
                mbar_expect_tx(&bars->full[s], (uint32_t)S::StageBytes);
                if (SCORE && maps.direct) {
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) {
                        tma_load_3d(dst + cb * S::KVBlock, &maps.stage_k, cb * 64, h, b * p.T + i_s, &bars->full[s]);
                        tma_load_3d(dst + cb * S::KVBlock + kWsKeys * 128, &maps.stage_v, cb * 64, h, b * p.T + i_s,
                                    &bars->full[s]);
                    }
                } else {
                    tma_load_5d(dst, &maps.stage, 0, h, b * p.T + i_s, 0, 0, &bars->full[s]);
                }
                mbar_arrive(&bars->full[s]);
            }
            ++idx;
        };
        if (t_hi >= 0) {
            // modified scores take the chunk first and backwards: a distance bias favours
            // near keys, and a reference maximum found at once need not move again
            if (SCORE)
                for (int i_s = i_last / kWsKeys * kWsKeys; i_s >= 0 && ok; i_s -= kWsKeys) issue_stage_tile(i_s);
            if (!paged) {
                for (int k = 0; k < sink_tiles && ok; ++k) issue_slot_tile(k * kWsKeys, kTileSink);
                // slot tiles with at least one key the CTA can see
                const int nslot = (C + kWsKeys - 1) / kWsKeys;
                for (int k = 0; k < nslot && ok; ++k) {
                    bool any = false;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        any |= slot_pos(k * kWsKeys + lane + 32 * u, false, READ) >= 0;
                    if (__any_sync(0xffffffffu, any)) issue_slot_tile(k * kWsKeys, kTileSlot);
                }
            } else if (t0 >= 0) {
                // paged: mapped and valid blocks holding positions <= t0, packed
                const int bs = p.bs, per = kWsKeys / bs;
                // (positions past the table hold no key; the append reports them)
                const int nlb = min(t0 / bs + 1, p.maxb);
                const int32_t* trow = p.table + (long long)b * p.maxb;
                int fill = 0, s = 0;
                int low = 0;                              // SCORE: the tile's lowest position
                for (int base = 0; base < nlb && ok; base += 32) {
                    const int lb = base + lane;
                    int phys = lb < nlb ? __ldcg(trow + lb) : -1;
                    if (phys >= p.num_blocks) {
                        set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                        phys = -1;
                    }
                    bool att = phys >= 0;
                    if (att && p.valid) att = (__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u;
                    if (SCORE && (long long)(lb + 1) * bs <= smin) att = false;
                    unsigned m = __ballot_sync(0xffffffffu, att);
                    while (m && ok) {
                        const int src = __ffs(m) - 1;
                        m &= m - 1;
                        const int ph = __shfl_sync(0xffffffffu, phys, src);
                        const int blb = base + src;
                        if (fill == 0) {
                            s = acquire();
                            low = blb * bs;
                        }
                        if (!ok) break;
                        if (Q8 && fill == 0 && lane == 0) meta[s].sc_off = 0;   // block rows: multiples of 8
                        // rows of this block: positions blb * bs + r, keys up to t0
                        for (int r = lane; r < bs; r += 32) {
                            const int q = blb * bs + r;
                            meta[s].pos[fill * bs + r] = q <= t0 && (!SCORE || q >= smin) ? q : -1;
                            if constexpr (SCORE) meta[s].rel[fill * bs + r] = (float)(q - pos0);
                        }
                        if (lane == 0) {
                            const int row = (int)(((long long)ph * p.Hkv + h) * bs);
                            if constexpr (Q8) {
                                mbar_expect_tx(&bars->full[s], (uint32_t)(2 * (D / 128) * bs * 128 + 2 * bs * 4));
#pragma unroll
                                for (int hh = 0; hh < D / 128; ++hh)
#pragma unroll
                                    for (int kv = 0; kv < 2; ++kv)
                                        tma_load_4d(code_at(s, hh, kv) + fill * bs * 128, &maps.block, 128 * hh, row, kv,
                                                    p.layer, &bars->full[s]);
#pragma unroll
                                for (int kv = 0; kv < 2; ++kv)
                                    bulk_load(sc_area + (s * 2 + kv) * S::ScRows + fill * bs,
                                              p.scales + p.sc_layer_off + kv * p.sc_kv_off + row, (uint32_t)(bs * 4),
                                              &bars->full[s]);
                            } else {
                                mbar_expect_tx(&bars->full[s], (uint32_t)(bs * D * 4));
                                unsigned char* dst = sm + S::OffStage + s * S::StageBytes + fill * bs * 128;
#pragma unroll
                                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                                    for (int kv = 0; kv < 2; ++kv)
                                        tma_load_4d(dst + cb * S::KVBlock + kv * kWsKeys * 128, &maps.block, cb * 64, row,
                                                    kv, p.layer, &bars->full[s]);
                            }
                        }
                        if (++fill == per) {
                            __syncwarp();
                            if (lane == 0) {
                                meta[s].kind = kTileBlocks;
                                // the last block's rows past t0 (SCORE: and rows below every start)
                                meta[s].any_absent = t0 < blb * bs + bs - 1 || (SCORE && low < smin);
                                // every cached key precedes every token of the chunk
                                meta[s].mask = (meta[s].any_absent || (SCORE && low < smax)) ? kMaskKeys : kMaskNone;
                                mbar_arrive(&bars->full[s]);
                            }
                            fill = 0;
                            ++idx;
                        }
                    }
                }
                if (ok && fill > 0) {
                    // a partial tile: the rest of its rows hold no key, and no copy lands there
                    for (int r = fill * bs + lane; r < kWsKeys; r += 32) meta[s].pos[r] = -1;
                    __syncwarp();
                    if (lane == 0) {
                        meta[s].kind = kTileBlocks;
                        meta[s].any_absent = 1;
                        meta[s].mask = kMaskKeys;
                        mbar_arrive(&bars->full[s]);
                    }
                    ++idx;
                }
            }
            if (!SCORE)
                for (int i_s = 0; i_s <= i_last && ok; i_s += kWsKeys) issue_stage_tile(i_s);
        }
        // end marker
        if (ok) {
            const int s = acquire();
            if (ok && lane == 0) {
                meta[s].kind = kTileEnd;
                mbar_arrive(&bars->full[s]);
            }
            if (ok) ++idx;
        }
        // never leave with copies landing in shared memory
        if (!ok && lane == 0)
            for (int k = (idx > NST ? idx - NST : 0); k < idx; ++k) mbar_wait(&bars->full[k % NST], (k / NST) & 1);
    } else if (warp == 2 || (!TWO && warp == 3)) {
        // ============================ fix-up ===============================
        const int ft = tid - 64;                       // 0 .. 63
        uint32_t fix_phase = 0;
        for (int j = 0;; ++j) {
            const int s = j % NST;
            if (!ws_wait(&bars->full[s], (j / NST) & 1, abort)) {
                give_up();
                break;
            }
            const int kind = meta[s].kind;
            unsigned char* st = sm + S::OffStage + s * S::StageBytes;
            if (kind != kTileEnd) {
                bool wrote = false;
                if constexpr (Q8) {
                    if (kind != kTileStage) {
                        // row ft of the cache tile: code x row scale to bf16, in the
                        // stage's K / V layout.  Column boxes go in order: box hh
                        // overwrites (in blocks 2 hh, 2 hh + 1) only this row's codes
                        // of boxes < hh and its own, each already read.
                        const float* scs = sc_area + s * 2 * S::ScRows + meta[s].sc_off;
                        const float scl[2] = {scs[ft], scs[S::ScRows + ft]};
#pragma unroll
                        for (int hh = 0; hh < D / 128; ++hh) {
#pragma unroll
                            for (int kv = 0; kv < 2; ++kv) {
                                const uint4* src = reinterpret_cast<const uint4*>(code_at(s, hh, kv) + ft * 128);
                                uint4 cw[8];
#pragma unroll
                                for (int q = 0; q < 8; ++q) cw[q] = src[q];
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    const uint32_t w4[4] = {cw[q].x, cw[q].y, cw[q].z, cw[q].w};
                                    const float2 sc2 = make_float2(scl[kv], scl[kv]);
#pragma unroll
                                    for (int hf = 0; hf < 2; ++hf) {
                                        uint32_t o[4];
#pragma unroll
                                        for (int e = 0; e < 2; ++e) {
                                            // code c as the fp32 2^23 + (c + 128) (the byte under
                                            // the exponent of 2^23), less 2^23 + 128: exact
                                            const uint32_t x = w4[2 * hf + e] ^ 0x80808080u;
#pragma unroll
                                            for (int h2 = 0; h2 < 2; ++h2) {
                                                float2 f = make_float2(
                                                    __int_as_float(__byte_perm(x, 0x4B000000u, 0x7540u | (uint32_t)(2 * h2))),
                                                    __int_as_float(__byte_perm(x, 0x4B000000u, 0x7540u | (uint32_t)(2 * h2 + 1))));
                                                f = __fmul2_rn(__fadd2_rn(f, make_float2(-8388736.f, -8388736.f)), sc2);
                                                o[2 * e + h2] = pack_bf16x2(f.x, f.y);
                                            }
                                        }
                                        const int ch = 16 * hh + 2 * q + hf;     // 8-column chunk of the row
                                        *reinterpret_cast<uint4*>(st + ws_off(ft, ch) + kv * (kWsKeys * 128)) =
                                            make_uint4(o[0], o[1], o[2], o[3]);
                                    }
                                }
                            }
                        }
                        wrote = true;
                    }
                }
                if (meta[s].any_absent) {
                    // V rows of absent keys to zero: 64 threads, one row each (32: two)
#pragma unroll 1
                    for (int r = ft; r < kWsKeys; r += TWO ? 32 : 64)
                        if (meta[s].pos[r] < 0) {
#pragma unroll
                            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                                for (int ch = 0; ch < 8; ++ch)
                                    *reinterpret_cast<uint4*>(st + cb * S::KVBlock + kWsKeys * 128 + r * 128 + ch * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                        }
                    wrote = true;
                }
                if constexpr (READ && Q8) {
                    // the rotation below reads rows other threads expanded
                    mbar_arrive(&bars->fixb);
                    if (!ws_wait(&bars->fixb, fix_phase & 1, abort)) {
                        give_up();
                        break;
                    }
                    ++fix_phase;
                }
                if constexpr (READ) {
                    // raw K rows rotated at their positions: thread ft takes the
                    // 16-byte chunk pair c (elements 8c .. 8c + 7 and their
                    // partners at + D/2) of rows r0 .. r0 + RUN - 1, in f32x2
                    // pairs; the angles advance by one step from row to row while
                    // positions are consecutive, else are computed afresh
                    constexpr int CP = D / 16, RG = 64 / CP, RUN = kWsKeys / RG;
                    const int c = ft % CP, r0 = (ft / CP) * RUN;
                    float2 cc[4], ss[4], stc[4], sts[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        rope_cos_sin(1, p.theta[8 * c + 2 * u], &stc[u].x, &sts[u].x);
                        rope_cos_sin(1, p.theta[8 * c + 2 * u + 1], &stc[u].y, &sts[u].y);
                        cc[u] = make_float2(1.f, 1.f);
                        ss[u] = make_float2(0.f, 0.f);
                    }
                    int prev = -2;
#pragma unroll 1
                    for (int r = r0; r < r0 + RUN; ++r) {
                        const int q = meta[s].pos[r];
                        if (q < 0) {
                            prev = -2;
                            continue;
                        }
                        if (q == prev + 1) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float2 c0 = cc[u];
                                cc[u] = __ffma2_rn(c0, stc[u], __fmul2_rn(ss[u], make_float2(-sts[u].x, -sts[u].y)));
                                ss[u] = __ffma2_rn(ss[u], stc[u], __fmul2_rn(c0, sts[u]));
                            }
                        } else {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                rope_cos_sin((long long)q, p.theta[8 * c + 2 * u], &cc[u].x, &ss[u].x);
                                rope_cos_sin((long long)q, p.theta[8 * c + 2 * u + 1], &cc[u].y, &ss[u].y);
                            }
                        }
                        prev = q;
                        uint4* plo = reinterpret_cast<uint4*>(st + ws_off(r, c));
                        uint4* phi = reinterpret_cast<uint4*>(st + ws_off(r, c + CP));
                        const uint4 wl = *plo, wh = *phi;
                        const uint32_t lw[4] = {wl.x, wl.y, wl.z, wl.w}, hw[4] = {wh.x, wh.y, wh.z, wh.w};
                        uint32_t ol[4], oh[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 x1 = make_float2(__uint_as_float(lw[u] << 16), __uint_as_float(lw[u] & 0xffff0000u));
                            const float2 x2 = make_float2(__uint_as_float(hw[u] << 16), __uint_as_float(hw[u] & 0xffff0000u));
                            const float2 y1 = __ffma2_rn(x1, cc[u], __fmul2_rn(x2, make_float2(-ss[u].x, -ss[u].y)));
                            const float2 y2 = __ffma2_rn(x1, ss[u], __fmul2_rn(x2, cc[u]));
                            ol[u] = pack_bf16x2(y1.x, y1.y);
                            oh[u] = pack_bf16x2(y2.x, y2.y);
                        }
                        *plo = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                        *phi = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                    }
                    wrote = true;
                }
                if (wrote) fence_proxy_async_smem();
            }
            // (one arrival a warp: arrivals on one barrier are made one after the other)
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->ready[s]);
            if (kind == kTileEnd) break;
        }
    } else if (TWO && (warp == 1 || (NQ == 2 && warp == 3))) {
        // ================== MMA issuers, one for each Q tile =================
        // S_i = Q_i K^T a tile ahead of O_i += P_i V.  (One thread for both took 3300 to
        // 4100 cycles a tile of both, 1460 of them on products: the waits and commits
        // of one now pass while the other's products run.)  The whole warp walks the
        // tiles, its values stay uniform; lane 0 issues.
        const int i = warp >> 1;
        const uint64_t qd = ws_sdesc(sm_u + S::OffQ + i * S::QBytes, 16, 1024);
        const uint64_t kd0 = ws_sdesc(sm_u + S::OffStage, 16, 1024);
        const uint64_t vd0 = ws_sdesc(sm_u + S::OffStage + kWsKeys * 128, S::KVBlock, 1024);
        const uint32_t s_t = tmem + S::SCol0 + (uint32_t)(i * 2 * kWsKeys), o_t = tmem + (uint32_t)(i * D);
        bool ok = ws_wait(&bars->q_ready[i], 0, abort);
        int ns = 0, npv = 0, nt = 0x7fffffff;              // S issued, P V issued, tiles
        long long c0 = clock64();
        while (ok && npv < nt) {
            // (each barrier's phases are asked for in order)
            if (ns < nt && ns < npv + 2 && ws_test(&bars->ready[ns % NST], (ns / NST) & 1)) {
                const int s = ns % NST;
                if (meta[s].kind == kTileEnd) {
                    nt = ns;
                } else {
                    ws_fence_after();
                    if (lane == 0) {
                        ws_issue_s<D, kWsRows * 128, S::KVBlock>(s_t + (uint32_t)((ns & 1) * kWsKeys), qd,
                                                                 kd0 + (uint64_t)((s * S::StageBytes) >> 4));
                        ws_commit(&bars->s_full[i][ns & 1]);
                    }
                    __syncwarp();
                    ++ns;
                }
                c0 = clock64();
                continue;
            }
            if (npv < ns && ws_test(&bars->p_full[i], npv & 1)) {
                ws_fence_after();
                const int s = npv % NST;
                if (lane == 0) {
                    // P_i in the S buffer it came from (bf16 pairs, 32 columns)
                    ws_issue_pv<D>(o_t, s_t + (uint32_t)((npv & 1) * kWsKeys),
                                   vd0 + (uint64_t)((s * S::StageBytes) >> 4), npv > 0);
                    ws_commit(&bars->o_done[i]);
                    ws_commit(&bars->empty[s]);            // this Q tile is done with the tile's K and V
                }
                __syncwarp();
                ++npv;
                c0 = clock64();
                continue;
            }
            if (*abort || clock64() - c0 > kWaitCycles) ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
            if (ok) {
                // the end: the softmax warps learn the tile count at the S slot they wait
                // on next (every S before it has been consumed)
                bars->ntiles = nt;
                mbar_arrive(&bars->s_full[i][nt & 1]);
            } else {
                give_up();
            }
            // every product this thread issued is done before TMEM is freed
            ws_commit(&bars->fin[i]);
            if (!mbar_wait(&bars->fin[i], 0)) set_error(p.err, 0x8u /* KVC_DEV_TIMEOUT */);
        }
        __syncwarp();
    } else if (warp == 1) {
        // =========================== MMA issuer =============================
        // the whole warp walks the tiles (its values stay uniform) and lane 0 issues
        bool ok = true;
        int nt = 0x7fffffff;
        uint64_t qd[NQ];
        for (int i = 0; i < NQ; ++i) qd[i] = ws_sdesc(sm_u + S::OffQ + i * S::QBytes, 16, 1024);
        const uint64_t kd0 = ws_sdesc(sm_u + S::OffStage, 16, 1024);
        const uint64_t vd0 = ws_sdesc(sm_u + S::OffStage + kWsKeys * 128, S::KVBlock, 1024);
        auto stage_d = [&](int j) { return (uint64_t)(((j % NST) * S::StageBytes) >> 4); };
        // S_i(j) = Q_i K_j^T
        auto issue_s = [&](int j) {
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if (!ok) break;
                if (j >= 2 && !ws_wait(&bars->s_free[i][j & 1], ((j >> 1) - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                ws_fence_after();
                const uint32_t d = tmem + S::SCol0 + (uint32_t)((i * 2 + (j & 1)) * kWsKeys);
                if (lane == 0) {
                    ws_issue_s<D, kWsRows * 128, S::KVBlock>(d, qd[i], kd0 + stage_d(j));
                    ws_commit(&bars->s_full[i][j & 1]);
                }
                __syncwarp();
            }
        };
        // S of tile t for every Q tile, once its keys are in place; false at
        // the end marker (nt = t) or when a wait gave up
        auto try_issue = [&](int t) -> bool {
            if (!ok || t >= nt) return false;
            if (!ws_wait(&bars->ready[t % NST], (t / NST) & 1, abort)) {
                ok = false;
                return false;
            }
            if (meta[t % NST].kind == kTileEnd) {
                nt = t;
                return false;
            }
            for (int i = 0; i < NQ && ok; ++i) {
                // q at position 0, and (read-time RoPE) again past the sink tiles
                if (t == 0 && !ws_wait(&bars->q_ready[i], 0, abort)) ok = false;
                if (READ && t > 0 && t == sink_tiles && !ws_wait(&bars->q_ready[i], 1, abort)) ok = false;
            }
            if (ok) issue_s(t);
            return ok;
        };
        // S runs LA tiles ahead of P V: each Q tile's next scores are queued
        // on the tensor cores while its softmax works on the current ones.
        // LA + 1 tiles are in flight, so the stages must hold them.
        constexpr int LA = NST >= 3 ? 2 : 1;
        int issued = 0;
        while (issued < LA && try_issue(issued)) ++issued;
        int j = 0;
        for (; ok && j < issued; ++j) {
            // O_i += P_i V_j
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if (!ws_wait(&bars->p_full[i], j & 1, abort)) {
                    ok = false;
                    break;
                }
                ws_fence_after();
                // P_i(j) in the S buffer it came from (bf16 pairs, 32 columns);
                // S of tile j + 2 reuses that buffer, issued after this P V
                const uint32_t p_t = tmem + S::SCol0 + (uint32_t)((i * 2 + (j & 1)) * kWsKeys);
                if (lane == 0) {
                    ws_issue_pv<D>(tmem + (uint32_t)(i * D), p_t, vd0 + stage_d(j), j > 0);
                    ws_commit(&bars->o_done[i]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) ws_commit(&bars->empty[j % NST]);       // K and V of tile j are done with
            if (issued == j + LA && try_issue(issued)) ++issued;
        }
        if (*abort) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        nt = j;
        if (lane == 0) {
            if (ok) {
                // the end: the softmax warps learn the tile count at the S slot
                // they wait on next (every S before it has been consumed)
                bars->ntiles = nt;
                for (int i = 0; i < NQ; ++i) mbar_arrive(&bars->s_full[i][nt & 1]);
            } else {
                give_up();
            }
            // every product this thread issued is done before TMEM is freed
            ws_commit(&bars->fin[0]);
            if (!mbar_wait(&bars->fin[0], 0)) set_error(p.err, 0x8u /* KVC_DEV_TIMEOUT */);
        }
        __syncwarp();
    } else if (warp >= kWsSoftmax0 && warp < kWsSoftmax0 + 4 * NQ) {
        // ============================ softmax ==============================
        const int qi = (warp - kWsSoftmax0) >> 2;     // Q tile
        const int r = tid - (kWsSoftmax0 + 4 * qi) * 32;   // row = TMEM lane
        const int tl = r / G;
        const int row_i = i0 + qi * tq + tl;
        const int row_h = h * G + r % G;
        const int row_t = pos0 + row_i;
        const bool row_ok = tl < tq && row_i < p.T && row_t >= 0;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        unsigned char* Qs = sm + S::OffQ + qi * S::QBytes;

        // The Q tile: rotated at its position (a sink tile's at min(t, C - 1)), scaled by
        // q_scale (softmax scale * log2 e, or 1), bf16.
        // 8-column chunk c of row rr and its partner c + D / 16 (lo, hi) to the tile,
        // [column block][128 rows][128 B], 128-byte swizzle; th(k): frequency of pair 8 c + k
        auto write_q_chunk = [&](int rr, int c, bool rok, long long qpos, auto rotated, auto th, uint4 lo, uint4 hi) {
            if (!SCORE || rotated.value) {
                const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
                uint32_t lo2[4], hi2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[2] = {__uint_as_float(lw[e] << 16), __uint_as_float(lw[e] & 0xffff0000u)};
                    float y[2] = {__uint_as_float(hw[e] << 16), __uint_as_float(hw[e] & 0xffff0000u)};
                    if (rotated.value && rok) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float cs, sn;
                            rope_cos_sin(qpos, th(2 * e + u), &cs, &sn);
                            const float x1 = x[u], x2 = y[u];
                            x[u] = x1 * cs - x2 * sn;
                            y[u] = x1 * sn + x2 * cs;
                        }
                    }
                    lo2[e] = pack_bf16x2(x[0] * p.q_scale, x[1] * p.q_scale);
                    hi2[e] = pack_bf16x2(y[0] * p.q_scale, y[1] * p.q_scale);
                }
                lo = make_uint4(lo2[0], lo2[1], lo2[2], lo2[3]);
                hi = make_uint4(hi2[0], hi2[1], hi2[2], hi2[3]);
            }
            const int c2 = c + D / 16;
            *reinterpret_cast<uint4*>(Qs + (c >> 3) * (kWsRows * 128) + rr * 128 + (((c ^ rr) & 7) << 4)) = lo;
            *reinterpret_cast<uint4*>(Qs + (c2 >> 3) * (kWsRows * 128) + rr * 128 + (((c2 ^ rr) & 7) << 4)) = hi;
        };
        // D / 16 lanes share a row, so that a load covers whole lines (unrotated, a row a
        // thread took 6 us of each CTA)
        constexpr int QLPR = D / 16, QRPW = 32 / QLPR;
        const int qc = lane % QLPR;                    // 8-column chunk, paired with qc + D / 16
        auto write_q_rows = [&](int it, bool at_sinks, auto rotated, const unsigned long long* th) {
            const int rr = (warp & 3) * 32 + it * QRPW + lane / QLPR;
            const int rtl = rr / G, ri = i0 + qi * tq + rtl, rt = pos0 + ri;
            const bool rok = rtl < tq && ri < p.T && rt >= 0;
            uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
            if (rok) {
                const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) +
                                            (((long long)b * p.T + ri) * p.Hq + h * G + (rr - rtl * G)) * D;
                lo = *reinterpret_cast<const uint4*>(qrow + 8 * qc);
                hi = *reinterpret_cast<const uint4*>(qrow + D / 2 + 8 * qc);
            }
            write_q_chunk(rr, qc, rok, at_sinks ? min(rt, C - 1) : rt, rotated, [&](int k) { return th[k]; }, lo, hi);
        };
        auto write_q = [&](bool at_sinks) {
            if (p.rope == kRopeNone) {
#pragma unroll 4
                for (int it = 0; it < 32 / QRPW; ++it) write_q_rows(it, at_sinks, std::false_type{}, nullptr);
            } else if constexpr (!READ && !SCORE) {
                // baked rows a thread each: the frequencies are then the same for the whole warp
                // (paged, 64 x 128 tokens: 1.129 ms by whole lines, 1.122 so; INT8 1.339 and 1.334;
                // ring, 8 x 128: 126 and 122.5 us.  Read-time RoPE is the other way round, 1.271
                // by lines against 1.293 ms; modified scores within 3 % either way)
                const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) +
                                            (((long long)b * p.T + (row_ok ? row_i : 0)) * p.Hq + row_h) * D;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                    if (row_ok) {
                        lo = *reinterpret_cast<const uint4*>(qrow + 8 * c);
                        hi = *reinterpret_cast<const uint4*>(qrow + D / 2 + 8 * c);
                    }
                    write_q_chunk(r, c, row_ok, row_t, std::true_type{}, [&](int k) { return p.theta[8 * c + k]; }, lo, hi);
                }
            } else {
                // (the lane's frequencies are read once: lanes read different ones; unrolled,
                // the rotations took 13 us more of each CTA)
                unsigned long long th[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) th[e] = p.theta[8 * qc + e];
#pragma unroll 1
                for (int it = 0; it < 32 / QRPW; ++it) write_q_rows(it, at_sinks, std::true_type{}, th);
            }
            fence_proxy_async_smem();
            mbar_arrive(&bars->q_ready[qi]);
        };
        write_q(sink_tiles > 0);

        float m_run = -INFINITY, l_run = 0.f;
        // SCORE: the row's slope (base 2), its bias at distance row_i, and its start
        float slope2 = 0.f, bias0 = 0.f;
        int start = 0;
        if constexpr (SCORE) {
            if (BIAS && row_ok) slope2 = p.score.slopes[row_h] * 1.4426950408889634f;
            bias0 = -slope2 * (float)row_i;
            if (row_ok && p.score.start) start = max(0, p.score.start[(long long)b * p.T + row_i]);
        }
        int j = 0;
        bool ok = true;
        for (;; ++j) {
            if (!ws_wait(&bars->s_full[qi][j & 1], (j >> 1) & 1, abort)) {
                ok = false;
                break;
            }
            if (j == *reinterpret_cast<volatile int*>(&bars->ntiles)) break;
            ws_fence_after();
            float sv[kWsKeys];
            const uint32_t scol = S::SCol0 + (uint32_t)((qi * 2 + (j & 1)) * kWsKeys);
            ws_ld32(lane_base + scol, sv);
            ws_ld32(lane_base + scol + 32, sv + 32);
            ws_wait_ld();
            ws_fence_before();
            __syncwarp();
            if (!TWO && lane == 0) mbar_arrive(&bars->s_free[qi][j & 1]);
            if (READ && j == sink_tiles - 1) write_q(false);     // S of the last sink tile is out of TMEM
            const int s = j % NST;
            if (!ws_wait(&bars->ready[s], (j / NST) & 1, abort)) {    // the stage's meta
                ok = false;
                break;
            }
            // masks: a key at position q is seen by the row at t iff q <= t and
            // (paged, or a sink q < S, or q in the window t - W + 1 .. t)
            const int mode = meta[s].mask;
            float mn, alpha;
            if constexpr (SCORE) {
                // keys that the row does not attend become -inf (if `on`)
                auto mask = [&](bool on) {
                    if (mode == kMaskRange) {
                        // the chunk's own rows: key k at kbase + k (the window holds every chunk token)
                        const int kb = meta[s].kbase;
                        int klo = row_ok ? (int)min((long long)start - kb, (long long)kWsKeys) : kWsKeys;
                        int khi = row_t - kb;
                        if (!on) {
                            klo = 0;
                            khi = kWsKeys;
                        }
                        if (!__all_sync(0xffffffffu, klo <= 0 && khi >= kWsKeys - 1)) ws_mask_range(sv, klo, khi);
                    } else if (on && !row_ok) {
#pragma unroll
                        for (int k = 0; k < kWsKeys; ++k) sv[k] = -INFINITY;
                    } else if (on && mode == kMaskKeys) {
                        const int from = paged ? start : max(start, row_t - p.window + 1);   // (sinks below it too)
#pragma unroll
                        for (int k = 0; k < kWsKeys; k += 4) {
                            const int4 q4 = *reinterpret_cast<const int4*>(&meta[s].pos[k]);
                            const int qk[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int q = qk[u];
                                const bool allowed = q >= 0 && q <= row_t && (q >= from || (q < p.sinks && q >= start));
                                sv[k + u] = allowed ? sv[k + u] : -INFINITY;
                            }
                        }
                    }
                };
                // s = A v + B in base 2: v = q . k, or with a cap v = -1 / (2^(cap_in q.k) + 1)
                // and s = 2 cap2 v + cap2 (cap tanh(x / cap) = cap - 2 cap / (e^(2 x / cap) + 1));
                // a distance bias differs from key to key and is added to every v
                float A = p.score.scale2, B = 0.f;
                if constexpr (CAP) {
                    const float nan = ws_cap(sv, p.score.cap_in);
                    // A NaN among a row's scores, which the cap passes on to its neighbours: the warp
                    // once more, the keys that such a row does not attend masked first; a NaN that
                    // is left is the row's own.  (Masked first in every tile with a mask: 8 rings of
                    // 4096, cap: 228 -> 262 us.)
                    if (__any_sync(0xffffffffu, nan != nan)) {
                        ws_ld32(lane_base + scol, sv);
                        ws_ld32(lane_base + scol + 32, sv + 32);
                        ws_wait_ld();
                        mask(nan != nan);
                        ws_cap(sv, p.score.cap_in);
                    }
                    A = 2.f * p.score.cap2;
                    B = p.score.cap2;
                }
                if constexpr (BIAS) {
                    // slope (p - t) = slope (p - pos0) - slope (t - pos0)
                    const float2 A2 = make_float2(A, A), sl = make_float2(slope2, slope2);
                    const float2 b2 = make_float2(bias0 + B, bias0 + B);
#pragma unroll
                    for (int k = 0; k < kWsKeys; k += 4) {
                        const float4 rel = *reinterpret_cast<const float4*>(&meta[s].rel[k]);
                        const float2 x0 = __ffma2_rn(make_float2(sv[k], sv[k + 1]), A2,
                                                     __ffma2_rn(make_float2(rel.x, rel.y), sl, b2));
                        const float2 x1 = __ffma2_rn(make_float2(sv[k + 2], sv[k + 3]), A2,
                                                     __ffma2_rn(make_float2(rel.z, rel.w), sl, b2));
                        sv[k] = x0.x;
                        sv[k + 1] = x0.y;
                        sv[k + 2] = x1.x;
                        sv[k + 3] = x1.y;
                    }
                    A = 1.f;
                    B = 0.f;
                }
                mask(true);
                mn = fmaxf(100.f - p.score.cap2, 0.f);
                mn = fminf(p.score.cap2, mn);
                alpha = 1.f;
                if constexpr (!FIXED) {
                    const float vmax = ws_max64(sv);
                    const float mx = vmax == -INFINITY ? -INFINITY : fmaf(vmax, A, B);
                    mn = m_run;
                    if (mx > m_run + kWsLazy) {
                        mn = mx;
                        alpha = m_run == -INFINITY ? 1.f : exp2f(m_run - mn);
                    }
                }
                // fp32 exponentials: on this part they cost what a pair of fp16 ones and
                // its conversions do
                const float ls = ws_exp64(sv, A, mn == -INFINITY ? 0.f : B - mn);
                l_run = l_run * alpha + ls;
                m_run = mn;
            } else {
                // (masks and maxima as the modified scores have them made read-time RoPE 1.25 ->
                // 1.32 ms and a paged INT8 batch 1.37 -> 1.53: this schedule is left alone)
                if (!row_ok) {
#pragma unroll
                    for (int k = 0; k < kWsKeys; ++k) sv[k] = -INFINITY;
                } else if (mode == kMaskRange) {
                    // the chunk's own rows: key k at kbase + k is seen iff 0 <= kbase + k <= t
                    // (the window holds every chunk token, the chunk being no longer than it)
                    const int kb = meta[s].kbase;
                    const int klo = -kb, khi = row_t - kb;
#pragma unroll
                    for (int k = 0; k < kWsKeys; ++k) sv[k] = (k >= klo && k <= khi) ? sv[k] : -INFINITY;
                } else if (mode == kMaskKeys) {
#pragma unroll
                    for (int k = 0; k < kWsKeys; ++k) {
                        const int q = meta[s].pos[k];
                        bool allowed = q >= 0 && q <= row_t;
                        if (!paged) allowed = allowed && (q < p.sinks || q > row_t - p.window);
                        sv[k] = allowed ? sv[k] : -INFINITY;
                    }
                }
                // four independent chains (latency, not issue slots, is what the
                // softmax warps wait on)
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < kWsKeys; k += 4)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mq[u] = fmaxf(mq[u], sv[k + u]);
                const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                mn = m_run;
                alpha = 1.f;
                if (mx > m_run + kWsLazy) {
                    mn = mx;
                    alpha = m_run == -INFINITY ? 1.f : exp2f(m_run - mn);
                }
                // p = 2^(s - m) (exactly 0 for a masked key: 2^-inf), summed in pairs
                const float nmn = mn == -INFINITY ? 0.f : -mn;
                float2 ls2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f)};
#pragma unroll
                for (int k = 0; k < kWsKeys; k += 2) {
                    const float2 d2 = __fadd2_rn(make_float2(sv[k], sv[k + 1]), make_float2(nmn, nmn));
                    const float2 e2 = ws_ex2_pair(d2.x, d2.y);
                    sv[k] = e2.x;
                    sv[k + 1] = e2.y;
                    ls2[(k >> 1) & 3] = __fadd2_rn(ls2[(k >> 1) & 3], e2);
                }
                const float2 lsa = __fadd2_rn(__fadd2_rn(ls2[0], ls2[1]), __fadd2_rn(ls2[2], ls2[3]));
                l_run = l_run * alpha + (lsa.x + lsa.y);
                m_run = mn;
            }
            // P V of the previous tile is done: P's buffer and O are free
            if (j > 0 && !ws_wait(&bars->o_done[qi], (j - 1) & 1, abort)) {
                ok = false;
                break;
            }
            ws_fence_after();
            if (!FIXED && j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    float ov[32];
                    ws_ld32(lane_base + (uint32_t)(qi * D + 32 * c4), ov);
                    ws_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) ov[k] *= alpha;
                    ws_st32(lane_base + (uint32_t)(qi * D + 32 * c4), ov);
                }
                ws_wait_st();
            }
            // P row r (bf16 pairs of the 64 keys) into the S buffer just read:
            // the A operand of P V, in tensor memory
            {
                float pw[kWsKeys / 2];
#pragma unroll
                for (int k2 = 0; k2 < kWsKeys / 2; ++k2) pw[k2] = __uint_as_float(pack_bf16x2(sv[2 * k2], sv[2 * k2 + 1]));
                ws_st32(lane_base + scol, pw);
            }
            ws_wait_st();
            ws_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[qi]);
        }
        if (!ok) give_up();
        // the last P V, then O / l to the output
        const int nt = j;
        bool have_o = false;
        if (ok && nt > 0) {
            if (ws_wait(&bars->o_done[qi], (nt - 1) & 1, abort))
                have_o = true;
            else
                give_up();
        }
        ws_fence_after();
        if (!*abort) {
            const float inv = (have_o && l_run > 0.f) ? 1.f / l_run : 0.f;
            // through the Q tile's shared memory (its products are done), so that
            // whole rows go out
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) {
                float ov[32];
                if (have_o) {
                    ws_ld32(lane_base + (uint32_t)(qi * D + 32 * c4), ov);
                    ws_wait_ld();
                }
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = (have_o && row_ok) ? pack_bf16x2(ov[8 * q4 + 2 * e] * inv, ov[8 * q4 + 2 * e + 1] * inv)
                                                  : 0u;
                    const int ch = 4 * c4 + q4;
                    *reinterpret_cast<uint4*>(Qs + (ch >> 3) * (kWsRows * 128) + r * 128 + (((ch ^ r) & 7) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();
            constexpr int LPR = D / 8, RPW = 32 / LPR;
            const int ch = lane % LPR;
#pragma unroll 4
            for (int it = 0; it < 32 / RPW; ++it) {
                const int rr = (warp & 3) * 32 + it * RPW + lane / LPR;
                const int rtl = rr / G, ri = i0 + qi * tq + rtl;
                if (rtl < tq && ri < p.T)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                              (((long long)b * p.T + ri) * p.Hq + h * G + (rr - rtl * G)) * D + 8 * ch) =
                        *reinterpret_cast<const uint4*>(Qs + (ch >> 3) * (kWsRows * 128) + rr * 128 +
                                                        (((ch ^ rr) & 7) << 4));
            }
        }
    }

    // the MMA thread has waited for all of its products (its last commit)
    ws_fence_before();
    __syncthreads();
    ws_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TmemCols) : "memory");
}

template <int D, bool READ, bool Q8, int MOD>
cudaError_t launch_prefill_ws_t(const PrefillParams& p, const PrefillMaps& maps, cudaStream_t stream) {
    constexpr int kSmem = ws_smem_bytes<D>();
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(prefill_ws_kernel<D, READ, Q8, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    const int tok = kWsRows / p.G * WsShape<D>::NQ;
    dim3 grid((p.T + tok - 1) / tok, p.Hkv, p.B);
    prefill_ws_kernel<D, READ, Q8, MOD><<<grid, WsShape<D>::Threads, kSmem, stream>>>(p, maps);
    return cudaGetLastError();
}

}  // namespace kvc
