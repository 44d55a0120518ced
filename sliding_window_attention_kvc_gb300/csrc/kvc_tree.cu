// kvc_tree_attention: attention of a tree of drafted tokens over a cache, as a
// step of speculative decoding verifies it.  Token i of sequence b continues
// token parent[i] (-1: the sequence itself); it stands at position
// t = pos0 + its depth and attends what a token there attends in the cache, its
// ancestors in the draft and itself.
//
// The (token, q head of the group) pairs of a kv head are the rows of one matrix
// product with the keys of that head, so the cache is read once for the whole
// draft.  A column is (sequence, kv head, up to NQ x 128 rows); its keys are cut
// into tiles of 64, the last tile the draft's own rows under the mask of
// ancestors.  A unit of work is a tile for one Q tile; all units of all columns,
// laid end to end, are split into nearly equal contiguous shares, one per CTA (one
// CTA per SM), so that one long sequence fills the GPU as a batch does.  The part of
// a column in a share is a segment and leaves one partial (m, l, o) per row;
// tree_combine_kernel joins them:  M = max m_i,
// out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M).
//
// Roles of a CTA's warps: 0 brings tiles in by TMA; 2 zeroes the V rows without a
// key (they may hold anything); 1 and 3 issue the products of a Q tile each,
// S = Q K^T a tile ahead of O += P V, accumulators in tensor memory; a warpgroup a
// Q tile does the softmax, a thread a row.  A column of one Q tile gives both
// warpgroups the same rows and alternate tiles, with sums of their own, which they join
// at the segment's end, half of the columns each.
// What bounds it: a tile is 64 rows of K and V (32 KB at head_dim 128) for
// 4 x 64 x 128 x D flops a Q tile: bytes up to one Q tile, the tensor pipe's turns
// beyond (a tile's S waits behind the P V before it).  Drafts of 32 tokens over 8 rings
// of 4096, 32 / 8 heads of 128 (139 MB): 40 us, half of it tiles at the rate of DRAM, then
// what comes once: the way to the first product, the rows' write, the combine.  64 tokens
// over 100,003 (411 MB, 105 GFLOP): 102 us, 0.59 of the bandwidth and 0.53 of the bf16 rate
// at once.  With baked keys the q rows are rotated one after the other before a CTA's first
// product, and the draft's keys by a launch of their own: 63 and 140 us.  At head_dim 64 31
// and 86 us, at 256 (two stages) 76 and 286.
#include <atomic>

#include "kvc_decode.cuh"
#include "kvc_tc.cuh"
#include "kvc_tree.h"

namespace kvc {

namespace {

constexpr int kTrSoftmax0 = 4;              // first softmax warp
constexpr int kTrMaxStages = 10;
constexpr float kTrLazy = 8.f;              // the reference maximum moves when a tile's exceeds it by more

__device__ __forceinline__ void tr_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void tr_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// FEW: drafts of one Q tile at head_dim 128: both warpgroups' products read one copy of it, which leaves room for a
// stage more.
template <int D, bool FEW = false>
struct TrShape {
    static constexpr int NQ = tree_q_tiles(D);
    static constexpr int QTiles = FEW ? 1 : NQ;
    // as many as there is room for (bytes on their way are what few rows are bound by: drafts of 8 over 64 rings
    // of 4096 took 219 us with four stages at head_dim 128, 203 with five, 196 with FEW's six)
    static constexpr int STAGES = D == 64 ? 10 : (D == 128 ? (FEW ? 6 : 5) : 2);
    static constexpr int CB = D / 64;                          // 64-column blocks of a row
    static constexpr int QBytes = kWsRows * D * 2;             // one Q tile
    // a stage: [8 rows of the tile][K|V][column block][8 rows x 128 bytes], so that one copy brings any
    // number of whole groups of 8 rows
    static constexpr int VOff = CB * 1024;
    static constexpr int Group = 2 * VOff;
    static constexpr int StageBytes = (kWsKeys / 8) * Group;
    static constexpr int OffQ = 0;
    static constexpr int OffStage = OffQ + QTiles * QBytes;
    static constexpr int OffMeta = OffStage + STAGES * StageBytes;
    static constexpr int TmemCols = 512;
    static constexpr int SCol0 = NQ * D;                       // S buffers after the O tiles
    static_assert(NQ * D + NQ * 2 * kWsKeys <= TmemCols, "TMEM columns");
    static constexpr int Threads = 32 * (kTrSoftmax0 + 4 * NQ);
};

// kTileOpen: every key of the tile that is there is attended by every token;
// kTileWindow: each row's window cuts it; kTileDraft: the draft's own rows.
enum : int { kTileOpen = 0, kTileWindow = 1, kTileDraft = 2 };

struct alignas(16) TrStageMeta {
    unsigned long long present;     // rows of the tile that hold a key
    int kind;
    int slot0;                      // kTileWindow: slot of the tile's first row
};

struct TrBars {
    uint64_t full[kTrMaxStages], ready[kTrMaxStages], empty[kTrMaxStages];
    // (of two tiles in turn: a warp hands over P of a tile before it asks for O of the tile before, and the
    // issuer may ask for a P once the next has been handed over; on one barrier each, a warp or an issuer held
    // up for a product's time would find the phase after the one it asks for, and wait for good)
    uint64_t s_full[2][2], p_full[2][2], o_done[2][2];
    // (an issuer's own: it counts the segments that bring it a tile.  On one barrier for both, a segment of one
    // tile, which only the first issuer asks for, left the second a phase behind: it began the next segment's
    // products on the q before; and asking for every phase it could find the one after, and wait for good)
    uint64_t q_ready[2], fin[2];
    uint64_t both[2];               // alternate tiles: both warpgroups' sums are there; both have read them
    uint32_t tmem;
    int abort;
    float2 ml[2][kWsRows];          // ... and their (m, l)
};

template <int D, bool FEW>
constexpr int tr_smem_bytes() {
    using S = TrShape<D, FEW>;
    static_assert(S::STAGES <= kTrMaxStages, "barriers of every stage");
    return S::OffMeta + S::STAGES * (int)sizeof(TrStageMeta) + (int)sizeof(TrBars);
}

// The token of a row of a column: row / G (exact for rows below 256; a division by a value that is not known at
// compile time is thirty instructions, and a cold one each).
__device__ __forceinline__ int tr_token(const TreeParams& p, int row) { return (row * p.inv_g) >> 16; }

// Cached rows of sequence b: live slots of a window layout, positions of a paged one.
__device__ __forceinline__ int tr_cached(const TreeParams& p, int pos) {
    if (pos <= 0) return 0;
    if (p.layout != kPaged) return pos < p.capacity ? pos : p.capacity;
    const long long lim = (long long)p.maxb * p.bs;
    return pos < lim ? pos : (int)lim;
}
__device__ __forceinline__ int tr_tiles(const TreeParams& p, int pos) {
    return (int)(((unsigned)tr_cached(p, pos) + kWsKeys - 1) / kWsKeys) + 1;      // (2^31 and more on the way)
}
__device__ __forceinline__ long long tr_seq_units(const TreeParams& p, int pos) {
    return (long long)tr_tiles(p, pos) * p.col_units * p.Hkv;
}

// What runs once a segment or once a kernel is kept short and out of line, one copy for
// all roles: it comes out of a cold instruction cache, a line of eight instructions at a
// time (inlined and unrolled, the way to a CTA's first product took 20 us, most of it the
// draft's ancestors).

// Where a share stands: the sequence and the units before it.
struct TrWalk {
    int b;
    long long before;
};
// Units of all sequences, and the shares they are cut into (a whole warp's call): one a
// CTA; fewer where the columns are alike and fewer than the CTAs: then each is cut into
// the same whole number of shares, and no CTA begins a second segment (its way to the
// first product, and a partial, cost 6 us).  Whole shares / all 152 CTAs, drafts of 32 over
// rings of 4096, 8 kv heads: 8 rings 41 / 46 us, 9 43 / 49, 10 54 / 53, 12 55 / 58, 14 56 / 63,
// 18 60 / 77.  From 77 columns on a column is one share: 10 and 11 rings leave 72 and 64 CTAs
// idle, which drafts of 8 (10 rings 55 / 46, 12 55 / 51) and of 64 (10 rings 78 / 71) and long
// rings (10 of 16384 170 / 126, 12 172 / 145, 18 191 / 206) are slower for; short ones are
// not (10 of 1024 24 / 33).
struct TrParts {
    long long units;
    int shares;
};
__device__ __noinline__ TrParts tr_partition(const TreeParams& p) {
    const int lane = threadIdx.x & 31;
    long long tot = 0;
    int lo = 0x7fffffff, hi = 0;                    // tiles of the shortest and of the longest column
    for (int base = 0; base < p.B; base += 32) {
        const int o = base + lane;
        if (o < p.B) {
            const int kt = tr_tiles(p, p.pos[o]);
            tot += (long long)kt * p.col_units * p.Hkv;
            lo = min(lo, kt);
            hi = max(hi, kt);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        tot += __shfl_xor_sync(0xffffffffu, tot, off);
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    TrParts r;
    r.units = tot;
    const long long s = (tot + kTreeMinTiles - 1) / kTreeMinTiles, cols = (long long)p.B * p.Hkv * p.ncol;
    r.shares = s < p.ctas ? (int)s : p.ctas;
    if (lo == hi && p.last_units * p.ncol == p.col_units && cols <= r.shares)
        r.shares = (int)cols * (r.shares / (int)cols);
    return r;
}

// The sequence that holds unit u (a whole warp's call).
__device__ __noinline__ TrWalk tr_find(const TreeParams& p, long long u) {
    const int lane = threadIdx.x & 31;
    TrWalk w{0, 0};
    long long run = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int o = base + lane;
        const long long n = o < p.B ? tr_seq_units(p, p.pos[o]) : 0;
        long long incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += a;
        }
        const unsigned in = __ballot_sync(0xffffffffu, o < p.B && run + incl > u);
        if (in) {
            const int src = __ffs(in) - 1;
            w.b = base + src;
            w.before = run + __shfl_sync(0xffffffffu, incl - n, src);
            return w;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    w.b = p.B - 1;                                  // (not reached: u lies below the total)
    return w;
}

// One segment: tiles tile0 .. tile0 + nt - 1 of a column.
struct TrSegment {
    int b, h, pos, n0, tokens;                 // sequence, kv head, its tokens in the cache; first token and tokens of the column
    int kt;                                    // tiles of the column, the last of them the draft
    int tile0, nt;                             // nt may be 0: one unit of a tile that begins in the share before
    int units;
    int first, last;                           // the column's first and last unit lie in this share
    int alt;                                   // one Q tile's rows: the warpgroups take alternate tiles
    long long col;                             // index of the column
    __device__ __forceinline__ int tiles(int i) const { return alt ? (nt + 1 - i) >> 1 : nt; }
};

// The segment that begins at unit u of a share ending at hi.
template <int D>
__device__ __noinline__ TrSegment tr_segment(const TreeParams& p, TrWalk& w, long long u, long long hi) {
    TrSegment s;
    s.pos = p.pos[w.b];
    for (long long n = tr_seq_units(p, s.pos); u >= w.before + n && w.b < p.B - 1;) {
        w.before += n;
        s.pos = p.pos[++w.b];
        n = tr_seq_units(p, s.pos);
    }
    s.b = w.b;
    s.kt = tr_tiles(p, s.pos);
    const long long hu = (long long)s.kt * p.col_units;
    long long v = u - w.before;
    s.h = (int)div_nonneg(v, hu);
    v -= s.h * hu;
    constexpr int NQ = TrShape<D>::NQ;
    int m = (int)div_nonneg(v, (long long)s.kt * NQ);          // every column but a head's last has NQ Q tiles
    if (m > p.ncol - 1) m = p.ncol - 1;
    v -= (long long)m * s.kt * NQ;
    s.n0 = m * p.mq;
    s.tokens = min(p.mq, p.T - s.n0);
    // units to tiles: a tile belongs to the share that holds its first unit
    const int per = m < p.ncol - 1 ? NQ : p.last_units;
    const int v0 = (int)v;                                     // (tiles of a column, times two at most)
    const int take = (int)min((long long)(s.kt * per - v0), hi - u);
    s.units = take;
    s.tile0 = per == 2 ? (v0 + 1) >> 1 : v0;
    s.nt = (per == 2 ? (v0 + take + 1) >> 1 : v0 + take) - s.tile0;
    s.alt = NQ == 2 && per == 1;
    s.first = v0 == 0;
    s.last = v0 + take == s.kt * per;
    s.col = ((long long)s.b * p.Hkv + s.h) * p.ncol + m;
    return s;
}

// The draft of sequence b, by a whole warp: lane l holds tokens l and l + 32, each
// with the tokens it attends in the draft (itself and its ancestors; 0: not a
// token, nor is what continues it).  Ancestors by doubling: after k rounds a token
// knows those up to 2^k steps above it.
struct TrDraft {
    unsigned long long see[2];
    __device__ __forceinline__ unsigned long long of(int t) const {
        const unsigned long long a = __shfl_sync(0xffffffffu, see[0], t & 31), c = __shfl_sync(0xffffffffu, see[1], t & 31);
        return t < 32 ? a : c;
    }
};
__device__ __noinline__ TrDraft tr_draft(const TreeParams& p, int b, int pos, bool report) {
    const int lane = threadIdx.x & 31;
    TrDraft d;
    int up[2];                                  // the token above those in `see`; -1: the sequence, -2: none
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = lane + 32 * e;
        int par = -2;
        if (i < p.T && pos >= 0) {
            par = __ldcg(p.parent + (long long)b * p.T + i);
            if (par >= i) {
                if (report) set_error(p.err, 0x10u /* KVC_DEV_BAD_ENTRY */);
                par = -2;
            }
            if (par < -2) par = -2;
        }
        up[e] = par;
        d.see[e] = 1ull << i;
    }
#pragma unroll 1
    while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {      // (parents lie below: at most six rounds)
        unsigned long long more[2];
        int next[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int src = up[e] & 31;
            const unsigned long long a = __shfl_sync(0xffffffffu, d.see[0], src), c = __shfl_sync(0xffffffffu, d.see[1], src);
            const int x = __shfl_sync(0xffffffffu, up[0], src), y = __shfl_sync(0xffffffffu, up[1], src);
            more[e] = up[e] < 0 ? 0ull : (up[e] < 32 ? a : c);
            next[e] = up[e] < 0 ? up[e] : (up[e] < 32 ? x : y);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            d.see[e] |= more[e];
            up[e] = next[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (up[e] != -1) d.see[e] = 0ull;
    return d;
}

// Bits lo .. hi of a word.
__device__ __forceinline__ unsigned long long tr_bits(int lo, int hi) {
    if (lo < 0) lo = 0;
    if (hi > 63) hi = 63;
    if (lo > hi) return 0ull;
    return (~0ull >> (63 - hi)) & (~0ull << lo);
}

// Age of the newest position at ring slot s >= sinks when pos tokens are cached (0: the last of them).
__device__ __forceinline__ int tr_age(const TreeParams& p, int pos, int s) {
    const int a = (int)(((long long)pos - 1 - s) % p.window);
    return a < 0 ? a + p.window : a;
}

// Keys of the tile of slots slot0 .. slot0 + 63 that the token at depth `depth`
// attends: sinks, and ages up to window - 2 - depth.  Ages fall by one a slot and
// go from 0 to window - 1 at one place.
__device__ __forceinline__ unsigned long long tr_window(const TreeParams& p, int pos, int slot0, int depth) {
    const int ks = max(0, p.sinks - slot0);
    if (ks >= 64) return ~0ull;
    const int a = tr_age(p, pos, slot0 + ks), lim = p.window - 2 - depth;
    return tr_bits(0, ks - 1) | tr_bits(ks + max(0, a - lim), min((long long)ks + a, 63LL)) |
           ((long long)ks + a + p.window - lim > 63 ? 0ull : tr_bits(ks + a + p.window - lim, 63));
}

// A wait that asks once without sleeping first: in the softmax's loop most have ended
// long before (a wait that may sleep costs 150 cycles even then, and a tile has three).
__device__ __forceinline__ bool tr_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return ws_test(bar, parity) || ws_wait(bar, parity, abort);
}

// Eight rotation pairs (elements of lo with those of hi) of a bf16 row at `pos`.
__device__ __noinline__ void tr_rotate8(uint4& lo, uint4& hi, long long pos, const unsigned long long* turns) {
    uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
        float y[2], z[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float x1 = __uint_as_float(w ? a[e] & 0xffff0000u : a[e] << 16);
            const float x2 = __uint_as_float(w ? b[e] & 0xffff0000u : b[e] << 16);
            float cs, sn;
            rope_cos_sin(pos, turns[2 * e + w], &cs, &sn);
            y[w] = x1 * cs - x2 * sn;
            z[w] = x1 * sn + x2 * cs;
        }
        a[e] = pack_bf16x2(y[0], y[1]);
        b[e] = pack_bf16x2(z[0], z[1]);
    }
    lo = make_uint4(a[0], a[1], a[2], a[3]);
    hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// BAKED: the draft's keys as the cache would store them, rotated at pos0 + depth.
// One CTA per sequence.
template <int D>
__global__ void __launch_bounds__(256) tree_stage_kernel(const __grid_constant__ TreeParams p) {
    __shared__ int s_depth[kTreeMax];
    tr_pdl_wait();
    tr_pdl_launch();
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int pos = p.pos[b];
    if (tid < 32) {
        const TrDraft d = tr_draft(p, b, pos, false);
        s_depth[lane] = __popcll(d.see[0]) - 1;
        s_depth[lane + 32] = __popcll(d.see[1]) - 1;
    }
    __syncthreads();
    constexpr int UPH = D / 16;
    const int units = p.T * p.Hkv * UPH;
    for (int u = tid; u < units; u += 256) {
        const int c = (u % UPH) * 8, row = u / UPH, t = row / p.Hkv;
        if (s_depth[t] < 0) continue;
        const long long at = ((long long)b * p.T * p.Hkv + row) * D + c;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.k_new) + at;
        uint4 x = __ldcg(reinterpret_cast<const uint4*>(src)), y = __ldcg(reinterpret_cast<const uint4*>(src + D / 2));
        tr_rotate8(x, y, (long long)pos + s_depth[t], p.theta + c);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.stage) + at;
        *reinterpret_cast<uint4*>(dst) = x;
        *reinterpret_cast<uint4*>(dst + D / 2) = y;
    }
}

// O[128 x D] (+)= P[128 x 64] V[64 x D]: P in tensor memory (bf16 pairs), vd: the descriptor of V's
// rows 0 .. 15 in a stage; `more`: accumulate onto O.
template <int D>
__device__ __forceinline__ void tr_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vd, uint32_t more) {
    constexpr uint32_t idesc = ws_idesc(kWsRows, D, 1);
#pragma unroll
    for (int ks = 0; ks < kWsKeys / 16; ++ks)
        ws_mma_ts(d_tmem, p_tmem + (uint32_t)(ks * 8), vd + (uint64_t)((ks * 2 * TrShape<D>::Group) >> 4), idesc,
                  ks > 0 ? 1u : more);
}

template <int D, bool FEW>
__global__ void __launch_bounds__(TrShape<D>::Threads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using S = TrShape<D, FEW>;
    constexpr int NQ = S::NQ, NST = S::STAGES, CB = S::CB;
    extern __shared__ __align__(1024) unsigned char sm[];          // (swizzled tiles: their blocks are 1024 bytes)
    const uint32_t sm_u = smem_u32(sm);
    TrStageMeta* meta = reinterpret_cast<TrStageMeta*>(sm + S::OffMeta);
    TrBars* bars = reinterpret_cast<TrBars*>(sm + S::OffMeta + NST * sizeof(TrStageMeta));
    volatile int* abort = &bars->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->ready[s], 1);
            mbar_init(&bars->empty[s], NQ);
        }
        for (int i = 0; i < 2; ++i) {
            for (int u = 0; u < 2; ++u) {
                mbar_init(&bars->s_full[i][u], 1);
                mbar_init(&bars->p_full[i][u], 4);
                mbar_init(&bars->o_done[i][u], 1);
            }
            mbar_init(&bars->q_ready[i], FEW ? 8 : 4);
            mbar_init(&bars->fin[i], 1);
            mbar_init(&bars->both[i], 4 * NQ);
        }
        bars->abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&maps.cache);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    tr_pdl_wait();
    tr_pdl_launch();
    if (sm_u & 1023u) {                              // (uniform; never seen: nothing else lies in shared memory)
        if (tid == 0) index_fault(p.err, 42, sm_u);
        return;
    }
    const TrParts parts = tr_partition(p);
    const long long units = parts.units;
    const int shares = parts.shares, x = blockIdx.x;
    if (x >= shares) return;                         // (uniform: before the tensor memory is taken)
    const long long lo = div_nonneg((long long)x * units, shares), hi = div_nonneg((long long)(x + 1) * units, shares);
    TrWalk walk = tr_find(p, lo);
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
        const bool paged = p.layout == kPaged;
        const int bs = p.bs;
        const int box = p.box;                                  // rows of one copy
        const int per = kWsKeys / box;                          // copies of a tile
        auto take_stage = [&](int s) -> bool {
            if (idx < NST || ws_wait(&bars->empty[s], ((idx / NST) - 1) & 1, abort)) return true;
            if (lane == 0) give_up();
            return ok = false;
        };
        for (long long u = lo; u < hi && ok;) {
            const TrSegment sg = tr_segment<D>(p, walk, u, hi);
            if (lane == 0) {                                    // for the combine: the column's first and last share
                if (sg.first) p.col_shares[sg.col].x = x;
                if (sg.last) p.col_shares[sg.col].y = x;
            }
            const int n = tr_cached(p, sg.pos);
            if (paged && n < sg.pos && lane == 0) set_error(p.err, 0x4u /* KVC_DEV_BAD_POSITION */);
            const int32_t* trow = p.table + (long long)sg.b * p.maxb;
            const int ncopy = (n + box - 1) / box;
            const int end = min(sg.tile0 + sg.nt, sg.kt - 1);   // past the segment's cached tiles
            // 32 copies at a time, one per lane: 32 / per tiles
            for (int t0 = sg.tile0; t0 < end && ok; t0 += 32 / per) {
                const int cp = t0 * per + lane;                 // this lane's copy: rows cp * box ..
                int row = -1;
                if (cp < ncopy) {
                    const int r0 = cp * box;
                    if (paged) {
                        const int lb = r0 / bs;
                        const int phys = __ldcg(trow + lb);
                        bool att = phys >= 0;
                        if (phys >= p.num_blocks) {
                            set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                            att = false;
                        }
                        if (att && p.valid) att = (__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u;
                        if (att) row = (int)(((long long)phys * p.Hkv + sg.h) * bs + (r0 - lb * bs));
                    } else {
                        row = (int)(((long long)sg.b * p.Hkv + sg.h) * p.capacity + r0);
                    }
                }
                const unsigned have = __ballot_sync(0xffffffffu, row >= 0);
                for (int k = 0; k < 32 / per && t0 + k < end; ++k) {
                    const int s = idx % NST;
                    if (!take_stage(s)) break;
                    const unsigned mine = (have >> (k * per)) & ((per == 32) ? 0xffffffffu : ((1u << per) - 1u));
                    const int j = lane - k * per;
                    if (j >= 0 && j < per && row >= 0) {
                        mbar_expect_tx(&bars->full[s], (uint32_t)(box * D * 4));
                        unsigned char* dst = sm + S::OffStage + s * S::StageBytes + j * (box / 8) * S::Group;
                        if (p.grouped)
                            tma_load_5d(dst, &maps.cache, 0, 0, 0, 0, row >> 3, &bars->full[s]);
                        else
                            tma_load_4d(dst, &maps.cache, 0, row, 0, 0, &bars->full[s]);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        const int s0 = (t0 + k) * kWsKeys, live = min(n - s0, kWsKeys);
                        unsigned long long present = 0;
                        for (int c = 0; c < per; ++c)
                            if ((mine >> c) & 1u) present |= (box == 64 ? ~0ull : ((1ull << box) - 1)) << (c * box);
                        present &= tr_bits(0, live - 1);
                        int kind = kTileOpen;
                        if (!paged) {
                            // open if even the deepest token's window holds the oldest of its rows
                            const int ks = max(0, p.sinks - s0);
                            if (ks < live) {
                                const int a = tr_age(p, sg.pos, s0 + ks);
                                if (a < live - 1 - ks || a > p.window - 1 - p.T) kind = kTileWindow;
                            }
                        }
                        meta[s].present = present;
                        meta[s].kind = kind;
                        meta[s].slot0 = s0;
                        mbar_arrive(&bars->full[s]);
                    }
                    ++idx;
                }
            }
            if (ok && sg.nt > 0 && sg.tile0 + sg.nt == sg.kt) {
                // the draft's own rows
                const TrDraft d = tr_draft(p, sg.b, sg.pos, true);
                const unsigned r0 = __ballot_sync(0xffffffffu, d.see[0] != 0ull), r1 = __ballot_sync(0xffffffffu, d.see[1] != 0ull);
                const int s = idx % NST;
                if (take_stage(s)) {
                    // (8 tokens a copy: a lane for K and one for V)
                    if (lane < kWsKeys / 4) {
                        mbar_expect_tx(&bars->full[s], (uint32_t)S::VOff);
                        tma_load_4d(sm + S::OffStage + s * S::StageBytes + (lane >> 1) * S::Group + (lane & 1) * S::VOff,
                                    (lane & 1) ? &maps.v : &maps.k, 0, sg.b * p.T + 8 * (lane >> 1), 0, sg.h, &bars->full[s]);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        meta[s].present = (unsigned long long)r0 | ((unsigned long long)r1 << 32);
                        meta[s].kind = kTileDraft;
                        meta[s].slot0 = 0;
                        mbar_arrive(&bars->full[s]);
                    }
                    ++idx;
                }
                __syncwarp();
            }
            u += sg.units;
        }
        // never leave with copies landing in shared memory
        if (!ok && lane == 0)
            for (int k = (idx > NST ? idx - NST : 0); k < idx; ++k) mbar_wait(&bars->full[k % NST], (k / NST) & 1);
    } else if (warp == 2) {
        // ============================ fix-up ===============================
        int j = 0;
        bool ok = true;
        for (long long u = lo; u < hi && ok;) {
            const TrSegment sg = tr_segment<D>(p, walk, u, hi);
            u += sg.units;
            for (const int end = j + sg.nt; j < end; ++j) {
                const int s = j % NST;
                if (!ws_wait(&bars->full[s], (j / NST) & 1, abort)) {
                    give_up();
                    ok = false;
                    break;
                }
                const unsigned long long present = meta[s].present;
                if (present != ~0ull) {
#pragma unroll 1
                    for (int r = lane; r < kWsKeys; r += 32) {
                        if ((present >> r) & 1ull) continue;
                        unsigned char* st = sm + S::OffStage + s * S::StageBytes + (r >> 3) * S::Group + S::VOff + (r & 7) * 128;
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                            for (int ch = 0; ch < 8; ++ch)
                                *reinterpret_cast<uint4*>(st + cb * 1024 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->ready[s]);
            }
        }
    } else if (warp == 1 || (NQ == 2 && warp == 3)) {
        // ========================== MMA issuers =============================
        // One warp for each Q tile: S_i = Q_i K^T a tile ahead of O_i += P_i V.  The
        // whole warp walks the tiles, its values stay uniform; lane 0 issues.
        const int i = warp >> 1;
        bool ok = true;
        int idx0 = 0, base = 0, loads = 0;             // tiles of the segments before; of this Q tile; its loads
        const uint64_t qd = ws_sdesc(sm_u + S::OffQ + (FEW ? 0 : i * S::QBytes), 16, 1024);
        const uint64_t kd0 = ws_sdesc(sm_u + S::OffStage, 16, S::Group);
        const uint64_t vd0 = ws_sdesc(sm_u + S::OffStage + S::VOff, 1024, S::Group);
        const uint32_t s0 = tmem + S::SCol0 + (uint32_t)(i * 2 * kWsKeys), o_t = tmem + (uint32_t)(i * D);
        for (long long u = lo; u < hi && ok;) {
            const TrSegment sg = tr_segment<D>(p, walk, u, hi);
            const int own = sg.tiles(i), others = sg.nt - own;
            if (own > 0) ok = ws_wait(&bars->q_ready[i], loads++ & 1, abort);
            int ns = 0, npv = 0, nother = 0;           // S issued, P V issued, the other Q tile's tiles passed
            long long t0 = clock64();
            while (ok && (npv < own || nother < others)) {
                // (each barrier's phases are asked for in order)
                if (ns < own && ns < npv + 2) {
                    const int t = idx0 + (sg.alt ? 2 * ns + i : ns), s = t % NST;
                    if (ws_test(&bars->ready[s], (t / NST) & 1)) {
                        ws_fence_after();
                        if (lane == 0) {
                            ws_issue_s<D, kWsRows * 128, 1024>(s0 + (uint32_t)(((base + ns) & 1) * kWsKeys), qd,
                                                                     kd0 + (uint64_t)((s * S::StageBytes) >> 4));
                            ws_commit(&bars->s_full[i][(base + ns) & 1]);
                        }
                        __syncwarp();
                        ++ns;
                        t0 = clock64();
                        continue;
                    }
                }
                if (npv < ns && ws_test(&bars->p_full[i][(base + npv) & 1], ((base + npv) >> 1) & 1)) {
                    ws_fence_after();
                    const int t = idx0 + (sg.alt ? 2 * npv + i : npv), s = t % NST;
                    if (lane == 0) {
                        // P_i in the S buffer it came from (bf16 pairs)
                        tr_issue_pv<D>(o_t, s0 + (uint32_t)(((base + npv) & 1) * kWsKeys),
                                       vd0 + (uint64_t)((s * S::StageBytes) >> 4), npv > 0);
                        ws_commit(&bars->o_done[i][(base + npv) & 1]);
                        ws_commit(&bars->empty[s]);        // this Q tile is done with the tile's K and V
                    }
                    __syncwarp();
                    ++npv;
                    t0 = clock64();
                    continue;
                }
                if (nother < others) {
                    const int t = idx0 + 2 * nother + (i ^ 1), s = t % NST;
                    if (ws_test(&bars->ready[s], (t / NST) & 1)) {
                        if (lane == 0) mbar_arrive(&bars->empty[s]);
                        __syncwarp();
                        ++nother;
                        t0 = clock64();
                        continue;
                    }
                }
                if (*abort || clock64() - t0 > kWaitCycles) ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok && lane == 0) give_up();
            __syncwarp();
            idx0 += sg.nt;
            base += own;
            u += sg.units;
        }
        if (lane == 0) {
            // every product this thread issued is done before TMEM is freed
            ws_commit(&bars->fin[i]);
            if (!mbar_wait(&bars->fin[i], 0)) set_error(p.err, 0x8u /* KVC_DEV_TIMEOUT */);
        }
        __syncwarp();
    } else if (warp >= kTrSoftmax0) {
        // ============================ softmax ==============================
        const int qi = (warp - kTrSoftmax0) >> 2;          // Q tile
        const int r = tid - (kTrSoftmax0 + 4 * qi) * 32;   // row = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        unsigned char* Qs = sm + S::OffQ + (FEW ? 0 : qi * S::QBytes);
        const int tl = tr_token(p, r);
        bool ok = true;
        int idx0 = 0, base = 0, at_b = -1, joins = 0;
        TrDraft draft{};
        for (long long u = lo; u < hi && ok;) {
            const TrSegment sg = tr_segment<D>(p, walk, u, hi);
            // (the draft's ancestors: before the q rows where those are rotated, else while the
            // first product runs)
            auto know_draft = [&]() {
                if (sg.b == at_b) return;
                draft = tr_draft(p, sg.b, sg.pos, false);
                at_b = sg.b;
            };
            if (p.rope != kRopeNone) know_draft();
            const int c0 = sg.alt ? 0 : qi * p.tq;         // the Q tile's first token in the column
            const bool row_ok = tl < p.tq && c0 + tl < sg.tokens;
            const int nt = sg.tiles(qi);                   // 0: the other warpgroup has the segment's one tile
            // Q rows, rotated at their positions when BAKED, unscaled bf16
            if (FEW || nt > 0) {
                // (D / 16 lanes share a row: a load covers whole lines; a batch is in flight at once.  Rows
                // behind the last token are its again: nothing is taken from them.)
                constexpr int ROWS = FEW ? 16 : 32;        // of a warp (FEW: a tile's among both warpgroups')
                constexpr int LPR = D / 16, RPW = 32 / LPR, NB = ROWS / RPW < 8 ? ROWS / RPW : 8;
                const int c = lane % LPR;                  // 8-column chunk, paired with c + D / 16
                const int q_r0 = (FEW ? warp - kTrSoftmax0 : warp & 3) * ROWS + lane / LPR, last_t = max(min(p.tq, sg.tokens - c0) - 1, 0);
                const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(p.q) +
                                          (((long long)sg.b * p.T + sg.n0 + c0) * p.Hq + sg.h * p.G) * D + 8 * c;
                // Q tile: [column block][128 rows][128 B], 128-byte swizzle; RPW rows on, bits 4 .. 6 change by a constant
                auto place = [&](int ch) { return (ch >> 3) * (kWsRows * 128) + q_r0 * 128 + (((ch ^ q_r0) & 7) << 4); };
                const int p1 = place(c), p2 = place(c + D / 16);
#pragma unroll 1
                for (int it0 = 0; it0 < ROWS / RPW; it0 += NB) {
                    uint4 a[NB], e[NB];
#pragma unroll
                    for (int it = 0; it < NB; ++it) {
                        const int rr = q_r0 + (it0 + it) * RPW, rtl = tr_token(p, rr);
                        const __nv_bfloat16* qrow = q0 + (long long)(min(rtl, last_t) * p.Hq + rr - rtl * p.G) * D;
                        a[it] = __ldcg(reinterpret_cast<const uint4*>(qrow));
                        e[it] = __ldcg(reinterpret_cast<const uint4*>(qrow + D / 2));
                    }
#pragma unroll
                    for (int it = 0; it < NB; ++it) {
                        const int on = (it0 + it) * RPW * 128, turn = ((it * RPW) & 7) << 4;
                        *reinterpret_cast<uint4*>(Qs + ((p1 + on) ^ turn)) = a[it];
                        *reinterpret_cast<uint4*>(Qs + ((p2 + on) ^ turn)) = e[it];
                    }
                }
                if (p.rope != kRopeNone) {
                    // each lane's own chunks, in place
#pragma unroll 1
                    for (int it = 0; it < ROWS / RPW; ++it) {
                        const int rr = q_r0 + it * RPW;
                        const int rtl = tr_token(p, rr);
                        const bool rok = rtl < p.tq && c0 + rtl < sg.tokens;
                        const unsigned long long mine = draft.of(rok ? sg.n0 + c0 + rtl : 0);
                        const int c1 = c, c2 = c + D / 16;
                        uint4* x = reinterpret_cast<uint4*>(Qs + (c1 >> 3) * (kWsRows * 128) + rr * 128 + (((c1 ^ rr) & 7) << 4));
                        uint4* y = reinterpret_cast<uint4*>(Qs + (c2 >> 3) * (kWsRows * 128) + rr * 128 + (((c2 ^ rr) & 7) << 4));
                        if (rok) tr_rotate8(*x, *y, (long long)sg.pos + max(__popcll(mine) - 1, 0), p.theta + 8 * c);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->q_ready[FEW ? 0 : qi]);
                    if (FEW && sg.nt > 1) mbar_arrive(&bars->q_ready[1]);      // (the second issuer has a tile)
                }
            }
            know_draft();
            const unsigned long long see = draft.of(row_ok ? sg.n0 + c0 + tl : 0);
            const bool real = row_ok && see != 0ull;
            const int depth = __popcll(see) - 1;
            float m_run = -INFINITY, l_run = 0.f;          // m in base-2 units of the scaled scores
            for (int lt = 0; lt < nt; ++lt) {
                const int j = base + lt;
                // the stage's meta, on the way to the scores
                const int gt = idx0 + (sg.alt ? 2 * lt + qi : lt);
                if (!tr_wait(&bars->ready[gt % NST], (gt / NST) & 1, abort)) {
                    ok = false;
                    break;
                }
                const TrStageMeta mt = meta[gt % NST];
                if (!tr_wait(&bars->s_full[qi][j & 1], (j >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                ws_fence_after();
                float sv[kWsKeys];
                const uint32_t scol = S::SCol0 + (uint32_t)((qi * 2 + (j & 1)) * kWsKeys);
                ws_ld32(lane_base + scol, sv);
                ws_ld32(lane_base + scol + 32, sv + 32);
                ws_wait_ld();
                if (mt.kind != kTileOpen || mt.present != ~0ull) {           // (uniform)
                    unsigned long long vis = mt.present;
                    if (mt.kind == kTileDraft)
                        vis &= see;
                    else if (mt.kind == kTileWindow)
                        vis &= tr_window(p, sg.pos, mt.slot0, depth);
                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int k = 0; k < kWsKeys; ++k)
                        sv[k] = (((k < 32 ? v0 : v1) >> (k & 31)) & 1u) ? sv[k] : -INFINITY;
                }
                const float mx = ws_max64(sv) * p.scale2;
                float mn = m_run, alpha = 1.f;
                if (mx > m_run + kTrLazy) {
                    mn = mx;
                    alpha = m_run == -INFINITY ? 1.f : exp2f(m_run - mn);
                }
                const float ls = ws_exp64(sv, p.scale2, mn == -INFINITY ? 0.f : -mn);
                l_run = l_run * alpha + ls;
                m_run = mn;
                // O is touched only once P V of the previous tile is done; where nothing is
                // rescaled, that is asked for after this tile's weights have been handed over
                const bool rescale = lt > 0 && __any_sync(0xffffffffu, alpha != 1.f);
                if (rescale) {
                    if (!tr_wait(&bars->o_done[qi][(j - 1) & 1], ((j - 1) >> 1) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    ws_fence_after();
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
                {
                    float pw[kWsKeys / 2];
#pragma unroll
                    for (int k2 = 0; k2 < kWsKeys / 2; ++k2)
                        pw[k2] = __uint_as_float(pack_bf16x2(sv[2 * k2], sv[2 * k2 + 1]));
                    ws_st32(lane_base + scol, pw);
                }
                ws_wait_st();
                ws_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[qi][j & 1]);
                if (lt > 0 && !rescale && !tr_wait(&bars->o_done[qi][(j - 1) & 1], ((j - 1) >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
            }
            if (!ok) {
                give_up();
                break;
            }
            // the last P V, then the partial (m, l, o) of each row
            if (nt > 0) {
                if (!ws_wait(&bars->o_done[qi][(base + nt - 1) & 1], ((base + nt - 1) >> 1) & 1, abort)) {
                    give_up();
                    break;
                }
                ws_fence_after();
            }
            // Alternate tiles: the two warpgroups' sums of a row become one, each warpgroup
            // joining half of the columns.  (f: what this row's sums enter with.)
            float f[2] = {1.f, 0.f};
            int cols = D, col0 = 0, o0 = qi * D;               // columns to write; O's column in tensor memory
            const bool other = sg.alt && sg.nt > 1;            // (the second warpgroup had a tile)
            if (sg.alt) {
                bars->ml[qi][r] = make_float2(m_run, l_run);
                ws_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->both[0]);
                if (!ws_wait(&bars->both[0], joins & 1, abort)) {
                    ok = false;
                    give_up();
                    break;
                }
                ws_fence_after();
                const float2 a = bars->ml[0][r], e = bars->ml[1][r];
                m_run = fmaxf(a.x, e.x);
                f[0] = a.x == -INFINITY && a.y == a.y ? 0.f : exp2f(a.x - m_run);
                f[1] = e.x == -INFINITY && e.y == e.y ? 0.f : exp2f(e.x - m_run);
                l_run = a.y * f[0] + e.y * f[1];
                cols = D / 2;
                col0 = qi * (D / 2);
                o0 = col0;
            }
            // a column in one piece goes to the output, others leave a partial of each row
            const bool whole = sg.first && sg.last;
            if (!real) {
                m_run = -INFINITY;
                l_run = 0.f;
            }
            const float inv = !whole ? 1.f : (l_run == 0.f ? 0.f : 1.f / l_run);
            const long long row_a = (x + sg.col) * p.rows + (sg.alt ? 0 : qi * p.tq * p.G);
            if (!whole && row_ok && (!sg.alt || qi == 0)) p.part_ml[row_a + r] = make_float2(m_run, l_run);
            if (nt > 0 || sg.alt) {
                // through the Q tile's shared memory (its products are done), each row in the
                // place of its own q (which this warp alone writes; FEW: a column block for each
                // warpgroup, and no q before both are done), CP columns at a time, so that whole
                // lines go out
                constexpr int CP = D == 64 || FEW ? 32 : 64, CPL = CP / 4;            // 16-byte chunks of a staged row
                auto stg = [&](int row, int ch) {
                    return reinterpret_cast<float4*>(Qs + (FEW ? qi : ch >> 3) * (kWsRows * 128) + row * 128 + (((ch ^ row) & 7) << 4));
                };
#pragma unroll 1
                for (int c6 = 0; c6 < cols; c6 += CP) {
#pragma unroll 1
                    for (int hf = 0; hf < CP / 32; ++hf) {
                        float ov[32];
                        ws_ld32(lane_base + (uint32_t)(o0 + c6 + 32 * hf), ov);
                        ws_wait_ld();
                        if (sg.alt) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) ov[k] = f[0] == 0.f ? 0.f : ov[k] * f[0];
                            if (other) {
                                float ow[32];
                                ws_ld32(lane_base + (uint32_t)(D + o0 + c6 + 32 * hf), ow);
                                ws_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) ov[k] = f[1] == 0.f ? ov[k] : fmaf(ow[k], f[1], ov[k]);
                            }
                        }
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) ov[k] = real ? ov[k] * inv : 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *stg(r, 8 * hf + k) = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int it = 0; it < CPL; ++it) {
                        const int rr = (warp & 3) * 32 + (32 / CPL) * it + lane / CPL, ch = lane % CPL;
                        const int rtl = tr_token(p, rr);
                        if (rtl < p.tq && c0 + rtl < sg.tokens) {
                            const float4 w = *stg(rr, ch);
                            if (whole) {
                                const long long row =
                                    ((long long)sg.b * p.T + sg.n0 + c0 + rtl) * p.Hq + sg.h * p.G + (rr - rtl * p.G);
                                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + col0 + c6 + 4 * ch) =
                                    make_uint2(pack_bf16x2(w.x, w.y), pack_bf16x2(w.z, w.w));
                            } else {
                                *reinterpret_cast<float4*>(p.part_o + (row_a + rr) * D + col0 + c6 + 4 * ch) = w;
                            }
                        }
                    }
                    __syncwarp();
                }
                // O is read: the next segment's first product may overwrite it
                // (it waits for this warpgroup's next P)
                ws_fence_before();
            }
            if (sg.alt) {
                // ... and for the other's reading of it
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->both[1]);
                if (!ws_wait(&bars->both[1], joins & 1, abort)) {
                    give_up();
                    break;
                }
                ++joins;
            }
            idx0 += sg.nt;
            base += nt;
            u += sg.units;
        }
    }

    // the MMA thread has waited for all of its products (its last commit)
    ws_fence_before();
    __syncthreads();
    ws_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::TmemCols) : "memory");
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
constexpr int kTrCombineThreads = 256;

// One CTA per (column, p.comb_rows of its rows); columns that one share held whole are
// done already.  D / 4 lanes a row, 16 bytes each; a batch of eight parts is in flight at
// once, joined to those before by the running maximum.
template <int D>
__global__ void __launch_bounds__(kTrCombineThreads) tree_combine_kernel(const __grid_constant__ TreeParams p) {
    constexpr int LPR = D / 4 < 32 ? D / 4 : 32, NC = D / 4 / LPR;        // lanes of a row; 16-byte chunks of a lane
    constexpr int U = NC == 1 ? 8 : 4;
    tr_pdl_launch();
    const int tid = threadIdx.x, lane = tid & 31;
    const int col = blockIdx.x, bh = col / p.ncol, m = col - bh * p.ncol, b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int tokens = min(p.mq, p.T - m * p.mq);
    tr_pdl_wait();
    const int2 sh = __ldcg(p.col_shares + col);
    if (!tree_shares_held(sh.x, sh.y, p.ctas)) {
        if (tid == 0) index_fault(p.err, 43, sh.x);
        return;
    }
    const int np = sh.y - sh.x + 1;
    if (np <= 1) return;                                                  // one share: written whole
    const long long slot = (long long)sh.x + col;
    const int c = lane % LPR;
#pragma unroll 1
    for (int row = blockIdx.y * p.comb_rows + tid / LPR; row < min(tokens * p.G, (int)(blockIdx.y + 1) * p.comb_rows);
         row += kTrCombineThreads / LPR) {
        float M = -INFINITY, L = 0.f;
        float4 acc[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < np; k0 += U) {
            float2 ml[U];
            float4 o[U][NC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long at = (slot + min(k0 + u, np - 1)) * p.rows + row;
                ml[u] = k0 + u < np ? __ldcg(p.part_ml + at) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    o[u][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + k * LPR + c);
            }
            float mn = M;
#pragma unroll
            for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
            const float a = M == -INFINITY ? 1.f : exp2f(M - mn);         // (nothing yet, or a sum of NaN)
            L *= a;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                acc[k].x *= a;
                acc[k].y *= a;
                acc[k].z *= a;
                acc[k].w *= a;
            }
            M = mn;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // (an empty part's o may hold anything; NaN scores leave no maximum, but a sum of NaN)
                if (ml[u].x == -INFINITY && ml[u].y == ml[u].y) continue;
                const float e = exp2f(ml[u].x - mn);
                L = fmaf(ml[u].y, e, L);
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    acc[k].x = fmaf(o[u][k].x, e, acc[k].x);
                    acc[k].y = fmaf(o[u][k].y, e, acc[k].y);
                    acc[k].z = fmaf(o[u][k].z, e, acc[k].z);
                    acc[k].w = fmaf(o[u][k].w, e, acc[k].w);
                }
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int t = tr_token(p, row);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                             (((long long)b * p.T + m * p.mq + t) * p.Hq + h * p.G + (row - t * p.G)) * D;
#pragma unroll
        for (int k = 0; k < NC; ++k)
            *reinterpret_cast<uint2*>(dst + 4 * (k * LPR + c)) =
                make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv), pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
    }
}

cudaLaunchConfig_t tr_config(dim3 grid, int threads, int smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int D, bool FEW = false>
cudaError_t launch_tree_t(const TreeParams& p, const TreeMaps& maps, cudaStream_t stream) {
    constexpr int kSmem = tr_smem_bytes<D, FEW>();
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(tree_kernel<D, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = tr_config(dim3(p.ctas), TrShape<D, FEW>::Threads, kSmem, stream, &attr);
    e = cudaLaunchKernelEx(&cfg, tree_kernel<D, FEW>, p, maps);
    if (e != cudaSuccess) return e;
    // a row a warp, or several where the CTAs would not be on the GPU together (four an SM): a second
    // wave of them cost the drafts over 8 rings 4 us
    TreeParams c = p;
    const long long cols = (long long)p.B * p.Hkv * p.ncol;
    const int rows = (p.T < p.mq ? p.T : p.mq) * p.G, pass = kTrCombineThreads / (D / 4 < 32 ? D / 4 : 32);
    const long long most = cols * ((rows + pass - 1) / pass), turns = (most + kTreeCtas * 4 - 1) / (kTreeCtas * 4);
    c.comb_rows = pass * (int)(turns < (rows + pass - 1) / pass ? turns : (rows + pass - 1) / pass);
    cfg = tr_config(dim3((unsigned)cols, (rows + c.comb_rows - 1) / c.comb_rows), kTrCombineThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D>, c);
}

}  // namespace

cudaError_t launch_tree(int D, const TreeParams& p, const TreeMaps& maps, cudaStream_t s) {
    if (D == 64) return launch_tree_t<64>(p, maps, s);
    if (D == 256) return launch_tree_t<256>(p, maps, s);
    // (one unit a tile: drafts of up to 128 rows)
    return p.col_units == 1 ? launch_tree_t<128, true>(p, maps, s) : launch_tree_t<128>(p, maps, s);
}

cudaError_t launch_tree_stage(int D, const TreeParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = tr_config(dim3(p.B), 256, 0, s, &attr);
    return D == 64    ? cudaLaunchKernelEx(&cfg, tree_stage_kernel<64>, p)
           : D == 128 ? cudaLaunchKernelEx(&cfg, tree_stage_kernel<128>, p)
                      : cudaLaunchKernelEx(&cfg, tree_stage_kernel<256>, p);
}

}  // namespace kvc
