// kvc_decode_attention_shared: decode attention of a paged batch whose groups
// of sequences share a prefix (the same physical blocks at the head of their
// tables).  softmax splits over any partition of the keys into partial results
// (m, l, o), so the shared keys are scored once for a whole group -- the rows
// of one matrix product are its members' q heads of a kv head -- and each
// sequence's own keys by the ordinary decode kernel; a combine kernel joins
// them:  M = max m_i,  out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M).
//
//   shared_plan_kernel    one CTA per sequence: its place in its group, and how
//                         many leading blocks its table shares with the first
//                         member's that has any; the last CTA to finish (an atomic
//                         ticket, no waiting) takes each group's minimum over the
//                         members that share and lays the work out.
//   (plan_rows_kernel)    the blocks behind the shared ones, per sequence.
//   shared_prefix_kernel  the shared keys, on tcgen05 (below).
//   (decode_mma_kernel)   the rest.
//   shared_combine_kernel one warp per (sequence, q head).
//
// Prefix work.  A column is (group, kv head, up to NQ x 128 rows of members x q
// heads); its keys are cut into tiles of 64, a unit of work for each Q tile.  All
// units of all columns, laid end to end, are split into nearly equal contiguous
// shares, one per CTA (one CTA per SM); the part of a column in a share is a
// segment and leaves one partial per row.
// What bounds it: a tile is 64 rows of K and V (32 KB at head_dim 128) for 4 x
// 64 x 128 x D flops a Q tile, so up to one Q tile the bytes bound, beyond it
// the softmax.
// Rows that are never there (members x heads below 128) cost nothing but
// tensor-core time.  A column of one Q tile gives both softmax warpgroups the
// same rows and alternate tiles, each with sums of its own (two partials): the
// latency of one tile's softmax, which a single warpgroup would wait out, is
// what a CTA with few rows spends its time on.
//
// Measured (32 / 8 heads of 128, blocks of 16), whole call: 64 sequences in groups
// of 8 with 2048 shared tokens and 2049 .. 8192 in all 185 us, 0.69 of the bytes'
// time (the plan 8 us, the prefix 25 to 35, the sequences' own keys 130 at 0.9 of
// bandwidth, the combine 5); 96 readers of one document 149 us, of which the prefix 75;
// six readers 41 us, five dependent launches.  Plain decode of the same batches, which
// takes a shared block from L2 for all sequences but the first (cold, us, plain / shared):
// 179 / 200, 1087 / 155, 30 / 52; the shared form pays from about 150,000 shared tokens
// mapped (sequences x prefix).
#include <atomic>

#include "kvc_decode.cuh"
#include "kvc_shared.h"
#include "kvc_tc.cuh"

namespace kvc {

namespace {

constexpr int kShPlanThreads = 256;
constexpr int kShSoftmax0 = 4;              // first softmax warp
constexpr float kShLazy = 8.f;

__device__ __forceinline__ void sh_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void sh_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
// Sums of three counts and a minimum over the CTA (every thread gets them).
struct ShScan {
    int below, rank, n, leader;
};
__device__ __forceinline__ ShScan sh_reduce(ShScan v, ShScan* s_w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        v.below += __shfl_xor_sync(0xffffffffu, v.below, off);
        v.rank += __shfl_xor_sync(0xffffffffu, v.rank, off);
        v.n += __shfl_xor_sync(0xffffffffu, v.n, off);
        v.leader = min(v.leader, __shfl_xor_sync(0xffffffffu, v.leader, off));
    }
    if (lane == 0) s_w[warp] = v;
    __syncthreads();
    ShScan r = s_w[0];
    for (int w = 1; w < kShPlanThreads / 32; ++w) {
        r.below += s_w[w].below;
        r.rank += s_w[w].rank;
        r.n += s_w[w].n;
        r.leader = min(r.leader, s_w[w].leader);
    }
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(kShPlanThreads) shared_plan_kernel(const __grid_constant__ SharedParams p) {
    __shared__ ShScan s_w[kShPlanThreads / 32];
    __shared__ int s_common, s_last;
    __shared__ long long s_u[kShPlanThreads / 32], s_r[kShPlanThreads / 32];
    __shared__ int s_g[kShPlanThreads / 32];
    const int tid = threadIdx.x, b = blockIdx.x;
    sh_pdl_wait();
    sh_pdl_launch();
    auto full_blocks = [&](int q) {                // blocks wholly at positions <= t of sequence q
        const int t = clamp_paged_t(p.pos[q], p.maxb, p.bs);
        return t < 0 ? 0 : (int)(((long long)t + 1) / p.bs);
    };
    // this sequence's place: the members of lower group ids before its group, its rank
    // in the group, the group's size, and the first member that has a block to share (an
    // idle one has none)
    const int gid = p.group[b];
    const bool grouped = gid >= 0 && gid < p.B;
    if (gid >= p.B && tid == 0) set_error(p.err, 0x10u /* KVC_DEV_BAD_ENTRY */);
    ShScan c{0, 0, 0, p.B};
    if (grouped) {
        for (int o = tid; o < p.B; o += kShPlanThreads) {
            const int og = p.group[o];
            if (og >= 0 && og < gid) ++c.below;
            if (og == gid) {
                ++c.n;
                if (o < b) ++c.rank;
                if (o < c.leader && full_blocks(o) > 0) c.leader = o;
            }
        }
    }
    c = sh_reduce(c, s_w);
    // leading blocks wholly at positions <= t here and for that member, whose entries
    // equal that member's
    const bool placed = grouped && c.n > 1 && c.leader < p.B;
    if (placed) {
        const int nb = min(full_blocks(b), full_blocks(c.leader));
        if (tid == 0) s_common = nb;
        __syncthreads();
        const int32_t* mine = p.table + (long long)b * p.maxb;
        const int32_t* lead = p.table + (long long)c.leader * p.maxb;
        int first = nb;
        for (int i = tid; i < nb; i += kShPlanThreads)
            if (mine[i] != lead[i]) {
                first = i;
                break;
            }
        if (first < nb) atomicMin(&s_common, first);
        __syncthreads();
    }
    if (tid == 0) {
        p.seq[b] = make_int4(placed ? c.below : -1, c.rank, c.n, placed ? s_common : 0);
        if (grouped) p.members[c.below + c.rank] = b;
        __threadfence();
        s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last CTA: the blocks that the members of a group have in common, how many have
    // any and the first of them, kept at the group's place in the member list.  Members
    // without (idle, or mapped elsewhere) take part in nothing but the tiles' rows: their
    // own keys begin at 0, and the join does not read their part of the prefix.
    for (int o = tid; o < p.B; o += kShPlanThreads) {
        p.gmin[o] = 0x7fffffff;
        p.start[o] = 0x7fffffff;
        p.seq_group[o].x = 0;
    }
    __syncthreads();
    for (int o = tid; o < p.B; o += kShPlanThreads) {
        const int4 s = __ldcg(&p.seq[o]);
        if (s.x >= 0 && s.w > 0) {
            atomicMin(&p.gmin[s.x], s.w);
            atomicMin(&p.start[s.x], o);
            atomicAdd(&p.seq_group[s.x].x, 1);
        }
    }
    __syncthreads();
    // groups with something to share, in member-list order: their units (tiles of
    // every column) and partial rows before them
    long long run_u = 0, run_r = 0;
    int run_g = 0;
    const int lane = tid & 31, warp = tid >> 5;
    for (int base = 0; base < p.B; base += kShPlanThreads) {
        const int o = base + tid;
        // place o of the member list begins a group iff two of its members share
        int4 s = make_int4(-1, 0, 0, 0);
        int lead = -1;
        if (o < p.B && __ldcg(&p.seq_group[o].x) > 1) {
            lead = __ldcg(&p.start[o]);
            s = __ldcg(&p.seq[lead]);
        }
        const int common = lead >= 0 ? __ldcg(&p.gmin[o]) : 0;
        const bool real = lead >= 0;
        SharedGroup g{};
        long long u = 0, r = 0;
        if (real) {
            g.n = s.z;
            g.off = o;
            g.leader = lead;
            g.rows = common * p.bs;
            g.kt = (g.rows + kWsKeys - 1) / kWsKeys;
            g.mt = (g.n + p.mq - 1) / p.mq;
            // the columns of a kv head: full ones of two units a tile, and a last one
            const int last = g.n - (g.mt - 1) * p.mq;
            g.hu = (long long)g.kt * ((g.mt - 1) * p.full_units + (last <= p.tq ? 1 : p.full_units));
            u = p.Hkv * g.hu;
            r = (long long)p.Hkv * g.n * p.G;
        }
        long long iu = u, ir = r;
        int ig = real ? 1 : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long a = __shfl_up_sync(0xffffffffu, iu, off), bb = __shfl_up_sync(0xffffffffu, ir, off);
            const int gg = __shfl_up_sync(0xffffffffu, ig, off);
            if (lane >= off) {
                iu += a;
                ir += bb;
                ig += gg;
            }
        }
        if (lane == 31) {
            s_u[warp] = iu;
            s_r[warp] = ir;
            s_g[warp] = ig;
        }
        __syncthreads();
        long long cu = run_u, cr = run_r;
        int cg = run_g;
        for (int w = 0; w < kShPlanThreads / 32; ++w) {
            if (w < warp) {
                cu += s_u[w];
                cr += s_r[w];
                cg += s_g[w];
            }
            run_u += s_u[w];
            run_r += s_r[w];
            run_g += s_g[w];
        }
        if (real) {
            g.units0 = cu + iu - u;
            g.rows0 = cr + ir - r;
            p.groups[cg + ig - 1] = g;
            p.gmin[o] = cg + ig - 1;          // its index, for the members below
        } else if (o < p.B) {
            p.gmin[o] = -1;
        }
        __syncthreads();
    }
    // each sequence's group and the position its own keys begin at
    for (int o = tid; o < p.B; o += kShPlanThreads) {
        const int4 s = __ldcg(&p.seq[o]);
        const int gi = s.x >= 0 && s.w > 0 ? p.gmin[s.x] : -1;
        p.seq_group[o] = make_int2(gi, s.y);
        p.start[o] = gi >= 0 ? p.groups[gi].rows : 0;
    }
    if (tid == 0) {
        p.head->units = run_u;
        p.head->ngroups = run_g;
        p.head->shares = (int)min((long long)p.ctas, (run_u + kSharedMinTiles - 1) / kSharedMinTiles);
        *p.ticket = 0u;                       // ready for the next call
    }
}

// ---------------------------------------------------------------------------
// prefix
// ---------------------------------------------------------------------------
template <int D>
struct PxShape {
    static constexpr int NQ = shared_q_tiles(D);
    static constexpr int STAGES = D == 64 ? 6 : (D == 128 ? 4 : 2);
    static constexpr int CB = D / 64;                          // 64-column blocks of a row
    static constexpr int QBytes = kWsRows * D * 2;             // one Q tile
    static constexpr int KVBlock = 2 * kWsKeys * 128;          // one column block of K and V
    static constexpr int StageBytes = CB * KVBlock;
    static constexpr int OffQ = 0;
    static constexpr int OffStage = OffQ + NQ * QBytes;
    static constexpr int OffMeta = OffStage + STAGES * StageBytes;
    static constexpr int TmemCols = 512;
    static constexpr int SCol0 = NQ * D;                       // S buffers after the O tiles
    static_assert(NQ * D + NQ * 2 * kWsKeys <= TmemCols, "TMEM columns");
    static constexpr int Threads = 32 * (kShSoftmax0 + 4 * NQ);
};

struct alignas(16) PxStageMeta {
    unsigned long long present;     // rows of the tile that hold a key
    unsigned long long pad;
};

struct PxBars {
    uint64_t full[6], ready[6], empty[6];
    uint64_t s_full[2][2], p_full[2], o_done[2], q_ready[2], fin[2];
    uint32_t tmem;
    int abort;
};

template <int D>
constexpr int px_smem_bytes() {
    using S = PxShape<D>;
    return S::OffMeta + S::STAGES * (int)sizeof(PxStageMeta) + (int)sizeof(PxBars) + 1024;
}

// Eight rotation pairs (elements of lo with those of hi) of a bf16 row at `pos`.
__device__ __forceinline__ void px_rotate8(uint4& lo, uint4& hi, long long pos, const unsigned long long* turns) {
    uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
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

// One segment: tiles tile0 .. tile0 + nt - 1 of a column.
struct PxSegment {
    int h, m0, members, off, leader, rows;     // kv head, first member's rank and members, the group's list and prefix
    int tile0, nt;                             // nt may be 0: one unit of a tile that begins in the share before
    long long units;
    int alt;                                   // one Q tile's rows: the warpgroups take alternate tiles
    long long row0;                            // partial row of the column's first row, before the share's own offset
    __device__ __forceinline__ int tiles(int i) const { return alt ? (nt + 1 - i) >> 1 : nt; }
};

// The segment that begins at unit u of a share ending at hi (a whole warp's call).
template <int D>
__device__ __forceinline__ PxSegment px_segment(const SharedParams& p, int ngroups, long long u, long long hi) {
    const int lane = threadIdx.x & 31;
    int gi = 0;
    for (int base = 0; base < ngroups; base += 32) {
        const unsigned le = __ballot_sync(0xffffffffu, base + lane < ngroups && __ldcg(&p.groups[base + lane].units0) <= u);
        if (le) gi = base + 31 - __clz(le);
        if (le != 0xffffffffu) break;
    }
    const SharedGroup* g = p.groups + gi;
    const int kt = __ldcg(&g->kt), n = __ldcg(&g->n);
    const long long hu = __ldcg(&g->hu);
    long long v = u - __ldcg(&g->units0);
    PxSegment s;
    s.h = (int)(v / hu);
    v -= s.h * hu;
    const int m = (int)(v / ((long long)kt * p.full_units));     // every column but a head's last is full
    v -= (long long)m * kt * p.full_units;
    s.m0 = m * p.mq;
    s.members = min(p.mq, n - s.m0);
    // units to tiles: a tile belongs to the share that holds its first unit
    const int per = s.members <= p.tq ? 1 : p.full_units;
    const long long take = min((long long)kt * per - v, hi - u);
    s.units = take;
    s.tile0 = (int)((v + per - 1) / per);
    s.nt = (int)((v + take + per - 1) / per) - s.tile0;
    s.off = __ldcg(&g->off);
    s.leader = __ldcg(&g->leader);
    s.rows = __ldcg(&g->rows);
    s.alt = PxShape<D>::NQ == 2 && s.members <= p.tq;
    s.row0 = __ldcg(&g->rows0) + ((long long)s.h * n + s.m0) * p.G;
    return s;
}

template <int D>
__global__ void __launch_bounds__(PxShape<D>::Threads, 1)
    shared_prefix_kernel(const __grid_constant__ SharedParams p, const __grid_constant__ CUtensorMap map) {
    using S = PxShape<D>;
    constexpr int NQ = S::NQ, NST = S::STAGES, CB = S::CB;
    extern __shared__ unsigned char px_raw[];
    const uint32_t raw_u = smem_u32(px_raw);
    unsigned char* sm = px_raw + (((raw_u + 1023u) & ~1023u) - raw_u);
    const uint32_t sm_u = smem_u32(sm);
    PxStageMeta* meta = reinterpret_cast<PxStageMeta*>(sm + S::OffMeta);
    PxBars* bars = reinterpret_cast<PxBars*>(sm + S::OffMeta + NST * sizeof(PxStageMeta));
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
            }
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->q_ready[i], kWsRows);
            mbar_init(&bars->fin[i], 1);
        }
        bars->abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&map);
    }
    sh_pdl_wait();
    sh_pdl_launch();
    const int ngroups = __ldcg(&p.head->ngroups), shares = __ldcg(&p.head->shares);
    const long long units = __ldcg(&p.head->units);
    const int x = blockIdx.x;
    if (x >= shares || units <= 0) return;           // (uniform: before the tensor memory is taken)
    const long long lo = div_nonneg((long long)x * units, shares), hi = div_nonneg((long long)(x + 1) * units, shares);
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
        const int bs = p.bs;
        const int box = bs < kWsKeys ? bs : kWsKeys;            // rows of one copy
        const int per = kWsKeys / box;                          // copies of a tile
        for (long long u = lo; u < hi && ok;) {
            const PxSegment sg = px_segment<D>(p, ngroups, u, hi);
            const int32_t* trow = p.table + (long long)sg.leader * p.maxb;
            const int ncopy = (sg.rows + box - 1) / box;        // of the whole prefix
            // 32 copies at a time, one per lane: 32 / per tiles
            for (int t0 = 0; t0 < sg.nt && ok; t0 += 32 / per) {
                const int cp = (sg.tile0 + t0) * per + lane;    // this lane's copy: rows cp * box ..
                int row = -1;
                if (cp < ncopy) {
                    const int r0 = cp * box, lb = r0 / bs;
                    const int phys = __ldcg(trow + lb);
                    bool att = phys >= 0;
                    if (phys >= p.num_blocks) {
                        set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                        att = false;
                    }
                    if (att && p.valid) att = (__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u;
                    if (att) row = (int)(((long long)phys * p.Hkv + sg.h) * bs + (r0 - lb * bs));
                }
                const unsigned have = __ballot_sync(0xffffffffu, row >= 0);
                for (int k = 0; k < 32 / per && t0 + k < sg.nt; ++k) {
                    const int s = idx % NST;
                    if (idx >= NST && !ws_wait(&bars->empty[s], ((idx / NST) - 1) & 1, abort)) {
                        if (lane == 0) give_up();
                        ok = false;
                        break;
                    }
                    const unsigned mine = (have >> (k * per)) & ((per == 32) ? 0xffffffffu : ((1u << per) - 1u));
                    const int j = lane - k * per;
                    if (j >= 0 && j < per && row >= 0) {
                        mbar_expect_tx(&bars->full[s], (uint32_t)(box * D * 4));
                        unsigned char* dst = sm + S::OffStage + s * S::StageBytes + j * box * 128;
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                            for (int kv = 0; kv < 2; ++kv)
                                tma_load_4d(dst + cb * S::KVBlock + kv * kWsKeys * 128, &map, cb * 64, row, kv,
                                            p.layer, &bars->full[s]);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        unsigned long long present = 0;
                        for (int c = 0; c < per; ++c)
                            if ((mine >> c) & 1u)
                                present |= (box == 64 ? ~0ull : ((1ull << box) - 1)) << (c * box);
                        meta[s].present = present;
                        mbar_arrive(&bars->full[s]);
                    }
                    ++idx;
                }
            }
            u += sg.units;
        }
        // never leave with copies landing in shared memory
        if (!ok && lane == 0)
            for (int k = (idx > NST ? idx - NST : 0); k < idx; ++k) mbar_wait(&bars->full[k % NST], (k / NST) & 1);
    } else if (warp == 2) {
        // ============================ fix-up ===============================
        // V rows without a key may hold anything: zero them
        int j = 0;
        bool ok = true;
        for (long long u = lo; u < hi && ok;) {
            const PxSegment sg = px_segment<D>(p, ngroups, u, hi);
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
                        unsigned char* st = sm + S::OffStage + s * S::StageBytes + kWsKeys * 128 + r * 128;
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                            for (int ch = 0; ch < 8; ++ch)
                                *reinterpret_cast<uint4*>(st + cb * S::KVBlock + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                // (one arrival a warp: arrivals on one barrier are made one after the other)
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->ready[s]);
            }
        }
    } else if (warp == 1 || (NQ == 2 && warp == 3)) {
        // ========================== MMA issuers =============================
        // One warp for each Q tile: S_i = Q_i K^T a tile ahead of O_i += P_i V.  (One
        // thread for both spent 3270 cycles a tile of both, 1460 of them on products:
        // the waits and commits of one now pass while the other's products run.)  The
        // whole warp walks the tiles, its values stay uniform; lane 0 issues.
        const int i = warp >> 1;
        bool ok = true;
        int idx0 = 0, base = 0, loads = 0;             // tiles of the segments before; of this Q tile; its loads
        const uint64_t qd = ws_sdesc(sm_u + S::OffQ + i * S::QBytes, 16, 1024);
        const uint64_t kd0 = ws_sdesc(sm_u + S::OffStage, 16, 1024);
        const uint64_t vd0 = ws_sdesc(sm_u + S::OffStage + kWsKeys * 128, S::KVBlock, 1024);
        const uint32_t s0 = tmem + S::SCol0 + (uint32_t)(i * 2 * kWsKeys), o_t = tmem + (uint32_t)(i * D);
        for (long long u = lo; u < hi && ok;) {
            const PxSegment sg = px_segment<D>(p, ngroups, u, hi);
            const int own = sg.tiles(i), others = sg.nt - own;
            if (own > 0) {
                ok = ws_wait(&bars->q_ready[i], loads & 1, abort);
                ++loads;
            }
            int ns = 0, npv = 0, nother = 0;           // S issued, P V issued, the other Q tile's tiles passed
            long long t0 = clock64();
            while (ok && (npv < own || nother < others)) {
                // (each barrier's phases are asked for in order)
                if (ns < own && ns < npv + 2) {
                    const int t = idx0 + (sg.alt ? 2 * ns + i : ns), s = t % NST;
                    if (ws_test(&bars->ready[s], (t / NST) & 1)) {
                        ws_fence_after();
                        if (lane == 0) {
                            ws_issue_s<D, kWsRows * 128, S::KVBlock>(s0 + (uint32_t)(((base + ns) & 1) * kWsKeys), qd,
                                                                     kd0 + (uint64_t)((s * S::StageBytes) >> 4));
                            ws_commit(&bars->s_full[i][(base + ns) & 1]);
                        }
                        __syncwarp();
                        ++ns;
                        t0 = clock64();
                        continue;
                    }
                }
                if (npv < ns && ws_test(&bars->p_full[i], (base + npv) & 1)) {
                    ws_fence_after();
                    const int t = idx0 + (sg.alt ? 2 * npv + i : npv), s = t % NST;
                    if (lane == 0) {
                        // P_i in the S buffer it came from (bf16 pairs)
                        ws_issue_pv<D>(o_t, s0 + (uint32_t)(((base + npv) & 1) * kWsKeys),
                                       vd0 + (uint64_t)((s * S::StageBytes) >> 4), npv > 0);
                        ws_commit(&bars->o_done[i]);
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
    } else if (warp >= kShSoftmax0) {
        // ============================ softmax ==============================
        const int qi = (warp - kShSoftmax0) >> 2;          // Q tile
        const int r = tid - (kShSoftmax0 + 4 * qi) * 32;   // row = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        unsigned char* Qs = sm + S::OffQ + qi * S::QBytes;
        const int tl = r / p.G, gq = r - tl * p.G;
        bool ok = true;
        int idx0 = 0, base = 0;
        for (long long u = lo; u < hi && ok;) {
            const PxSegment sg = px_segment<D>(p, ngroups, u, hi);
            const int ml = (sg.alt ? 0 : qi * p.tq) + tl;  // the row's member of the column
            const bool row_ok = tl < p.tq && ml < sg.members;
            const int nt = sg.tiles(qi);                   // 0: the other warpgroup has the segment's one tile
            // Q row, rotated at its position when BAKED, unscaled bf16
            if (nt > 0) {
                // (D / 16 lanes share a row: a load covers whole lines)
                constexpr int LPR = D / 16, RPW = 32 / LPR;
                const int c = lane % LPR;                  // 8-column chunk, paired with c + D / 16
#pragma unroll 4
                for (int it = 0; it < 32 / RPW; ++it) {
                    const int rr = (warp & 3) * 32 + it * RPW + lane / LPR;
                    const int rtl = rr / p.G, rm = (sg.alt ? 0 : qi * p.tq) + rtl;
                    const bool rok = rtl < p.tq && rm < sg.members;
                    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
                    if (rok) {
                        const int mb = __ldcg(p.members + sg.off + sg.m0 + rm);
                        const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) +
                                                    ((long long)mb * p.Hq + sg.h * p.G + (rr - rtl * p.G)) * D;
                        a = *reinterpret_cast<const uint4*>(qrow + 8 * c);
                        b = *reinterpret_cast<const uint4*>(qrow + D / 2 + 8 * c);
                        if (p.rope != kRopeNone)
                            px_rotate8(a, b, clamp_paged_t(p.pos[mb], p.maxb, p.bs), p.theta + 8 * c);
                    }
                    // Q tile: [column block][128 rows][128 B], 128-byte swizzle
                    const int c1 = c, c2 = c + D / 16;
                    *reinterpret_cast<uint4*>(Qs + (c1 >> 3) * (kWsRows * 128) + rr * 128 + (((c1 ^ rr) & 7) << 4)) = a;
                    *reinterpret_cast<uint4*>(Qs + (c2 >> 3) * (kWsRows * 128) + rr * 128 + (((c2 ^ rr) & 7) << 4)) = b;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars->q_ready[qi]);
            }
            float m_run = -INFINITY, l_run = 0.f;          // m in base-2 units of the scaled scores
            for (int lt = 0; lt < nt; ++lt) {
                const int j = base + lt;
                if (!ws_wait(&bars->s_full[qi][j & 1], (j >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                ws_fence_after();
                float sv[kWsKeys];
                const uint32_t scol = S::SCol0 + (uint32_t)((qi * 2 + (j & 1)) * kWsKeys);
                ws_ld32(lane_base + scol, sv);
                ws_ld32(lane_base + scol + 32, sv + 32);
                ws_wait_ld();
                const int gt = idx0 + (sg.alt ? 2 * lt + qi : lt);
                if (!ws_wait(&bars->ready[gt % NST], (gt / NST) & 1, abort)) {    // the stage's meta
                    ok = false;
                    break;
                }
                const unsigned long long present = meta[gt % NST].present;
                if (present != ~0ull) {
#pragma unroll
                    for (int k = 0; k < kWsKeys; ++k) sv[k] = ((present >> k) & 1ull) ? sv[k] : -INFINITY;
                }
                const float mx = ws_max64(sv) * p.scale2;
                float mn = m_run, alpha = 1.f;
                if (mx > m_run + kShLazy) {
                    mn = mx;
                    alpha = m_run == -INFINITY ? 1.f : exp2f(m_run - mn);
                }
                // (fp32 exponentials: taken two at once in fp16 they cost the same and are
                // off by up to 2^-7)
                const float ls = ws_exp64(sv, p.scale2, mn == -INFINITY ? 0.f : -mn);
                l_run = l_run * alpha + ls;
                m_run = mn;
                // P V of the previous tile is done: O is free
                if (lt > 0 && !ws_wait(&bars->o_done[qi], (j - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                if (lt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
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
                if (lane == 0) mbar_arrive(&bars->p_full[qi]);
            }
            if (!ok) {
                give_up();
                break;
            }
            // the last P V, then the partial (m, l, o) of each row
            if (nt > 0) {
                if (!ws_wait(&bars->o_done[qi], (base + nt - 1) & 1, abort)) {
                    give_up();
                    break;
                }
                ws_fence_after();
            }
            const long long prow = sg.row0 + (long long)x * (NQ * kWsRows) + (sg.alt ? 0 : qi * p.tq * p.G) +
                                   (long long)tl * p.G + gq + (sg.alt && qi ? p.alt_rows : 0);
            if (row_ok) p.part_ml[prow] = make_float2(m_run, l_run);
            if (nt > 0) {
                // through the Q tile's shared memory (its products are done), each row in the
                // place of its own q (which this warp alone writes), CP columns at a time, so
                // that whole lines go out
                constexpr int CP = D == 64 ? 32 : 64, CPL = CP / 4;            // 16-byte chunks of a staged row
                auto stg = [&](int row, int ch) {
                    return reinterpret_cast<float4*>(Qs + (ch >> 3) * (kWsRows * 128) + row * 128 + (((ch ^ row) & 7) << 4));
                };
                const long long row_a = prow - ((long long)tl * p.G + gq);     // the column's row 0 of this Q tile
#pragma unroll 1
                for (int c6 = 0; c6 < D / CP; ++c6) {
#pragma unroll
                    for (int hf = 0; hf < CP / 32; ++hf) {
                        float ov[32];
                        ws_ld32(lane_base + (uint32_t)(qi * D + CP * c6 + 32 * hf), ov);
                        ws_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *stg(r, 8 * hf + k) = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int it = 0; it < CPL; ++it) {
                        const int rr = (warp & 3) * 32 + (32 / CPL) * it + lane / CPL, ch = lane % CPL;
                        const int rtl = rr / p.G;
                        if (rtl < p.tq && (sg.alt ? 0 : qi * p.tq) + rtl < sg.members)
                            *reinterpret_cast<float4*>(p.part_o + (row_a + rr) * D + CP * c6 + 4 * ch) =
                                *stg(rr, ch);
                    }
                    __syncwarp();
                }
                // O is read: the next segment's first product may overwrite it
                // (it waits for this warpgroup's next P)
                ws_fence_before();
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
constexpr int kShCombineWarps = 8;

// One warp per (sequence, q head): lane l holds D / 32 columns.  The parts
// are the decode kernel's slots of the sequence, then the shares of its prefix
// column (two each when its warpgroups took alternate tiles).
template <int D>
__global__ void __launch_bounds__(kShCombineWarps * 32)
    shared_combine_kernel(const __grid_constant__ SharedParams p, const __grid_constant__ SharedDecode dp) {
    constexpr int NC = D / 32;
    sh_pdl_launch();
    sh_pdl_wait();
    const int lane = threadIdx.x & 31;
    const int w = blockIdx.x * kShCombineWarps + (threadIdx.x >> 5);
    // ready the decode kernel's counters and the reader counts for the next call
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < dp.num_blocks;
         i += (long long)gridDim.x * blockDim.x)
        dp.refs[i] = 0u;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < dp.ncounters; i += blockDim.x) dp.counters[i] = 0u;
    if (w >= p.B * p.Hq) return;
    const int b = w / p.Hq, qh = w - b * p.Hq;
    // the decode slots of sequence b, as its kernel cut them
    long long tot = 0, before = 0, rb = 0;
    for (int base = 0; base < p.B; base += 32) {
        const long long st = base + lane < p.B ? (long long)__ldcg(dp.seq_rows + base + lane) : 0;
        tot += st;
        if (base + lane < b) before += st;
        if (base + lane == b) rb += st;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        tot += __shfl_xor_sync(0xffffffffu, tot, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
        rb += __shfl_xor_sync(0xffffffffu, rb, off);
    }
    const int2 fl = paged_seq_shares(before, rb, tot, paged_share_count(tot, dp.nsplit));
    const int first = fl.x + b;
    int nd = fl.y - fl.x + 1;
    if (first < 0 || nd < 1 || first + nd > dp.max_items) {
        if (lane == 0) index_fault(p.err, 21, first);
        return;
    }
    // the shares of its prefix column
    const int2 sg = __ldcg(p.seq_group + b);
    int np = 0, fx = 0, alt = 0;
    long long prow = 0;
    if (sg.x >= 0) {
        const SharedGroup* g = p.groups + sg.x;
        const int kt = __ldcg(&g->kt), n = __ldcg(&g->n), h = qh / p.G;
        const int m = sg.y / p.mq;
        const long long units = __ldcg(&p.head->units);
        const int shares = __ldcg(&p.head->shares);
        const bool one = min(p.mq, n - m * p.mq) <= p.tq;
        const long long u0 = __ldcg(&g->units0) + h * __ldcg(&g->hu) + (long long)m * kt * p.full_units;
        fx = streamk_share_of(u0, units, shares);
        np = streamk_share_of(u0 + (long long)kt * (one ? 1 : p.full_units) - 1, units, shares) - fx + 1;
        alt = shared_q_tiles(D) == 2 && one;
        prow = __ldcg(&g->rows0) + ((long long)h * n + sg.y) * p.G + qh % p.G;
        if (alt) np *= 2;
    }
    const int parts = nd + np;
    constexpr int RT = shared_q_tiles(D) * kWsRows;
    auto slot = [&](int k, const float2** ml) -> const float* {
        if (k < nd) {
            const long long s = (long long)(first + k) * p.Hq + qh;
            *ml = dp.part_ml + s;
            return dp.part_o + s * D;
        }
        const int j = k - nd, sx = fx + (alt ? j >> 1 : j);
        const long long s = prow + (long long)sx * RT + ((alt && (j & 1)) ? p.alt_rows : 0);
        *ml = p.part_ml + s;
        return p.part_o + s * D;
    };
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32) {
        const float2* ml;
        slot(k, &ml);
        M = fmaxf(M, __ldcg(ml).x);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f, acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = 0.f;
    for (int base = 0; base < parts; base += 32) {
        float e = 0.f;
        if (base + lane < parts) {
            const float2* ml;
            slot(base + lane, &ml);
            const float2 v = __ldcg(ml);
            if (v.x != -INFINITY || v.y != v.y) {      // (NaN scores leave no maximum, but a sum of NaN)
                e = exp2f(v.x - M);
                L += v.y * e;
            }
        }
        const int cnt = min(32, parts - base);
        // eight parts' loads in flight; an empty part's o may hold anything: not read
        constexpr int U = NC == 8 ? 4 : 8;
        for (int k0 = 0; k0 < cnt; k0 += U) {
            float v[U][NC], ek[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ek[u] = __shfl_sync(0xffffffffu, e, (k0 + u) & 31);
                if (k0 + u >= cnt) ek[u] = 0.f;
                const float2* ml;
                const float* o = slot(base + k0 + u, &ml) + lane * NC;
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    float2 w2 = make_float2(0.f, 0.f);
                    if (ek[u] != 0.f) w2 = __ldcg(reinterpret_cast<const float2*>(o + c));
                    v[u][c] = w2.x;
                    v[u][c + 1] = w2.y;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c] = fmaf(v[u][c], ek[u], acc[c]);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(dp.out) + ((long long)b * p.Hq + qh) * D + lane * NC;
#pragma unroll
    for (int c = 0; c < NC; c += 2)
        *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
}

cudaLaunchConfig_t sh_config(dim3 grid, int threads, int smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
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

template <int D>
cudaError_t launch_prefix_t(const SharedParams& p, const CUtensorMap& map, cudaStream_t stream) {
    constexpr int kSmem = px_smem_bytes<D>();
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(shared_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = sh_config(dim3(p.ctas), PxShape<D>::Threads, kSmem, stream, &attr);
    return cudaLaunchKernelEx(&cfg, shared_prefix_kernel<D>, p, map);
}

template <int D>
cudaError_t launch_combine_t(const SharedParams& p, const SharedDecode& dp, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const long long warps = (long long)p.B * p.Hq;
    const cudaLaunchConfig_t cfg = sh_config(dim3((unsigned)((warps + kShCombineWarps - 1) / kShCombineWarps)),
                                             kShCombineWarps * 32, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, shared_combine_kernel<D>, p, dp);
}

}  // namespace

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = sh_config(dim3(p.B), kShPlanThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, shared_plan_kernel, p);
}

cudaError_t launch_shared_prefix(int D, const SharedParams& p, const CUtensorMap& map, cudaStream_t stream) {
    return D == 64 ? launch_prefix_t<64>(p, map, stream)
                   : (D == 128 ? launch_prefix_t<128>(p, map, stream) : launch_prefix_t<256>(p, map, stream));
}

cudaError_t launch_shared_combine(int D, const SharedParams& p, const SharedDecode& dp, cudaStream_t stream) {
    return D == 64 ? launch_combine_t<64>(p, dp, stream)
                   : (D == 128 ? launch_combine_t<128>(p, dp, stream) : launch_combine_t<256>(p, dp, stream));
}

}  // namespace kvc
