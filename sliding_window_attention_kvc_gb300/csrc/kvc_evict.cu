// Caches kept in part: how much attention weight each block received, and the
// lightest blocks given back.
#include <cooperative_groups.h>

#include "kvc_decode.cuh"
#include "kvc_select.h"

namespace kvc {

namespace {

__device__ __forceinline__ void ev_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void ev_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// weights of blocks
// ---------------------------------------------------------------------------
constexpr int kWeighThreads = 256;
constexpr int kWeighRows = 256;                     // positions of a CTA, where a block has no more
constexpr int kWeighParts = kWeighThreads / (kWeighRows / 4);   // head groups that share a position

// One CTA per (`per` blocks, sequence).  A thread adds up the weights
// 2^(s - M) / L of four positions (one 16-byte load a head) over a quarter of the q
// heads, in head order; the quarters, then the rows of each block, are added in
// order: the same sums whatever the decode's shares were.  What bounds it: 4 bytes a
// row and head, which the decode has just left in L2, and an exponential for each
// (64 sequences, 32 heads, 277,000 rows: 13 us launched alone on cold caches; its way to
// position and table passes while the combine runs).
__global__ void __launch_bounds__(kWeighThreads, 6) weigh_kernel(const __grid_constant__ WeighParams p) {
    __shared__ float4 s_part[kWeighThreads];
    __shared__ float s_row[kWeighRows];
    __shared__ float s_warp[kWeighThreads / 32];
    constexpr int U = 4;                            // heads in flight
    const int tid = threadIdx.x, b = blockIdx.y;
    const int lb0 = blockIdx.x * p.per;
    const int32_t* trow = p.table + (long long)b * p.maxb;
    // (positions, table and valid bits were final before the decode could start the kernels
    // behind it: they are read while it runs)
    ev_pdl_launch();
    const int t = clamp_paged_t(__ldcg(p.pos + b), p.maxb, p.bs);
    const float* sc = p.scores + (long long)b * p.Hq * p.stride;
    const float2* ml = p.ml + (long long)b * p.Hq;
    float* wrow = p.weights + (long long)b * p.maxb;
    auto attended = [&](int lb) {
        const int phys = __ldcg(trow + lb);
        return phys >= 0 && phys < p.num_blocks && (!p.valid || ((__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u));
    };
    auto store = [&](int lb, float sum) { wrow[lb] = p.decay == 0.f ? sum : fmaf(p.decay, wrow[lb], sum); };
    // weights of positions pos .. pos + 3 (pos a multiple of 4, within the row) over heads h0 .. h1 - 1; what lies
    // behind the position, or in a block that is not attended, is whatever was there
    auto weights4 = [&](long long pos, int h0, int h1) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int h = h0; h < h1; h += U) {
            float4 s[U];
            float2 m[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = min(h + u, h1 - 1);
                s[u] = __ldcg(reinterpret_cast<const float4*>(sc + x * p.stride + pos));
                m[u] = __ldcg(ml + x);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u < h1) {
                    a.x = fmaf(exp2f(s[u].x - m[u].x), m[u].y, a.x);
                    a.y = fmaf(exp2f(s[u].y - m[u].x), m[u].y, a.y);
                    a.z = fmaf(exp2f(s[u].z - m[u].x), m[u].y, a.z);
                    a.w = fmaf(exp2f(s[u].w - m[u].x), m[u].y, a.w);
                }
        }
        return a;
    };
    // positions p0 .. p0 + kWeighRows - 1 (p0 a multiple of 4) into s_row
    constexpr int QUADS = kWeighRows / 4;
    const int quad = tid % QUADS, part = tid / QUADS;
    const int h0 = (int)((long long)p.Hq * part / kWeighParts), h1 = (int)((long long)p.Hq * (part + 1) / kWeighParts);
    auto rows = [&](long long p0) {
        const long long pos = p0 + 4 * quad;
        s_part[tid] = pos <= t ? weights4(pos, h0, h1) : make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
        if (tid < QUADS) {
            float4 a = s_part[tid];
            for (int k = 1; k < kWeighParts; ++k) {
                const float4 c = s_part[k * QUADS + tid];
                a.x += c.x;
                a.y += c.y;
                a.z += c.z;
                a.w += c.w;
            }
            *reinterpret_cast<float4*>(s_row + 4 * tid) = a;
        }
        __syncthreads();
    };
    const long long pos0 = (long long)lb0 * p.bs, lead = pos0 & 3;    // rows read in front of the first
    if (p.per == 1) {                               // one block, its rows in turn
        float a = 0.f;
        const bool on = pos0 <= t && attended(lb0); // (uniform)
        ev_pdl_wait();
        if (on) {
            const long long end = min(pos0 + p.bs - 1, (long long)t);
            for (long long r0 = pos0 - lead; r0 <= end; r0 += kWeighRows) {
                rows(r0);
                const long long r = r0 + tid;
                if (r >= pos0 && r <= end) a += s_row[tid];
                __syncthreads();
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
        if ((tid & 31) == 0) s_warp[tid >> 5] = a;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWeighThreads / 32; ++w) a += s_warp[w];
            store(lb0, a);
        }
        return;
    }
    const bool mine = tid < p.per && lb0 + tid < p.maxb;
    const bool on = mine && pos0 + (long long)tid * p.bs <= t && attended(lb0 + tid);
    ev_pdl_wait();
    if (pos0 <= t) rows(pos0 - lead);               // (uniform)
    if (mine) {
        float sum = 0.f;
        if (on) {
            const int end = (int)min((long long)p.bs - 1, t - (pos0 + (long long)tid * p.bs));
            for (int r = 0; r <= end; ++r) sum += s_row[(int)lead + tid * p.bs + r];
        }
        store(lb0 + tid, sum);
    }
}

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------
constexpr int kEvictThreads = 1024;             // at most; at least 256
constexpr int kEvictWarps = kEvictThreads / 32;

// Order of weights as unsigned integers: -0 counts as 0, NaN as the heaviest.
__device__ __forceinline__ uint32_t weight_key(float x) {
    if (!(x == x)) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the CTA of one count, and over the threads before this one.
__device__ __forceinline__ int evict_scan(int v, int* s_w, int* tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += a;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (int)(blockDim.x >> 5) ? s_w[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += a;
        }
        s_w[lane] = w;
    }
    __syncthreads();
    const int ex = x - v + (warp > 0 ? s_w[warp - 1] : 0);
    *tot = s_w[(blockDim.x >> 5) - 1];
    __syncthreads();
    return ex;
}

// A cluster of CTAs per sequence, a contiguous part of its blocks each: the excess
// over `keep` of its mapped blocks, lightest first, ties by the lowest index, from a
// radix search of the excess-th lightest (four digits at most: it ends where a digit
// takes all of its keys; every CTA counts its own keys, kept in shared memory, and
// adds up the cluster's counts).  Blocks whose count reaches zero are marked; the
// last cluster to finish (an atomic ticket, no waiting) puts the marked ones on the
// free list in ascending order and clears their resident bits.
// What bounds it: a dozen dependent trips to L2, barriers and a cold instruction
// cache, for long tables the atomics too: 12.5 us for 64 sequences of up to 512 blocks,
// 32 for two of up to 62,500 (309 with a single CTA a sequence; 83 with the free list
// written a word of 32 marks a thread, 32 lines a store; 42 with one counter a digit, its
// additions in turn, and 1024 threads whatever the table; 37 with the free list staged in
// shared memory, 256 words at a time).
constexpr int kEvictKeys = 8192;                // keys a CTA keeps
constexpr uint32_t kKeyStays = 0xffffffffu;     // not among the blocks that may go

// CTAs of a sequence at most (16 brought two of up to 62,500 blocks from 34 to 32 us, and a call that gives
// nothing back from 10 to 13).
constexpr int kEvictCluster = 8;

// CLM: the most CTAs of a cluster (1: no cluster, nothing is gathered).
template <int CLM>
__global__ void __launch_bounds__(kEvictThreads) block_evict_kernel(const __grid_constant__ EvictParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = CLM > 1 ? (int)cluster.num_blocks() : 1, rank = CLM > 1 ? (int)cluster.block_rank() : 0;
    __shared__ int s_hist[4][256];              // this CTA's counts of each pass
    __shared__ __align__(16) int s_part[256 * 8];   // a pass's counts, a column for every eighth lane
    __shared__ int s_w[kEvictWarps];
    __shared__ int s_count[2];                  // mapped, and those that may go
    __shared__ int s_digit, s_beyond, s_in, s_cut, s_last;
    __shared__ uint32_t s_key[kEvictKeys];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x / CL;
    auto sync_all = [&]() {
        if (CLM > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    for (int i = tid; i < 256 * 8; i += nt) s_part[i] = 0;
    if (tid < 2) s_count[tid] = 0;
    __syncthreads();
    ev_pdl_wait();
    ev_pdl_launch();
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    int32_t* trow = p.table + (long long)b * p.maxb;
    float* wrow = p.weights + (long long)b * p.maxb;
    const int hi = nb - p.recent;               // blocks first .. hi - 1 may go
    const int lo_i = (int)((long long)nb * rank / CL), hi_i = (int)((long long)nb * (rank + 1) / CL);
    const bool kept = hi_i - lo_i <= kEvictKeys;
    int live = 0, loose = 0;
#pragma unroll 1
    for (int base = lo_i; base < hi_i; base += 4 * nt) {
        int e[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = base + u * nt + tid;
            e[u] = i < hi_i ? trow[i] : -1;
            w[u] = i < hi_i ? wrow[i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = base + u * nt + tid;
            const bool may = e[u] >= 0 && i >= p.first && i < hi;
            live += e[u] >= 0;
            loose += may;
            if (kept && i < hi_i) s_key[i - lo_i] = may ? weight_key(w[u]) : kKeyStays;
        }
    }
    live = __reduce_add_sync(0xffffffffu, live);
    loose = __reduce_add_sync(0xffffffffu, loose);
    if (lane == 0) {
        atomicAdd(&s_count[0], live);
        atomicAdd(&s_count[1], loose);
    }
    sync_all();
    // a value of each CTA of the cluster (all on their way together)
    auto of_all = [&](int* mine, int (&v)[CLM]) {
#pragma unroll
        for (int c = 0; c < CLM; ++c) v[c] = CLM == 1 ? *mine : (c < CL ? *cluster.map_shared_rank(mine, c) : 0);
    };
    int nlive = 0, nloose = 0;
    {
        int v[CLM], w[CLM];
        of_all(&s_count[0], v);
        of_all(&s_count[1], w);
#pragma unroll
        for (int c = 0; c < CLM; ++c) {
            nlive += v[c];
            nloose += w[c];
        }
    }
    // this thread's key of index i (a long table's keys are worked out again)
    auto key_of = [&](int i) -> uint32_t {
        if (i >= hi_i) return kKeyStays;
        if (kept) return s_key[i - lo_i];
        return i >= p.first && i < hi && trow[i] >= 0 ? weight_key(wrow[i]) : kKeyStays;
    };
    int want = min(nlive - p.keep, nloose);
    if (want > 0) {                             // (the same in every CTA of the cluster)
        uint32_t prefix = 0, mask = 0;
        int digit = 0, pass = 0;
#pragma unroll 1
        for (;; ++pass) {
            const int shift = 24 - 8 * pass;
#pragma unroll 1
            for (int base = lo_i; base < hi_i; base += nt) {
                const uint32_t key = key_of(base + tid);
                const bool in = key != kKeyStays && (key & mask) == prefix;
                // (most weights share a few digits: eight lanes that add to one of them meet four at a time)
                if (in) atomicAdd(&s_part[((key >> shift) & 255u) * 8 + (lane & 7)], 1);
            }
            __syncthreads();
            if (tid < 256) {
                int4* c = reinterpret_cast<int4*>(s_part + tid * 8);
                const int4 x = c[0], y = c[1];
                s_hist[pass][tid] = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
                c[0] = c[1] = make_int4(0, 0, 0, 0);
            }
            sync_all();
            // a thread a digit: its keys in the cluster, and those of smaller digits
            int mine = 0, incl = 0;
            if (tid < 256) {
                int v[CLM];
                of_all(&s_hist[pass][tid], v);
#pragma unroll
                for (int c = 0; c < CLM; ++c) mine += v[c];
                incl = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int a = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += a;
                }
                if (lane == 31) s_w[warp] = incl;
            }
            __syncthreads();
            if (tid < 256) {
                for (int w = 0; w < warp; ++w) incl += s_w[w];
                if (incl >= want && incl - mine < want) {
                    s_digit = tid;
                    s_beyond = incl - mine;
                    s_in = mine;
                }
            }
            __syncthreads();
            digit = s_digit;
            want -= s_beyond;
            prefix |= (uint32_t)digit << shift;
            mask |= 255u << shift;
            if (pass == 3 || s_in == want) break;       // all that begin with these digits go, or all four are known
            __syncthreads();
        }
        // keys whose digits lie below `prefix` go, and the first `want` of those that begin with it: so many of
        // them lie in the CTAs before
        int before = 0;
        {
            int v[CLM];
            of_all(&s_hist[pass][digit], v);
#pragma unroll
            for (int c = 0; c < CLM; ++c) before += c < rank ? v[c] : 0;
        }
        const int own = s_hist[pass][digit];
        const int take = before >= want ? 0 : min(own, want - before);      // of this CTA's
        int cut = take > 0 ? hi_i : lo_i;       // those in front of it
        if (take > 0 && take < own) {           // (uniform) a contiguous run of keys a thread: one scan
            const int run = (hi_i - lo_i + nt - 1) / nt, a0 = lo_i + tid * run, a1 = min(a0 + run, hi_i);
            auto same = [&](int i) {
                const uint32_t key = key_of(i);
                return key != kKeyStays && (key & mask) == prefix;
            };
            int n = 0, tot;
            for (int i = a0; i < a1; ++i) n += same(i);
            int k = evict_scan(n, s_w, &tot);
            if (k < take && k + n >= take) {
                int i = a0;
                for (;; ++i)
                    if (same(i) && ++k == take) break;
                s_cut = i + 1;
            }
            __syncthreads();
            cut = s_cut;
        }
#pragma unroll 1
        for (int base = lo_i; base < hi_i; base += 4 * nt) {
            int phys[4], old[4];
            unsigned goes = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = base + u * nt + tid;
                const uint32_t key = key_of(i), top = key & mask;
                const bool g = key != kKeyStays && (top < prefix || (top == prefix && i < cut));
                goes |= (unsigned)g << u;
                phys[u] = g ? trow[i] : 0;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if ((goes >> u) & 1u) {
                    const int i = base + u * nt + tid;
                    trow[i] = -1;
                    wrow[i] = 0.f;
                    old[u] = 0;
                    if (phys[u] >= p.num_blocks)
                        set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                    else
                        old[u] = atomicSub(&p.refcount[phys[u]], 1);
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (((goes >> u) & 1u) && old[u] == 1) atomicOr(&p.back[phys[u] >> 5], 1u << (phys[u] & 31));
        }
    }
    __threadfence();
    sync_all();                                 // the cluster's marks are made, its counts read
    if (rank == 0 && tid == 0) s_last = atomicAdd(p.ticket, 1u) == (unsigned)(gridDim.x / CL) - 1u;
    sync_all();
    if (!(CLM > 1 ? *cluster.map_shared_rank(&s_last, 0) : s_last)) {
        sync_all();                             // (no CTA leaves while it is read)
        return;
    }
    // the last cluster: its CTAs share the words of marks
    __threadfence();
    const int words = (p.num_blocks + 31) / 32;
    const int w0 = (int)((long long)words * rank / CL), w1 = (int)((long long)words * (rank + 1) / CL);
    const int free0 = *p.free_count;
    const bool short_ = w1 - w0 <= 256 * 8;     // the words stay in shared memory
    int mine = 0;
#pragma unroll 1
    for (int i = w0 + tid; i < w1; i += nt) {
        const uint32_t w = __ldcg(p.back + i);
        if (short_) s_part[i - w0] = (int)w;
        mine += __popc(w);
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (tid == 0) s_count[0] = 0;
    __syncthreads();
    if (lane == 0 && mine) atomicAdd(&s_count[0], mine);
    sync_all();
    int at = free0, all = free0;                // list entries before this CTA's, and in the end
    {
        int v[CLM];
        of_all(&s_count[0], v);
#pragma unroll
        for (int c = 0; c < CLM; ++c) {
            at += c < rank ? v[c] : 0;
            all += v[c];
        }
    }
    // 2048 words at a time: a scan places them, then a warp a word writes its marked blocks side by side
    static_assert(kEvictKeys >= 256 * 8, "a place for each word");
#pragma unroll 1
    for (int base = w0; base < w1; base += 256 * 8) {
        const int n = min(w1 - base, 256 * 8);
        if (!short_) {
            for (int k = tid; k < n; k += nt) s_part[k] = (int)__ldcg(p.back + base + k);
            __syncthreads();
        }
        const int run = (n + nt - 1) / nt, a0 = min(tid * run, n), a1 = min(a0 + run, n);
        int c = 0, tot;
        for (int k = a0; k < a1; ++k) c += __popc(s_part[k]);
        int k0 = at + evict_scan(c, s_w, &tot);
        for (int k = a0; k < a1; ++k) {
            s_key[k] = (uint32_t)k0;
            k0 += __popc(s_part[k]);
        }
        for (int k = tid; k < n; k += nt) {
            const uint32_t w = (uint32_t)s_part[k];
            if (w) {
                p.back[base + k] = 0u;
                if (p.valid) atomicAnd(&p.valid[base + k], ~w);
            }
        }
        __syncthreads();
        const uint32_t below = (1u << lane) - 1u;
        for (int k = 32 * warp; k < n; k += nt) {
            const uint32_t word = k + lane < n ? (uint32_t)s_part[k + lane] : 0u, place = k + lane < n ? s_key[k + lane] : 0u;
            if (!__any_sync(0xffffffffu, word != 0u)) continue;
            const int id = 32 * (base + k) + lane;
#pragma unroll 8
            for (int x = 0; x < 32; ++x) {
                const uint32_t w = __shfl_sync(0xffffffffu, word, x);
                const uint32_t j = __shfl_sync(0xffffffffu, place, x) + __popc(w & below);
                if (((w >> lane) & 1u) && j < (uint32_t)p.num_blocks) p.free_list[j] = id + 32 * x;
            }
        }
        if (tid == 0 && (at < 0 || at + tot > p.num_blocks)) index_fault(p.err, 41, at + tot);
        at += tot;
        __syncthreads();
    }
    sync_all();                                 // (the counts have been read)
    if (rank == 0 && tid == 0) {
        *p.free_count = min(all, p.num_blocks);
        *p.ticket = 0u;                         // ready for the next call
    }
}

cudaLaunchConfig_t ev_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& p, cudaStream_t s) {
    WeighParams q = p;
    // blocks of a CTA: their rows, and up to 3 in front of them, at most kWeighRows
    q.per = p.bs > kWeighRows / 2 ? 1 : (p.bs % 4 ? kWeighRows - 3 : kWeighRows) / p.bs;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = ev_config(dim3((p.maxb + q.per - 1) / q.per, p.B), kWeighThreads, s, &attr);
    return cudaLaunchKernelEx(&cfg, weigh_kernel, q);
}

cudaError_t launch_block_evict(const EvictParams& p, cudaStream_t s) {
    // up to four keys a thread, as far as a cluster goes; no more threads than keys: their barriers are
    // what a short table waits for
    int cl = 1, threads = 256;
    while (threads < kEvictThreads && threads < p.maxb) threads *= 2;
    while (cl < kEvictCluster && (long long)cl * 4 * threads < p.maxb) cl *= 2;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = ev_config(dim3((unsigned)(p.B * cl)), threads, s, attr);
    if (cl == 1) return cudaLaunchKernelEx(&cfg, block_evict_kernel<1>, p);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, block_evict_kernel<kEvictCluster>, p);
}

}  // namespace kvc
