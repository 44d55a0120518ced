// Caches kept in part: how much attention weight each block received, and the
// lightest blocks given back.
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

// One CTA per (`per` blocks, sequence), a thread a position: the weights
// 2^(s - M) / L of its row over all q heads, added up in head order, then the
// rows of each block in row order: the same sums whatever the decode's shares were.
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(const __grid_constant__ WeighParams p) {
    __shared__ float s_row[kWeighThreads];
    __shared__ float s_warp[kWeighThreads / 32];
    constexpr int U = 8;                            // heads in flight
    const int tid = threadIdx.x, b = blockIdx.y;
    const int lb0 = blockIdx.x * p.per;
    ev_pdl_wait();
    ev_pdl_launch();
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int32_t* trow = p.table + (long long)b * p.maxb;
    const float* sc = p.scores + (long long)b * p.Hq * p.stride;
    const float2* ml = p.ml + (long long)b * p.Hq;
    float* wrow = p.weights + (long long)b * p.maxb;
    auto attended = [&](int lb) {
        const int phys = __ldg(trow + lb);
        return phys >= 0 && phys < p.num_blocks && (!p.valid || ((__ldg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u));
    };
    auto row_weight = [&](long long pos) {
        float a = 0.f;
        for (int h0 = 0; h0 < p.Hq; h0 += U) {
            float s[U];
            float2 m[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = min(h0 + u, p.Hq - 1);
                s[u] = __ldcg(sc + h * p.stride + pos);
                m[u] = __ldcg(ml + h);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h0 + u < p.Hq) a = fmaf(exp2f(s[u] - m[u].x), m[u].y, a);
        }
        return a;
    };
    auto store = [&](int lb, float sum) { wrow[lb] = p.decay == 0.f ? sum : fmaf(p.decay, wrow[lb], sum); };
    if (p.bs > kWeighThreads) {                     // one block, its rows in turn
        float a = 0.f;
        if ((long long)lb0 * p.bs <= t && attended(lb0))
            for (long long r = tid; r < p.bs; r += kWeighThreads)
                if (lb0 * (long long)p.bs + r <= t) a += row_weight(lb0 * (long long)p.bs + r);
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
    const int i = tid / p.bs, lb = lb0 + i;         // block of this thread's position
    const long long pos = (long long)lb0 * p.bs + tid;
    float a = 0.f;
    if (i < p.per && lb < p.maxb && pos <= t && attended(lb)) a = row_weight(pos);
    s_row[tid] = a;
    __syncthreads();
    if (tid < p.per && lb0 + tid < p.maxb) {
        float sum = 0.f;
        for (int r = 0; r < p.bs; ++r) sum += s_row[tid * p.bs + r];
        store(lb0 + tid, sum);
    }
}

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;

// Order of weights as unsigned integers: -0 counts as 0, NaN as the heaviest.
__device__ __forceinline__ uint32_t weight_key(float x) {
    if (!(x == x)) return 0xffffffffu;
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
        int w = s_w[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += a;
        }
        s_w[lane] = w;
    }
    __syncthreads();
    const int ex = x - v + (warp > 0 ? s_w[warp - 1] : 0);
    *tot = s_w[kEvictWarps - 1];
    __syncthreads();
    return ex;
}

// One CTA per sequence: the excess over `keep` of its mapped blocks, lightest
// first, ties by the lowest index, from a radix search of the excess-th lightest
// (four digits).  Blocks whose count reaches zero are marked; the last CTA to
// finish (an atomic ticket, no waiting) puts the marked ones on the free list in
// ascending order and clears their resident bits.
__global__ void __launch_bounds__(kEvictThreads) block_evict_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int s_hist[256];
    __shared__ int s_w[kEvictWarps];
    __shared__ int s_digit, s_beyond, s_last;
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
    ev_pdl_wait();
    ev_pdl_launch();
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    int32_t* trow = p.table + (long long)b * p.maxb;
    float* wrow = p.weights + (long long)b * p.maxb;
    const int hi = nb - p.recent;                   // blocks first .. hi - 1 may go
    int live = 0, loose = 0;
    for (int i = tid; i < nb; i += kEvictThreads) {
        const int on = trow[i] >= 0;
        live += on;
        loose += on && i >= p.first && i < hi;
    }
    int nlive, nloose;
    evict_scan(live, s_w, &nlive);
    evict_scan(loose, s_w, &nloose);
    int want = min(nlive - p.keep, nloose);
    if (want > 0) {
        uint32_t prefix = 0, mask = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kEvictThreads) s_hist[i] = 0;
            __syncthreads();
            for (int base = p.first; base < hi; base += kEvictThreads) {
                const int i = base + tid;
                const bool in0 = i < hi && trow[i] >= 0;
                const uint32_t key = in0 ? weight_key(wrow[i]) : 0u;
                const bool in = in0 && (key & mask) == prefix;
                const uint32_t digit = (key >> shift) & 255u;
                const unsigned act = __ballot_sync(0xffffffffu, in);
                if (in) {
                    const unsigned same = __match_any_sync(act, digit);
                    if (lane == __ffs(same) - 1) atomicAdd(&s_hist[digit], __popc(same));
                }
            }
            __syncthreads();
            if (tid < 32) {
                int c[8], sum = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    c[k] = s_hist[lane * 8 + k];
                    sum += c[k];
                }
                int incl = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int a = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += a;
                }
                int run = incl - sum;
                if (run < want && incl >= want) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (run < want && run + c[k] >= want) {
                            s_digit = lane * 8 + k;
                            s_beyond = run;
                        }
                        run += c[k];
                    }
                }
            }
            __syncthreads();
            want -= s_beyond;
            prefix |= (uint32_t)s_digit << shift;
            mask |= 255u << shift;
            __syncthreads();
        }
        int run = 0;                                // equal keys before this pass
        for (int base = p.first; base < hi; base += kEvictThreads) {
            const int i = base + tid;
            const int phys = i < hi ? trow[i] : -1;
            const uint32_t key = phys >= 0 ? weight_key(wrow[i]) : 0xffffffffu;
            const int same = phys >= 0 && key == prefix;
            int tot;
            const int ex = evict_scan(same, s_w, &tot);
            if (phys >= 0 && (key < prefix || (same && run + ex < want))) {
                trow[i] = -1;
                wrow[i] = 0.f;
                if (phys >= p.num_blocks)
                    set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                else if (atomicSub(&p.refcount[phys], 1) == 1)
                    atomicOr(&p.back[phys >> 5], 1u << (phys & 31));
            }
            run += tot;
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const int words = (p.num_blocks + 31) / 32;
    int at = *p.free_count;
    for (int base = 0; base < words; base += kEvictThreads) {
        const int i = base + tid;
        uint32_t w = i < words ? __ldcg(p.back + i) : 0u;
        int tot;
        int k = at + evict_scan(__popc(w), s_w, &tot);
        if (w) {
            p.back[i] = 0u;
            if (p.valid) p.valid[i] &= ~w;
        }
        while (w) {
            const int f = i * 32 + __ffs(w) - 1;
            w &= w - 1u;
            if (k >= 0 && k < p.num_blocks)
                p.free_list[k] = f;
            else
                index_fault(p.err, 41, k);
            ++k;
        }
        at += tot;
    }
    if (tid == 0) {
        *p.free_count = min(at, p.num_blocks);
        *p.ticket = 0u;                             // ready for the next call
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
    q.per = p.bs > kWeighThreads ? 1 : kWeighThreads / p.bs;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = ev_config(dim3((p.maxb + q.per - 1) / q.per, p.B), kWeighThreads, s, &attr);
    return cudaLaunchKernelEx(&cfg, weigh_kernel, q);
}

cudaError_t launch_block_evict(const EvictParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = ev_config(dim3(p.B), kEvictThreads, s, &attr);
    return cudaLaunchKernelEx(&cfg, block_evict_kernel, p);
}

}  // namespace kvc
