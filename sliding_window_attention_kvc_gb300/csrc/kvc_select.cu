// Caches read in part: bounds of each block's keys, blocks chosen by what the
// bounds allow a query's scores to be, and the lists that a decode over the
// chosen blocks walks.
//
// For a block and kv head, hi_d and lo_d are the largest and smallest key
// value of channel d.  For any key of the block
//     q . k = sum q_d k_d <= sum max(q_d hi_d, q_d lo_d) = U,
// so a block whose U is small holds no key that the query attends much.  hi and
// lo are kept as 8-bit codes of one step s = max(|hi|, |lo|) / 127, hi rounded
// up and lo down, so that the codes' bound is a bound still; q enters as codes
// too (step max|q| / 127).  U is then s s_q u, u an integer below 127 127 256 <
// 2^24: its products run four to an instruction (dp4a), and no order of the
// sums, here or in any other program, gives another score.
#include "kvc_decode.cuh"
#include "kvc_select.h"

namespace kvc {

namespace {

__device__ __forceinline__ void sl_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void sl_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

cudaLaunchConfig_t sl_config(dim3 grid, int threads, int smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
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

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------
constexpr int kBoundsThreads = 128;
constexpr int kBoundsWarps = 152 * 48;         // warps that keep the GPU full

// 16 bytes of a key row as floats.
template <typename Elt>
__device__ __forceinline__ void key_values(const uint4& w, float scale, float* f) {
    if constexpr (sizeof(Elt) == 1) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = (float)(int8_t)(x[i >> 2] >> (8 * (i & 3))) * scale;
    } else {
        EltTraits<Elt>::unpack(w, f);
    }
}

// The larger and the smaller of 16 bytes of values, kept as they come (bf16 pairs) or as floats.
template <typename Elt>
struct Ends {
    static constexpr int VPL = 16 / (int)sizeof(Elt);
    static constexpr bool kPacked = sizeof(Elt) == 2;
    static constexpr int N = kPacked ? VPL / 2 : VPL;
    float f[kPacked ? 1 : N];
    uint32_t w[kPacked ? N : 1];
    __device__ __forceinline__ void init(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if constexpr (kPacked)
                w[i] = pack_bf16x2(x, x);
            else
                f[i] = x;
    }
    template <bool MAX>
    static __device__ __forceinline__ uint32_t pair(uint32_t a, uint32_t b) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a), y = *reinterpret_cast<const __nv_bfloat162*>(&b);
        const __nv_bfloat162 z = MAX ? __hmax2(x, y) : __hmin2(x, y);
        return *reinterpret_cast<const uint32_t*>(&z);
    }
    template <bool MAX>
    __device__ __forceinline__ void join(const uint4& v, float scale) {
        if constexpr (kPacked) {
            w[0] = pair<MAX>(w[0], v.x);
            w[1] = pair<MAX>(w[1], v.y);
            w[2] = pair<MAX>(w[2], v.z);
            w[3] = pair<MAX>(w[3], v.w);
        } else {
            float x[VPL];
            key_values<Elt>(v, scale, x);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = MAX ? fmaxf(f[i], x[i]) : fminf(f[i], x[i]);
        }
    }
    // joined with what lane ^ off has
    template <bool MAX>
    __device__ __forceinline__ void exchange(int off) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if constexpr (kPacked) {
                w[i] = pair<MAX>(w[i], __shfl_xor_sync(0xffffffffu, w[i], off));
            } else {
                const float o = __shfl_xor_sync(0xffffffffu, f[i], off);
                f[i] = MAX ? fmaxf(f[i], o) : fminf(f[i], o);
            }
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (kPacked)
            return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else
            return f[i];
    }
};

// One warp per touched block of a sequence and `heads` kv heads.  A lane keeps the
// ends of 16 bytes of the row (32 on rows of 1 KB); 512 / row bytes rows pass at
// once.  The block is read whole from its first row, so that the result does not
// depend on what was there before.  Where lanes are left over, one group of them
// makes the codes of the largest values and the next those of the smallest.
template <typename Elt, int D>
__global__ void __launch_bounds__(kBoundsThreads) block_bounds_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int VPL = 16 / (int)sizeof(Elt);            // values of a chunk
    constexpr int CPR = D / VPL;                          // chunks of a row
    constexpr int LPR = CPR < 32 ? CPR : 32;              // lanes of a row
    constexpr int NCH = CPR / LPR;                        // chunks of a lane
    constexpr int RPW = 32 / LPR;                         // rows at once
    constexpr int U = NCH > 1 ? 4 : 8;                    // loads in flight
    sl_pdl_wait();
    sl_pdl_launch();
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const int slot = unit / p.parts, h0 = (unit - slot * p.parts) * p.heads, b = blockIdx.y;
    if (slot >= p.slots) return;
    const long long t0 = p.pos[b];
    int n = p.n_new;
    if (p.n_tok) n = max(0, min(n, p.n_tok[b]));
    const long long end = t0 + n, first = t0 > 0 ? t0 : 0;
    const long long lb = first / p.bs + slot;
    if (end <= first || lb * p.bs >= end) return;
    if (lb >= p.maxb) {
        if (lane == 0) set_error(p.err, 0x4u /* KVC_DEV_BAD_POSITION */);
        return;
    }
    const int phys = p.table[(long long)b * p.maxb + lb];
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) set_error(p.err, phys < 0 ? 0x2u : 0x1u);
        return;
    }
    const int rows = (int)min((long long)p.bs, end - lb * p.bs);
    const int c = lane % LPR, r0 = lane / LPR;
#pragma unroll 1
    for (int h = h0; h < min(h0 + p.heads, p.Hkv); ++h) {
        const long long row0 = ((long long)phys * p.Hkv + h) * p.bs;
        const Elt* src = static_cast<const Elt*>(p.cache) + p.layer_off + row0 * D;
        const float* sc = sizeof(Elt) == 1 ? p.scales + p.sc_layer_off + row0 : nullptr;
        Ends<Elt> hi[NCH], lo[NCH];
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
            hi[k].init(-INFINITY);
            lo[k].init(INFINITY);
        }
#pragma unroll 1
        for (int base = r0; base < rows; base += U * RPW) {
            uint4 w[U][NCH];
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = min(base + u * RPW, rows - 1);  // (a row twice changes nothing)
#pragma unroll
                for (int k = 0; k < NCH; ++k)
                    w[u][k] = __ldg(reinterpret_cast<const uint4*>(src + (long long)r * D + (k * LPR + c) * VPL));
                s[u] = sizeof(Elt) == 1 ? __ldg(sc + r) : 1.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < NCH; ++k) {
                    hi[k].template join<true>(w[u][k], s[u]);
                    lo[k].template join<false>(w[u][k], s[u]);
                }
        }
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                hi[k].template exchange<true>(off);
                lo[k].template exchange<false>(off);
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) a = fmaxf(a, fmaxf(fabsf(hi[k].value(i)), fabsf(lo[k].value(i))));
        }
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const float step = __fdiv_rn(a, 127.f);
        const long long at = (long long)phys * p.Hkv + h;
        if (lane == 0) p.steps[at] = step;
        // codes: lanes below LPR the largest, the next LPR the smallest (where a row takes the whole warp, both)
        constexpr int BOTH = RPW == 1 ? 2 : 1;
        if (r0 < 2) {
#pragma unroll
            for (int k = 0; k < NCH; ++k)
#pragma unroll
                for (int q = 0; q < BOTH; ++q) {
                    const int e = BOTH == 2 ? q : r0;
                    uint32_t w[VPL / 4];
#pragma unroll
                    for (int i = 0; i < VPL / 4; ++i) w[i] = 0u;
#pragma unroll
                    for (int i = 0; i < VPL; ++i) {
                        const float x = step > 0.f ? __fdiv_rn(e ? lo[k].value(i) : hi[k].value(i), step) : 0.f;
                        const int code = e ? (int)fmaxf(floorf(x), -127.f) : (int)fminf(ceilf(x), 127.f);
                        w[i >> 2] |= (uint32_t)(code & 0xff) << (8 * (i & 3));
                    }
                    int8_t* d = p.codes + at * 2 * D + e * D + (k * LPR + c) * VPL;
                    if constexpr (VPL == 4)
                        *reinterpret_cast<uint32_t*>(d) = w[0];
                    else if constexpr (VPL == 8)
                        *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
    }
}

template <typename Elt, int D>
cudaError_t launch_bounds_t(const BoundsParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    BoundsParams q = p;
    // a warp walks several heads of its block where there are more than enough warps: the
    // way to the block (position, table) is paid once
    q.heads = 1;
    while (q.heads < 8 && 2 * q.heads <= p.Hkv && (long long)p.B * p.slots * p.Hkv / (2 * q.heads) >= kBoundsWarps)
        q.heads *= 2;
    q.parts = (p.Hkv + q.heads - 1) / q.heads;
    const long long units = (long long)p.slots * q.parts;
    constexpr int W = kBoundsThreads / 32;
    const cudaLaunchConfig_t cfg =
        sl_config(dim3((unsigned)((units + W - 1) / W), p.B), kBoundsThreads, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, block_bounds_kernel<Elt, D>, q);
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
constexpr int kScoreThreads = 128;
constexpr int kScoreCtas = 152 * 8;            // CTAs that keep the GPU full

// Order of floats as unsigned integers; -0 counts as 0, NaN as the least.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (!(x == x)) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (chunk of blocks, kv head, sequence).  The group's q heads as
// codes in shared memory, positive and negative parts apart: hi meets the one
// and lo the other.  A warp scores groups of 32 blocks, a lane keeping track of
// each; D / 16 lanes hold a block's codes, 16 channels of each end a lane, U x 512 / D
// blocks at once, and the next ones (the first while the queries are made codes)
// are on their way meanwhile.
template <typename Act, int D>
__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int LPB = D / 16, BPW = 32 / LPB, U = D == 64 ? 2 : 4, NP = D / 64, W = kScoreThreads / 32;
    constexpr int IT = 32 / (U * BPW);                                // steps of a group
    extern __shared__ __align__(16) unsigned char s_q[];              // [G][2][D] codes, then [G] steps
    int8_t* codes = reinterpret_cast<int8_t*>(s_q);
    float* s_step = reinterpret_cast<float*>(s_q + (size_t)p.G * 2 * D);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, b = blockIdx.z;
    sl_pdl_wait();
    sl_pdl_launch();
    const int c0 = blockIdx.x * kScoreChunk * p.groups;
    const int32_t* trow = p.table + (long long)b * p.maxb;
    // this lane's block of a group: its entry as it stands
    auto entry = [&](int lb) { return lb < p.maxb ? __ldg(trow + lb) : -1; };
    int raw = entry(c0 + warp * 32 + lane);
    const int traw = p.pos[b];
    const int t = clamp_paged_t(traw, p.maxb, p.bs);
    if ((traw < 0 || traw != t) && blockIdx.x == 0 && h == 0 && tid == 0) set_error(p.err, 0x4u /* KVC_DEV_BAD_POSITION */);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    const int c1 = min(nb, c0 + kScoreChunk * p.groups);
    if (c0 >= c1) return;
    auto resident = [&](int lb, int phys) -> int {
        if (lb >= c1) return -1;
        if (phys >= p.num_blocks) {
            set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
            return -1;
        }
        return phys >= 0 && p.valid && !((__ldg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u) ? -1 : phys;
    };
    int lb = c0 + warp * 32 + lane;
    int phys = resident(lb, raw);
    const int ln = lane % LPB, sub = lane / LPB;
    uint4 hi[U], lo[U];
    float step[U];
    auto load = [&](int it) {                                         // the ends of U BPW blocks of the group
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ph = __shfl_sync(0xffffffffu, phys, (it * U + u) * BPW + sub);
            const long long at = (long long)max(ph, 0) * p.Hkv + h;
            const uint4* src = reinterpret_cast<const uint4*>(p.codes + at * 2 * D);
            hi[u] = lo[u] = make_uint4(0u, 0u, 0u, 0u);
            step[u] = 0.f;
            if (ph >= 0) {
                hi[u] = __ldg(src + ln);
                lo[u] = __ldg(src + LPB + ln);
                step[u] = __ldg(p.steps + at);
            }
        }
    };
    load(0);
#pragma unroll 1
    for (int g = warp; g < p.G; g += W) {
        const Act* qr = static_cast<const Act*>(p.q) + ((long long)b * p.Hq + h * p.G + g) * D;
        float x[2 * NP], a = 0.f;
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int i = lane + 32 * m;
            x[2 * m] = EltTraits<Act>::to_f32(qr[i]);
            x[2 * m + 1] = EltTraits<Act>::to_f32(qr[i + D / 2]);
        }
        if (p.rope != kRopeNone) {
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                float cs, sn;
                rope_cos_sin((long long)t, p.theta[lane + 32 * m], &cs, &sn);
                const float x1 = x[2 * m], x2 = x[2 * m + 1];
                x[2 * m] = x1 * cs - x2 * sn;
                x[2 * m + 1] = x1 * sn + x2 * cs;
            }
        }
#pragma unroll
        for (int m = 0; m < 2 * NP; ++m) a = fmaxf(a, fabsf(x[m]));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const float sq = __fdiv_rn(a, 127.f);
#pragma unroll
        for (int m = 0; m < 2 * NP; ++m) {
            const int code = q8_code(x[m], sq);
            int8_t* d = codes + (size_t)g * 2 * D + lane + 32 * (m >> 1) + (m & 1) * (D / 2);
            d[0] = (int8_t)max(code, 0);
            d[D] = (int8_t)min(code, 0);
        }
        if (lane == 0) s_step[g] = sq;
    }
    __syncthreads();
    uint32_t* keys = p.keys + ((long long)b * p.Hkv + h) * p.maxb;
#pragma unroll 1
    for (;;) {
        const int next = lb + W * 32, next_raw = next - lane < c1 ? entry(next) : -1;
        const int cur = phys;
        float score = -INFINITY;                                      // of this lane's own block
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            uint4 h4[U], l4[U];
            float st[U], best[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                h4[u] = hi[u];
                l4[u] = lo[u];
                st[u] = step[u];
                best[u] = -INFINITY;
            }
            if (it == IT - 1) phys = resident(next, next_raw);
            if (it < IT - 1 || next - lane < c1) load(it < IT - 1 ? it + 1 : 0);
#pragma unroll 1
            for (int g = 0; g < p.G; ++g) {
                const uint4 qp = *reinterpret_cast<const uint4*>(codes + (size_t)g * 2 * D + 16 * ln);
                const uint4 qn = *reinterpret_cast<const uint4*>(codes + (size_t)g * 2 * D + D + 16 * ln);
                const float sq = s_step[g];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    int a = __dp4a((int)h4[u].x, (int)qp.x, 0);
                    int e = __dp4a((int)l4[u].x, (int)qn.x, 0);
                    a = __dp4a((int)h4[u].y, (int)qp.y, a);
                    e = __dp4a((int)l4[u].y, (int)qn.y, e);
                    a = __dp4a((int)h4[u].z, (int)qp.z, a);
                    e = __dp4a((int)l4[u].z, (int)qn.z, e);
                    a = __dp4a((int)h4[u].w, (int)qp.w, a);
                    e = __dp4a((int)l4[u].w, (int)qn.w, e);
                    a += e;
#pragma unroll
                    for (int off = 1; off < LPB; off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
                    best[u] = fmaxf(best[u], __fmul_rn((float)a, __fmul_rn(sq, st[u])));
                }
            }
            // the lane of each block takes its score
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = lane - (it * U + u) * BPW;              // this lane's block among these BPW
                const float x = __shfl_sync(0xffffffffu, best[u], (j & (BPW - 1)) * LPB);
                if (j >= 0 && j < BPW) score = x;
            }
        }
        if (lb < c1)
            keys[lb] = cur < 0 ? 0u : (lb < p.first || lb >= nb - p.recent) ? 0xffffffffu : score_key(score);
        if (next - lane >= c1) break;                                 // (uniform in the warp)
        lb = next;
    }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;

// Sums over the CTA's threads before this one, of two counts at once; totals in *tot.
__device__ __forceinline__ int2 pick_scan(int2 v, int2* s_w, int2* tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int2 x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, off), c = __shfl_up_sync(0xffffffffu, x.y, off);
        if (lane >= off) {
            x.x += a;
            x.y += c;
        }
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    int2 before = make_int2(0, 0), all = before;
    for (int w = 0; w < nw; ++w) {
        const int2 s = s_w[w];
        if (w < warp) {
            before.x += s.x;
            before.y += s.y;
        }
        all.x += s.x;
        all.y += s.y;
    }
    __syncthreads();
    *tot = all;
    return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// Counts key `key`'s digit among the warp's (one addition for lanes of one digit).
__device__ __forceinline__ void pick_count(int* hist, bool in, uint32_t digit) {
    const unsigned act = __ballot_sync(0xffffffffu, in);
    if (in) {
        const unsigned same = __match_any_sync(act, digit);
        if ((threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
    }
}

// The digit that holds the want-th key (1-based) from the top (DOWN) or the
// bottom; how many keys lie beyond it on that side goes to *beyond.  By warp 0.
template <bool DOWN>
__device__ __forceinline__ void pick_digit(const int* hist, int want, int* digit, int* beyond) {
    const int lane = threadIdx.x & 31;
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = lane * 8 + i;
        c[i] = hist[DOWN ? 255 - d : d];
        sum += c[i];
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
        for (int i = 0; i < 8; ++i) {
            if (run < want && run + c[i] >= want) {
                *digit = DOWN ? 255 - (lane * 8 + i) : lane * 8 + i;
                *beyond = run;
            }
            run += c[i];
        }
    }
}

// One CTA per (kv head, sequence): the k largest keys, ties by the lowest index,
// by a radix search of the k-th largest (four digits at most: it ends where a digit
// takes all of its keys), then the kept indices in ascending order.  A thread keeps
// the first kPickKeys of its keys in registers; longer tables are read again.
// What bounds it: one trip to the keys, then barriers.
constexpr int kPickKeys = 4;

__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const __grid_constant__ SelectParams p) {
    __shared__ int s_hist[4][256];
    __shared__ int2 s_w[kPickWarps];
    __shared__ int s_digit[4], s_beyond[4];
    const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
    for (int i = tid; i < 4 * 256; i += kPickThreads) s_hist[0][i] = 0;
    if (tid < 4) s_digit[tid] = -1;
    sl_pdl_wait();
    sl_pdl_launch();
    const uint32_t* keys = p.keys + ((long long)b * p.Hkv + h) * p.maxb;
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    int32_t* out = p.blocks + ((long long)b * p.Hkv + h) * p.k;
    uint32_t mine[kPickKeys];
#pragma unroll
    for (int u = 0; u < kPickKeys; ++u) {
        const int i = u * kPickThreads + tid;
        mine[u] = i < nb ? __ldcg(keys + i) : 0u;
    }
    const int tail = kPickKeys * kPickThreads;
    __syncthreads();
    // keys above `low` are kept, and the first `ties` of those equal to it
    uint32_t prefix = 0, mask = 0, low = 0;
    int want = p.k, ties = 0x7fffffff;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
#pragma unroll
        for (int u = 0; u < kPickKeys; ++u)
            if (u * kPickThreads < nb)         // (uniform)
                pick_count(s_hist[pass], mine[u] != 0u && (mine[u] & mask) == prefix, (mine[u] >> shift) & 255u);
        for (int base = tail; base < nb; base += kPickThreads) {
            const uint32_t key = base + tid < nb ? __ldcg(keys + base + tid) : 0u;
            pick_count(s_hist[pass], key != 0u && (key & mask) == prefix, (key >> shift) & 255u);
        }
        __syncthreads();
        if (tid < 32) pick_digit<true>(s_hist[pass], want, &s_digit[pass], &s_beyond[pass]);
        __syncthreads();
        const int digit = s_digit[pass];
        if (digit < 0) {                       // fewer candidates than k (seen in the first pass): all of them
            low = 0u;
            ties = 0;
            break;
        }
        want -= s_beyond[pass];
        prefix |= (uint32_t)digit << shift;
        mask |= 255u << shift;
        if (s_hist[pass][digit] == want) {     // all that begin with these digits
            low = prefix ? prefix - 1u : 0u;   // (candidates' keys are above 0)
            ties = 0;
            break;
        }
        low = prefix;
        ties = want;
    }
    int2 run = make_int2(0, 0);                // keys above `low`, keys equal to it, before this pass
    auto emit = [&](int i, uint32_t key) {
        const bool more = key > low, same = key == low && key != 0u;
        int2 tot;
        const int2 ex = pick_scan(make_int2(more, same), s_w, &tot);
        const int above = run.x + ex.x, equal = run.y + ex.y;
        if (more || (same && equal < ties)) {
            const int at = above + min(equal, ties);
            if (at < p.k)
                out[at] = i;
            else
                index_fault(p.err, 40, at);
        }
        run.x += tot.x;
        run.y += tot.y;
    };
#pragma unroll
    for (int u = 0; u < kPickKeys; ++u)
        if (u * kPickThreads < nb) emit(u * kPickThreads + tid, mine[u]);
    for (int base = tail; base < nb; base += kPickThreads)
        emit(base + tid, base + tid < nb ? __ldcg(keys + base + tid) : 0u);
    for (int i = run.x + min(run.y, ties) + tid; i < p.k; i += kPickThreads) out[i] = -1;
}

// ---------------------------------------------------------------------------
// lists of a selected decode
// ---------------------------------------------------------------------------
constexpr int kListThreads = 256;

// One CTA per (kv head, sequence): its blocks, checked, as physical ones without
// gaps.  Entries ascend; one that does not lie above those before it (a block
// named twice) or past the table is reported and left out, negative ones are no
// entries.  Blocks that are unmapped, not resident or past the position are not
// attended.
__global__ void __launch_bounds__(kListThreads) select_list_kernel(const __grid_constant__ SelectPlanParams p) {
    constexpr int NW = kListThreads / 32;
    __shared__ int s_max[NW], s_cnt[NW], s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, b = blockIdx.y;
    sl_pdl_wait();
    sl_pdl_launch();
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int last = t < 0 ? -1 : t / p.bs;
    const int32_t* src = p.blocks + ((long long)b * p.Hkv + h) * p.k;
    const int32_t* trow = p.table + (long long)b * p.maxb;
    int32_t* dst = p.list + ((long long)h * p.B + b) * p.k;
    if (tid == 0) s_last = 0;
    int top = -1, n = 0;                  // largest entry and attended blocks before this pass
    for (int base = 0; base < p.k; base += kListThreads) {
        const int i = base + tid;
        int lb = i < p.k ? __ldcg(src + i) : -1;
        if (lb >= p.maxb) {
            set_error(p.err, 0x10u /* KVC_DEV_BAD_ENTRY */);
            lb = -1;
        }
        int m = lb;                       // largest entry up to here
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, m, off);
            if (lane >= off) m = max(m, a);
        }
        if (lane == 31) s_max[warp] = m;
        int before = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) before = -1;
        __syncthreads();
        before = max(before, top);
        int all = top;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before = max(before, s_max[w]);
            all = max(all, s_max[w]);
        }
        top = all;
        int phys = -1;
        if (lb >= 0 && lb <= before) {
            set_error(p.err, 0x10u);
        } else if (lb >= 0 && lb <= last) {
            phys = __ldg(trow + lb);
            if (phys >= p.num_blocks) {
                set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                phys = -1;
            }
            if (phys >= 0 && p.valid && !((__ldg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u)) phys = -1;
        }
        const unsigned have = __ballot_sync(0xffffffffu, phys >= 0);
        if (lane == 0) s_cnt[warp] = __popc(have);
        if (phys >= 0 && lb == last) s_last = 1;
        __syncthreads();
        int at = n + __popc(have & ((1u << lane) - 1u));
        for (int w = 0; w < NW; ++w) {
            if (w < warp) at += s_cnt[w];
            n += s_cnt[w];
        }
        if (phys >= 0) dst[at] = phys;
        __syncthreads();
    }
    // every attended block but the position's own holds bs rows
    if (tid == 0) p.rows[h * p.B + b] = n * p.bs - (s_last ? p.bs - (t - last * p.bs + 1) : 0);
}

}  // namespace

cudaError_t launch_block_bounds(int dtype, int D, const BoundsParams& p, cudaStream_t s) {
#define KVC_CASE(T, E, DD) \
    if (dtype == T && D == DD) return launch_bounds_t<E, DD>(p, s);
    KVC_CASE(0, float, 64) KVC_CASE(0, float, 128) KVC_CASE(0, float, 256)
    KVC_CASE(1, __nv_bfloat16, 64) KVC_CASE(1, __nv_bfloat16, 128) KVC_CASE(1, __nv_bfloat16, 256)
    KVC_CASE(2, int8_t, 128) KVC_CASE(2, int8_t, 256)
#undef KVC_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_select(int dtype, int D, const SelectParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const int smem = p.G * (2 * D + 4);
    // a CTA walks several chunks where there are more than enough of them
    SelectParams sp = p;
    const long long chunks = (p.maxb + kScoreChunk - 1) / kScoreChunk, units = chunks * p.Hkv * p.B;
    sp.groups = 1;
    while (sp.groups < 8 && units / (2 * sp.groups) >= kScoreCtas) sp.groups *= 2;
    cudaLaunchConfig_t cfg = sl_config(dim3((unsigned)((chunks + sp.groups - 1) / sp.groups), p.Hkv, p.B), kScoreThreads,
                                       smem, s, &attr);
    cudaError_t e = cudaErrorInvalidValue;
    // (above 48 KB, groups of more than 93 heads of 256, a kernel asks for its shared memory)
#define KVC_CASE(F, A, DD)                                                                                   \
    if ((dtype == 0) == F && D == DD) {                                                                      \
        e = smem > 48 * 1024 ? cudaFuncSetAttribute(block_score_kernel<A, DD>,                               \
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize, smem)       \
                             : cudaSuccess;                                                                  \
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, block_score_kernel<A, DD>, sp);                    \
    }
    KVC_CASE(true, float, 64) KVC_CASE(true, float, 128) KVC_CASE(true, float, 256)
    KVC_CASE(false, __nv_bfloat16, 64) KVC_CASE(false, __nv_bfloat16, 128) KVC_CASE(false, __nv_bfloat16, 256)
#undef KVC_CASE
    if (e != cudaSuccess) return e;
    cfg = sl_config(dim3(p.Hkv, p.B), kPickThreads, 0, s, &attr);
    return cudaLaunchKernelEx(&cfg, block_pick_kernel, sp);
}

cudaError_t launch_select_plan(const SelectPlanParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = sl_config(dim3(p.Hkv, p.B), kListThreads, 0, s, &attr);
    return cudaLaunchKernelEx(&cfg, select_list_kernel, p);
}

}  // namespace kvc
