// Caches read in part: bounds of each block's keys, blocks chosen by what the
// bounds allow a query's scores to be, and the lists that a decode over the
// chosen blocks walks.
//
// For a block and kv head, hi_d and lo_d are the largest and smallest key
// value of channel d.  For any key of the block
//     q . k = sum q_d k_d <= sum max(q_d hi_d, q_d lo_d) = U,
// so a block whose U is small holds no key that the query attends much.  hi and
// lo are kept as 8-bit codes of one step s = max(|hi|, |lo|) / 127, hi rounded
// up and lo down, so that the codes' bound is a bound still, but for the fp32
// roundings of s and of the quotients (2^-23 of 127 s at most); q enters as codes
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
// What bounds it: a prompt's bytes (8 ragged chunks, 107 MB of bf16: 22 us, 0.72 of the
// measured bandwidth; ends kept as floats, a head a warp: 38); a step's call the trips to
// position, table and rows (64 sequences, 8 kv heads: 3.1 us).  The same calls on fp32 caches:
// 39 us (0.79) and 3.6; on INT8 ones, whose every code becomes a float times its row's step,
// 57 us (0.15) and 5.8.
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
                    w[u][k] = __ldcg(reinterpret_cast<const uint4*>(src + (long long)r * D + (k * LPR + c) * VPL));
                s[u] = sizeof(Elt) == 1 ? __ldcg(sc + r) : 1.f;
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
constexpr int kScoreThreads = 128;             // a block of the cache a thread

// Order of floats as unsigned integers; -0 counts as 0, NaN as the least.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (!(x == x)) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sums of N values over the W lanes that share them, in log2(W) steps of which each
// halves the values that a lane still holds (N = 8, W = 8: 7 exchanges against 24 of a
// sum at a time): lane bit `off` keeps the upper half where it is set.  Afterwards a lane
// holds v[0 .. max(1, N / W) - 1] of the values whose index begins with its bits, from
// the highest down; lanes beyond N hold the same.
template <int N, int W>
__device__ __forceinline__ void spread_sum(int (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int off = W / 2; off >= 1; off >>= 1) {
        if (n > 1) {
            n >>= 1;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const bool up = lane & off;
                    const int send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
}

__device__ __noinline__ float2 score_angle(int t, unsigned long long turns) {
    float2 r;
    rope_cos_sin((long long)t, turns, &r.x, &r.y);
    return r;
}

// One CTA per (128 blocks, kv head, sequence): a warp scores 32 blocks, a lane keeping
// track of each.  The group's q heads are codes in shared memory, positive and negative
// parts apart: hi meets the one and lo the other.  D / 16 lanes hold a block's codes, 16
// channels of each end a lane, two blocks at a time; the next ones (the first while
// the queries are made codes) are on their way meanwhile, and four q heads share their
// sums' shuffles.
// What bounds it: 2 D + 4 bytes a block and kv head from DRAM against 2 D / 4 products of
// four for each q head and what surrounds them: at four heads a group the instructions,
// so that addresses are one product and absent blocks are read like others (block 0) and
// left out at the end.  64 sequences of up to 1024 blocks, 8 kv heads, 77 MB: 27 us with
// the choice behind it (43 with the codes brought by bulk copies, all kv heads a CTA;
// 29 with a sum at a time).
template <typename Act, int D>
__global__ void __launch_bounds__(kScoreThreads) block_score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int LPB = D / 16, BPW = 32 / LPB, U = 2, W = kScoreThreads / 32;
    constexpr int IT = 32 / (U * BPW);                                // steps of a warp
    constexpr int HB = LPB / 4;                                       // lanes of a q head after the sums
    extern __shared__ __align__(16) unsigned char s_q[];              // [G4][2][D] codes, then [G4] steps; G4: G in fours
    const int G4 = (p.G + 3) & ~3;
    int8_t* codes = reinterpret_cast<int8_t*>(s_q);
    float* s_step = reinterpret_cast<float*>(s_q + (size_t)G4 * 2 * D);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, b = blockIdx.z;
    sl_pdl_wait();
    sl_pdl_launch();
    const int lb0 = (blockIdx.x * W + warp) * 32;                     // this warp's blocks
    int phys = lb0 + lane < p.maxb ? __ldcg(p.table + (long long)b * p.maxb + lb0 + lane) : -1;
    const int traw = p.pos[b];
    const int t = clamp_paged_t(traw, p.maxb, p.bs);
    if ((traw < 0 || traw != t) && blockIdx.x == 0 && h == 0 && tid == 0) set_error(p.err, 0x4u /* KVC_DEV_BAD_POSITION */);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    if ((int)blockIdx.x * W * 32 >= nb) return;                       // (uniform)
    if (lb0 + lane >= nb) phys = -1;
    if (phys >= p.num_blocks) {
        set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
        phys = -1;
    }
    if (phys >= 0 && p.valid && !((__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u)) phys = -1;
    const unsigned have = __ballot_sync(0xffffffffu, phys >= 0);
    const int ln = lane % LPB, sub = lane / LPB;
    const uint32_t unit = (uint32_t)max(phys, 0) * (uint32_t)p.Hkv + (uint32_t)h;      // (fits: the steps are an array of them)
    const float step = have ? __ldcg(p.steps + unit) : 0.f;
    const uint4* src = reinterpret_cast<const uint4*>(p.codes) + ln;
    uint4 hi[2][U], lo[2][U];
    auto load = [&](int it) {                                         // the ends of U BPW blocks
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint4* at = src + (size_t)__shfl_sync(0xffffffffu, unit, (it * U + u) * BPW + sub) * (2 * LPB);
            hi[it & 1][u] = __ldcg(at);
            lo[it & 1][u] = __ldcg(at + LPB);
        }
    };
    if (have) load(0);
    // q heads as codes: D / 16 lanes a row, 8 channels of each half a lane
#pragma unroll 1
    for (int g = warp * BPW; g < G4; g += W * BPW) {
        // (behind the last head it stands again: the largest of the scores is what counts)
        const Act* qr = static_cast<const Act*>(p.q) + ((long long)b * p.Hq + h * p.G + min(g + sub, p.G - 1)) * D + 8 * ln;
        constexpr int CH = 8 * (int)sizeof(Act) / 16, V = 16 / (int)sizeof(Act);
        float x[2][8], a = 0.f;                                       // halves of the head
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                EltTraits<Act>::unpack(__ldcg(reinterpret_cast<const uint4*>(qr + e * (D / 2)) + c), x[e] + c * V);
        if (p.rope != kRopeNone) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 cs = score_angle(t, p.theta[8 * ln + i]);
                const float x1 = x[0][i], x2 = x[1][i];
                x[0][i] = x1 * cs.x - x2 * cs.y;
                x[1][i] = x1 * cs.y + x2 * cs.x;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));
#pragma unroll
        for (int off = 1; off < LPB; off <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const float sq = __fdiv_rn(a, 127.f);
        if (g + sub < G4) {
            int8_t* d = codes + (size_t)(g + sub) * 2 * D + 8 * ln;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t up[2] = {0u, 0u}, down[2] = {0u, 0u};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int code = q8_code(x[e][i], sq);
                    up[i >> 2] |= (uint32_t)max(code, 0) << (8 * (i & 3));
                    down[i >> 2] |= (uint32_t)(min(code, 0) & 0xff) << (8 * (i & 3));
                }
                *reinterpret_cast<uint2*>(d + e * (D / 2)) = make_uint2(up[0], up[1]);
                *reinterpret_cast<uint2*>(d + D + e * (D / 2)) = make_uint2(down[0], down[1]);
            }
            if (ln == 0) s_step[g + sub] = sq;
        }
    }
    __syncthreads();
    if (lb0 >= nb) return;
    uint32_t* keys = p.keys + ((long long)b * p.Hkv + h) * p.key_stride + lb0;
    if (!have) {
        if (lb0 + lane < nb) keys[lane] = 0u;
        return;
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        if (it + 1 < IT) load(it + 1);
        float best[U];
#pragma unroll
        for (int u = 0; u < U; ++u) best[u] = -INFINITY;
        // the step of this lane's block after the sums (LPB == 4: of both)
        float st[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            st[u] = LPB == 4 || u == 0
                        ? __shfl_sync(0xffffffffu, step,
                                      (it * U + (LPB == 4 ? u : (ln & (HB / 2)) != 0)) * BPW + sub)
                        : 0.f;
#pragma unroll 1
        for (int g = 0; g < G4; g += 4) {
            int v[4 * U];                                             // [head][block]
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint4 qp = *reinterpret_cast<const uint4*>(codes + (size_t)(g + y) * 2 * D + 16 * ln);
                const uint4 qn = *reinterpret_cast<const uint4*>(codes + (size_t)(g + y) * 2 * D + D + 16 * ln);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 a4 = hi[it & 1][u], b4 = lo[it & 1][u];
                    int a = __dp4a((int)a4.x, (int)qp.x, 0);
                    a = __dp4a((int)b4.x, (int)qn.x, a);
                    a = __dp4a((int)a4.y, (int)qp.y, a);
                    a = __dp4a((int)b4.y, (int)qn.y, a);
                    a = __dp4a((int)a4.z, (int)qp.z, a);
                    a = __dp4a((int)b4.z, (int)qn.z, a);
                    a = __dp4a((int)a4.w, (int)qp.w, a);
                    a = __dp4a((int)b4.w, (int)qn.w, a);
                    v[y * U + u] = a;
                }
            }
            spread_sum<4 * U, LPB>(v, lane);
            // this lane's head of the four: its upper two bits among the LPB; block: the next one, or both
            const float sq = s_step[g + (ln / HB & 3)];
#pragma unroll
            for (int u = 0; u < (LPB == 4 ? U : 1); ++u) best[u] = fmaxf(best[u], __fmul_rn((float)v[u], __fmul_rn(sq, st[u])));
        }
        // the largest over the heads; a lane of each block stores its key
#pragma unroll
        for (int u = 0; u < (LPB == 4 ? U : 1); ++u) {
            best[u] = fmaxf(best[u], __shfl_xor_sync(0xffffffffu, best[u], HB));
            best[u] = fmaxf(best[u], __shfl_xor_sync(0xffffffffu, best[u], 2 * HB));
            const int j = (it * U + (LPB == 4 ? u : (ln & (HB / 2)) != 0)) * BPW + sub, lb = lb0 + j;
            if ((LPB == 4 ? ln == 0 : (ln & ~(HB / 2)) == 0) && lb < nb)
                keys[j] = !((have >> j) & 1u)                     ? 0u
                          : (lb < p.first || lb >= nb - p.recent) ? 0xffffffffu
                                                                  : score_key(best[u]);
        }
    }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
constexpr int kPickThreads = 1024;             // at most
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

// Counts the digits of the warp's keys (one addition where all lanes have the same).
__device__ __forceinline__ void pick_count(int* hist, bool in, uint32_t digit) {
    const unsigned act = __ballot_sync(0xffffffffu, in);
    if (!act) return;
    const int lead = __ffs(act) - 1;
    const uint32_t d0 = __shfl_sync(0xffffffffu, digit, lead);
    const bool alike = __all_sync(0xffffffffu, !in || digit == d0);
    if (alike) {
        if ((int)(threadIdx.x & 31) == lead) atomicAdd(&hist[d0], __popc(act));
    } else if (in) {
        atomicAdd(&hist[digit], 1);
    }
}

// The digit that holds the want-th key (1-based) from the top; how many keys lie
// above it goes to *beyond.  By warp 0.
__device__ __forceinline__ void pick_digit(const int* hist, int want, int* digit, int* beyond) {
    const int lane = threadIdx.x & 31;
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - (lane * 8 + i)];
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
                *digit = 255 - (lane * 8 + i);
                *beyond = run;
            }
            run += c[i];
        }
    }
}

// One CTA per (kv head, sequence): the k largest keys, ties by the lowest index,
// by a radix search of the k-th largest (four digits at most: it ends where a digit
// takes all of its keys), then the kept indices in ascending order.  A thread keeps
// four neighbouring keys in registers; what is behind those is read again.
// What bounds it: one trip to the keys, then barriers: 8 us, launched alone on cold
// caches, for 512 rows of up to 1024 keys as for 8 of up to 2048.
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const __grid_constant__ SelectParams p) {
    __shared__ int s_hist[4][256];
    __shared__ int2 s_w[kPickWarps];
    __shared__ int s_digit[4], s_beyond[4];
    const int tid = threadIdx.x, nt = blockDim.x, h = blockIdx.x, b = blockIdx.y;
    for (int i = tid; i < 4 * 256; i += nt) s_hist[0][i] = 0;
    if (tid < 4) s_digit[tid] = -1;
    sl_pdl_wait();
    sl_pdl_launch();
    const uint4* keys = reinterpret_cast<const uint4*>(p.keys + ((long long)b * p.Hkv + h) * p.key_stride);
    const int t = clamp_paged_t(p.pos[b], p.maxb, p.bs);
    const int nb = t < 0 ? 0 : t / p.bs + 1;
    int32_t* out = p.blocks + ((long long)b * p.Hkv + h) * p.k;
    // four keys from index i on (0 behind the last)
    auto four = [&](int i, uint32_t (&k)[4]) {
        const uint4 w = i < nb ? __ldcg(keys + (i >> 2)) : make_uint4(0u, 0u, 0u, 0u);
        k[0] = w.x;
        k[1] = i + 1 < nb ? w.y : 0u;
        k[2] = i + 2 < nb ? w.z : 0u;
        k[3] = i + 3 < nb ? w.w : 0u;
    };
    uint32_t mine[4];
    four(4 * tid, mine);
    __syncthreads();
    // keys above `low` are kept, and the first `ties` of those equal to it
    uint32_t prefix = 0, mask = 0, low = 0;
    int want = p.k, ties = 0x7fffffff;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
#pragma unroll 1
        for (int base = 0; base < nb; base += 4 * nt) {
            uint32_t k[4] = {mine[0], mine[1], mine[2], mine[3]};
            if (base > 0) four(base + 4 * tid, k);
#pragma unroll
            for (int u = 0; u < 4; ++u) pick_count(s_hist[pass], k[u] != 0u && (k[u] & mask) == prefix, (k[u] >> shift) & 255u);
        }
        __syncthreads();
        if (tid < 32) pick_digit(s_hist[pass], want, &s_digit[pass], &s_beyond[pass]);
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
#pragma unroll 1
    for (int base = 0; base < nb; base += 4 * nt) {
        uint32_t k[4] = {mine[0], mine[1], mine[2], mine[3]};
        if (base > 0) four(base + 4 * tid, k);
        int2 n = make_int2(0, 0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            n.x += k[u] > low;
            n.y += k[u] == low && k[u] != 0u;
        }
        int2 tot;
        const int2 ex = pick_scan(n, s_w, &tot);
        int above = run.x + ex.x, equal = run.y + ex.y;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool more = k[u] > low, same = k[u] == low && k[u] != 0u;
            if (more || (same && equal < ties)) {
                const int at = above + min(equal, ties);
                if (at < p.k)
                    out[at] = base + 4 * tid + u;
                else
                    index_fault(p.err, 40, at);
            }
            above += more;
            equal += same;
        }
        run.x += tot.x;
        run.y += tot.y;
    }
    for (int i = run.x + min(run.y, ties) + tid; i < p.k; i += nt) out[i] = -1;
}

// ---------------------------------------------------------------------------
// lists of a selected decode
// ---------------------------------------------------------------------------
constexpr int kListThreads = 256;

// One CTA per (kv head, sequence): its blocks, checked, as physical ones without
// gaps.  Entries ascend; one that does not lie above those before it (a block
// named twice) or past the table is reported and left out, negative ones are no
// entries.  Blocks that are unmapped, not resident or past the position are not
// attended.  What bounds it: the trips to position, list and table (6 us alone on cold
// caches, 64 sequences, 8 kv heads, 128 blocks each).
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
            phys = __ldcg(trow + lb);
            if (phys >= p.num_blocks) {
                set_error(p.err, 0x1u /* KVC_DEV_BAD_BLOCK */);
                phys = -1;
            }
            if (phys >= 0 && p.valid && !((__ldcg(p.valid + (phys >> 5)) >> (phys & 31)) & 1u)) phys = -1;
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

template <typename Act, int D>
cudaError_t launch_score_t(const SelectParams& p, cudaStream_t s) {
    const int smem = ((p.G + 3) & ~3) * (2 * D + 4);
    // (above 48 KB, groups of more than 92 heads of 256, a kernel asks for its shared memory)
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(block_score_kernel<Act, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        sl_config(dim3((unsigned)((p.maxb + kScoreThreads - 1) / kScoreThreads), p.Hkv, p.B), kScoreThreads, smem, s, &attr);
    return cudaLaunchKernelEx(&cfg, block_score_kernel<Act, D>, p);
}

cudaError_t launch_select(int dtype, int D, const SelectParams& p, cudaStream_t s) {
    cudaError_t e = cudaErrorInvalidValue;
#define KVC_CASE(F, A, DD) \
    if ((dtype == 0) == F && D == DD) e = launch_score_t<A, DD>(p, s);
    KVC_CASE(true, float, 64) KVC_CASE(true, float, 128) KVC_CASE(true, float, 256)
    KVC_CASE(false, __nv_bfloat16, 64) KVC_CASE(false, __nv_bfloat16, 128) KVC_CASE(false, __nv_bfloat16, 256)
#undef KVC_CASE
    if (e != cudaSuccess) return e;
    // four keys a thread, as far as a CTA goes
    int threads = 128;
    while (threads < kPickThreads && 4 * threads < p.maxb) threads *= 2;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = sl_config(dim3(p.Hkv, p.B), threads, 0, s, &attr);
    return cudaLaunchKernelEx(&cfg, block_pick_kernel, p);
}

cudaError_t launch_select_plan(const SelectPlanParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = sl_config(dim3(p.Hkv, p.B), kListThreads, 0, s, &attr);
    return cudaLaunchKernelEx(&cfg, select_list_kernel, p);
}

}  // namespace kvc
