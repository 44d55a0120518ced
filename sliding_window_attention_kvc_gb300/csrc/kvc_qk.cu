// kvc_append_qk: the step between a layer's projection and its attention, in
// one pass -- norms of queries and keys for each head, rotary positions, and
// the append of keys and values to the cache.
//
// For a row x of D values (one head of one token):
//     x' = x / sqrt(mean(x^2) + eps) * (w + offset)            (q and k, optional)
//     (y_a, y_b) = m (x'_a cos - x'_b sin, x'_a sin + x'_b cos)
// over the pairs (a, b) of the first `dim` values, at the angle
// position * f_i; q rows go to q_out, k and v rows to the token's slot.
//
// Bound: bytes (each row is read and written once; a prompt) or launch
// latency (one token).  A lane owns 8 consecutive values of a row, so a row
// is one 16-byte load (two for fp32) for each of D / 8 lanes, its norm a
// butterfly over those lanes, and its pair partners either the lane's own
// (neighbour pairs) or one shuffle away (halves of whole 8-value chunks; other
// rotated widths go through shared memory).  The angles of a token are reduced
// exactly and their sines and cosines taken once per CTA, in shared memory,
// while the rows' loads are in flight, and serve every head.
//
// One token a CTA of two warps, twelve CTAs an SM: eight ragged prompt
// chunks of up to 2048 tokens, 32 / 8 heads of 128, bf16 paged, 303 MB: 61 us (65 replayed from a graph), 0.73 of
// the measured copy bandwidth.  Four
// warps took 96 us, CTAs that walk several tokens 117 us (their loads waited for the
// rows before).  One token of each of 64 sequences: 6.2 us, of which the launch and one
// dependent load each of position, table and rows are most.
#include "kvc_device.cuh"
#include "kvc_host.h"

namespace kvc {

namespace {

constexpr int kQkThreads = 64;
constexpr int kQkCtas = 12;          // CTAs an SM
constexpr int kQkBatch = 4;          // rows a thread keeps in flight
// How a row's pairs lie: neighbours; halves of whole 8-value chunks; any halves.
enum : int { kRotNone = 0, kRotPairs = 1, kRotChunks = 2, kRotAny = 3 };

struct QkParams {
    const void* q;
    const void* k;
    const void* v;
    const void* qw;                  // norm weights [D], null: that side is not normed
    const void* kw;
    void* q_out;                     // [B, n_new, Hq, D]
    void* cache;
    float* scales;                   // INT8 cache, else null
    const int32_t* pos;
    const int32_t* n_tok;            // may be null
    const int32_t* table;
    uint32_t* err;
    long long layer_off, kv_off, sc_layer_off, sc_kv_off;
    long long q_stride, k_stride, v_stride;    // elements between tokens
    int n_new, Hq, Hkv;
    int layout, window, sinks, capacity, bs, num_blocks, maxb;
    int rows_per_z;                  // rows (heads of q, k, v) of one CTA
    int rot;                         // rotated values of a row (even), 0: none
    int mode;                        // kRotNone ...
    float eps, offset, mag;
    unsigned long long turns[kMaxHalfDim];
};

template <typename Act> struct QkVec;
template <> struct QkVec<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const { EltTraits<__nv_bfloat16>::unpack(w, f); }
    __device__ __forceinline__ void put(const float (&f)[8]) {
        w = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
template <> struct QkVec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};

// A row of K (from f) or V (as loaded, in x; INT8: from f) to element offset `at` of the K
// half; every lane of a warp calls.
template <typename Act, int D, bool Q8>
__device__ __forceinline__ void qk_store(const QkParams& p, QkVec<Act>& x, const float (&f)[8], long long at, bool v,
                                         bool write, int lr) {
    const long long off = p.layer_off + at + (v ? p.kv_off : 0);
    if constexpr (Q8) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
#pragma unroll
        for (int o = D / 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (!write) return;
        const float sc = __fdiv_rn(amax, 127.f);
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo |= ((uint32_t)q8_code(f[j], sc) & 0xffu) << (8 * j);
            hi |= ((uint32_t)q8_code(f[4 + j], sc) & 0xffu) << (8 * j);
        }
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(p.cache) + off + lr * 8) = make_uint2(lo, hi);
        if (lr == 0) p.scales[p.sc_layer_off + at / D + (v ? p.sc_kv_off : 0)] = sc;
    } else if (write) {
        if (!v) x.put(f);
        x.store(static_cast<Act*>(p.cache) + off + lr * 8);
    }
}

// One head's row in 8 values a lane, by every lane of a warp at once: norm (ss: the
// row's sum of squares over its lanes), then rotation.  w: this lane's weights; c,
// s: its cosines and (signed) sines, interleaved: of its four pairs.
template <int D>
__device__ __forceinline__ void qk_row(float (&f)[8], bool norm, const float (&w)[8], float eps, int mode,
                                       const float (&c)[8], const float (&s)[8], int src, bool rotated, float* row,
                                       int lr, int half, int rot) {
    constexpr int LPR = D / 8;
    float2* const g = reinterpret_cast<float2*>(f);
    if (norm) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) q = __ffma2_rn(g[j], g[j], q);
        float ss = q.x + q.y;
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float rs = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            g[j] = __fmul2_rn(__fmul2_rn(g[j], make_float2(rs, rs)), make_float2(w[2 * j], w[2 * j + 1]));
    }
    if (mode == kRotPairs) {
        if (rotated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f[2 * j], y = f[2 * j + 1];
                f[2 * j] = x * c[j] - y * s[j];
                f[2 * j + 1] = x * s[j] + y * c[j];
            }
        }
    } else if (mode == kRotChunks) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, f[j], src, LPR);
        if (rotated) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * c[j] + o[j] * s[j];
        }
    } else if (mode == kRotAny) {
#pragma unroll
        for (int j = 0; j < 8; ++j) row[lr * 8 + j] = f[j];
        __syncwarp();
        if (rotated) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = lr * 8 + j;
                if (e < rot) f[j] = f[j] * c[j] + row[e < half ? e + half : e - half] * s[j];
            }
        }
        __syncwarp();
    }
}

// Act: element type of q, k, v, q_out and the weights; Q8: an INT8 cache.  Two
// warps a token: what a lane needs for every row (weights, sines, cosines) is in
// registers and serves a dozen rows.  With eight warps a token, three rows a
// thread, a prompt of 11.5k tokens spent 67% of the issue slots at 3.3 TB/s.
template <typename Act, int D, bool Q8>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) append_qk_kernel(const __grid_constant__ QkParams p) {
    constexpr int LPR = D / 8;                    // lanes of a row
    constexpr int RP = kQkThreads / LPR;          // rows the CTA visits at once
    __shared__ float2 s_cs[kMaxHalfDim];
    __shared__ float s_row[RP][D + 8];            // rotated widths off the 8-value chunks
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x;
    const int lr = tid % LPR, r0 = tid / LPR;
    const int i_tok = blockIdx.x, b = blockIdx.y;
    const int first = blockIdx.z * p.rows_per_z, end = min(p.Hq + 2 * p.Hkv, first + p.rows_per_z);
    const long long tok = (long long)b * p.n_new + i_tok;
    // the CTA's heads of q, of k and of v
    const int q0 = first, q1 = min(end, p.Hq);
    const int k0 = max(first, p.Hq) - p.Hq, k1 = min(end, p.Hq + p.Hkv) - p.Hq;
    const int v0 = max(first - p.Hq - p.Hkv, 0), v1 = end - p.Hq - p.Hkv;
    const Act* const qs = static_cast<const Act*>(p.q) + tok * p.q_stride + lr * 8;
    const Act* const ks = static_cast<const Act*>(p.k) + tok * p.k_stride + lr * 8;
    const Act* const vs = static_cast<const Act*>(p.v) + tok * p.v_stride + lr * 8;
    QkVec<Act> x[kQkBatch];
    auto load = [&](const Act* src, int base, int hi) {
#pragma unroll
        for (int u = 0; u < kQkBatch; ++u)
            if (base + u * RP + r0 < hi) x[u].load(src + (long long)(base + u * RP + r0) * D);
    };
    // the first rows need neither the count nor the position
    if (q0 < q1) load(qs, q0, q1);

    const int n = p.n_tok ? min(p.n_tok[b], p.n_new) : p.n_new;
    const int t0 = p.pos[b];
    const long long pos = (long long)t0 + i_tok;
    if (i_tok >= n || pos < 0) return;            // right and left padding: nothing is written

    // where the token goes in the cache (element offset of kv head 0 in the K half)
    bool keep = true;
    long long row_base = 0, head_stride = 0;
    if (p.layout != kPaged) {
        // a window token that a later one of this call overwrites is not written
        const long long last = (long long)t0 + n - 1;
        keep = pos < p.sinks || pos + p.window > last;
        const long long slot = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
        row_base = ((long long)b * p.Hkv * p.capacity + slot) * D;
        head_stride = (long long)p.capacity * D;
    } else {
        const long long lb = pos / p.bs;
        int phys = -1;
        uint32_t bad = 0;
        if (lb >= p.maxb) {
            bad = 0x4u;   // KVC_DEV_BAD_POSITION
        } else {
            phys = p.table[(long long)b * p.maxb + lb];
            if (phys < 0) bad = 0x2u;                       // KVC_DEV_UNMAPPED_APPEND
            else if (phys >= p.num_blocks) bad = 0x1u;      // KVC_DEV_BAD_BLOCK
        }
        if (bad) {
            keep = false;
            if (tid == 0 && blockIdx.z == 0) set_error(p.err, bad);
        }
        row_base = ((long long)phys * p.Hkv * p.bs + pos % p.bs) * D;
        head_stride = (long long)p.bs * D;
    }

    // the token's sines and cosines, once for all its heads
    const int half = p.rot >> 1;
    const int hc = half >> 3;                     // halves of whole chunks: chunks of a half
    float c[8], s[8];
    bool rotated = false;
    if (p.mode != kRotNone) {
        for (int i = tid; i < half; i += kQkThreads) {
            float cc, ss;
            rope_cos_sin(pos, p.turns[i], &cc, &ss);
            s_cs[i] = make_float2(cc * p.mag, ss * p.mag);
        }
        __syncthreads();
        rotated = lr * 8 < p.rot;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            int i = -1;
            float sign = 1.f;
            if (p.mode == kRotPairs) {
                if (j < 4 && lr * 8 + 2 * j < p.rot) i = lr * 4 + j;
            } else if (lr * 8 + j < p.rot) {
                // y_a = x_a cos - x_b sin, y_b = x_b cos + x_a sin
                const int e = lr * 8 + j;
                i = e < half ? e : e - half;
                sign = e < half ? -1.f : 1.f;
            }
            if (i >= 0) {
                const float2 cs = s_cs[i];
                c[j] = cs.x;
                s[j] = cs.y * sign;
            }
        }
    }
    const int src = lr < hc ? lr + hc : (lr < 2 * hc ? lr - hc : lr);
    float w[8];
    auto weights = [&](const void* wp) {
        if (!wp) return;
        QkVec<Act> wv;
        wv.load(static_cast<const Act*>(wp) + lr * 8);
        wv.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += p.offset;
    };

    if (q0 < q1) {
        weights(p.qw);
        Act* const dst = static_cast<Act*>(p.q_out) + tok * p.Hq * D + lr * 8;
        for (int base = q0; base < q1; base += kQkBatch * RP) {
            if (base != q0) load(qs, base, q1);
#pragma unroll
            for (int u = 0; u < kQkBatch; ++u) {
                if (base + u * RP >= q1) break;   // (uniform: a warp's rows share its shuffles)
                const int r = base + u * RP + r0;
                float f[8];
                x[u].get(f);
                qk_row<D>(f, p.qw, w, p.eps, p.mode, c, s, src, rotated, s_row[r0], lr, half, p.rot);
                if (r < q1) {
                    x[u].put(f);
                    x[u].store(dst + (long long)r * D);
                }
            }
        }
    }
    if (k0 < k1) {
        weights(p.kw);
        for (int base = k0; base < k1; base += kQkBatch * RP) {
            load(ks, base, k1);
#pragma unroll
            for (int u = 0; u < kQkBatch; ++u) {
                if (base + u * RP >= k1) break;
                const int r = base + u * RP + r0;
                float f[8];
                x[u].get(f);
                qk_row<D>(f, p.kw, w, p.eps, p.mode, c, s, src, rotated, s_row[r0], lr, half, p.rot);
                qk_store<Act, D, Q8>(p, x[u], f, row_base + r * head_stride, false, keep && r < k1, lr);
            }
        }
    }
    for (int base = v0; base < v1; base += kQkBatch * RP) {
        load(vs, base, v1);
#pragma unroll
        for (int u = 0; u < kQkBatch; ++u) {
            if (base + u * RP >= v1) break;
            const int r = base + u * RP + r0;
            float f[8];
            if constexpr (Q8) x[u].get(f);
            qk_store<Act, D, Q8>(p, x[u], f, row_base + r * head_stride, true, keep && r < v1, lr);
        }
    }
}

template <typename Act, int D, bool Q8>
cudaError_t launch_qk(const QkParams& p, dim3 grid, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kQkThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_qk_kernel<Act, D, Q8>, p);
}

// The grid: one CTA per token; few tokens: a token's rows over several CTAs, so
// that every SM has eight.
cudaError_t dispatch_qk(int dtype, int D, int B, QkParams& p, cudaStream_t s) {
    const int R = p.Hq + 2 * p.Hkv, RP = kQkThreads / (D / 8);
    const long long tokens = (long long)B * p.n_new;
    int parts = (R + RP - 1) / RP;
    if (tokens * parts > 8 * 152) parts = (int)((8 * 152 + tokens - 1) / tokens);
    if (parts > 65535) parts = 65535;
    p.rows_per_z = ((R + parts - 1) / parts + RP - 1) / RP * RP;
    const dim3 grid(p.n_new, B, (R + p.rows_per_z - 1) / p.rows_per_z);
    cudaError_t e = cudaErrorInvalidValue;
#define KVC_QK(DD)                                                               \
    if (D == DD)                                                                 \
        e = dtype == KVC_F32 ? launch_qk<float, DD, false>(p, grid, s)           \
            : dtype == KVC_BF16 ? launch_qk<__nv_bfloat16, DD, false>(p, grid, s) \
                                : launch_qk<__nv_bfloat16, DD, true>(p, grid, s);
    KVC_QK(64)
    KVC_QK(128)
    KVC_QK(256)
#undef KVC_QK
    return e;
}

}  // namespace

cudaError_t launch_append_rows(int dtype, const AppendParams& a, cudaStream_t stream) {
    QkParams p{};
    p.k = a.k_new;
    p.v = a.v_new;
    p.cache = a.cache;
    p.scales = a.scales;
    p.pos = a.pos;
    p.table = a.table;
    p.err = a.err;
    p.layer_off = a.layer_off;
    p.kv_off = a.kv_off;
    p.sc_layer_off = a.sc_layer_off;
    p.sc_kv_off = a.sc_kv_off;
    p.k_stride = p.v_stride = (long long)a.Hkv * a.D;
    p.n_new = a.n_new;
    p.Hkv = a.Hkv;
    p.layout = a.layout;
    p.window = a.window;
    p.sinks = a.sinks;
    p.capacity = a.capacity;
    p.bs = a.bs;
    p.num_blocks = a.num_blocks;
    p.maxb = a.maxb;
    return dispatch_qk(dtype, a.D, a.B, p, stream);
}

}  // namespace kvc

using namespace kvc;

extern "C" {

KVC_API int kvc_rotary_init(kvc_rotary* r) {
    if (!r) return KVC_ERR_NULL;
    r->ready = 0;
    if (r->magnitude == r->filled) r->magnitude = 0.f;     // the last call's value, not the caller's
    r->filled = 0.f;
    if (r->pairs != KVC_PAIRS_HALF && r->pairs != KVC_PAIRS_INTERLEAVED) return KVC_ERR_ARG;
    if (r->dim < 0 || r->dim > 2 * kMaxHalfDim || (r->dim & 1)) return KVC_ERR_ARG;
    if (r->scaling < KVC_SCALING_NONE || r->scaling > KVC_SCALING_BANDS) return KVC_ERR_ARG;
    if (!(r->base > 1.f) || !std::isfinite(r->base)) return KVC_ERR_ARG;
    if (!(r->magnitude >= 0.f) || !std::isfinite(r->magnitude)) return KVC_ERR_ARG;
    if (r->scaling != KVC_SCALING_NONE && (!(r->factor > 0.f) || !std::isfinite(r->factor))) return KVC_ERR_ARG;
    const bool ranged = r->scaling == KVC_SCALING_YARN || r->scaling == KVC_SCALING_BANDS;
    if (ranged && (r->original_len < 1 || !(r->slow > 0.f) || !(r->fast > r->slow) || !std::isfinite(r->fast)))
        return KVC_ERR_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    const int n = r->dim;
    const double base = r->base, orig = r->original_len;
    double low = 0.0, high = 0.0;
    if (r->scaling == KVC_SCALING_YARN && n > 0) {
        // the (fractional) pair that makes `turns` turns within the original length
        auto pair_of = [&](double turns) { return n * std::log(orig / (turns * two_pi)) / (2.0 * std::log(base)); };
        low = std::fmax(std::floor(pair_of(r->fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(r->slow)), n - 1.0);
    }
    for (int i = 0; i < n / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / n);
        double g = f;
        if (r->scaling == KVC_SCALING_LINEAR) {
            g = f / r->factor;
        } else if (r->scaling == KVC_SCALING_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            g = f / r->factor * ramp + f * (1.0 - ramp);
        } else if (r->scaling == KVC_SCALING_BANDS) {
            const double turns = orig * f / two_pi;
            const double keep = std::fmin(std::fmax((turns - r->slow) / ((double)r->fast - r->slow), 0.0), 1.0);
            g = f / r->factor * (1.0 - keep) + f * keep;
        }
        double turn = g / two_pi;
        turn -= std::floor(turn);                  // whole turns change nothing
        r->turns[i] = (uint64_t)std::ldexp(turn, 64);
    }
    if (r->magnitude == 0.f)
        r->magnitude = r->filled = (r->scaling == KVC_SCALING_YARN && r->factor > 1.f)
                                       ? (float)(0.1 * std::log((double)r->factor) + 1.0) : 1.f;
    r->ready = 1;
    return KVC_OK;
}

KVC_API int kvc_append_qk(const kvc_desc* d, void* cache, int32_t layer, const void* q, const void* k_new,
                          const void* v_new, int32_t q_stride, int32_t k_stride, int32_t v_stride, int32_t n_new,
                          const int32_t* pos, const int32_t* n_tok, const int32_t* block_table, const kvc_qk* qk,
                          void* q_out, void* workspace, size_t workspace_bytes, void* stream) {
    Geo g;
    const int rc = check_desc(d, &g);
    if (rc) return rc;
    if (!cache || !q || !k_new || !v_new || !pos || !qk || !q_out || !workspace) return KVC_ERR_NULL;
    if (d->layout == KVC_LAYOUT_PAGED && !block_table) return KVC_ERR_NULL;
    const kvc_rotary* rot = qk->rotary;
    if (rot && (!rot->ready || rot->dim > d->head_dim)) return KVC_ERR_ARG;
    const bool rotates = rot && rot->dim > 0;
    // a cache that rotates keys itself (baked, or when they are read) takes the norms alone,
    // and a baked one not even these: its decode would rotate the queries again
    if (d->rope == KVC_ROPE_BAKED || (d->rope == KVC_ROPE_READ_INCACHE && rotates)) return KVC_ERR_UNSUPPORTED;
    if (!(qk->eps >= 0.f)) return KVC_ERR_ARG;
    if (layer < 0 || layer >= d->layers || n_new < 1 || n_new > 0x7fffffff / 2) return KVC_ERR_ARG;
    const int wq = d->q_heads * d->head_dim, wk = d->kv_heads * d->head_dim;
    if (!q_stride) q_stride = wq;
    if (!k_stride) k_stride = wk;
    if (!v_stride) v_stride = wk;
    if (q_stride < wq || k_stride < wk || v_stride < wk) return KVC_ERR_ARG;
    const int per16 = 16 / g.act_elt;
    if (!aligned16(cache) || !aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) ||
        !aligned16(workspace) || !aligned16(qk->q_weight) || !aligned16(qk->k_weight) || q_stride % per16 ||
        k_stride % per16 || v_stride % per16)
        return KVC_ERR_ALIGN;
    const WorkspaceLayout w = ws_layout(d, g);
    if (workspace_bytes < w.total) return KVC_ERR_WORKSPACE;

    QkParams p{};
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.qw = qk->q_weight;
    p.kw = qk->k_weight;
    p.q_out = q_out;
    p.cache = cache;
    p.pos = pos;
    p.n_tok = n_tok;
    p.table = block_table;
    p.err = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + w.err);
    p.layer_off = (long long)layer * 2 * g.half_elems;
    p.kv_off = g.half_elems;
    if (d->dtype == KVC_I8) {
        const long long half_rows = g.half_elems / d->head_dim;
        p.scales = reinterpret_cast<float*>(static_cast<char*>(cache) + (size_t)d->layers * 2 * (size_t)g.half_elems);
        p.sc_layer_off = (long long)layer * 2 * half_rows;
        p.sc_kv_off = half_rows;
    }
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_new = n_new;
    p.Hq = d->q_heads;
    p.Hkv = d->kv_heads;
    p.layout = d->layout;
    p.window = d->window;
    p.sinks = d->layout == KVC_LAYOUT_SINK_RING ? d->sinks : 0;
    p.capacity = g.C;
    p.bs = d->block_size;
    p.num_blocks = d->num_blocks;
    p.maxb = d->max_blocks_per_seq;
    p.eps = qk->eps;
    p.offset = qk->weight_offset;
    if (rotates) {
        p.rot = rot->dim;
        p.mode = rot->pairs == KVC_PAIRS_INTERLEAVED ? kRotPairs : (rot->dim % 16 == 0 ? kRotChunks : kRotAny);
        p.mag = rot->magnitude;
        for (int i = 0; i < rot->dim / 2; ++i) p.turns[i] = rot->turns[i];
    }
    const cudaError_t e = dispatch_qk(d->dtype, d->head_dim, d->batch, p, (cudaStream_t)stream);
    return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

}  // extern "C"
