// Host-side building blocks shared by the C-ABI translation units: descriptor
// checks, the workspace carve-up, RoPE frequency tables and the tensor-map
// encoder.
#pragma once

#include <cmath>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "kvc.h"
#include "kvc_params.h"

namespace kvc {

struct Geo {
    int elt;        // bytes per cache element (INT8: the codes)
    int act_elt;    // bytes per element of q, out, k_new, v_new
    int C;          // window layouts: slots per (sequence, kv head)
    int G, GH, nsub;
    long long half_elems;   // elements of one K (or V) half of one layer
};

// rows of K/V one pipeline stage holds: fp32 kernel 8 KiB per K stage;
// bf16 tensor-core kernel 4 (2 for head_dim 256) sub-tiles of 16 rows
inline int rows_per_stage(int elt, int D) { return elt == 4 ? 8192 / (D * elt) : (D == 256 ? 32 : 64); }

inline int check_desc(const kvc_desc* d, Geo* g) {
    if (!d) return KVC_ERR_NULL;
    if (d->layout < 0 || d->layout > 2 || d->rope < 0 || d->rope > 2 || d->dtype < 0 || d->dtype > 2)
        return KVC_ERR_DESC;
    if (d->layers < 1 || d->batch < 1 || d->kv_heads < 1 || d->q_heads < 1 || d->q_heads % d->kv_heads)
        return KVC_ERR_DESC;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return KVC_ERR_UNSUPPORTED;
    if (d->num_splits < 0) return KVC_ERR_DESC;
    if (d->rope != KVC_ROPE_NONE && !(d->rope_base > 0.f)) return KVC_ERR_DESC;
    if (d->softmax_scale < 0.f) return KVC_ERR_DESC;
    g->elt = d->dtype == KVC_F32 ? 4 : (d->dtype == KVC_BF16 ? 2 : 1);
    g->act_elt = d->dtype == KVC_F32 ? 4 : 2;
    if (d->dtype == KVC_I8 && d->head_dim < 128) return KVC_ERR_UNSUPPORTED;
    g->G = d->q_heads / d->kv_heads;
    g->GH = (g->G % 4 == 0) ? 4 : ((g->G % 2 == 0) ? 2 : 1);
    g->nsub = g->G / g->GH;
    // launch-grid limits: sequences on x, (kv head, q-head group) pairs on y,
    // and a 32-bit count of (sequence, pair) units
    const long long pairs = (long long)d->kv_heads * g->nsub;
    if (d->batch > 65535 || pairs > 65535 || d->batch * pairs > 0x7fffffffLL) return KVC_ERR_DESC;
    if (d->layout == KVC_LAYOUT_PAGED) {
        if (d->block_size < 1 || d->num_blocks < 1 || d->max_blocks_per_seq < 1) return KVC_ERR_DESC;
        if ((long long)d->block_size * d->max_blocks_per_seq > 0x7fffffffLL) return KVC_ERR_DESC;
        if (d->rope == KVC_ROPE_READ_INCACHE) return KVC_ERR_UNSUPPORTED;
        g->C = 0;
        g->half_elems = (long long)d->num_blocks * d->kv_heads * d->block_size * d->head_dim;
    } else {
        if (d->window < 1) return KVC_ERR_DESC;
        if (d->layout == KVC_LAYOUT_RING && d->sinks != 0) return KVC_ERR_DESC;
        if (d->layout == KVC_LAYOUT_SINK_RING && d->sinks < 1) return KVC_ERR_DESC;
        if ((long long)d->window + d->sinks > 0x3fffffffLL) return KVC_ERR_DESC;
        g->C = d->window + d->sinks;
        g->half_elems = (long long)d->batch * d->kv_heads * g->C * d->head_dim;
    }
    // INT8 scale tensor maps: rows of a half in multiples of 4 (16-byte strides)
    if (d->dtype == KVC_I8 && (g->half_elems / d->head_dim) % 4) return KVC_ERR_UNSUPPORTED;
    return KVC_OK;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline WorkspaceLayout ws_layout(const kvc_desc* d, const Geo& g) {
    WorkspaceLayout w{};
    const int units = d->batch * d->kv_heads * g.nsub;
    const int groups = d->kv_heads * g.nsub;
    // stream-K shares per (kv head, q-head group): bf16 kernels, and the paged
    // plan.  bf16: a persistent grid of about two CTAs per SM claims them in turn.
    // the persistent grid: 152 SMs times the decode kernel's resident CTAs
    // (at least two: kernels held to one CTA per SM keep two shares per SM)
    const int per_sm = decode_ctas_per_sm(d->dtype == KVC_I8, d->layout == KVC_LAYOUT_PAGED,
                                          d->rope == KVC_ROPE_READ_INCACHE, d->head_dim);
    const int stream_ctas = kStreamCtas / 2 * (per_sm > 2 ? per_sm : 2);
    const int persist = (stream_ctas + groups - 1) / groups;
    if (d->layout == KVC_LAYOUT_PAGED || d->dtype != KVC_F32) {
        const bool bf16 = d->dtype != KVC_F32;     // tensor-core kernel (bf16 or INT8 cache)
        const int factor = (bf16 && d->layout == KVC_LAYOUT_PAGED && d->batch >= kPagedShareBatch)
                               ? kPagedShareFactor : 1;
        w.shares = d->num_splits > 0 ? d->num_splits : factor * persist;
        w.ctas = bf16 ? (persist < w.shares ? persist : w.shares) : w.shares;
        w.items = w.shares + d->batch;     // slot x + b of segment (share x, sequence b)
        w.nsplit = 0;
    } else {
        const int T = rows_per_stage(g.elt, d->head_dim);
        int maxs = g.C / (2 * T);
        if (maxs < 1) maxs = 1;
        int ns = d->num_splits > 0 ? d->num_splits : (kTargetCtas + units - 1) / units;
        if (d->num_splits <= 0 && ns > maxs) ns = maxs;
        if (ns < 1) ns = 1;
        w.nsplit = ns;
        w.items = d->batch * ns;
    }
    size_t off = 0;
    w.err = off;
    off += 256;
    w.counters = off;
    off = align_up(off + (size_t)(units + 1) * 4, 256);
    w.part_ml = off;
    off = align_up(off + (size_t)w.items * d->q_heads * 8, 256);
    w.part_o = off;
    off = align_up(off + (size_t)w.items * d->q_heads * d->head_dim * 4, 256);
    w.plan_seq = w.plan_acc = w.plan_items = w.plan_info = w.plan_total = w.plan_cta = w.plan_dir = w.plan_refs = w.blocks = off;
    if (d->layout == KVC_LAYOUT_PAGED) {
        w.plan_seq = off;
        off = align_up(off + (size_t)d->batch * 8, 256);
        w.plan_acc = off;
        off = align_up(off + (size_t)d->batch * 12, 256);
        w.plan_items = off;
        off = align_up(off + (size_t)w.items * 16, 256);
        w.plan_info = off;
        off = align_up(off + (size_t)w.items * 16, 256);
        w.plan_cta = off;
        off = align_up(off + (size_t)w.shares * 8, 256);
        w.plan_dir = off;
        off = align_up(off + (size_t)d->batch * ((d->max_blocks_per_seq + 31) / 32) * 8, 256);
        w.plan_refs = off;
        off = align_up(off + (size_t)d->num_blocks * 4, 256);
        w.blocks = off;
        off = align_up(off + align_up((size_t)d->batch * 5 * 4, 16) + (size_t)d->batch * 16 + 16 +
                           (size_t)d->num_blocks * 4, 256);
        w.plan_total = off;
        off += 256;
    }
    w.total = off;
    return w;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// theta_i = base^(-2i/D); passed as fp32 (small in-tile angles) and as the
// 64-bit fixed-point fraction of a turn theta_i / (2 pi) * 2^64 used for
// exact reduction of pos * theta_i on the device.
inline void fill_theta(int D, float base, unsigned long long* turns, float* theta_f) {
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < D / 2; ++i) {
        const double th = std::pow((double)base, -2.0 * i / D);
        turns[i] = (unsigned long long)std::ldexp(th / two_pi, 64);
        if (theta_f) theta_f[i] = (float)th;
    }
}

// cuTensorMapEncodeTiled, looked up once through the runtime's driver entry
// point (no link against the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

}  // namespace kvc
