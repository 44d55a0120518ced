// kvc_append_path: the keys and values of the accepted path of a tree of
// drafted tokens, gathered out of the draft's rows and appended.
#include "kvc_decode.cuh"
#include "kvc_tree.h"

namespace kvc {

namespace {

constexpr int kPathThreads = 128;

// One CTA per (path place, sequence).  A thread takes 16 bytes of the first and
// of the second half of a row, which are rotated with each other when BAKED (as
// kvc_append rotates them), of K and of V: four loads in flight, whole sectors
// written.  INT8: a warp a kv head.  A handful of rows: the latency of one
// dependent chain (count, index, row) is what it costs: 2.1 us for up to 8 of 32
// tokens of 64 sequences, 8 kv heads of 128, bf16, replayed from a graph.
template <typename Elt, int D>
__global__ void __launch_bounds__(kPathThreads) append_path_kernel(const __grid_constant__ PathParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int j = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int t0 = p.pos[b];
    int n = p.n_path ? p.n_path[b] : p.P;
    const int tok = p.path[(long long)b * p.P + j];
    if (n > p.P) {
        if (j == 0 && tid == 0) set_error(p.err, 0x10u /* KVC_DEV_BAD_ENTRY */);
        n = p.P;
    }
    if (t0 < 0 || j >= n) return;
    if (tok < 0 || tok >= p.T) {
        if (tid == 0) set_error(p.err, 0x10u);
        return;
    }
    const long long pos = (long long)t0 + j, last = (long long)t0 + n - 1;
    long long row_base, head_stride;           // elements of the K half to kv head 0's row; between kv heads
    if (p.layout != kPaged) {
        // a row that a later one of this call overwrites is not written
        if (pos >= p.sinks && pos + p.window <= last) return;
        const long long slot = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
        row_base = ((long long)b * p.Hkv * p.capacity + slot) * D;
        head_stride = (long long)p.capacity * D;
    } else {
        const long long lb = pos / p.bs;
        if (lb >= p.maxb) {
            if (tid == 0) set_error(p.err, 0x4u /* KVC_DEV_BAD_POSITION */);
            return;
        }
        const int phys = p.table[(long long)b * p.maxb + lb];
        if (phys < 0 || phys >= p.num_blocks) {
            if (tid == 0) set_error(p.err, phys < 0 ? 0x2u : 0x1u);
            return;
        }
        row_base = ((long long)phys * p.Hkv * p.bs + (pos % p.bs)) * D;
        head_stride = (long long)p.bs * D;
    }
    const long long src = ((long long)b * p.T + tok) * p.Hkv * D;
    if constexpr (sizeof(Elt) == 1) {
        const __nv_bfloat16* ks = static_cast<const __nv_bfloat16*>(p.k_new) + src;
        const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(p.v_new) + src;
        const int lane = tid & 31;
        for (int h = tid >> 5; h < p.Hkv; h += kPathThreads / 32) {
            int8_t* kd = static_cast<int8_t*>(p.cache) + p.layer_off + row_base + h * head_stride;
            float* sd = p.scales + p.sc_layer_off + (row_base + h * head_stride) / D;
            int8_t kq[D / 32], vq[D / 32];
            float sk, sv;
            q8_store_token_warp<D / 64>(ks + (long long)h * D, vs + (long long)h * D, kd, kd + p.kv_off, sd,
                                        sd + p.sc_kv_off, p.rope, pos, p.theta, lane, kq, vq, &sk, &sv);
        }
    } else {
        using TR = EltTraits<Elt>;
        constexpr int CH = 16 / (int)sizeof(Elt), UPH = D / (2 * CH);     // values of 16 bytes; units of a head
        const Elt* ks = static_cast<const Elt*>(p.k_new) + src;
        const Elt* vs = static_cast<const Elt*>(p.v_new) + src;
        Elt* kc = static_cast<Elt*>(p.cache) + p.layer_off + row_base;
        for (int u = tid; u < p.Hkv * UPH; u += kPathThreads) {
            const int h = u / UPH, c = (u - h * UPH) * CH;
            const Elt* kr = ks + (long long)h * D + c;
            const Elt* vr = vs + (long long)h * D + c;
            uint4 a = __ldcg(reinterpret_cast<const uint4*>(kr)), e = __ldcg(reinterpret_cast<const uint4*>(kr + D / 2));
            const uint4 x = __ldcg(reinterpret_cast<const uint4*>(vr)), y = __ldcg(reinterpret_cast<const uint4*>(vr + D / 2));
            if (p.rope == kRopeBaked) {
                float f[CH], g[CH];
                TR::unpack(a, f);
                TR::unpack(e, g);
                alignas(16) Elt lo[CH], hi[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float cs, sn;
                    rope_cos_sin(pos, p.theta[c + i], &cs, &sn);
                    lo[i] = TR::from_f32(f[i] * cs - g[i] * sn);
                    hi[i] = TR::from_f32(f[i] * sn + g[i] * cs);
                }
                a = *reinterpret_cast<const uint4*>(lo);
                e = *reinterpret_cast<const uint4*>(hi);
            }
            Elt* kd = kc + h * head_stride + c;
            *reinterpret_cast<uint4*>(kd) = a;
            *reinterpret_cast<uint4*>(kd + D / 2) = e;
            *reinterpret_cast<uint4*>(kd + p.kv_off) = x;
            *reinterpret_cast<uint4*>(kd + p.kv_off + D / 2) = y;
        }
    }
}

template <typename Elt, int D>
cudaError_t launch_path_t(const PathParams& p, cudaStream_t s) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.P, p.B);
    cfg.blockDim = dim3(kPathThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_path_kernel<Elt, D>, p);
}

}  // namespace

cudaError_t launch_append_path(int dtype, int D, const PathParams& p, cudaStream_t s) {
#define KVC_CASE(T, E, DD) \
    if (dtype == T && D == DD) return launch_path_t<E, DD>(p, s);
    KVC_CASE(0, float, 64) KVC_CASE(0, float, 128) KVC_CASE(0, float, 256)
    KVC_CASE(1, __nv_bfloat16, 64) KVC_CASE(1, __nv_bfloat16, 128) KVC_CASE(1, __nv_bfloat16, 256)
    KVC_CASE(2, int8_t, 128) KVC_CASE(2, int8_t, 256)
#undef KVC_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kvc
