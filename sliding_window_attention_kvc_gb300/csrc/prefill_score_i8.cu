// The warp-specialised tcgen05 prefill with modified scores, INT8 caches
// (kvc_prefill_ws.cuh).
#include "kvc_prefill_ws.cuh"

namespace kvc {

cudaError_t launch_prefill_score_i8(int head_dim, const PrefillParams& p, const PrefillMaps& maps,
                                    cudaStream_t stream) {
    if (p.G < 1 || p.G > kWsRows || p.rope == kRopeRead) return cudaErrorInvalidValue;
    const int mod = (p.score.cap2 > 0.f ? kModCap : 0) | (p.score.slopes ? kModBias : 0) |
                    (p.score.cap2 > 0.f && p.score.cap2 <= kWsFixedCap && !p.score.slopes ? kModFixed : 0);
#define KVC_WS(DD, M) \
    if (head_dim == DD && mod == (M)) return launch_prefill_ws_t<DD, false, true, kModScore | (M)>(p, maps, stream);
#define KVC_WS_ALL(DD) KVC_WS(DD, 0) KVC_WS(DD, kModCap) KVC_WS(DD, kModBias) KVC_WS(DD, kModCap | kModBias) \
    KVC_WS(DD, kModCap | kModFixed)
    KVC_WS_ALL(128)
    KVC_WS_ALL(256)
#undef KVC_WS_ALL
#undef KVC_WS
    return cudaErrorInvalidValue;
}

}  // namespace kvc
