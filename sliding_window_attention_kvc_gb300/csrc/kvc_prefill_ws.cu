// The warp-specialised tcgen05 prefill, plain scores (kvc_prefill_ws.cuh).
#include "kvc_prefill_ws.cuh"

namespace kvc {

cudaError_t launch_prefill_ws(int head_dim, bool q8, const PrefillParams& p, const PrefillMaps& maps,
                              cudaStream_t stream) {
    if (p.G < 1 || kWsRows % p.G) return cudaErrorInvalidValue;
    const bool rd = p.rope == kRopeRead;
#define KVC_WS(DD, RD, Q) \
    if (head_dim == DD && rd == RD && q8 == Q) return launch_prefill_ws_t<DD, RD, Q, kModPlain>(p, maps, stream);
    KVC_WS(64, false, false) KVC_WS(64, true, false)
    KVC_WS(128, false, false) KVC_WS(128, true, false) KVC_WS(128, false, true) KVC_WS(128, true, true)
    KVC_WS(256, false, false) KVC_WS(256, true, false) KVC_WS(256, false, true) KVC_WS(256, true, true)
#undef KVC_WS
    return cudaErrorInvalidValue;
}

}  // namespace kvc
