// Paged attention, fp16 queries over an 8-bit (E4M3) cache.
#include "attn.cuh"

namespace w4g {

template <>
int launch_attn_typed<0, true>(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_attn_dp<0, true, 64>(ctx, a, stream);
    if (a.head_dim <= 128) return launch_attn_dp<0, true, 128>(ctx, a, stream);
    return launch_attn_dp<0, true, 256>(ctx, a, stream);
}

}  // namespace w4g
