// Paged attention, bf16 queries over a cache of the same type.
#include "attn.cuh"

namespace w4g {

template <>
int launch_attn_typed<1, false>(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_attn_dp<1, false, 64>(ctx, a, stream);
    if (a.head_dim <= 128) return launch_attn_dp<1, false, 128>(ctx, a, stream);
    return launch_attn_dp<1, false, 256>(ctx, a, stream);
}

}  // namespace w4g
