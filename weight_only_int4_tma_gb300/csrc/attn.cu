// Paged attention: the workspace's size and the choice of the instance (attn.cuh).
#include "attn.cuh"

namespace w4g {

template <> int launch_attn_typed<0, false>(const DeviceCtx&, const AttnArgs&, cudaStream_t);
template <> int launch_attn_typed<0, true>(const DeviceCtx&, const AttnArgs&, cudaStream_t);
template <> int launch_attn_typed<1, false>(const DeviceCtx&, const AttnArgs&, cudaStream_t);
template <> int launch_attn_typed<1, true>(const DeviceCtx&, const AttnArgs&, cudaStream_t);

size_t attn_workspace_bytes(const DeviceCtx& ctx, int q_heads, int kv_heads, int head_dim) {
    const int ctas = ctx.num_sms;
    const int rows = q_heads / kv_heads <= 8 ? 8 : 16;
    const int dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    return attn_counter_bytes(ctas) + 2ull * ctas * attn_part_floats(rows, dp) * 4;
}

int launch_attn(const DeviceCtx& ctx, const AttnArgs& a, int dtype, bool e4m3, cudaStream_t stream) {
    if (dtype == 0)
        return e4m3 ? launch_attn_typed<0, true>(ctx, a, stream) : launch_attn_typed<0, false>(ctx, a, stream);
    return e4m3 ? launch_attn_typed<1, true>(ctx, a, stream) : launch_attn_typed<1, false>(ctx, a, stream);
}

}  // namespace w4g
