// Attention of drafted tokens: the workspace's size and the choice of the instance (tree.cuh).
#include "tree.cuh"

namespace w4g {

template <> int launch_tree_typed<0, false>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<0, true>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<1, false>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<1, true>(const DeviceCtx&, const TreeArgs&, cudaStream_t);

size_t tree_workspace_bytes(const DeviceCtx& ctx, int head_dim) {
    return tree_workspace(ctx.num_sms, tree_dp(head_dim));
}

int launch_tree(const DeviceCtx& ctx, const TreeArgs& a, int dtype, bool e4m3, cudaStream_t stream) {
    if (dtype == 0)
        return e4m3 ? launch_tree_typed<0, true>(ctx, a, stream) : launch_tree_typed<0, false>(ctx, a, stream);
    return e4m3 ? launch_tree_typed<1, true>(ctx, a, stream) : launch_tree_typed<1, false>(ctx, a, stream);
}

}  // namespace w4g
