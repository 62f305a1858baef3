// Attention of drafted tokens, bf16 queries over a cache of the same type.
#include "tree.cuh"

namespace w4g {

template <>
int launch_tree_typed<1, false>(const DeviceCtx& ctx, const TreeArgs& a, cudaStream_t stream) {
    return launch_tree_dp<1, false>(ctx, a, stream);
}

}  // namespace w4g
