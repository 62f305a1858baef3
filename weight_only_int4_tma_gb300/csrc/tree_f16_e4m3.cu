// Attention of drafted tokens, fp16 queries over an 8-bit cache.
#include "tree.cuh"

namespace w4g {

template <>
int launch_tree_typed<0, true>(const DeviceCtx& ctx, const TreeArgs& a, cudaStream_t stream) {
    return launch_tree_dp<0, true>(ctx, a, stream);
}

}  // namespace w4g
