// Attention of drafted tokens: the workspace's size and the choice of the instance (tree.cuh).
#include "tree.cuh"

namespace w4g {

template <> int launch_tree_typed<0, false>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<0, true>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<1, false>(const DeviceCtx&, const TreeArgs&, cudaStream_t);
template <> int launch_tree_typed<1, true>(const DeviceCtx&, const TreeArgs&, cudaStream_t);

bool tree_map(CUtensorMap* map, const TreeArgs& a, const KvView& kv, bool e4m3, int dp, int box) {
    const EncodeTiledFn encode = tensor_map_encoder();
    if (!encode) return false;
    const uint64_t es = e4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), static_cast<cuuint64_t>(a.page_size),
                                static_cast<cuuint64_t>(a.kv_heads), static_cast<cuuint64_t>(a.num_pages)};
    cuuint64_t strides[3] = {kv.slot_stride * es, kv.head_stride * es, kv.page_stride * es};
    for (int i = 0; i < 3; ++i) {
        if (dims[i + 1] == 1) strides[i] = 16;  // never taken
        if (strides[i] == 0 || strides[i] >= 1ull << 40) return false;
    }
    const cuuint32_t shape[4] = {static_cast<cuuint32_t>(e4m3 ? dp : 64), static_cast<cuuint32_t>(box), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, kv.p, dims, strides,
                  shape, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tree_query_map(CUtensorMap* map, const TreeArgs& a, int box) {
    const EncodeTiledFn encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), static_cast<cuuint64_t>(a.q_heads),
                                static_cast<cuuint64_t>(a.T), 1};
    const cuuint64_t token = static_cast<cuuint64_t>(a.ldq) * 2;
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.head_dim) * 2, token, token};
    if (token >= 1ull << 40) return false;
    const cuuint32_t shape[4] = {64, static_cast<cuuint32_t>(a.q_heads / a.kv_heads), static_cast<cuuint32_t>(box), 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<uint16_t*>(a.q), dims, strides, shape, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t tree_workspace_bytes(const DeviceCtx& ctx, int head_dim) {
    return tree_workspace(ctx.num_sms, tree_dp(head_dim));
}

int launch_tree(const DeviceCtx& ctx, const TreeArgs& a, int dtype, bool e4m3, cudaStream_t stream) {
    if (dtype == 0)
        return e4m3 ? launch_tree_typed<0, true>(ctx, a, stream) : launch_tree_typed<0, false>(ctx, a, stream);
    return e4m3 ? launch_tree_typed<1, true>(ctx, a, stream) : launch_tree_typed<1, false>(ctx, a, stream);
}

}  // namespace w4g
