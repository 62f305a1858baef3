// Attention of drafted tokens over a paged key-value cache (include/decode.h): one CTA per
// (sequence, query head), one row after another.  Each warp takes 32 tokens at a time, a lane per
// token for the scores and a lane per value for the output, with a running maximum.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kTreeWarps = 4;

template <int DT, bool E4M3>
__device__ __forceinline__ float kv_value(const void* p, int64_t at) {
    if constexpr (E4M3)
        return __half2float(__ushort_as_half(static_cast<uint16_t>(
            dec_e4m3x2_to_f16x2(static_cast<const uint8_t*>(p)[at]) & 0xFFFFu)));
    else
        return dec_to_f32<DT>(static_cast<const uint16_t*>(p)[at]);
}

template <int DT, bool E4M3>
__global__ void __launch_bounds__(32 * kTreeWarps) tree_kernel(TreeArgs a) {
    __shared__ float sq[256], so[kTreeWarps][256], sm[kTreeWarps], sl[kTreeWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = a.head_dim;
    grid_dep_wait();
    const int64_t units = static_cast<int64_t>(a.B) * a.q_heads;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int b = static_cast<int>(u / a.q_heads), h = static_cast<int>(u % a.q_heads);
        const int first = a.starts[b], last = a.starts[b + 1];
        if (first == last && first >= 0 && first <= a.T) continue;
        const int len = a.lens[b], n = last - first;
        if (first < 0 || last < first || last > a.T || n > 64 || len < n ||
            len > a.max_pages * a.page_size) {
            if (tid == 0) record_status(a.status, kDecInvalidArg);
            continue;
        }
        const int g = h / (a.q_heads / a.kv_heads), ctx = len - n;
        const float scale = a.scale * (E4M3 && a.kc.scale ? a.kc.scale[g] : 1.0f);
        const float vs = E4M3 && a.vc.scale ? a.vc.scale[g] : 1.0f;
        for (int i = 0; i < n; ++i) {
            const uint64_t all = n == 64 ? ~0ull : (1ull << n) - 1;
            const uint64_t w = (a.mask ? a.mask[first + i] : ~0ull >> (63 - i)) & all;
            const int from = a.window ? ctx + __popcll(w) - a.window : 0;
            __syncthreads();
            const uint16_t* q = a.q + static_cast<int64_t>(first + i) * a.ldq + static_cast<int64_t>(h) * D;
            for (int d = tid; d < D; d += 32 * kTreeWarps) sq[d] = dec_to_f32<DT>(q[d]);
            __syncthreads();
            float m = -INFINITY, l = 0.0f, o[8] = {};
            for (int j0 = warp * 32; j0 < len; j0 += 32 * kTreeWarps) {
                const int j = j0 + lane;
                bool seen = j < len && (j >= ctx ? (w >> (j - ctx)) & 1 : j < a.sinks || j >= from);
                const int page = seen ? a.block_table[b * a.ld_table + j / a.page_size] : 0;
                if (seen && (page < 0 || page >= a.num_pages)) {
                    record_status(a.status, kDecInvalidArg);
                    seen = false;
                }
                const int64_t kat = static_cast<int64_t>(page) * a.kc.page_stride + (j % a.page_size) * a.kc.slot_stride + g * a.kc.head_stride;
                const int64_t vat = static_cast<int64_t>(page) * a.vc.page_stride + (j % a.page_size) * a.vc.slot_stride + g * a.vc.head_stride;
                float s = -INFINITY;
                if (seen) {
                    s = 0.0f;
                    for (int d = 0; d < D; ++d) s = fmaf(sq[d], kv_value<DT, E4M3>(a.kc.p, kat + d), s);
                    s *= scale;
                }
                float top = s;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    const float x = __shfl_xor_sync(0xFFFFFFFFu, top, d);
                    top = x > top || x != x ? x : top;
                }
                top = top > m || top != top || m == -INFINITY ? top : m;
                if (m != m) top = m;
                if (top == -INFINITY) continue;
                const float f = m == -INFINITY ? 0.0f : expf(m - top);
                const float p = s == -INFINITY ? 0.0f : expf(s - top);
                m = top;
                l = l * f + warp_sum(p);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= f;
                for (int t = 0; t < 32; ++t) {
                    const float pt = __shfl_sync(0xFFFFFFFFu, p, t);
                    const int64_t at = __shfl_sync(0xFFFFFFFFu, vat, t);
                    if (!(pt == 0.0f)) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (lane + 32 * e < D) o[e] = fmaf(pt, kv_value<DT, E4M3>(a.vc.p, at + lane + 32 * e), o[e]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (lane + 32 * e < D) so[warp][lane + 32 * e] = o[e];
            if (lane == 0) sm[warp] = m, sl[warp] = l;
            __syncthreads();
            float top = -INFINITY, sum = 0.0f;
            for (int x = 0; x < kTreeWarps; ++x) top = sm[x] > top || sm[x] != sm[x] ? sm[x] : top;
            for (int x = 0; x < kTreeWarps; ++x) sum += sm[x] == -INFINITY ? 0.0f : sl[x] * expf(sm[x] - top);
            const int64_t row = first + i;
            for (int d = tid; d < D; d += 32 * kTreeWarps) {
                float v = 0.0f;
                for (int x = 0; x < kTreeWarps; ++x)
                    if (sm[x] != -INFINITY) v += so[x][d] * expf(sm[x] - top);
                a.out[row * a.ldo + static_cast<int64_t>(h) * D + d] = dec_from_f32<DT>(sum == 0.0f ? 0.0f : v * (vs / sum));
            }
            if (a.lse && tid == 0)
                a.lse[row * a.q_heads + h] = sum > 0.0f ? top + logf(sum) : sum == 0.0f ? -INFINITY : top;
        }
    }
}

}  // namespace

size_t tree_workspace_bytes(const DeviceCtx&, int) { return 16; }

int launch_tree(const DeviceCtx& ctx, const TreeArgs& a, int dtype, bool e4m3, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(a.B) * a.q_heads;
    const int64_t most = static_cast<int64_t>(ctx.num_sms) * 64;
    const dim3 grid(static_cast<unsigned>(units < most ? units : most));
    auto kern = dtype == 0 ? (e4m3 ? tree_kernel<0, true> : tree_kernel<0, false>)
                           : (e4m3 ? tree_kernel<1, true> : tree_kernel<1, false>);
    return launch_dependent(kern, grid, dim3(32 * kTreeWarps), 0, stream, a);
}

}  // namespace w4g
