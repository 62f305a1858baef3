// Attention of one new token per sequence over a paged key-value cache (include/decode.h):
//   s_j = scale q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j)  over the visible tokens.
// One pass with the running maximum m and sum l of the softmax: a new score s moves the
// reference to m' = max(m, s), and l and the weighted sum of values are multiplied by
// exp(m - m') first, so the result is that of the two-pass formula.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kMaxD = 256;

template <int DT, bool E4M3>
__device__ __forceinline__ float attn_load(const void* p, int64_t off) {
    if constexpr (E4M3) {
        const uint32_t h2 = dec_e4m3x2_to_f16x2(static_cast<const uint8_t*>(p)[off]);
        return __half2float(__ushort_as_half(static_cast<uint16_t>(h2)));
    } else {
        return dec_to_f32<DT>(static_cast<const uint16_t*>(p)[off]);
    }
}

// One CTA per (query head, sequence); its warps take the tokens in turn.
template <int DT, bool E4M3>
__global__ void __launch_bounds__(32 * kAttnWarps) attn_kernel(AttnArgs a) {
    __shared__ float sm[kAttnWarps], sl[kAttnWarps], so[kAttnWarps][kMaxD];
    grid_dep_wait();
    const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.x);
    const int g = h / (a.q_heads / a.kv_heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.head_dim;
    const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
    int64_t len = a.lens[b];
    if (len < 0 || len > most) {
        if (threadIdx.x == 0) record_status(a.status, kDecInvalidArg);
        len = len < 0 ? 0 : most;
    }
    const int64_t first = a.window > 0 && len > a.window ? len - a.window : 0;
    const float ks = E4M3 && a.kc.scale ? a.kc.scale[g] : 1.0f;
    const float vs = E4M3 && a.vc.scale ? a.vc.scale[g] : 1.0f;
    float q[kMaxD / 32], o[kMaxD / 32];
    for (int i = 0; i < kMaxD / 32; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? dec_to_f32<DT>(a.q[b * a.ldq + static_cast<int64_t>(h) * D + d]) : 0.0f;
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = first + warp; j < len; j += kAttnWarps) {
        const int page = a.block_table[b * a.ld_table + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) record_status(a.status, kDecInvalidArg);
            continue;
        }
        const int64_t slot = j % a.page_size;
        const int64_t ko = page * a.kc.page_stride + slot * a.kc.slot_stride + g * a.kc.head_stride;
        const int64_t vo = page * a.vc.page_stride + slot * a.vc.slot_stride + g * a.vc.head_stride;
        float s = 0.0f;
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int d = lane + 32 * i;
            if (d < D) s += q[i] * attn_load<DT, E4M3>(a.kc.p, ko + d);
        }
        s = warp_sum(s) * ks * a.scale;
        const float m2 = fmaxf(m, s);
        const float c = __expf(m - m2), p = __expf(s - m2);
        l = l * c + p;
        for (int i = 0; i < kMaxD / 32; ++i) {
            const int d = lane + 32 * i;
            if (d < D) o[i] = o[i] * c + p * attn_load<DT, E4M3>(a.vc.p, vo + d);
        }
        m = m2;
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    for (int i = 0; i < kMaxD / 32; ++i)
        if (lane + 32 * i < D) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kAttnWarps; ++w) L += M == -INFINITY ? 0.0f : sl[w] * __expf(sm[w] - M);
    for (int d = threadIdx.x; d < D; d += 32 * kAttnWarps) {
        float v = 0.0f;
        for (int w = 0; w < kAttnWarps; ++w)
            v += M == -INFINITY ? 0.0f : so[w][d] * __expf(sm[w] - M);
        a.out[b * a.ldo + static_cast<int64_t>(h) * D + d] =
            dec_from_f32<DT>(L > 0.0f ? v / L * vs : 0.0f);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<int64_t>(b) * a.q_heads + h] = L > 0.0f ? M + logf(L) : -INFINITY;
}

}  // namespace

size_t attn_workspace_bytes(const DeviceCtx&, int, int, int, bool) { return 16; }

int launch_attn(const DeviceCtx& ctx, const AttnArgs& a, int dtype, bool e4m3,
                cudaStream_t stream) {
    (void)ctx;
    const dim3 grid(static_cast<unsigned>(a.q_heads), static_cast<unsigned>(a.B));
    auto kern = dtype == 0 ? (e4m3 ? attn_kernel<0, true> : attn_kernel<0, false>)
                           : (e4m3 ? attn_kernel<1, true> : attn_kernel<1, false>);
    return launch_dependent(kern, grid, 32 * kAttnWarps, 0, stream, a);
}

}  // namespace w4g
