// Root-mean-square norm with the residual's addition (include/decode.h):
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight,
// written in the input's type, as int8 with one scale per row (max |y| / 127), or as E4M3
// with one power-of-two scale per 32 values.  Everything between the loads and the stores
// is fp32; h is rounded only for residual_out.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kNormThreads = 256;

// E8M0 exponent of a block whose largest magnitude is `most`: floor(log2(most)) - 8 (8 is
// the exponent of E4M3's largest value), at least -127; -127 for a zero block.  Below the
// normal numbers the floor of the logarithm is under -126 and the clamp decides.
__device__ __forceinline__ int norm_mx_exponent(float most) {
    const int e = static_cast<int>((__float_as_uint(most) >> 23) & 0xFFu) - 127 - 8;
    return most > 0.0f ? max(e, -127) : -127;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float norm_pow2(int e) {
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float norm_block_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) s += red[w];
    __syncthreads();
    return s;
}
__device__ __forceinline__ float norm_block_max(float v, float* red) {
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) s = fmaxf(s, red[w]);
    __syncthreads();
    return s;
}

// One CTA per row, one value per thread and step.
template <int DT, int OUT>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
    __shared__ float red[kNormThreads / 32];
    grid_dep_wait();
    const int m = static_cast<int>(blockIdx.x);
    const uint16_t* x = a.x + m * a.ldx;
    const uint16_t* res = a.residual ? a.residual + m * a.ldr : nullptr;
    uint16_t* res_out = a.residual_out ? a.residual_out + m * a.ldr : nullptr;
    auto value = [&](int i) {
        float h = dec_to_f32<DT>(x[i]);
        if (res) h += dec_to_f32<DT>(res[i]);
        return h;
    };
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.H; i += kNormThreads) {
        const float h = value(i);
        ss += h * h;
    }
    ss = norm_block_sum(ss, red);
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
    auto normed = [&](int i, float h) {
        const float w = a.weight ? dec_to_f32<DT>(a.weight[i]) : 1.0f;
        return h * r * w;
    };
    if constexpr (OUT == kNormSame) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.ldy;
        for (int i = threadIdx.x; i < a.H; i += kNormThreads) {
            const float h = value(i);
            const uint16_t out = dec_from_f32<DT>(normed(i, h));
            if (res_out) res_out[i] = dec_from_f32<DT>(h);
            y[i] = out;
        }
    } else if constexpr (OUT == kNormI8) {
        float most = 0.0f;
        for (int i = threadIdx.x; i < a.H; i += kNormThreads)
            most = fmaxf(most, fabsf(normed(i, value(i))));
        most = norm_block_max(most, red);
        const float s = most > 0.0f ? __fdiv_rn(most, 127.0f) : 1.0f;
        int8_t* y = static_cast<int8_t*>(a.y) + static_cast<int64_t>(m) * a.H;
        for (int i = threadIdx.x; i < a.H; i += kNormThreads) {
            const float h = value(i);
            const int q = __float2int_rn(__fdiv_rn(normed(i, h), s));
            if (res_out) res_out[i] = dec_from_f32<DT>(h);
            y[i] = static_cast<int8_t>(max(-127, min(127, q)));
        }
        if (threadIdx.x == 0) static_cast<float*>(a.scales)[m] = s;
    } else {
        uint8_t* y = static_cast<uint8_t*>(a.y) + static_cast<int64_t>(m) * a.H;
        uint8_t* sc = static_cast<uint8_t*>(a.scales) + static_cast<int64_t>(m) * (a.H / 32);
        for (int i = threadIdx.x; i < a.H; i += kNormThreads) {  // H % 32 == 0: whole warps
            const float h = value(i);
            const float v = normed(i, h);
            const float most = warp_max(fabsf(v));
            const int e = norm_mx_exponent(most);
            if (res_out) res_out[i] = dec_from_f32<DT>(h);
            y[i] = static_cast<uint8_t>(dec_e4m3x2(v * norm_pow2(-e), 0.0f));
            if ((i & 31) == 0) sc[i / 32] = static_cast<uint8_t>(e + 127);
        }
    }
}

template <int DT>
int launch_norm_dt(const NormArgs& a, int M, int out, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(M));
    if (out == kNormSame)
        return launch_dependent(norm_kernel<DT, kNormSame>, grid, kNormThreads, 0, stream, a);
    if (out == kNormI8)
        return launch_dependent(norm_kernel<DT, kNormI8>, grid, kNormThreads, 0, stream, a);
    return launch_dependent(norm_kernel<DT, kNormMx>, grid, kNormThreads, 0, stream, a);
}

}  // namespace

int launch_norm(const DeviceCtx& ctx, const NormArgs& a, int M, int dtype, int out,
                cudaStream_t stream) {
    (void)ctx;
    return dtype == 0 ? launch_norm_dt<0>(a, M, out, stream) : launch_norm_dt<1>(a, M, out, stream);
}

}  // namespace w4g
