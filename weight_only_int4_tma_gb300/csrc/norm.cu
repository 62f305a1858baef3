// Root-mean-square norm with the residual's addition (include/decode.h):
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight,
// written in the input's type, as int8 with one scale per row (max |y| / 127), or as E4M3
// with one power-of-two scale per 32 values.  Everything between the loads and the stores
// is fp32; h is rounded only for residual_out.
//
// A row is read once: its threads hold it in registers, in 16-byte pieces of 8 values, from
// the loads over the reduction to the stores.  Bound by HBM for many rows, by the latency of
// one load, one block reduction and one store for few.  With residual, on the device: 4096 x
// 8192 bf16 41.5 us, 6.5 TB/s; to int8 42.6 us, 5.5 TB/s; to MX 38.7 us, 6.1 TB/s; 1 x 8192 2.5 us, 8 x
// 8192 to int8 2.7 us and to MX 2.6 us in a graph.  (Rows of up to 1024 threads leave a thread 64
// registers: with four pieces each it spills 70 to 84 bytes.)
#include "decode.cuh"

namespace w4g {
namespace {

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

template <int DT>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] & 0xFFFFu));
        f[2 * j + 1] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] >> 16));
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(dec_pack2<DT>(f[0], f[1]), dec_pack2<DT>(f[2], f[3]),
                      dec_pack2<DT>(f[4], f[5]), dec_pack2<DT>(f[6], f[7]));
}

// The sum of `sum` and, with MAX, the largest `most` (magnitudes) over the warps of one row (warps
// row_warp0 .. + row_warps - 1 of the CTA); every thread of the CTA takes part, `red` holds a
// pair per warp.
template <bool MAX>
__device__ __forceinline__ void row_reduce(float& sum, float& most, float2* red, int row_warp0,
                                           int row_warps) {
    sum = warp_sum(sum);
    if (MAX) most = warp_max(most);
    if (row_warps == 1) return;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(sum, most);
    __syncthreads();
    const float2 v = lane < row_warps ? red[row_warp0 + lane] : make_float2(0.0f, 0.0f);
    sum = warp_sum(v.x);
    if (MAX) most = warp_max(v.y);
}

// `row_threads` (a multiple of 32) threads per row, rows_per_cta rows per CTA, V pieces per
// thread: piece p of a row is held by thread p % row_threads.
template <int DT, int OUT, int V>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a, int M, int row_threads) {
    __shared__ float2 red[32];
    const int in_cta = static_cast<int>(threadIdx.x) / row_threads;
    const int t = static_cast<int>(threadIdx.x) - in_cta * row_threads;
    const int rows_per_cta = static_cast<int>(blockDim.x) / row_threads;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * rows_per_cta + in_cta;
    const int row_warps = row_threads >> 5, row_warp0 = in_cta * row_warps;
    const int pieces = a.H >> 3;
    const bool live = m < M;
    float h[V][8];
    uint4 xv[V], rv[V], wv[V];
    grid_dep_wait();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int p = t + j * row_threads;
        const bool in = live && p < pieces;
        xv[j] = rv[j] = wv[j] = make_uint4(0, 0, 0, 0);
        if (in) {
            xv[j] = reinterpret_cast<const uint4*>(a.x + m * a.ldx)[p];
            if (a.residual) rv[j] = reinterpret_cast<const uint4*>(a.residual + m * a.ldr)[p];
        }
    }
    if (a.weight) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = t + j * row_threads;
            if (p < pieces) wv[j] = reinterpret_cast<const uint4*>(a.weight)[p];
        }
    }
    grid_dep_launch();
    // h, and in its place h * weight once the sum has it: y = (h * weight) * r.  Rounding is
    // monotone, so the row's largest |y| is (the largest |h * weight|) * r to the bit, and one
    // reduction gives both the sum and what an int8 row's scale needs.
    float ss = 0.0f, most = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float r8[8], w8[8];
        const int p = t + j * row_threads;
        unpack8<DT>(xv[j], h[j]);
        unpack8<DT>(rv[j], r8);
        unpack8<DT>(wv[j], w8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[j][e] += r8[e];
            ss = fmaf(h[j][e], h[j][e], ss);
        }
        if (a.residual_out && live && p < pieces)
            reinterpret_cast<uint4*>(a.residual_out + m * a.ldr)[p] = pack8<DT>(h[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.weight) h[j][e] *= w8[e];
            if (OUT == kNormI8) most = fmaxf(most, fabsf(h[j][e]));
        }
    }
    row_reduce<OUT == kNormI8>(ss, most, red, row_warp0, row_warps);
    float r = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
    // infinite for a zero row with eps = 0, whose 8-bit forms are zeros all the same: any finite r does
    if (OUT != kNormSame && r == INFINITY) r = 1.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] *= r;
    if constexpr (OUT == kNormSame) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = t + j * row_threads;
            if (live && p < pieces)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + m * a.ldy)[p] =
                    pack8<DT>(h[j]);
        }
    } else if constexpr (OUT == kNormI8) {
        most *= r;
        // NaN with an infinity or a NaN in the row, as r or r times the infinity is
        const float s = most == 0.0f ? 1.0f : __fdiv_rn(most, 127.0f);
        // y / s as y * (127 / most): 2^-23 off, like y itself; the division for each value took
        // half of the kernel's time.  The sum with 1.5 * 2^23 rounds to the nearest integer
        // (ties to even) and leaves it in the low byte.
        const float up = most < 1e-30f ? 0x1p64f : 1.0f;  // keeps the factor finite
        const float inv = most > 0.0f ? __fdiv_rn(127.0f, most * up) : 0.0f;
        uint2* y = reinterpret_cast<uint2*>(static_cast<int8_t*>(a.y) + m * a.H);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = t + j * row_threads;
            uint32_t q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(fmaf(h[j][e] * up, inv, 12582912.0f));
            const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
            if (live && p < pieces) y[p] = make_uint2(lo, hi);
        }
        if (live && t == 0) static_cast<float*>(a.scales)[m] = s;
    } else {
        uint2* y = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + m * a.H);
        uint8_t* sc = static_cast<uint8_t*>(a.scales) + m * (a.H / 32);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int p = t + j * row_threads;
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(h[j][e]));
            // a block of 32 is the pieces of four neighbouring lanes
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int e2 = norm_mx_exponent(top);
            const float f = norm_pow2(-e2);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = dec_e4m3x2(h[j][2 * e] * f, h[j][2 * e + 1] * f);
            if (live && p < pieces) {
                y[p] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
                if ((p & 3) == 0) sc[p >> 2] = static_cast<uint8_t>(e2 + 127);
            }
        }
    }
}

constexpr int kNormThreads = 256;

// Rows that are not 16-byte aligned, of a length that is no multiple of 8, or longer than
// 32768: one CTA per row, one value per thread and step, the row read twice (the second time
// from L1 or L2).  Bound by its many short loads: 800 x 4100 bf16 with residual 7.4 us, 3.5 TB/s.
template <int DT>
__global__ void __launch_bounds__(kNormThreads) norm_any_kernel(NormArgs a) {
    __shared__ float2 red[kNormThreads / 32];
    grid_dep_wait();
    const int64_t m = blockIdx.x;
    const uint16_t* x = a.x + m * a.ldx;
    const uint16_t* res = a.residual ? a.residual + m * a.ldr : nullptr;
    uint16_t* res_out = a.residual_out ? a.residual_out + m * a.ldr : nullptr;
    uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.ldy;
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
    float none = 0.0f;
    row_reduce<false>(ss, none, red, 0, kNormThreads / 32);
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.H) + a.eps);
    for (int i = threadIdx.x; i < a.H; i += kNormThreads) {
        const float h = value(i);
        const float w = a.weight ? dec_to_f32<DT>(a.weight[i]) : 1.0f;
        if (res_out) res_out[i] = dec_from_f32<DT>(h);
        y[i] = dec_from_f32<DT>(h * w * r);
    }
}

template <int DT, int OUT, int V>
int launch_norm_v(const NormArgs& a, int M, int row_threads, cudaStream_t stream) {
    // several short rows share a CTA
    const int rows = row_threads >= 256 ? 1 : 256 / row_threads;
    return launch_dependent(norm_kernel<DT, OUT, V>, dim3(blocks_for(M, rows)),
                            rows * row_threads, 0, stream, a, M, row_threads);
}

template <int DT, int OUT>
int launch_norm_out(const DeviceCtx& ctx, const NormArgs& a, int M, cudaStream_t stream) {
    const int pieces = a.H / 8;
    // Few rows: one piece per thread where 1024 threads suffice (latency).  Rows for every SM: two
    // (bf16 with residual, 800 x 4096: 4.6 us against 5.2 with one and 5.7 with four).  Long
    // rows, many of them: four, the most loads under way (4096 x 8192: 41.3 us against 47.5 and
    // 43.5; at 400 x 8192 5.7 against 5.8 and 4.9).
    int V = M <= ctx.num_sms || pieces < 64 ? 1 : pieces > 512 && M > 8 * ctx.num_sms ? 4 : 2;
    if (V * 1024 < pieces) V = pieces <= 2048 ? 2 : 4;
    const int row_threads = ((pieces + V - 1) / V + 31) / 32 * 32;
    if (V == 1) return launch_norm_v<DT, OUT, 1>(a, M, row_threads, stream);
    if (V == 2) return launch_norm_v<DT, OUT, 2>(a, M, row_threads, stream);
    return launch_norm_v<DT, OUT, 4>(a, M, row_threads, stream);
}

template <int DT>
int launch_norm_dt(const DeviceCtx& ctx, const NormArgs& a, int M, int out, cudaStream_t stream) {
    const uintptr_t bases = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                            reinterpret_cast<uintptr_t>(a.weight) |
                            reinterpret_cast<uintptr_t>(a.residual_out);
    if (out == kNormI8) return launch_norm_out<DT, kNormI8>(ctx, a, M, stream);
    if (out == kNormMx) return launch_norm_out<DT, kNormMx>(ctx, a, M, stream);
    const bool pieces = a.H % 8 == 0 && a.H <= 32768 && a.ldx % 8 == 0 && a.ldr % 8 == 0 &&
                        a.ldy % 8 == 0 && (bases | reinterpret_cast<uintptr_t>(a.y)) % 16 == 0;
    if (pieces) return launch_norm_out<DT, kNormSame>(ctx, a, M, stream);
    return launch_dependent(norm_any_kernel<DT>, dim3(static_cast<unsigned>(M)), kNormThreads, 0,
                            stream, a);
}

}  // namespace

int launch_norm(const DeviceCtx& ctx, const NormArgs& a, int M, int dtype, int out,
                cudaStream_t stream) {
    return dtype == 0 ? launch_norm_dt<0>(ctx, a, M, out, stream)
                      : launch_norm_dt<1>(ctx, a, M, out, stream);
}

}  // namespace w4g
