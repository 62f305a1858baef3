// Log probabilities of given tokens, entropy and largest logits (include/decode.h): one CTA per
// row; one pass for the maximum, one for the sums, one for each of the largest.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kLpThreads = 256;

template <int DT>
__device__ __forceinline__ float logit(const void* x, int64_t at) {
    if constexpr (DT == 2) return static_cast<const float*>(x)[at];
    else return dec_to_f32<DT>(static_cast<const uint16_t*>(x)[at]);
}

// Order of the largest: NaN above all, -0 as 0, the lower index first.
__device__ __forceinline__ uint64_t order_key(float v, int i) {
    uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
    b = v != v ? 0xFFFFFFFFu : b >> 31 ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(b) << 32 | (0x7FFFFFFFu - static_cast<uint32_t>(i));
}

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* red, F f) {
    for (int d = 16; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kLpThreads / 32; ++w) v = f(v, red[w]);
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(LogprobArgs a) {
    __shared__ float redf[kLpThreads / 32];
    __shared__ double redd[kLpThreads / 32];
    __shared__ uint64_t redk[kLpThreads / 32];
    grid_dep_wait();
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x, row = t * a.ld;
    const float f = a.factor ? a.factor[t] : 1.0f;
    const bool fine = f > 0.0f && f < INFINITY;
    float m = -INFINITY;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float v = logit<DT>(a.x, row + i) * f;
        m = v > m || v != v ? v : m;
    }
    m = block_reduce(m, redf, [](float x, float y) { return x != x ? x : y > x || y != y ? y : x; });
    double sum = 0.0, part = 0.0;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float z = logit<DT>(a.x, row + i) * f - m;
        const float e = expf(z);
        sum += e;
        if (e != 0.0f) part += e * z;
    }
    sum = block_reduce(sum, redd, [](double x, double y) { return x + y; });
    part = block_reduce(part, redd, [](double x, double y) { return x + y; });
    double lse = m + log(sum), entropy = log(sum) - part / sum;
    if (m == -INFINITY) lse = -INFINITY, entropy = 0.0;
    if (m == INFINITY) lse = INFINITY, entropy = NAN;
    if (m != m || !fine) lse = entropy = NAN;
    auto logprob = [&](float x) {
        return m == -INFINITY && fine ? -INFINITY : static_cast<float>(static_cast<double>(x * f) - lse);
    };
    if (tid == 0) {
        if (a.lse) a.lse[t] = static_cast<float>(lse);
        if (a.entropy) a.entropy[t] = static_cast<float>(entropy);
    }
    for (int c = tid; c < a.n_ids; c += kLpThreads) {
        const int id = a.ids[t * a.n_ids + c];
        if (id >= a.V) record_status(a.status, kDecInvalidArg);
        a.logprobs[t * a.n_ids + c] = id < 0 ? 0.0f : id >= a.V ? NAN : logprob(logit<DT>(a.x, row + id));
    }
    uint64_t below = ~0ull;
    for (int c = 0; c < a.top; ++c) {
        uint64_t best = 0;
        for (int i = tid; i < a.V; i += kLpThreads) {
            const uint64_t k = order_key(logit<DT>(a.x, row + i), i);
            if (k < below && k > best) best = k;
        }
        below = block_reduce(best, redk, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
        const int id = static_cast<int>(0x7FFFFFFFu - static_cast<uint32_t>(below));
        if (tid == 0) {
            a.top_ids[t * a.top + c] = id;
            if (a.top_logprobs) a.top_logprobs[t * a.top + c] = logprob(logit<DT>(a.x, row + id));
        }
    }
}

}  // namespace

int launch_logprob(const DeviceCtx&, const LogprobArgs& a, int dtype, cudaStream_t stream) {
    auto kern = dtype == 0 ? logprob_kernel<0> : dtype == 1 ? logprob_kernel<1> : logprob_kernel<2>;
    return launch_dependent(kern, dim3(static_cast<unsigned>(a.T)), dim3(kLpThreads), 0, stream, a);
}

}  // namespace w4g
