// Rotary positions with the append to a paged key-value cache, and the table of cosines and
// sines (include/decode.h).  Pair j of a head turns by pos * f(j): (a cos - b sin, b cos +
// a sin), in fp32 from the table's fp32 cosines and sines, rounded once to the stored type.
#include "decode.cuh"

namespace w4g {
namespace {

// f(j) = base^(-2j/rot), scaled; the angle, its cosine and sine in fp64 (a position of 10^5
// or more times a frequency near 1 needs the bits), rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(RopeTableArgs a) {
    grid_dep_wait();
    const int half = a.rot_dim / 2;
    const int64_t n = static_cast<int64_t>(a.table_len) * half;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
        const int64_t pos = i / half;
        const int j = static_cast<int>(i - pos * half);
        double base = a.base;
        if (a.kind == 2) base *= pow(a.factor, a.rot_dim / (a.rot_dim - 2.0));
        double f = pow(base, -2.0 * j / a.rot_dim);
        if (a.kind == 1) f /= a.factor;
        if (a.kind == 3) {
            const double turns = a.original_len * f / 6.283185307179586476925286766559;
            const double w = fmin(1.0, fmax(0.0, (turns - a.low) / (a.high - a.low)));
            f = w * f + (1.0 - w) * f / a.factor;
        }
        double s, c;
        sincos(static_cast<double>(pos) * f, &s, &c);
        float* row = a.table + pos * a.rot_dim;
        row[j] = static_cast<float>(a.magnitude * c);
        row[half + j] = static_cast<float>(a.magnitude * s);
    }
}

constexpr int kRopeThreads = 256;

// One value per thread: heads 0..q_heads-1 are queries, then keys, then values.
template <int DT, bool E4M3>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    grid_dep_wait();
    const int t = static_cast<int>(blockIdx.x);
    const int D = a.head_dim, half = a.rot_dim / 2;
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.table_len) {
        if (threadIdx.x == 0) record_status(a.status, kDecInvalidArg);
        return;
    }
    int64_t slot = -1;
    if (a.kc.p) {
        slot = a.slots[t];
        if (slot >= a.num_slots) {
            if (threadIdx.x == 0) record_status(a.status, kDecInvalidArg);
            slot = -1;
        }
    }
    const int64_t page = slot >= 0 ? slot / a.page_size : 0;
    const int64_t in_page = slot >= 0 ? slot - page * a.page_size : 0;
    const float* cs = a.table + static_cast<int64_t>(pos) * a.rot_dim;
    const int units = (a.q_heads + 2 * a.kv_heads) * (D / 2);
    // a unit is a pair of one head: the rotated pairs first, then pairs of neighbours
    for (int u = threadIdx.x; u < units; u += kRopeThreads) {
        const int head = u / (D / 2), j = u - head * (D / 2);
        const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.kv_heads;
        const int h = is_q ? head : is_v ? head - a.q_heads - a.kv_heads : head - a.q_heads;
        if (is_v && slot < 0) continue;
        const uint16_t* src = is_q ? a.q + t * a.ldq : is_v ? a.v + t * a.ldv : a.k + t * a.ldk;
        src += static_cast<int64_t>(h) * D;
        int i0 = 2 * j, i1 = 2 * j + 1;
        if (j < half && a.layout == 0) { i0 = j; i1 = j + half; }
        float x0 = dec_to_f32<DT>(src[i0]), x1 = dec_to_f32<DT>(src[i1]);
        if (j < half && !is_v) {
            const float c = cs[j], s = cs[half + j];
            const float y0 = x0 * c - x1 * s;
            x1 = x1 * c + x0 * s;
            x0 = y0;
        }
        if (is_q || (!is_v && a.k_out)) {
            uint16_t* dst = (is_q ? a.q_out + t * a.ldqo : a.k_out + t * a.ldko) +
                            static_cast<int64_t>(h) * D;
            dst[i0] = dec_from_f32<DT>(x0);
            dst[i1] = dec_from_f32<DT>(x1);
        }
        if (!is_q && slot >= 0) {
            const KvView& c = is_v ? a.vc : a.kc;
            const int64_t off = page * c.page_stride + in_page * c.slot_stride + h * c.head_stride;
            if constexpr (E4M3) {
                const float s = c.scale ? c.scale[h] : 1.0f;
                const uint32_t p = dec_e4m3x2(__fdiv_rn(x0, s), __fdiv_rn(x1, s));
                static_cast<uint8_t*>(c.p)[off + i0] = static_cast<uint8_t>(p);
                static_cast<uint8_t*>(c.p)[off + i1] = static_cast<uint8_t>(p >> 8);
            } else {
                static_cast<uint16_t*>(c.p)[off + i0] = dec_from_f32<DT>(x0);
                static_cast<uint16_t*>(c.p)[off + i1] = dec_from_f32<DT>(x1);
            }
        }
    }
}

}  // namespace

int launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
    const int64_t n = (static_cast<int64_t>(a.table_len) * (a.rot_dim / 2) + 255) / 256;
    const unsigned blocks = static_cast<unsigned>(n < 16384 ? n : 16384);
    return launch_dependent(rope_table_kernel, dim3(blocks), 256, 0, stream, a);
}

int launch_rope(const DeviceCtx& ctx, const RopeArgs& a, int dtype, bool e4m3,
                cudaStream_t stream) {
    (void)ctx;
    const dim3 grid(static_cast<unsigned>(a.T));
    auto kern = dtype == 0 ? (e4m3 ? rope_kernel<0, true> : rope_kernel<0, false>)
                           : (e4m3 ? rope_kernel<1, true> : rope_kernel<1, false>);
    return launch_dependent(kern, grid, kRopeThreads, 0, stream, a);
}

}  // namespace w4g
