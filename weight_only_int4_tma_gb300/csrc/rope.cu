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

// Any rot_dim: one pair per thread; heads 0..q_heads-1 are queries, then keys, then values.  Bound by
// its 2-byte loads and stores and a division per pair (4096 tokens of 32 + 32 + 32 heads of 96 with 24
// turned, bf16: 0.15 GB in 78 us, 1.9 TB/s).
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

// x / s, rounded to nearest, given inv = 1 / s rounded to nearest: the product with inv, corrected by
// its remainder (Markstein: exact rounding for normal results).  x * inv alone moves one code in a
// million to the neighbour.  1003 tokens of 96 heads: 10.0 us, 9.3 by x * inv, 11.1 by division.
// Only quotients of 2^-12 .. 2^10 are corrected, beyond which E4M3 has no two numbers to choose
// from: an infinity would become a NaN, and -0 lose its sign.  inv has to be a normal number and the
// remainder's last bit (2^-48 of x) representable: 2^-80 <= |s| <= 2^80.
__device__ __forceinline__ float rope_quotient(float x, float s, float inv) {
    const float q = x * inv;
    const uint32_t lo = __float_as_uint(0x1p-12f), hi = __float_as_uint(0x1p10f);
    return __float_as_uint(fabsf(q)) - lo < hi - lo ? fmaf(fmaf(-q, s, x), inv, q) : q;
}

// Eight neighbouring values of a head, read once (evicted first: 1003 tokens of 96 heads 7 %
// less time).
template <int DT>
__device__ __forceinline__ void rope_load8(const uint16_t* p, float (&f)[8]) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] & 0xFFFFu));
        f[2 * j + 1] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] >> 16));
    }
}
template <int DT>
__device__ __forceinline__ uint4 rope_pack8(const float (&f)[8]) {
    return make_uint4(dec_pack2<DT>(f[0], f[1]), dec_pack2<DT>(f[2], f[3]),
                      dec_pack2<DT>(f[4], f[5]), dec_pack2<DT>(f[6], f[7]));
}

// How a token's work is cut: a unit is two 16-byte chunks of one head (one, where their number
// is odd), the two that a rotation in the half layout needs, or neighbours.  A CTA has
// blockDim.x threads (a multiple of 32) for each of blockDim.y tokens; grid: (groups of
// tokens, CTAs per group).
struct RopeUnits {
    int per_head;         // units of a head
    int rot_units;        // of those, the first ones, pairs (c, c + rot/16) of the half layout
    int chunks;           // chunks of a head
    int heads;            // queries, keys and, with a cache, values (without one v may be null)
    int head_shift;       // log2 of per_head, or -1; likewise of the page size: a division by
    int page_shift;       // a run-time number is a fifth of a unit's instructions
};

// One unit per thread, loaded and stored in 16-byte pieces; a token's position, slot and table
// row come through L1, which its threads share.  Bound by HBM for many tokens (2 + 2 bytes per
// value: 4096 tokens of 64 + 8 + 8 heads of 128, bf16, 0.17 GB in 30.7 us, 5.5 TB/s; with two tokens a
// thread 30.1 against 30.5; to an 8-bit cache 30.9, 5.2 TB/s), by the chain position -> table row -> store for few (one token 1.5 us in a
// graph).
template <int DT, bool E4M3>
__global__ void __launch_bounds__(128) rope_units_kernel(RopeArgs a, RopeUnits n) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int unit = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
    const int head = n.head_shift >= 0 ? unit >> n.head_shift : unit / n.per_head;
    const int u = unit - head * n.per_head;
    grid_dep_wait();
    if (t >= a.T || head >= n.heads) return;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.kv_heads;
    const int h = is_q ? head : is_v ? head - a.q_heads - a.kv_heads : head - a.q_heads;
    const int D = a.head_dim, half = a.rot_dim / 2;
    // the unit's chunks c0, c1 (c1 < 0: none) and whether each turns
    const bool paired = !is_v && u < n.rot_units;
    int c0 = paired ? u : 2 * u, c1 = paired ? u + n.rot_units : 2 * u + 1;
    if (c1 >= n.chunks) c1 = -1;
    const uint16_t* src = (is_q ? a.q + t * a.ldq : is_v ? a.v + t * a.ldv : a.k + t * a.ldk) +
                          static_cast<int64_t>(h) * D;
    float x0[8], x1[8];
    rope_load8<DT>(src + 8 * c0, x0);
    if (c1 >= 0) rope_load8<DT>(src + 8 * c1, x1);
    const int pos = a.positions[t];
    const int64_t wanted = a.kc.p && !is_q ? a.slots[t] : -1;
    if (pos < 0 || pos >= a.table_len) {
        record_status(a.status, kDecInvalidArg);
        return;
    }
    if (wanted >= a.num_slots && a.kc.p) record_status(a.status, kDecInvalidArg);
    const int64_t slot = wanted < a.num_slots ? wanted : -1;
    const float* cs = a.table + static_cast<int64_t>(pos) * a.rot_dim;
    if (paired) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 c = *reinterpret_cast<const float4*>(cs + 8 * u + 4 * q);
            const float4 s = *reinterpret_cast<const float4*>(cs + half + 8 * u + 4 * q);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = x0[4 * q + e], r = x1[4 * q + e];
                x0[4 * q + e] = p * cc[e] - r * ss[e];
                x1[4 * q + e] = r * cc[e] + p * ss[e];
            }
        }
    } else if (!is_v && a.layout == 1) {
        auto turn = [&](float (&x)[8], int chunk) {
            if (8 * chunk >= a.rot_dim) return;
            const float4 c = *reinterpret_cast<const float4*>(cs + 4 * chunk);
            const float4 s = *reinterpret_cast<const float4*>(cs + half + 4 * chunk);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = x[2 * e], r = x[2 * e + 1];
                x[2 * e] = p * cc[e] - r * ss[e];
                x[2 * e + 1] = r * cc[e] + p * ss[e];
            }
        };
        turn(x0, c0);
        if (c1 >= 0) turn(x1, c1);
    }
    if (is_q || (!is_v && a.k_out)) {
        uint16_t* dst = (is_q ? a.q_out + t * a.ldqo : a.k_out + t * a.ldko) + static_cast<int64_t>(h) * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = rope_pack8<DT>(x0);
        if (c1 >= 0) *reinterpret_cast<uint4*>(dst + 8 * c1) = rope_pack8<DT>(x1);
    }
    if (slot < 0) return;
    const KvView& kv = is_v ? a.vc : a.kc;
    const int64_t page = n.page_shift >= 0 ? slot >> n.page_shift : slot / a.page_size;
    const int64_t off = page * kv.page_stride + (slot - page * a.page_size) * kv.slot_stride + h * kv.head_stride;
    if constexpr (E4M3) {
        float s = kv.scale ? kv.scale[h] : 1.0f;
        if (!(fabsf(s) >= 0x1p-80f && fabsf(s) <= 0x1p80f)) {
            // the same quotients of numbers by a power of two off, exact where a quotient is in range
            const float by = fabsf(s) < 1.0f ? 0x1p100f : 0x1p-100f;
            s *= by;
#pragma unroll
            for (int e = 0; e < 8; ++e) x0[e] *= by, x1[e] *= by;
        }
        const float inv = __frcp_rn(s);
        auto pack = [&](const float (&x)[8]) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = dec_e4m3x2(rope_quotient(x[2 * e], s, inv), rope_quotient(x[2 * e + 1], s, inv));
            return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        };
        uint8_t* dst = static_cast<uint8_t*>(kv.p) + off;
        *reinterpret_cast<uint2*>(dst + 8 * c0) = pack(x0);
        if (c1 >= 0) *reinterpret_cast<uint2*>(dst + 8 * c1) = pack(x1);
    } else {
        uint16_t* dst = static_cast<uint16_t*>(kv.p) + off;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = rope_pack8<DT>(x0);
        if (c1 >= 0) *reinterpret_cast<uint4*>(dst + 8 * c1) = rope_pack8<DT>(x1);
    }
}

}  // namespace

int launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
    const int64_t n = (static_cast<int64_t>(a.table_len) * (a.rot_dim / 2) + 255) / 256;
    const unsigned blocks = static_cast<unsigned>(n < 16384 ? n : 16384);
    return launch_dependent(rope_table_kernel, dim3(blocks), dim3(256), 0, stream, a);
}

int launch_rope(const DeviceCtx& ctx, const RopeArgs& a, int dtype, bool e4m3,
                cudaStream_t stream) {
    (void)ctx;
    // Whole chunks turn: rot_dim / 2 of whole chunks in the half layout, rot_dim in the other.
    const bool whole = a.layout == 0 ? a.rot_dim % 16 == 0 : a.rot_dim % 8 == 0;
    if (whole) {
        RopeUnits n{};
        n.chunks = a.head_dim / 8;
        n.rot_units = a.layout == 0 ? a.rot_dim / 16 : 0;
        n.per_head = (n.chunks + 1) / 2;
        n.heads = a.q_heads + a.kv_heads * (a.kc.p ? 2 : 1);
        const int units = n.per_head * n.heads;
        n.head_shift = power_of_two(n.per_head);
        n.page_shift = power_of_two(a.page_size);
        // as few idle threads as whole warps allow: 640 units (64 + 8 + 8 heads of 128) in five
        // CTAs of 128 rather than three of 224 (4096 tokens: 30.7 against 33.7 us)
        const int blocks = (units + 127) / 128;
        const int threads = ((units + blocks - 1) / blocks + 31) / 32 * 32;
        const int tokens = blocks > 1 ? 1 : 128 / threads;
        auto kern = dtype == 0 ? (e4m3 ? rope_units_kernel<0, true> : rope_units_kernel<0, false>)
                               : (e4m3 ? rope_units_kernel<1, true> : rope_units_kernel<1, false>);
        if (blocks <= 65535)
            return launch_dependent(kern, dim3(blocks_for(a.T, tokens),
                                               static_cast<unsigned>(blocks)),
                                    dim3(threads, tokens), 0, stream, a, n);
    }
    const dim3 grid(static_cast<unsigned>(a.T));
    auto kern = dtype == 0 ? (e4m3 ? rope_kernel<0, true> : rope_kernel<0, false>)
                           : (e4m3 ? rope_kernel<1, true> : rope_kernel<1, false>);
    return launch_dependent(kern, grid, dim3(kRopeThreads), 0, stream, a);
}

}  // namespace w4g
