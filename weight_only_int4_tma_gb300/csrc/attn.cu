// Attention of one new token per sequence over a paged key-value cache (include/decode.h):
//   s_j = scale q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j)  over the visible tokens.
//
// The keys and values are read once and nothing else of size is: with G query heads per
// key-value head the work is 2 G operations per cached 16-bit value, far below what the
// tensor cores do in the time of the read, so the kernel is built to keep loads in flight.
//
// Data path.  A warp takes steps of 16 R tokens.  Its keys and values go from global memory
// straight into the registers of an mma.sync operand, 16 bytes a lane and load, with no
// shared memory and no barrier between the warps:
//   S^T = K Q^T   (tokens are the MMA's 16 rows, query heads its 8 columns): lane 4g + i
//                 holds tokens g and g + 8; the 16 bytes it loads of a key row are two (four
//                 for 8-bit caches) of the MMA's K steps.  The K index of an MMA is a sum's
//                 index, so any order serves if the queries use the same one.
//   O^T = V^T P^T (head dimensions are the rows): lane 4g + i holds tokens 2i, 2i+1, 2i+8,
//                 2i+9 at eight neighbouring dimensions; byte permutes pair the tokens.
//                 Dimension pairs of an MMA's rows g, g + 8 are (2j, 2j + 1) of the lane's
//                 eight, an order that only the store has to know.
// The probabilities leave S^T with tokens in rows and are wanted with tokens as the K index:
// one 8 x 8 transpose of 16-bit pairs (movmatrix).  They are split in a high and a low
// 16-bit part, each multiplied with V: a single 16-bit rounding of P (2^-9 for bf16) would
// show in the result as much as the result's own.
//
// Softmax.  One pass with a running reference m per query head: weights are exp2(s - m), and
// when a score passes m by more than 2^8 the sums so far are scaled to the new reference
// (a warp vote finds out; exact in the end, since numerator and denominator share it).
//
// Work split.  The steps of all (sequence, head, row tile) items stand in one line that is
// cut into equal shares, one per CTA, whatever the lengths; every CTA finds its share from
// the lengths on the device.  An item inside one CTA is finished there; one that is cut
// leaves (m, l, O) in fp32 in the workspace, and the CTA that arrives last joins the parts
// in their order.
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kMaxCtasPerSm = 6;   // no instance runs more (the workspace's layout)
constexpr float kLag = 8.0f;       // scores may pass the reference by 2^8

__device__ __forceinline__ uint4 ldg16(const char* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg8(const char* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// D += A B, 16 x 8 x 16, fp32 accumulate; BF: bf16 operands, else fp16.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// DT: 0 fp16, 1 bf16 (queries, output).  E4M3: 8-bit cache.  DP: head dimension rounded up
// to 64, 128 or 256.  NT: tiles of 8 query heads that a CTA takes at once.  R: groups of 16
// tokens per step.  P16: the page size is a multiple of 16, so a group lies in one page.
template <int DT_, bool E4M3_, int DP_, int NT_, int R_, bool P16_, int OCC_>
struct AttnShape {
    static constexpr int DT = DT_, DP = DP_, NT = NT_, R = R_, OCC = OCC_;
    static constexpr bool E4M3 = E4M3_, P16 = P16_;
    static constexpr bool BF = DT == 1 && !E4M3;  // type of the MMA's operands
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int ROWS = 8 * NT;
    static constexpr int STEP = 16 * R;
    static constexpr int KL = DP * ES / 64;   // 16-byte loads of a key row per lane
    static constexpr int VC = DP / 64;        // loads of a value row per lane (16 or 8 bytes)
    static constexpr int VW = E4M3 ? 2 : 4;   // words of one
    static constexpr int MS = DP / 16;        // MMA steps over the head dimension
    static constexpr int Q_BYTES = NT * MS * 32 * 8;
    static constexpr int O_FLOATS = kAttnWarps * ROWS * DP;
    static constexpr int SMEM = Q_BYTES + 4 * O_FLOATS;
    // a join keeps one factor per part and row where the warps' sums stood before
    static_assert(kAttnWarps * DP >= 64, "at most 57 parts in one round");
};

// Where the parts of one CTA stand in the workspace: counters first (three times as many
// as any instance has CTAs, so that calls of different instances may share a workspace), then for each CTA two
// parts (its first item if that began in an earlier CTA, its last if that ends in a later
// one) of m[ROWS], l[ROWS], O[ROWS][DP].
__host__ __device__ constexpr size_t part_floats(int rows, int dp) {
    return static_cast<size_t>(rows) * (dp + 2);
}
__host__ __device__ constexpr size_t counter_bytes(int ctas) {
    return (static_cast<size_t>(ctas) * 4 + 127) / 128 * 128;
}

// Visible tokens [first, len) of sequence b.
struct Span {
    int first, len;
};
__device__ __forceinline__ Span visible(const AttnArgs& a, int b, bool report) {
    int len = a.lens[b];
    const int most = a.max_pages * a.page_size;
    if (len < 0 || len > most) {
        if (report) record_status(a.status, kDecInvalidArg);
        len = len < 0 ? 0 : most;
    }
    return {a.window > 0 && len > a.window ? len - a.window : 0, len};
}
template <int STEP>
__device__ __forceinline__ int span_steps(Span s) {
    return s.len == 0 ? 0 : (s.len + STEP - 1) / STEP - s.first / STEP;
}

// a / b; the long division only where 32 bits do not hold the numbers.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0)
        return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

template <class S>
__global__ void __launch_bounds__(kAttnThreads, S::OCC) attn_kernel(AttnArgs a, int page_shift) {
    constexpr int NT = S::NT, R = S::R, DP = S::DP, ROWS = S::ROWS, STEP = S::STEP;
    extern __shared__ __align__(16) unsigned char smem[];
    uint2* qs = reinterpret_cast<uint2*>(smem);                  // [NT][MS][32] B fragments
    float* so = reinterpret_cast<float*>(smem + S::Q_BYTES);     // [warp][ROWS][DP]
    __shared__ float sfct[ROWS];                                 // score factor of each row
    __shared__ float sm_m[kAttnWarps][ROWS], sm_l[kAttnWarps][ROWS];
    __shared__ float row_m[ROWS], row_l[ROWS];
    __shared__ long long scan[kAttnWarps];
    __shared__ int find_b;
    __shared__ long long find_u;
    __shared__ int is_last;

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, i = lane & 3;
    const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    const int G = a.q_heads / a.kv_heads;
    const int row_tiles = (G + ROWS - 1) / ROWS;
    const int items_per_seq = a.kv_heads * row_tiles;

    grid_dep_wait();
    // ---- this CTA's share of the line of steps ----
    const int per_thread = (a.B + kAttnThreads - 1) / kAttnThreads;
    const int b_lo = min(a.B, tid * per_thread), b_hi = min(a.B, b_lo + per_thread);
    long long mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += span_steps<STEP>(visible(a, b, cta == 0));
    mine *= items_per_seq;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    // whole rounds of the warps: a share of fewer steps would take as long
    const long long rounds = quotient(total + ctas * kAttnWarps - 1, ctas * kAttnWarps);
    const long long share = max(rounds, 1ll) * kAttnWarps;
    long long u = share * cta;
    const long long u_end = min(total, u + share);
    const long long excl = before + incl - mine;
    if (u < u_end && excl <= u && u < excl + mine) {  // one thread at most
        long long at = excl;
        int b = b_lo;
        for (; b + 1 < b_hi; ++b) {
            const long long n = static_cast<long long>(span_steps<STEP>(visible(a, b, false))) * items_per_seq;
            if (u < at + n) break;
            at += n;
        }
        find_b = b;
        find_u = u - at;
    }
    // rows with nothing to attend to
    for (int b = cta; b < a.B; b += ctas) {
        if (visible(a, b, false).len != 0) continue;
        uint16_t* o = a.out + b * a.ldo;
        for (int e = tid; e < a.q_heads * a.head_dim; e += kAttnThreads) o[e] = 0;
        if (a.lse)
            for (int h = tid; h < a.q_heads; h += kAttnThreads)
                a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
    }
    __syncthreads();
    if (u >= u_end) return;
    int b = find_b;
    Span span = visible(a, b, false);
    int n_steps = span_steps<STEP>(span);
    int item = static_cast<int>(quotient(find_u, n_steps));
    int step = static_cast<int>(find_u - static_cast<long long>(item) * n_steps);

    int* counters = static_cast<int*>(a.workspace);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + counter_bytes(3 * a.max_ctas));
    const uint32_t row_bytes = static_cast<uint32_t>(a.head_dim) * S::ES;

    while (u < u_end) {
        // ---- one item's steps [step, step_end) ----
        const int step_end = static_cast<int>(min(static_cast<long long>(n_steps), step + (u_end - u)));
        const int kvh = item / row_tiles, row0 = (item - kvh * row_tiles) * ROWS;
        const int rows = min(ROWS, G - row0);
        const int head0 = kvh * G + row0;
        const float ks = S::E4M3 && a.kc.scale ? a.kc.scale[kvh] : 1.0f;
        const float vs = S::E4M3 && a.vc.scale ? a.vc.scale[kvh] : 1.0f;

        // queries as B fragments: lane (g, i) of MMA step st holds four values of row 8 nt + g.
        // With an 8-bit cache the MMA is fp16: bf16 queries are scaled there by a power of
        // two per row that brings the largest to 2^8..2^9, undone in the row's factor.
        const uint16_t* qrow = a.q + b * a.ldq + static_cast<int64_t>(head0) * a.head_dim;
        for (int r = warp; r < ROWS; r += kAttnWarps) {
            float f = a.scale * 1.4426950408889634f * ks, qscale = 1.0f;
            if constexpr (S::E4M3 && S::DT == 1) {
                float most = 0.0f;
                if (r < rows)
                    for (int d = lane; d < a.head_dim; d += 32)
                        most = fmaxf(most, fabsf(dec_to_f32<1>(qrow[static_cast<int64_t>(r) * a.head_dim + d])));
                most = warp_max(most);
                const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
                if (most > 0.0f && e > -119) {
                    qscale = __uint_as_float(static_cast<uint32_t>(8 - e + 127) << 23);
                    f *= __uint_as_float(static_cast<uint32_t>(e - 8 + 127) << 23);
                }
            }
            for (int n = lane; n < S::MS * 4; n += 32) {  // (MMA step, i) of this row
                const int st = n >> 2, qi = n & 3;
                const int col = S::E4M3 ? 64 * (st >> 2) + 16 * qi + 4 * (st & 3)
                                        : 32 * (st >> 1) + 8 * qi + 4 * (st & 1);
                uint2 v = make_uint2(0, 0);
                if (r < rows && col < a.head_dim)
                    v = *reinterpret_cast<const uint2*>(qrow + static_cast<int64_t>(r) * a.head_dim + col);
                if constexpr (S::E4M3 && S::DT == 1) {
                    v.x = dec_pack2<0>(__uint_as_float(v.x << 16) * qscale,
                                       __uint_as_float(v.x & 0xFFFF0000u) * qscale);
                    v.y = dec_pack2<0>(__uint_as_float(v.y << 16) * qscale,
                                       __uint_as_float(v.y & 0xFFFF0000u) * qscale);
                }
                qs[((r >> 3) * S::MS + st) * 32 + 4 * (r & 7) + qi] = v;
            }
            if (lane == 0) sfct[r] = f;
        }
        __syncthreads();
        float fct[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) fct[nt][c] = sfct[8 * nt + 2 * i + c];

        // ---- the warp's steps ----
        float m[NT][2], l[NT][2], o[NT][S::MS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) m[nt][c] = -INFINITY, l[nt][c] = 0.0f;
#pragma unroll
            for (int s = 0; s < S::MS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.0f;
        }
        uint32_t kr[R][2][4 * S::KL], vr[R][4][S::VC * S::VW];
        const int32_t* table = a.block_table + b * a.ld_table;
        const char* kbase = static_cast<const char*>(a.kc.p) + kvh * a.kc.head_stride * S::ES;
        const char* vbase = static_cast<const char*>(a.vc.p) + kvh * a.vc.head_stride * S::ES;
        const int64_t kss = a.kc.slot_stride * S::ES, vss = a.vc.slot_stride * S::ES;
        const int64_t kps = a.kc.page_stride * S::ES, vps = a.vc.page_stride * S::ES;
        const int st0 = span.first / STEP + step, st1 = span.first / STEP + step_end;

        // Page numbers one step ahead of the loads that need them.  P16: one per group,
        // the same in every lane; else lane t's is that of the step's token t.
        constexpr int NP = S::P16 ? R : 1;
        int pid[NP];
        auto page_of = [&](int tok) { return page_shift >= 0 ? tok >> page_shift : tok / a.page_size; };
        auto fetch_pages = [&](int st) {
#pragma unroll
            for (int r = 0; r < NP; ++r) {
                const int tok = S::P16 ? st * STEP + 16 * r : st * STEP + lane;
                const bool in = st < st1 && tok < span.len &&
                                (S::P16 ? tok + 16 > span.first : lane < STEP && tok >= span.first);
                pid[r] = in ? table[page_of(tok)] : 0;
            }
        };
        // Addresses of a step's rows.  P16: per group, the pointers of its first row (null:
        // nothing to read); else per lane, those of its own token's rows.
        const char* kp[NP];
        const char* vp[NP];
        auto locate = [&](int st) {
#pragma unroll
            for (int r = 0; r < NP; ++r) {
                const int tok = S::P16 ? st * STEP + 16 * r : st * STEP + lane;
                const bool in = tok < span.len &&
                                (S::P16 ? tok + 16 > span.first : lane < STEP && tok >= span.first);
                const bool ok = in && static_cast<unsigned>(pid[r]) < static_cast<unsigned>(a.num_pages);
                if (in && !ok) record_status(a.status, kDecInvalidArg);
                const int slot = tok - page_of(tok) * a.page_size;
                kp[r] = ok ? kbase + pid[r] * kps + slot * kss : nullptr;
                vp[r] = ok ? vbase + pid[r] * vps + slot * vss : nullptr;
            }
        };
        auto row_ptr = [&](const char* const (&p)[NP], int64_t stride, int r, int t) -> const char* {
            if constexpr (S::P16) {
                return p[r] ? p[r] + t * stride : nullptr;
            } else {
                return reinterpret_cast<const char*>(
                    __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(p[0]), 16 * r + t));
            }
        };
        auto in_span = [&](int tok) { return tok >= span.first && tok < span.len; };
        auto load_k = [&](int st) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = g + 8 * h;
                    const char* p = row_ptr(kp, kss, r, t);
                    const bool ok = p != nullptr && in_span(st * STEP + 16 * r + t);
#pragma unroll
                    for (int c = 0; c < S::KL; ++c) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (ok && 64 * c + 16 * i < row_bytes) v = ldg16(p + 64 * c + 16 * i);
                        kr[r][h][4 * c] = v.x, kr[r][h][4 * c + 1] = v.y;
                        kr[r][h][4 * c + 2] = v.z, kr[r][h][4 * c + 3] = v.w;
                    }
                }
        };
        auto load_v = [&](int st) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int t = 2 * i + (h & 1) + 8 * (h >> 1);
                    const char* p = row_ptr(vp, vss, r, t);
                    const bool ok = p != nullptr && in_span(st * STEP + 16 * r + t);
#pragma unroll
                    for (int c = 0; c < S::VC; ++c) {
                        if constexpr (S::E4M3) {
                            uint2 v = make_uint2(0, 0);
                            if (ok && 64 * c + 8 * g < row_bytes) v = ldg8(p + 64 * c + 8 * g);
                            vr[r][h][2 * c] = v.x, vr[r][h][2 * c + 1] = v.y;
                        } else {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (ok && 128 * c + 16 * g < row_bytes) v = ldg16(p + 128 * c + 16 * g);
                            vr[r][h][4 * c] = v.x, vr[r][h][4 * c + 1] = v.y;
                            vr[r][h][4 * c + 2] = v.z, vr[r][h][4 * c + 3] = v.w;
                        }
                    }
                }
        };

        int st = st0 + warp;
        if (st < st1) {
            fetch_pages(st);
            locate(st);
            load_k(st);
            load_v(st);
            fetch_pages(st + kAttnWarps);
        }
        for (; st < st1; st += kAttnWarps) {
            const bool more = st + kAttnWarps < st1;
            // tokens of this step that count, bit 2r + h: group r, row g + 8h
            uint32_t live = 0;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool there = row_ptr(kp, 0, r, g + 8 * h) != nullptr;
                    if (there && in_span(st * STEP + 16 * r + g + 8 * h)) live |= 1u << (2 * r + h);
                }
            float s[R][NT][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][nt][e] = 0.0f;
#pragma unroll
                for (int ms = 0; ms < S::MS; ++ms) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (S::E4M3) {
                        a0 = dec_e4m3x2_to_f16x2(kr[r][0][ms]);
                        a1 = dec_e4m3x2_to_f16x2(kr[r][1][ms]);
                        a2 = dec_e4m3x2_to_f16x2(kr[r][0][ms] >> 16);
                        a3 = dec_e4m3x2_to_f16x2(kr[r][1][ms] >> 16);
                    } else {
                        a0 = kr[r][0][2 * ms], a1 = kr[r][1][2 * ms];
                        a2 = kr[r][0][2 * ms + 1], a3 = kr[r][1][2 * ms + 1];
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = qs[(nt * S::MS + ms) * 32 + lane];
                        mma16816<S::BF>(s[r][nt], a0, a1, a2, a3, q.x, q.y);
                    }
                }
            }
            if (more) {
                locate(st + kAttnWarps);
                load_k(st + kAttnWarps);
                fetch_pages(st + 2 * kAttnWarps);
            }
            // scores in units of log 2; those of tokens that do not count are -inf
            bool passed = false;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool counts = (live >> (2 * r + (e >> 1))) & 1u;
                        s[r][nt][e] = counts ? s[r][nt][e] * fct[nt][e & 1] : -INFINITY;
                        passed |= s[r][nt][e] > m[nt][e & 1] + kLag;
                    }
            if (__any_sync(0xFFFFFFFFu, passed)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = m[nt][c];
#pragma unroll
                        for (int r = 0; r < R; ++r) top = fmaxf(top, fmaxf(s[r][nt][c], s[r][nt][c + 2]));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const float f = top == m[nt][c] ? 1.0f : exp2_fast(m[nt][c] - top);
                        m[nt][c] = top;
                        l[nt][c] *= f;
#pragma unroll
                        for (int ms = 0; ms < S::MS; ++ms) {
                            o[nt][ms][c] *= f;
                            o[nt][ms][c + 2] *= f;
                        }
                    }
            }
            // weights, split in 16-bit parts, as B fragments.  fp16 keeps 2^-14 as its
            // smallest full number: its weights are scaled by 2^7 (at most 2^15 with the lag).
            constexpr float kShift = S::BF ? 0.0f : 7.0f;
            uint32_t ph[R][NT][2], pl[R][NT][2];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p[2], low[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float ref = m[nt][c] == -INFINITY ? 0.0f : m[nt][c] - kShift;
                            p[c] = exp2_fast(s[r][nt][2 * h + c] - ref);
                            l[nt][c] += p[c];
                        }
                        const uint32_t hi = dec_pack2<S::BF ? 1 : 0>(p[0], p[1]);
                        low[0] = p[0] - dec_to_f32<S::BF ? 1 : 0>(static_cast<uint16_t>(hi & 0xFFFFu));
                        low[1] = p[1] - dec_to_f32<S::BF ? 1 : 0>(static_cast<uint16_t>(hi >> 16));
                        ph[r][nt][h] = transpose8x8(hi);
                        pl[r][nt][h] = transpose8x8(dec_pack2<S::BF ? 1 : 0>(low[0], low[1]));
                    }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int ms = 0; ms < S::MS; ++ms) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (S::E4M3) {
                        const int w = 2 * (ms >> 2) + ((ms >> 1) & 1);
                        const uint32_t sel = (ms & 1) ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(vr[r][0][w], vr[r][1][w], sel);
                        const uint32_t y = __byte_perm(vr[r][2][w], vr[r][3][w], sel);
                        a0 = dec_e4m3x2_to_f16x2(x), a1 = dec_e4m3x2_to_f16x2(x >> 16);
                        a2 = dec_e4m3x2_to_f16x2(y), a3 = dec_e4m3x2_to_f16x2(y >> 16);
                    } else {
                        a0 = __byte_perm(vr[r][0][ms], vr[r][1][ms], 0x5410);
                        a1 = __byte_perm(vr[r][0][ms], vr[r][1][ms], 0x7632);
                        a2 = __byte_perm(vr[r][2][ms], vr[r][3][ms], 0x5410);
                        a3 = __byte_perm(vr[r][2][ms], vr[r][3][ms], 0x7632);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<S::BF>(o[nt][ms], a0, a1, a2, a3, ph[r][nt][0], ph[r][nt][1]);
                        mma16816<S::BF>(o[nt][ms], a0, a1, a2, a3, pl[r][nt][0], pl[r][nt][1]);
                    }
                }
            if (more) load_v(st + kAttnWarps);
        }

        // ---- join the warps ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[nt][c];
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
                const int row = 8 * nt + 2 * i + c;
                if (g == 0) sm_m[warp][row] = m[nt][c], sm_l[warp][row] = v;
                if (row < rows) {
                    float* dst = so + (warp * ROWS + row) * DP;
#pragma unroll
                    for (int ms = 0; ms < S::MS; ++ms)
                        *reinterpret_cast<float2*>(dst + 64 * (ms >> 2) + 8 * g + 2 * (ms & 3)) =
                            make_float2(o[nt][ms][c], o[nt][ms][c + 2]);
                }
            }
        __syncthreads();
        const bool begins = step == 0, ends = step_end == n_steps;
        const bool whole = begins && ends;
        float* part = parts + (2 * cta + (begins ? 1 : 0)) * part_floats(ROWS, DP);
        if (tid < ROWS) {
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sm_m[w][tid]);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = top == -INFINITY ? 0.0f : exp2_fast(sm_m[w][tid] - top);
                sum += sm_l[w][tid] * f;
                sm_m[w][tid] = f;  // from here on the warp's factor
            }
            row_m[tid] = top;
            row_l[tid] = sum;
            if (!whole) part[tid] = top, part[ROWS + tid] = sum;
        }
        __syncthreads();
        const int words = a.head_dim / 2;  // stores of two values
        auto store = [&](int row, int d, float x, float y, float sum) {
            const float f = sum > 0.0f ? vs / sum : 0.0f;
            uint16_t* dst = a.out + b * a.ldo + static_cast<int64_t>(head0 + row) * a.head_dim + d;
            *reinterpret_cast<uint32_t*>(dst) = dec_pack2<S::DT>(x * f, y * f);
        };
        auto store_lse = [&](int row, float top, float sum) {
            constexpr float kShift = S::BF ? 0.0f : 7.0f;
            if (a.lse)
                a.lse[static_cast<int64_t>(b) * a.q_heads + head0 + row] =
                    sum > 0.0f ? (top - kShift) * 0.69314718055994531f + logf(sum) : -INFINITY;
        };
        for (int e = tid; e < rows * words; e += kAttnThreads) {
            const int row = e / words, d = 2 * (e - row * words);
            float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float2 x = *reinterpret_cast<const float2*>(so + (w * ROWS + row) * DP + d);
                v.x += x.x * sm_m[w][row];
                v.y += x.y * sm_m[w][row];
            }
            if (whole) store(row, d, v.x, v.y, row_l[row]);
            else *reinterpret_cast<float2*>(part + 2 * ROWS + row * DP + d) = v;
        }
        if (whole) {
            if (tid < rows) store_lse(tid, row_m[tid], row_l[tid]);
        } else {
            // ---- join the CTAs: the last one to arrive reads the others' parts, in order ----
            // Many parts are joined in two rounds, runs of `fan` first: one CTA reads about
            // 0.1 TB/s, and 456 parts of 8 rows and 128 dimensions are 1.9 MB.
            const int c0 = static_cast<int>(quotient(u - step, share));
            const int n = static_cast<int>(quotient(u - step + n_steps - 1, share)) - c0 + 1;
            const int fan = n <= 16 ? n : n <= 256 ? 16 : 32;
            auto part_of = [&](int k) {  // part k of the item
                return parts + (2 * (c0 + k) + (k == 0 ? 1 : 0)) * part_floats(ROWS, DP);
            };
            // true in every thread of the CTA that completes the counter's `want` arrivals
            auto arrive = [&](int* counter, int want) {
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    is_last = atomicAdd(counter, 1) == want - 1;
                    if (is_last) *counter = 0;  // ready for the next call
                    __threadfence();
                }
                __syncthreads();
                return is_last != 0;
            };
            // parts k0, k0 + stride, ... (count of them) into one: written over part k0, or
            // stored as the result
            auto join = [&](int k0, int stride, int count, bool final) {
                for (int row = warp; row < rows; row += kAttnWarps) {
                    float top = -INFINITY;
                    for (int k = lane; k < count; k += 32)
                        top = fmaxf(top, __ldcg(part_of(k0 + k * stride) + row));
                    top = warp_max(top);
                    float sum = 0.0f;
                    for (int k = lane; k < count; k += 32) {
                        const float* p = part_of(k0 + k * stride);
                        const float f = top == -INFINITY ? 0.0f : exp2_fast(__ldcg(p + row) - top);
                        sum += f * __ldcg(p + ROWS + row);
                        so[k * ROWS + row] = f;  // count <= kMaxFan of them
                    }
                    sum = warp_sum(sum);
                    if (lane == 0) row_m[row] = top, row_l[row] = sum;
                }
                __syncthreads();
                float* to = part_of(k0);
                for (int e = tid; e < rows * (DP / 4); e += kAttnThreads) {
                    const int row = e / (DP / 4), d = 4 * (e % (DP / 4));
                    if (d >= a.head_dim) continue;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int k = 0; k < count; k += 8) {
                        float4 x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = k + j < count ? __ldcg(reinterpret_cast<const float4*>(
                                                       part_of(k0 + (k + j) * stride) + 2 * ROWS + row * DP + d))
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float f = k + j < count ? so[(k + j) * ROWS + row] : 0.0f;
                            v.x += x[j].x * f, v.y += x[j].y * f;
                            v.z += x[j].z * f, v.w += x[j].w * f;
                        }
                    }
                    if (final) {
                        store(row, d, v.x, v.y, row_l[row]);
                        store(row, d + 2, v.z, v.w, row_l[row]);
                    } else {
                        *reinterpret_cast<float4*>(to + 2 * ROWS + row * DP + d) = v;
                    }
                }
                if (tid < rows) {
                    if (final) store_lse(tid, row_m[tid], row_l[tid]);
                    else to[tid] = row_m[tid], to[ROWS + tid] = row_l[tid];
                }
            };
            const int mine_k = cta - c0, run = mine_k / fan, runs = (n + fan - 1) / fan;
            // counters by the CTA of the run's first part.  That CTA may end one item and
            // begin another, so first runs, later runs and second rounds count apart.
            int* first = counters + (run == 0 ? 0 : a.max_ctas) + c0 + run * fan;
            if (arrive(first, min(fan, n - run * fan))) {
                join(run * fan, 1, min(fan, n - run * fan), runs == 1);
                if (runs > 1 && arrive(counters + 2 * a.max_ctas + c0, runs)) join(0, fan, runs, true);
            }
        }
        // ---- the next item ----
        u += step_end - step;
        step = 0;
        if (ends && ++item == items_per_seq && u < u_end) {
            item = 0;
            do {
                ++b;
                span = visible(a, b, false);
                n_steps = span_steps<STEP>(span);
            } while (n_steps == 0 && b + 1 < a.B);
        }
        __syncthreads();
    }
}

template <class S>
int launch_attn_shape(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    if (S::SMEM > 48 * 1024 &&
        cudaFuncSetAttribute(attn_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) !=
            cudaSuccess)
        return -3;
    int shift = -1;
    if ((a.page_size & (a.page_size - 1)) == 0)
        for (shift = 0; (1 << shift) < a.page_size;) ++shift;
    return launch_dependent(attn_kernel<S>, dim3(static_cast<unsigned>(ctx.num_sms * S::OCC)),
                            kAttnThreads, S::SMEM, stream, a, shift);
}

template <int DT, bool E4M3, int DP, int NT, bool P16>
int launch_attn_nt(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    // a step's keys fill 32 registers a lane, or 16 or 64 at the ends of the range
    constexpr int kRegs16 = DP * (E4M3 ? 1 : 2) / 8;  // of 16 tokens
    constexpr int R = kRegs16 >= 32 ? 1 : 2;
    constexpr int kOcc = DP == 256 ? (NT == 1 ? 2 : 1) : NT == 2 ? 2 : DP == 64 ? 4 : 3;
    return launch_attn_shape<AttnShape<DT, E4M3, DP, NT, R, P16, kOcc>>(ctx, a, stream);
}

template <int DT, bool E4M3, int DP>
int launch_attn_dp(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    const bool p16 = a.page_size % 16 == 0;
    if (a.q_heads / a.kv_heads <= 8)
        return p16 ? launch_attn_nt<DT, E4M3, DP, 1, true>(ctx, a, stream)
                   : launch_attn_nt<DT, E4M3, DP, 1, false>(ctx, a, stream);
    return p16 ? launch_attn_nt<DT, E4M3, DP, 2, true>(ctx, a, stream)
               : launch_attn_nt<DT, E4M3, DP, 2, false>(ctx, a, stream);
}

template <int DT, bool E4M3>
int launch_attn_dt(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_attn_dp<DT, E4M3, 64>(ctx, a, stream);
    if (a.head_dim <= 128) return launch_attn_dp<DT, E4M3, 128>(ctx, a, stream);
    return launch_attn_dp<DT, E4M3, 256>(ctx, a, stream);
}

}  // namespace

size_t attn_workspace_bytes(const DeviceCtx& ctx, int q_heads, int kv_heads, int head_dim, bool) {
    const int ctas = ctx.num_sms * kMaxCtasPerSm;
    const int rows = q_heads / kv_heads <= 8 ? 8 : 16;
    const int dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    return counter_bytes(3 * ctas) + 2ull * ctas * part_floats(rows, dp) * 4;
}

int launch_attn(const DeviceCtx& ctx, const AttnArgs& args, int dtype, bool e4m3,
                cudaStream_t stream) {
    AttnArgs a = args;
    a.max_ctas = ctx.num_sms * kMaxCtasPerSm;
    if (dtype == 0)
        return e4m3 ? launch_attn_dt<0, true>(ctx, a, stream) : launch_attn_dt<0, false>(ctx, a, stream);
    return e4m3 ? launch_attn_dt<1, true>(ctx, a, stream) : launch_attn_dt<1, false>(ctx, a, stream);
}

}  // namespace w4g
