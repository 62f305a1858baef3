// Log probabilities of given tokens, entropy and largest logits (include/decode.h):
//   lse = f m + ln S,  S = sum 2^t,  t = (x - m) f log2 e,  entropy = ln 2 (log2 S - sum 2^t t / S).
//
// A row is read once, in 16-byte pieces, by a cluster of 1, 2, 4 or 8 CTAs (the fewer the
// more rows there are); a thread carries its own reference m, S and sum of 2^t t in fp32, rescaled only when a
// value passes m by more than 2^10, and they are joined at the end.  Differences x - m are taken before
// they are scaled, and where f is at most 1 of halves, with 2 f, so that logits of any size are right: a difference
// that fp32 does not reach then is one whose product with f it does not reach either.  (Halves are
// exact but for the last bit of subnormal numbers, so the results are the same bits wherever x - m is finite.)
//
// The largest logits need no second pass over the row either: every thread keeps the largest of its own
// pieces.  Every logit that is not below the top-th largest of those maxima belongs to a thread whose
// maximum is not below it either.  So only these threads' pieces, `top` in 256 and a few more
// where maxima are equal, are read again, from L2, whatever the order of the logits is.  Where many
// are equal, the index of each thread's first decides.
//
// What bounds it: many rows without largest logits memory (2048 of 128000 bf16: 525 MB in 85 us, 6.1 TB/s of
// the 6.8 that a plain copy reaches); with the largest their search, which runs once per row at cold
// instructions' speed (301 of 50001 fp32 with 20: 18 us, 9 for the bytes; 2048 of 128000 with 20: 139 us); one row
// the chain of launch, loads, joins of threads, CTAs and cluster (128000 with 5: 7.9 us, of which 0.04 for the bytes).
#include "decode.cuh"

namespace w4g {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpTop = 32;          // largest number of largest logits
constexpr int kLpCluster = 8;
constexpr int kLpCandidates = 1024;
constexpr int kLpFew = 64;          // threads whose pieces are read again without looking at indexes
constexpr float kLpLag = 10.0f;     // t may pass 0 by 10: sums stay far from fp32's limits
constexpr float kLog2e = 1.4426950408889634f;

template <int DT>
__device__ __forceinline__ float logit(const void* x, int64_t at) {
    if constexpr (DT == 2) return static_cast<const float*>(x)[at];
    else return dec_to_f32<DT>(static_cast<const uint16_t*>(x)[at]);
}
template <int DT>
__device__ __forceinline__ void unpack_logits(uint4 v, float (&f)[DT == 2 ? 4 : 8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == 2) {
            f[j] = __uint_as_float(w[j]);
        } else {
            f[2 * j] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] & 0xFFFFu));
            f[2 * j + 1] = dec_to_f32<DT>(static_cast<uint16_t>(w[j] >> 16));
        }
    }
}

// Order of the largest: NaN above all, -0 as 0; with the index, the lower one first.  0 is below every key.
__device__ __forceinline__ uint32_t order_value(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v != v ? 0xFFFFFFFFu : b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(float v, int i) {
    return static_cast<uint64_t>(order_value(v)) << 32 | (0x7FFFFFFFu - static_cast<uint32_t>(i));
}
// The logit of a key (0 for -0, which makes no difference to its log probability).
__device__ __forceinline__ float key_logit(uint64_t k) {
    const uint32_t v = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(v == 0xFFFFFFFFu ? 0x7FFFFFFFu : v >> 31 ? v & 0x7FFFFFFFu : ~v);
}
__device__ __forceinline__ int key_index(uint64_t k) {
    return static_cast<int>(0x7FFFFFFFu - static_cast<uint32_t>(k));
}
__device__ __forceinline__ float lp_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lp_max(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// m: the largest x or a little less; s = sum 2^t, w = sum 2^t t, t = (x - m) c; x: logits or their halves.
struct LpSums {
    float m, s, w;
    __device__ __forceinline__ void shift(float to, float c) {  // to a larger m
        if (m == -INFINITY) {  // nothing but logits of -infinity so far
            s = w = 0.0f;
        } else {
            const float d = fmaxf((m - to) * c, -200.0f), e = lp_exp2(d);
            w = e * fmaf(d, s, w);
            s *= e;
        }
        m = to;
    }
    __device__ __forceinline__ void join(LpSums o, float c) {
        const float top = lp_max(m, o.m);
        shift(top, c);
        o.shift(top, c);
        s += o.s, w += o.w;
    }
};

// Where a row's pieces stand: elements 0 .. head - 1 one by one, then pieces of PER, then the rest one by one.
struct LpRow {
    int head, pieces, tail;
};

struct LpShared {
    LpSums part[kLpWarps];
    LpSums ranks[kLpCluster];
    uint32_t sorted[32][kLpWarps];         // the warps' maxima in descending order
    uint64_t best[kLpCluster][kLpTop];     // at the leader: the largest of every CTA
    uint64_t cand[kLpCandidates + kLpTop];
    uint64_t red[kLpWarps];
    int chosen[kLpThreads];                // threads whose pieces are read again
    uint64_t least_key;                    // no logit below this is among the largest
    uint32_t least;                        // of the chosen threads' maxima
    int n_chosen, n_cand;
};

template <int DT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_kernel(LogprobArgs a, int cluster) {
    constexpr int PER = DT == 2 ? 4 : 8, U = 4;
    __shared__ LpShared sh;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x / cluster;
    const int rank = static_cast<int>(blockIdx.x - t * cluster);
    if (cluster > 1) cluster_arrive_relaxed();
    grid_dep_wait();
    const float f = a.factor ? a.factor[t] : 1.0f;
    const bool fine = f > 0.0f && f <= 0x1p127f;   // (f log2 e is finite)
    // what the sums have are logits times `half`, whose factor then is `ff`; fp16's differences are always finite
    const bool halved = DT != 0 && f <= 1.0f;
    const float half = halved ? 0.5f : 1.0f, ff = halved ? f + f : f, c = ff * kLog2e;
    const char* base = static_cast<const char*>(a.x) + t * a.ld * (DT == 2 ? 4 : 2);
    LpRow row;
    row.head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / (DT == 2 ? 4 : 2);
    row.head = min(row.head, a.V);
    row.pieces = (a.V - row.head) / PER;
    row.tail = a.V - row.head - row.pieces * PER;
    const uint4* body = reinterpret_cast<const uint4*>(base + row.head * (DT == 2 ? 4 : 2));
    const int per_cta = (row.pieces + cluster - 1) / cluster;
    const int p_lo = min(row.pieces, rank * per_cta), p_hi = min(row.pieces, p_lo + per_cta);
    const int tail0 = row.head + row.pieces * PER;

    // the given token of this thread and its logit, under way from the start
    const bool has_id = rank == 0 && tid < a.n_ids;
    const int my_id = has_id ? a.ids[t * a.n_ids + tid] : -1;
    const float my_logit = my_id >= 0 && my_id < a.V ? logit<DT>(base, my_id) : 0.0f;

    // ---- one pass: this thread's sums and its largest logit ----
    LpSums sum{-INFINITY, 0.0f, 0.0f};
    float bv = -INFINITY;   // NaN once there was one
    int at = -1;            // where bv stood first: a piece's number, or one of the single logits' index
    auto add = [&](float x) {
        if (!((x - sum.m) * c <= kLpLag)) sum.shift(lp_max(sum.m, x), c);  // (NaN while m is -infinity)
        const float d = fmaxf((x - (sum.m == -INFINITY ? 0.0f : sum.m)) * c, -200.0f);
        const float e = lp_exp2(d);
        sum.s += e;
        sum.w = fmaf(e, d, sum.w);
    };
    auto single = [&](int i) {
        const float x = logit<DT>(base, i);
        add(x * half);
        if (TOP) {
            if (at == -1 || (!(x <= bv) && bv == bv)) at = -2 - i;
            bv = lp_max(bv, x);
        }
    };
    if (rank == 0 && tid < row.head) single(tid);
    constexpr uint32_t kNone = DT == 0 ? 0xFC00FC00u : DT == 1 ? 0xFF80FF80u : 0xFF800000u;
    uint4 now[U], next[U];
    auto load = [&](uint4 (&v)[U], int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {  // pieces past the end are logits of -infinity
            v[u] = make_uint4(kNone, kNone, kNone, kNone);
            if (p0 + u * kLpThreads < p_hi) v[u] = __ldcs(body + p0 + u * kLpThreads);
        }
    };
    load(now, p_lo + tid);
    for (int p0 = p_lo + tid; p0 < p_hi; p0 += U * kLpThreads) {
        load(next, p0 + U * kLpThreads);
        float x[U][PER];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unpack_logits<DT>(now[u], x[u]);
#pragma unroll
            for (int e = 0; e < PER; e += 2) top = max3_nan(top, x[u][e], x[u][e + 1]);
        }
        if (TOP && (at == -1 || (!(top <= bv) && bv == bv))) {
            bv = lp_max(bv, top);
            at = p0;
        }
        top *= half;
        if (!((top - sum.m) * c <= kLpLag)) sum.shift(lp_max(sum.m, top), c);
        const float m = sum.m == -INFINITY ? 0.0f : sum.m;
        const uint64_t m2 = pack_f2(-m, -m), c2 = pack_f2(c, c), half2 = pack_f2(half, half);
        uint64_t s2 = 0, w2 = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                float d0, d1;
                const uint64_t pair = pack_f2(x[u][e], x[u][e + 1]);
                unpack_f2(mul_f2(DT == 0 ? add_f2(pair, m2) : fma_f2(pair, half2, m2), c2), d0, d1);
                // 2^-200 is 0; a product of 0 and -infinity would be NaN
                const uint64_t d = pack_f2(fmaxf(d0, -200.0f), fmaxf(d1, -200.0f));
                unpack_f2(d, d0, d1);
                const uint64_t y = pack_f2(lp_exp2(d0), lp_exp2(d1));
                s2 = add_f2(s2, y);
                w2 = fma_f2(y, d, w2);
            }
        float lo, hi;
        unpack_f2(s2, lo, hi);
        sum.s += lo + hi;
        unpack_f2(w2, lo, hi);
        sum.w += lo + hi;
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
    }
    if (rank == cluster - 1 && tid < row.tail) single(tail0 + tid);

    // ---- the CTA's sums, in warp 0 ----
    // (From here on loops stay loops: code that runs once per row is fetched as it runs, at some 20
    // cycles an instruction: 60 rows of 32000 with 20 alternatives 16.0 us with them unrolled.)
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1)
        sum.join({__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d),
                  __shfl_xor_sync(0xFFFFFFFFu, sum.w, d)}, c);
    if (lane == 0) sh.part[warp] = sum;
    if (tid == 0) sh.n_chosen = sh.n_cand = 0, sh.least = 0xFFFFFFFFu;

    auto cta_sums = [&]() {   // by one warp, beside what the others do
        if (warp != kLpWarps - 1) return;
        sum = sh.part[lane & (kLpWarps - 1)];
#pragma unroll 1
        for (int d = kLpWarps / 2; d > 0; d >>= 1)
            sum.join({__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d),
                      __shfl_xor_sync(0xFFFFFFFFu, sum.w, d)}, c);
        if (lane == 0) sh.part[0] = sum;
    };

    // ---- the CTA's largest logits ----
    if (TOP) {
        const int k = a.top;
        const uint32_t mine = at == -1 ? 0u : order_value(bv);
        uint32_t key = mine;   // bitonic sort of the warp's, the largest in lane 0
#pragma unroll 1
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll 1
            for (int d = size >> 1; d > 0; d >>= 1) {
                const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
                key = ((lane & d) == 0) == ((lane & size) == 0) ? max(key, o) : min(key, o);
            }
        sh.sorted[lane][warp] = key;
        __syncthreads();
        cta_sums();
        // how many maxima are larger than this thread's: a binary search in every warp's list
        int lo[kLpWarps];
#pragma unroll
        for (int w = 0; w < kLpWarps; ++w) lo[w] = 0;
#pragma unroll 1
        for (int step = 16; step > 0; step >>= 1)
#pragma unroll
            for (int w = 0; w < kLpWarps; ++w)
                if (sh.sorted[lo[w] + step - 1][w] > mine) lo[w] += step;
        int above = 0;
#pragma unroll
        for (int w = 0; w < kLpWarps; ++w) above += lo[w] + (lo[w] == 31 && sh.sorted[31][w] > mine);
        // the threads whose maximum is not below the top-th largest (all that have logits, if they are fewer)
        const bool in = mine != 0 && above < k;
        if (in) {
            sh.chosen[atomicAdd(&sh.n_chosen, 1)] = tid;
            atomicMin(&sh.least, mine);
        }
        __syncthreads();
        int chosen = sh.n_chosen;
        uint64_t least = chosen < k ? 0 : static_cast<uint64_t>(sh.least) << 32;
        if (chosen > kLpFew) {  // many equal maxima: those of the lowest indexes
            uint64_t exact = 0;
            if (in) {
                int i = -2 - at;
                if (at >= 0) {
                    i = -1;
#pragma unroll 1
                    for (int u = 0; u < U && i < 0; ++u) {
                        float x[PER];
                        const int p = at + u * kLpThreads;
                        unpack_logits<DT>(body[p], x);
#pragma unroll
                        for (int e = PER - 1; e >= 0; --e)
                            if (order_value(x[e]) == mine) i = row.head + p * PER + e;
                    }
                }
                exact = static_cast<uint64_t>(mine) << 32 | (0x7FFFFFFFu - static_cast<uint32_t>(i));
            }
            sh.cand[tid] = exact;
            __syncthreads();
            int larger = 0;
            if (in)
#pragma unroll 2
                for (int j = 0; j < kLpThreads; ++j) larger += sh.cand[j] > exact;
            if (in && larger < k) sh.chosen[larger] = tid;
            if (in && larger == k - 1) sh.least_key = exact;
            __syncthreads();
            chosen = k;
            least = sh.least_key;
        }
        // the chosen threads' logits
        const int each_has = (p_hi - p_lo + kLpThreads - 1) / kLpThreads;
        auto each = [&](auto&& use) {
            if (tid < chosen) {
                const int who = sh.chosen[tid];
                if (rank == 0 && who < row.head) use(logit<DT>(base, who), who);
                if (rank == cluster - 1 && who < row.tail) use(logit<DT>(base, tail0 + who), tail0 + who);
            }
            for (int n = tid; n < chosen * each_has; n += kLpThreads) {
                const int nth = n / each_has, p = p_lo + sh.chosen[nth] + (n - nth * each_has) * kLpThreads;
                if (p >= p_hi) continue;
                float x[PER];
                unpack_logits<DT>(body[p], x);
#pragma unroll
                for (int e = 0; e < PER; ++e) use(x[e], row.head + p * PER + e);
            }
        };
        auto keep = [&](bool some, uint64_t key_of) {   // by whole warps: one addition for all lanes
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, some);
            if (who == 0) return;
            int at0 = 0;
            if (lane == 0) at0 = atomicAdd(&sh.n_cand, __popc(who));
            at0 = __shfl_sync(0xFFFFFFFFu, at0, 0) + __popc(who & ((1u << lane) - 1));
            if (some && at0 < kLpCandidates) sh.cand[at0] = key_of;
        };
        if (row.head + row.tail > 0) {   // single logits of chosen threads
            const int who = tid < chosen ? sh.chosen[tid] : kLpThreads;
            const bool head = rank == 0 && who < row.head, tail = rank == cluster - 1 && who < row.tail;
            uint64_t key_of = head ? order_key(logit<DT>(base, who), who) : 0;
            keep(head && key_of >= least, key_of);
            key_of = tail ? order_key(logit<DT>(base, tail0 + who), tail0 + who) : 0;
            keep(tail && key_of >= least, key_of);
        }
        const uint32_t least_value = static_cast<uint32_t>(least >> 32);
#pragma unroll 1
        for (int n0 = tid - lane; n0 < chosen * each_has; n0 += kLpThreads) {
            const int n = n0 + lane, nth = n / each_has;
            const int p = n < chosen * each_has ? p_lo + sh.chosen[nth] + (n - nth * each_has) * kLpThreads : p_hi;
            uint4 piece = make_uint4(0, 0, 0, 0);
            uint32_t hits = 0;
            if (p < p_hi) {
                float x[PER];
                piece = body[p];
                unpack_logits<DT>(piece, x);
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (order_value(x[e]) >= least_value) hits |= 1u << e;
            }
            while (__any_sync(0xFFFFFFFFu, hits != 0)) {   // one of each lane's at a time: few have any
                const int e = __ffs(hits) - 1;
                uint64_t key_of = 0;
                if (hits) {
                    const int word = DT == 2 ? e : e >> 1;
                    const uint32_t w = word == 0 ? piece.x : word == 1 ? piece.y : word == 2 ? piece.z : piece.w;
                    const float x = DT == 2 ? __uint_as_float(w)
                                            : dec_to_f32<DT == 2 ? 0 : DT>(static_cast<uint16_t>(e & 1 ? w >> 16 : w & 0xFFFFu));
                    key_of = order_key(x, row.head + p * PER + e);
                }
                keep(hits != 0 && key_of >= least, key_of);
                hits &= hits - 1;
            }
        }
        __syncthreads();
        int n = sh.n_cand;
        if (n > kLpCandidates) {
            // Too many in few threads' pieces: one after another, each the largest below the one before.
            uint64_t below = ~0ull;
            for (n = 0; n < k; ++n) {
                uint64_t most = 0;
                each([&](float x, int i) {
                    const uint64_t key_of = order_key(x, i);
                    if (key_of < below && key_of > most) most = key_of;
                });
#pragma unroll 1
                for (int d = 16; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
                __syncthreads();
                if (lane == 0) sh.red[warp] = most;
                __syncthreads();
                most = sh.red[lane & (kLpWarps - 1)];
#pragma unroll 1
                for (int d = 16; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
                if (tid == 0) sh.cand[n] = most;
                below = most;
            }
            __syncthreads();
        }
        // in order, to the leader; places that stay empty (a short row's) are 0
        const uint32_t to = smem_addr(&sh.best[rank][0]);
        const uint32_t dst = cluster > 1 ? map_to_rank(to, 0) : to;
        if (cluster > 1) cluster_wait_acquire();
        auto put = [&](int at, uint64_t v) {
            if (cluster > 1) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst + 8 * at), "l"(v) : "memory");
            else sh.best[0][at] = v;
        };
        for (int i = tid; i < n; i += kLpThreads) {
            const uint64_t own = sh.cand[i];
            int larger = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) larger += sh.cand[j] > own;
            if (larger < k) put(larger, own);
        }
        if (tid >= n && tid < k) put(tid, 0);
    } else {
        __syncthreads();
        cta_sums();
        if (cluster > 1) cluster_wait_acquire();
    }

    // ---- the row's ----
    if (warp == kLpWarps - 1 && lane == 0) {
        sum = sh.part[0];
        if (cluster > 1) {
            const uint32_t dst = map_to_rank(smem_addr(&sh.ranks[rank]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(sum.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 4), "f"(sum.s) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 8), "f"(sum.w) : "memory");
        } else {
            sh.ranks[0] = sum;
        }
    }
    if (cluster > 1) {
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    sum = sh.ranks[0];
#pragma unroll 1
    for (int r = 1; r < cluster; ++r) sum.join(sh.ranks[r], c);
    // ln S = a_s + b_s: its exponent times 355 / 512, ln 2's leading bits, exact, and the rest (the reduction
    // of Cody and Waite, Software Manual for the Elementary Functions, 1980); and sums with the error of
    // each rounding, so that a result is within little more than its own last rounding however large m
    // is.  (In fp64 these few operations took 6000 cycles, a third of a single row's time.)
    const float m = sum.m;
    const int s_bits = __float_as_int(sum.s);
    const float s_exp = static_cast<float>((s_bits >> 23) - 127);
    const float a_s = s_exp * 0.693359375f;
    const float b_s = fmaf(s_exp, -2.12194440054690583e-4f, logf(__int_as_float((s_bits & 0x007FFFFF) | 0x3F800000)));
    auto two_sum = [](float x, float y, float& err) {
        const float s = x + y, z = s - x;
        err = (x - (s - z)) + (y - z);
        return s;
    };
    auto logprob = [&](float x) {   // (x half - m) ff - ln S
        if (!fine || m != m) return NAN;
        if (m == -INFINITY) return -INFINITY;
        if (m == INFINITY) return x == INFINITY ? NAN : -INFINITY;
        if (x == -INFINITY) return x;
        float d_err, s_err;
        const float d = two_sum(x * half, -m, d_err), p = d * ff;
        const float s = two_sum(p, -a_s, s_err);
        return fabsf(p) < 1e30f ? s + (s_err + (fmaf(d, ff, -p) + d_err * ff - b_s)) : p;
    };
    if (tid == 0) {
        float lse = NAN, entropy = NAN;
        if (fine && m == m) {
            lse = m, entropy = m == INFINITY ? NAN : 0.0f;   // (where m is infinite)
            if (fabsf(m) < INFINITY) {
                float err;
                const float p = m * ff, s = two_sum(p, a_s, err);
                lse = fabsf(p) < 1e30f ? s + (err + (fmaf(m, ff, -p) + b_s)) : p;
                entropy = a_s + fmaf(-0.69314718055994531f, sum.w / sum.s, b_s);
            }
        }
        if (a.lse) a.lse[t] = lse;
        if (a.entropy) a.entropy[t] = entropy;
    }
    auto given = [&](int i, int id, float x) {
        if (id >= a.V) record_status(a.status, kDecInvalidArg);
        a.logprobs[t * a.n_ids + i] = id < 0 ? 0.0f : id >= a.V ? NAN : logprob(x);
    };
    if (has_id) given(tid, my_id, my_logit);
    for (int i = tid + kLpThreads; i < a.n_ids; i += kLpThreads) {
        const int id = a.ids[t * a.n_ids + i];
        given(i, id, id >= 0 && id < a.V ? logit<DT>(base, id) : 0.0f);
    }
    if (TOP) {
        // the CTAs' largest, each CTA's in order: a thread per key counts the larger ones
        const int r = tid / kLpTop, n = tid % kLpTop;
        static_assert(kLpThreads == kLpCluster * kLpTop, "a thread for each key");
        const uint64_t mine = r < cluster && n < a.top ? sh.best[r][n] : 0;
        int larger = n;
        if (cluster > 1) {
            larger = 0;
            if (mine != 0)
#pragma unroll 1
                for (int o = 0; o < cluster; ++o)
#pragma unroll 8
                    for (int j = 0; j < a.top; ++j) larger += sh.best[o][j] > mine;
        }
        if (mine != 0 && larger < a.top) {
            const int id = key_index(mine);
            a.top_ids[t * a.top + larger] = id;
            if (a.top_logprobs) a.top_logprobs[t * a.top + larger] = logprob(key_logit(mine));
        }
    }
}

template <int DT, bool TOP>
int launch_logprob_as(const DeviceCtx& ctx, const LogprobArgs& a, cudaStream_t stream) {
    // CTAs for a row: up to two on an SM, each with at least 32 logits for every thread.  More of them share the
    // code that runs once per row badly: 60 rows of 32000 with 20 largest take 9.4 us with 2 CTAs a
    // row, 10.9 with 4, 17.8 with 8; 64 of 128000 16.0 with 2, 14.5 with 4; one of 32000 7.8 with 2, 7.6 with 8.
    int cluster = 1;
    while (cluster < kLpCluster && 2ll * cluster * a.T <= 2ll * ctx.num_sms &&
           a.V / (2 * cluster) >= kLpThreads * 32)
        cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T) * static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<DT, TOP>, a, cluster) == cudaSuccess ? 0 : -3;
}

}  // namespace

int launch_logprob(const DeviceCtx& ctx, const LogprobArgs& a, int dtype, cudaStream_t stream) {
    if (a.top)
        return dtype == 0 ? launch_logprob_as<0, true>(ctx, a, stream)
             : dtype == 1 ? launch_logprob_as<1, true>(ctx, a, stream) : launch_logprob_as<2, true>(ctx, a, stream);
    return dtype == 0 ? launch_logprob_as<0, false>(ctx, a, stream)
         : dtype == 1 ? launch_logprob_as<1, false>(ctx, a, stream) : launch_logprob_as<2, false>(ctx, a, stream);
}

}  // namespace w4g
