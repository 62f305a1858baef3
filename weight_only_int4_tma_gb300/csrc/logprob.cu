// Log probabilities of given tokens, entropy and largest logits (include/decode.h):
//   lse = f m + ln S,  S = sum 2^t,  t = (x - m) f log2 e,  entropy = ln 2 (log2 S - sum 2^t t / S).
//
// A row is read once, in 16-byte pieces, by a cluster of 1, 2, 4 or 8 CTAs (as many as keep all SMs
// busy); a thread carries its own reference m, S and sum of 2^t t in fp32, rescaled only when a
// value passes m by more than 2^10, and they are joined at the end.  Differences x - m are taken before
// they are scaled, so that logits of any size are right.
//
// The largest logits need no second pass over the row either: every thread keeps the largest of its own
// pieces.  Every logit that is not below the top-th largest of those maxima belongs to a thread whose
// maximum is not below it either.  So only these threads' pieces, `top` in 256 and a few more
// where maxima are equal, are read again, from L2, whatever the order of the logits is.  Where many
// are equal, the index of each thread's first decides.
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

// m: the largest logit or a little less; s = sum 2^t, w = sum 2^t t, t = (x - m) c.
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
    const bool fine = f > 0.0f && f < INFINITY;
    const float c = f * kLog2e;
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
        add(x);
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
        if (!((top - sum.m) * c <= kLpLag)) sum.shift(lp_max(sum.m, top), c);
        const float m = sum.m == -INFINITY ? 0.0f : sum.m;
        const uint64_t m2 = pack_f2(-m, -m), c2 = pack_f2(c, c);
        uint64_t s2 = 0, w2 = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                float d0, d1;
                unpack_f2(mul_f2(add_f2(pack_f2(x[u][e], x[u][e + 1]), m2), c2), d0, d1);
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
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum.join({__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d),
                  __shfl_xor_sync(0xFFFFFFFFu, sum.w, d)}, c);
    if (lane == 0) sh.part[warp] = sum;
    if (tid == 0) sh.n_chosen = sh.n_cand = 0, sh.least = 0xFFFFFFFFu;

    // ---- the CTA's largest logits ----
    if (TOP) {
        const int k = a.top;
        const uint32_t mine = at == -1 ? 0u : order_value(bv);
        uint32_t key = mine;   // bitonic sort of the warp's, the largest in lane 0
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int d = size >> 1; d > 0; d >>= 1) {
                const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
                key = ((lane & d) == 0) == ((lane & size) == 0) ? max(key, o) : min(key, o);
            }
        sh.sorted[lane][warp] = key;
        __syncthreads();
        // how many maxima are larger than this thread's: a binary search in every warp's list
        int lo[kLpWarps];
#pragma unroll
        for (int w = 0; w < kLpWarps; ++w) lo[w] = 0;
#pragma unroll
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
        each([&](float x, int i) {
            const uint64_t key_of = order_key(x, i);
            if (key_of >= least) {
                const int slot = atomicAdd(&sh.n_cand, 1);
                if (slot < kLpCandidates) sh.cand[slot] = key_of;
            }
        });
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
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
                __syncthreads();
                if (lane == 0) sh.red[warp] = most;
                __syncthreads();
                most = sh.red[lane & (kLpWarps - 1)];
#pragma unroll
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
            for (int j = 0; j < n; ++j) larger += sh.cand[j] > own;
            if (larger < k) put(larger, own);
        }
        if (tid >= n && tid < k) put(tid, 0);
    } else {
        if (cluster > 1) cluster_wait_acquire();
        __syncthreads();
    }

    // ---- the row's ----
    if (warp == 0) {
        sum = sh.part[lane & (kLpWarps - 1)];
        if (lane >= kLpWarps) sum = LpSums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum.join({__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d),
                      __shfl_xor_sync(0xFFFFFFFFu, sum.w, d)}, c);
        if (cluster > 1 && lane == 0) {
            const uint32_t dst = map_to_rank(smem_addr(&sh.ranks[rank]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(sum.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 4), "f"(sum.s) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 8), "f"(sum.w) : "memory");
        } else if (lane == 0) {
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
    for (int r = 1; r < cluster; ++r) sum.join(sh.ranks[r], c);
    // ln S by its exponent, in fp64, and its mantissa: within 2^-24 of the result's last bits however
    // large S is, without a logarithm in fp64
    const float m = sum.m;
    const int s_bits = __float_as_int(sum.s);
    const double log_s = ((s_bits >> 23) - 127) * 0.69314718055994530942 +
                         logf(__int_as_float((s_bits & 0x007FFFFF) | 0x3F800000));
    auto logprob = [&](float x) {
        if (!fine || m != m) return NAN;
        if (m == -INFINITY) return -INFINITY;
        if (m == INFINITY) return x == INFINITY ? NAN : -INFINITY;
        return static_cast<float>((static_cast<double>(x) - m) * f - log_s);
    };
    if (tid == 0) {
        float lse = NAN, entropy = NAN;
        if (fine && m == m) {
            lse = m, entropy = m == INFINITY ? NAN : 0.0f;
            if (fabsf(m) < INFINITY) {
                lse = static_cast<float>(static_cast<double>(m) * f + log_s);
                entropy = static_cast<float>(log_s - 0.69314718055994530942 * static_cast<double>(sum.w) / sum.s);
            }
        }
        if (a.lse) a.lse[t] = lse;
        if (a.entropy) a.entropy[t] = entropy;
    }
    for (int i = tid; i < a.n_ids; i += kLpThreads) {
        const int id = a.ids[t * a.n_ids + i];
        if (id >= a.V) record_status(a.status, kDecInvalidArg);
        a.logprobs[t * a.n_ids + i] = id < 0 ? 0.0f : id >= a.V ? NAN : logprob(logit<DT>(base, id));
    }
    if (TOP) {
        // the CTAs' largest, each CTA's in order: a thread per key counts the larger ones
        const int r = tid / kLpTop, n = tid % kLpTop;
        static_assert(kLpThreads == kLpCluster * kLpTop, "a thread for each key");
        const uint64_t mine = r < cluster && n < a.top ? sh.best[r][n] : 0;
        int larger = n;
        for (int o = 0; o < cluster; ++o) {
            int lo = 0;  // of CTA o's: a binary search
            if (o != r && mine != 0) {
#pragma unroll
                for (int step = kLpTop / 2; step > 0; step >>= 1)
                    if (lo + step <= a.top && sh.best[o][lo + step - 1] > mine) lo += step;
                if (lo < a.top && sh.best[o][lo] > mine) ++lo;
            }
            larger += lo;
        }
        if (mine != 0 && larger < a.top) {
            const int id = key_index(mine);
            a.top_ids[t * a.top + larger] = id;
            if (a.top_logprobs) a.top_logprobs[t * a.top + larger] = logprob(logit<DT>(base, id));
        }
    }
}

template <int DT, bool TOP>
int launch_logprob_as(const DeviceCtx& ctx, const LogprobArgs& a, cudaStream_t stream) {
    // CTAs for a row: as many as fit on the device together (four on an SM), each with at least a
    // few pieces for every thread
    int cluster = 1;
    while (cluster < kLpCluster && 2ll * cluster * a.T <= 4ll * ctx.num_sms &&
           a.V / (2 * cluster) >= kLpThreads * 8)
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
