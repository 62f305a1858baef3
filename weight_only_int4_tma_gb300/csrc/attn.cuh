// Attention of one new token per sequence over a paged key-value cache (include/decode.h):
//   s_j = scale q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j)  over the visible tokens.
//
// The keys and values are read once and nothing else of size is: with G query heads per
// key-value head the work is 2 G operations per cached 16-bit value, far below what the
// tensor cores do in the time of the read, so the kernel is built to keep loads in flight.
// Measured on several devices (a copy reaches 6.78 TB/s):
//   64 sequences of up to 16384 tokens, 8 heads of 128, bf16: 2.37 GB in 342 to 355 us, 6.7 to 6.9
//   TB/s; with 8 bits 1.18 GB in 190 to 208 us, 5.7 to 6.2 TB/s;
//   16 sequences of up to 4096 tokens, 32 heads of 128, fp16: 0.54 GB in 86 to 88 us, 6.2 TB/s;
//   one sequence of 131072 tokens, 8 heads of 128, bf16: 0.54 GB in 81 to 84 us, 6.4 to 6.6 TB/s;
//   33 windows of up to 4096 tokens, 4 heads of 64, 8-bit: 0.049 GB in 22.0 us, 2.2 TB/s: a round of
//   the warps' steps takes 2.0 us, of conversions and MMAs that wait for one another (16
//   consumer warps with half the step each: 25.9 us);
//   64 of 8000 tokens of it: 0.26 GB in 88 to 92 us, 2.9 TB/s, as DRAM fetches such short rows that
//   stand apart at 1.6 times their bytes;
//   one sequence of 777 tokens: 8.9 to 9.3 us, which is lengths, page table, keys and the join, one
//   after another.
//
// Data path.  Steps of 16 R tokens go through a ring in shared memory of 128 KB (one CTA per
// SM): eight producer warps (or four) fill it with asynchronous copies, eight consumer warps
// (or four) take its steps in turn, each working alone.  mma.sync suffices: the tcgen05 form would need the
// 128-row tiles that one token's few query heads do not fill.  ldmatrix turns a step into its
// operands:
//   S^T = K Q^T   tokens are the MMA's 16 rows, query heads its 8 columns (with 8 heads or
//                 fewer per key-value head half of a 16-row query tile would be padding);
//   O^T = V^T P^T head dimensions are the rows; ldmatrix's transposed form reads V^T.
// 8-bit caches are converted to fp16 between ldmatrix and MMA (exact), two values at a time.
// The probabilities leave S^T with tokens in rows and are wanted with tokens as the K index:
// one 8 x 8 transpose of 16-bit pairs (movmatrix).  They are split in a high and a low
// 16-bit part, each multiplied with V: a single 16-bit rounding of P (2^-9 for bf16) would
// show in the result as much as the result's own.  Both parts are positive (together within 2^-16
// of the weight for bf16, 2^-21 for fp16), as 16-bit values may be infinite; 8-bit ones are not.
//
// Softmax.  One pass with a running reference m per query head: weights are exp2(s - m), and
// when a score passes m by more than 2^8 the sums so far are scaled to the new reference
// (a warp vote finds out; exact in the end, since numerator and denominator share it).  All maxima
// carry a NaN: from the step on in which a score is one it stands in m and in every sum.  With
// an infinite score m is infinite and the sums are NaN, as inf / inf is.
//
// Work split.  All (sequence, head, row tile) items stand in one line, each as long as its steps
// and kItemCost more for what an item costs by itself.  The line is cut in equal shares, one per
// CTA, whatever the lengths; every CTA finds its own from the lengths on the device.  The
// producers run on into the next item while the consumers finish one.  An item whose steps lie
// in one share is finished there; one that is cut leaves (m, l, O) of each part in fp32 in the
// workspace, and the CTA that completes an item's count of parts joins them, in their order.
// (SMs do not get equal bandwidth, so shares of falling size claimed by whoever is free end more
// evenly; but each more part costs more than that gives: 24 sequences of 8192 tokens, 4 heads of
// 128 with 16 rows: 77 us with equal shares, 87 to 92 with claimed ones; 64 sequences up to
// 16384 tokens: 355 and 349 us.)
#pragma once
#include "decode.cuh"

namespace w4g {

// Of an item by itself, in steps: some 2 us.  (52 ragged sequences of 32 heads, 8-bit, pages of 8:
// 42 us; 91 with shares of steps alone.)
constexpr int kItemCost = 8;
constexpr float kLag = 8.0f;       // scores may pass the reference by 2^8
// The workspace: three counters per CTA, then for each CTA two parts (its first item if that began in
// an earlier share, its last if that ends in a later one) of m[rows], l[rows], O[rows][dp].
__host__ __device__ constexpr size_t attn_part_floats(int rows, int dp) {
    return static_cast<size_t>(rows) * (dp + 2);
}
__host__ __device__ constexpr size_t attn_counter_bytes(int ctas) {
    return (static_cast<size_t>(ctas) * 12 + 127) / 128 * 128;
}

namespace {

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
// The larger, or NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}
// Two weights >= 0 to 16 bits, each below the weight itself (by at most 2^-7 of it in bf16, 2^-9 and
// 2^-23 in fp16), so that what is left of it is positive: a product of either part with an
// infinite value is that infinity, not NaN.  0 stays 0; of a weight under 2^-22 fp16's high part may be 0.
template <int DT>
__device__ __forceinline__ uint32_t pack_below(float lo, float hi) {
    if constexpr (DT == 0) {
        constexpr float kLess = 1.0f - 0x1p-10f;
        uint32_t r;
        asm("cvt.rz.relu.f16x2.f32 %0, %1, %2;"
            : "=r"(r) : "f"(fmaf(hi, kLess, -0x1p-24f)), "f"(fmaf(lo, kLess, -0x1p-24f)));
        return r;
    } else {
        constexpr float kLess = 1.0f - 0x1p-23f;
        return __byte_perm(__float_as_uint(lo * kLess), __float_as_uint(hi * kLess), 0x7632);
    }
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes global -> shared, asynchronously; zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
// Arrives on the barrier once this thread's copies so far are there.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Barrier of the consumer warps alone.
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}
// D += A B, 16 x 8 x 16, fp32 accumulate; BF: bf16 operands, else fp16.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// DT: 0 fp16, 1 bf16 (queries, output).  E4M3: 8-bit cache.  DP: head dimension rounded up
// to 64, 128 or 256.  NT: tiles of 8 query heads that a CTA takes at once.  PG: 16 or 8 where
// the page size is a multiple of that, so that PG tokens that begin at a multiple of PG lie in
// one page; else 1.
template <int DT_, bool E4M3_, int DP_, int NT_, int PG_>
struct AttnShape {
    static constexpr int DT = DT_, DP = DP_, NT = NT_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int PG = PG_;
    static constexpr bool GROUPS = PG > 1;
    static constexpr bool BF = DT == 1 && !E4M3;  // type of the MMA's operands
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int ROWS = 8 * NT;
    static constexpr int PITCH = DP * ES;         // bytes of a token's row in the ring
    static constexpr int CH = PITCH / 16;         // 16-byte chunks of it
    // 16 R tokens per step: 4 KB of keys where that is at most 64 tokens; 32 where every
    // lane looks up the page of one token
    static constexpr int R = PITCH >= 256 ? 1 : PITCH == 128 ? 2 : (GROUPS ? 4 : 2);
    static constexpr int NG = GROUPS ? 16 * R / PG : 1;   // groups of a step
    static constexpr int STEP = 16 * R;
    static constexpr int SLOT = STEP * PITCH;     // bytes of a step's keys, or values
    // Consumer warps.  Four where two tiles of 256 values need the registers of the others (16
    // sequences of 4000 tokens, 4 heads with 16 rows, bf16 92.8 us with eight, 69.1 with four; 8-bit
    // 107.9 and 64.2; with one tile four are 2 % slower).  They spill a little all the same: 32 to
    // 68 bytes at 255 registers, and with eight warps two tiles of 8-bit heads of 128 60 to 72 at 168.
    static constexpr int W = DP == 256 && NT == 2 ? 4 : 8;
    // Producer warps.  Eight where the consumers need no more than the 128 registers that leaves them
    // (8 sequences of 2000 tokens, 8 heads of 128: bf16 21.6 us with four, 20.0 with eight, 8-bit
    // 16.7 and 14.4; two query tiles spill then: 14 of 2000 tokens 21.9 and 29.1).
    static constexpr int PW = NT == 1 && DP <= 128 ? 8 : 4;
    static constexpr int MS = DP / 16;            // MMA steps over the head dimension
    static constexpr int OP = DP + 4;             // row of the warps' sums, in floats
    static constexpr int SO_BYTES = W * ROWS * OP * 4;   // the warps' sums
    // Steps of the ring: 128 KB of them, in a multiple of W and of PW.  (192 KB leave room for half the
    // warps' sums at a time: 64 sequences of up to 16384 tokens 353 us against 368, one of 131072
    // 84.2 and 90.3; 64 KB: 352 against 343 in another run.)  A stage then has the same producer in every round, and the same consumer
    // within an item: nobody waits for a stage two rounds ahead of it, which the barriers' one
    // bit of phase could not tell from the round at hand.
    static constexpr int NST = (128 << 10) / (2 * SLOT);
    // Joining an item's parts, in the warps' rounds.  By row one round of the steps is 2.0 us (64 bytes;
    // 1 leaves 33 windows of up to 4096 tokens whole: 23.2 us against 22.5), 1.3, 1.05, 1.0.  With
    // 16 rows the join is longer (64 bytes, one sequence of 1000 tokens 12.1 us with 0, 10.4 with 2).
    static constexpr int WHOLE = PITCH == 64 ? (NT == 1 ? 0 : 2) : PITCH == 256 || W == 4 ? 4 : 3;
    static constexpr int THREADS = 32 * (W + PW);
    static constexpr int RING = NST * 2 * SLOT;
    static constexpr int SMEM = RING + SO_BYTES + NST * (4 + 3 * 8);
    static_assert(NST % W == 0 && NST % PW == 0, "a stage's producer and consumer are fixed");
    static_assert(SMEM <= 219 * 1024, "the ring fits");
};

// Byte offset of chunk c of token row r in a slot: the chunks of eight rows that ldmatrix
// reads together stand in different 16-byte columns of 128.
template <int CH>
__device__ __forceinline__ constexpr uint32_t ring_at(int r, int c) {
    return static_cast<uint32_t>(r * CH * 16 + ((CH >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
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

// One item's steps [step, step_end) of n_steps, as one CTA takes them.
struct Segment {
    int b, item, step, step_end, n_steps;
    int rest;   // what the CTA's share holds after this item
    Span span;
};

// A part of an item that several CTAs hold: the item's are those of CTAs c0 .. c0 + n - 1.
struct Cut {
    int c0, n, at, b, head0, rows, last;  // at: the part written here; last: it completes its run
    float vs;
};

// The line and its shares, the same in every CTA.
struct Line {
    long long end, share;
    bool apart;   // a share is a part of one item
    bool whole;   // a share is the items that begin in it, to their ends
};
// parts that an item of n_steps is cut in (`apart`)
__device__ __forceinline__ int parts_of(const Line& line, int n_steps) {
    return static_cast<int>(quotient(n_steps + line.share - 1, line.share));
}

// Fills `line` and prefix[thread], what lies before each thread's sequences (thread t has
// sequences t * per_thread ...); by all threads of a CTA, which then meet at a barrier.
template <int STEP, int THREADS, int WARPS, int WHOLE>
__device__ __forceinline__ void lay_line(const AttnArgs& a, int items_per_seq, int ctas, bool report,
                                         Line& line, long long* prefix, long long* scan, int* tops) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int per_thread = (a.B + THREADS - 1) / THREADS;
    const int b_lo = min(a.B, tid * per_thread), b_hi = min(a.B, b_lo + per_thread);
    // their length in the line in the low bits, the number that have any steps above: below 2^27
    // sequences, whose 2^39 tokens are 2^35 steps of 16, and 8 for each sequence
    constexpr int kSeqBit = 36;
    static_assert((1ll << 35) + (1ll << 27) * kItemCost < (1ll << kSeqBit), "the lengths stay below the count");
    constexpr long long kLow = (1ll << kSeqBit) - 1;
    long long mine = 0;
    int top = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = span_steps<STEP>(visible(a, b, report));
        if (n) mine += n + kItemCost + (1ll << kSeqBit);
        top = max(top, n);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl, tops[warp] = top;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) incl += scan[w];
        total += scan[w];
        top = max(top, tops[w]);
    }
    prefix[tid] = ((incl - mine) & kLow) * items_per_seq;
    if (tid == 0) {
        const long long items = (total >> kSeqBit) * items_per_seq;
        total = (total & kLow) * items_per_seq;
        line.end = total;
        line.share = max(quotient(total + ctas - 1, ctas), 1ll);
        // Few items: shares cut from one item each, in whole rounds of the warps, so that no CTA has
        // two partial items to write and join, if that takes few rounds more.  (Heads of 128: 14
        // sequences of 4000 tokens, 4 heads with 16 rows, five more: 26.7 us with equal shares, 22.4
        // so; with rows of 64 bytes 7 of 4000, two more, 16.7 and 18.8.)
        line.apart = false;
        long long rounds = (line.share + WARPS - 1) / WARPS;
        if (2 * items <= ctas) {
            const long long steps = total - items * kItemCost;
            const int slots = ctas * WARPS, left = static_cast<int>(ctas - items) * WARPS;
            const long long r = max(quotient(steps + left - 1, left), 1ll);
            line.apart = r <= max(quotient(steps + slots - 1, slots), 1ll) + 1 + WHOLE;
            if (line.apart) rounds = r, line.share = r * WARPS;
        }
        // No item is cut where the longest takes not many rounds more than a share: joining takes some
        // WHOLE of them, with items cut anywhere one more.  (8 heads of 128, one sequence of 400
        // tokens, four rounds: 8.7 us whole, 9.5 in parts; of 600, five: 10.3 and 9.7; 16 sequences
        // of 300 tokens: 8.0 and 14.4 us, of 500 9.6 and 15.4.)
        if (items <= ctas && (top + WARPS - 1) / WARPS < rounds + WHOLE + (line.apart ? 0 : 1)) {
            line.apart = true;
            line.share = max((top + WARPS - 1) / WARPS * WARPS, 1);
        }
        // Nor where there are more items than CTAs and whole ones make the fullest share at most kOver
        // steps longer: by the mean length, with none that is longer than that by itself, and none
        // over 4 kOver, as a share's last item may lie beyond it in full.  (Heads of 128, 8 of them:
        // 32 sequences of 700 tokens 25.5 us cut, 21.7 whole, of 1500 41.4 and 36.6; 24 of 1500, 75
        // steps over, 34.0 and 35.7.)
        constexpr int kOver = (WHOLE + 2) * WARPS;
        line.whole = items > ctas && top + kItemCost <= min(4ll * kOver, line.share + kOver) &&
                     quotient(items + ctas - 1, ctas) * quotient(total, items) <= line.share + kOver;
    }
}

// One row of a finished item, four of its values.
template <int DT>
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int head, int d, float4 v, float f) {
    uint16_t* dst = a.out + b * a.ldo + static_cast<int64_t>(head) * a.head_dim + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(dec_pack2<DT>(v.x * f, v.y * f), dec_pack2<DT>(v.z * f, v.w * f));
}
// m and l of a row to its log-sum-exp; `shift`: see the weights in attn_kernel.  l is NaN only where m
// is +inf or NaN, which the log-sum-exp then is too.
__device__ __forceinline__ void store_lse(const AttnArgs& a, int b, int head, float m, float l, float shift) {
    if (a.lse)
        a.lse[static_cast<int64_t>(b) * a.q_heads + head] =
            l > 0.0f ? (m - shift) * 0.69314718055994531f + logf(l) : l == 0.0f ? -INFINITY : m;
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, 1) attn_kernel(AttnArgs a, int page_shift) {
    constexpr int NT = S::NT, R = S::R, DP = S::DP, ROWS = S::ROWS, STEP = S::STEP, W = S::W;
    constexpr int NST = S::NST, MS = S::MS, CH = S::CH;
    constexpr int T = S::BF ? 1 : 0;                  // type of the weights
    constexpr float kShift = S::BF ? 0.0f : 7.0f;     // see the weights below
    extern __shared__ __align__(1024) unsigned char smem[];
    float* so = reinterpret_cast<float*>(smem + S::RING);        // [W][ROWS][OP]
    // per step of the ring: its keys are there, its values are there, it may be refilled
    uint64_t* bars = reinterpret_cast<uint64_t*>(so + W * ROWS * S::OP);
    uint32_t* metas = reinterpret_cast<uint32_t*>(bars + 3 * NST);   // which tokens have a page
    __shared__ int abort_flag;
    __shared__ float sm_m[W][ROWS], sm_l[W][ROWS];
    __shared__ Line line;
    __shared__ long long scan[W + S::PW];
    __shared__ int tops[W + S::PW];
    __shared__ long long prefix[S::THREADS];
    __shared__ Segment segs[2];                // the current one and the one after it, in turn
    __shared__ int share_n;
    __shared__ Cut cuts[2];                    // an item begun by an earlier CTA, one left to a later

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, i = lane & 3;
    const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    const int G = a.q_heads / a.kv_heads;
    const int row_tiles = (G + ROWS - 1) / ROWS;
    const int items_per_seq = a.kv_heads * row_tiles;
    const int row_bytes = a.head_dim * S::ES;
    int* counters = static_cast<int*>(a.workspace);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + attn_counter_bytes(ctas));

    if (row_bytes < S::PITCH) {  // columns past the head dimension are never copied: zero
        for (int e = tid; e < S::RING / 16; e += S::THREADS)
            reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
    }
    const uint32_t full_k = smem_addr(bars), full_v = full_k + 8 * NST, empty = full_v + 8 * NST;
    if (tid < NST) {
        mbar_init(full_k + 8 * tid, 33);  // 32 lanes' copies, and the word of `metas`
        mbar_init(full_v + 8 * tid, 32);
        mbar_init(empty + 8 * tid, 1);
    }
    if (tid == 0) abort_flag = 0;
    grid_dep_wait();
    lay_line<STEP, S::THREADS, W, S::WHOLE>(a, items_per_seq, ctas, cta == 0, line, prefix, scan, tops);
    const int per_thread = (a.B + S::THREADS - 1) / S::THREADS;
    // rows with nothing to attend to
    for (int b = cta; b < a.B; b += ctas) {
        if (visible(a, b, false).len != 0) continue;
        uint16_t* o = a.out + b * a.ldo;
        for (int e = tid; e < a.q_heads * a.head_dim; e += S::THREADS) o[e] = 0;
        if (a.lse)
            for (int h = tid; h < a.q_heads; h += S::THREADS)
                a.lse[static_cast<int64_t>(b) * a.q_heads + h] = -INFINITY;
    }
    __syncthreads();  // line, prefix, the barriers, and the zeroed ring

    // the segment after `s`, where more_after(s): the next item's first steps
    auto after = [&](const Segment& s) {
        Segment n = s;
        if (++n.item == items_per_seq) {
            n.item = 0;
            do {
                ++n.b;
                n.span = visible(a, n.b, false);
                n.n_steps = span_steps<STEP>(n.span);
            } while (n.n_steps == 0 && n.b + 1 < a.B);
        }
        n.step = 0;
        n.step_end = line.whole ? n.n_steps : min(n.n_steps, s.rest - kItemCost);
        n.rest = s.rest - kItemCost - n.n_steps;
        return n;
    };

    auto more_after = [&](const Segment& s) { return s.rest > (line.whole ? 0 : kItemCost); };

    // The first segment of the CTA's share; false: there is none.  By all lanes of a warp.
    const long long share_end = min(line.end, line.share * (cta + 1));   // in the line (not `apart`)
    auto locate = [&](Segment& first) {
        if (line.apart) {  // the cta-th part of all items
            int done = 0;
            bool found = false;
            for (int b0 = 0; b0 < a.B && !found; b0 += 32) {
                const int b = b0 + lane, share = static_cast<int>(line.share);
                const Span span = b < a.B ? visible(a, b, false) : Span{0, 0};
                const int n_steps = span_steps<STEP>(span), per = parts_of(line, n_steps);
                int incl = per * items_per_seq;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= d) incl += o;
                }
                const int at = cta - done - (incl - per * items_per_seq);
                const bool here = at >= 0 && at < per * items_per_seq;
                const int step = here ? at % per * share : 0;
                const unsigned who = __ballot_sync(0xFFFFFFFFu, here);
                if (who) {
                    const int from = __ffs(who) - 1;
                    auto get = [&](int v) { return __shfl_sync(0xFFFFFFFFu, v, from); };
                    first = Segment{get(b), get(here ? at / per : 0), get(step), get(min(n_steps, step + share)),
                                    get(n_steps), 0, Span{get(span.first), get(span.len)}};
                    found = true;
                }
                done += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            return found;
        }
        const long long u = line.share * cta;
        if (u >= line.end) return false;
        // the thread whose sequences hold place u, then the sequence
        int t = 0;
        for (int t0 = 0; t0 < S::THREADS && t0 * per_thread < a.B; t0 += 32)
            t += __popc(__ballot_sync(0xFFFFFFFFu, prefix[t0 + lane] <= u));
        --t;
        long long at = prefix[t];
        int b = t * per_thread;
        Span span = visible(a, b, false);
        int n_steps = span_steps<STEP>(span);
        auto length = [&]() { return n_steps ? static_cast<long long>(n_steps + kItemCost) * items_per_seq : 0ll; };
        while (at + length() <= u && b + 1 < a.B) {
            at += length();
            span = visible(a, ++b, false);
            n_steps = span_steps<STEP>(span);
        }
        const int item = static_cast<int>(quotient(u - at, n_steps + kItemCost));
        const long long begin = at + static_cast<long long>(item) * (n_steps + kItemCost);
        const int step = max(static_cast<int>(u - begin) - kItemCost, 0);
        const int rest = static_cast<int>(share_end - begin) - kItemCost - n_steps;
        first = Segment{b, item, step, min(n_steps, n_steps + rest), n_steps, rest, span};
        if (line.whole ? u == begin : first.step < first.step_end) {
            if (line.whole) first.step_end = n_steps;
            return true;
        }
        if (!more_after(first)) return false;   // the share ends before any step
        first = after(first);
        return true;
    };

    const uint32_t ring = smem_addr(smem);
    if (warp >= W) {
        // ---- producers: steps pw, pw + PW, ... of the share ----
        const int pw = warp - W;
        Segment ld{};
        constexpr int RPI = 32 / CH;   // token rows that one instruction of the warp copies
        static_assert(CH <= 32, "a row is one instruction at most");
        const int lrow = lane / CH, lchunk = lane % CH;
        const bool column = 16 * lchunk < row_bytes;    // this lane's chunk is within the head
        const int64_t kss = a.kc.slot_stride * S::ES, vss = a.vc.slot_stride * S::ES;
        const int64_t kps = a.kc.page_stride * S::ES, vps = a.vc.page_stride * S::ES;
        const uint32_t lane_at = ring_at<CH>(lrow, lchunk);
        auto page_of = [&](int tok) { return page_shift >= 0 ? tok >> page_shift : tok / a.page_size; };
        auto wanted = [&](int tok) {
            return tok < ld.span.len && tok + S::PG > ld.span.first;
        };
        // Page numbers.  Groups: lane n NG + r has that of group r of the warp's n-th step from the
        // batch's first on, 32 / NG steps at a time and the next ones under way; else lane t
        // has that of token t of the next step.
        constexpr int NG = S::NG, PB = S::GROUPS ? 32 / NG : 1;
        const int32_t* table;
        const char* kbase;
        const char* vbase;
        int first_st = 0, pid = 0, pid_next = 0, in_batch = 0;
        auto fetch_pages = [&](int st) {
            const int s_ = S::GROUPS ? st + lane / NG * S::PW : st;
            const int tok = s_ * STEP + (S::GROUPS ? S::PG * (lane % NG) : lane);
            int p = 0;
            if (s_ < first_st + ld.step_end && (S::GROUPS || lane < STEP) && wanted(tok)) p = table[page_of(tok)];
            return p;
        };
        auto open = [&](int st) {  // begins segment ld at token step ld's first + st
            const int head = ld.item / row_tiles;
            first_st = ld.span.first / STEP;
            table = a.block_table + ld.b * a.ld_table;
            kbase = static_cast<const char*>(a.kc.p) + head * a.kc.head_stride * S::ES + lrow * kss + 16 * lchunk;
            vbase = static_cast<const char*>(a.vc.p) + head * a.vc.head_stride * S::ES + lrow * vss + 16 * lchunk;
            pid = fetch_pages(first_st + st);
            pid_next = fetch_pages(first_st + st + PB * S::PW);
            in_batch = 0;
        };
        // one side's copies of a step: rows of `at` (bytes from base: of each group's first row,
        // or of the lane's token); of a partial step those with `lo` <= token < `hi` and a page,
        // zeros for the others
        auto copy = [&](uint32_t dst, const char* base, const int64_t (&at)[NG], int64_t stride,
                        uint32_t there, int lo, int hi, bool partial) {
            if constexpr (S::GROUPS) {
                auto all = [&](auto ok_of) {
#pragma unroll
                    for (int r = 0; r < NG; ++r) {
                        const char* p = base + at[r];
#pragma unroll
                        for (int j = 0; j < S::PG / RPI; ++j) {
                            const uint32_t to = (dst ^ (CH >= 8 ? ((RPI * j) & 7) << 4 : 0)) + (S::PG * r + RPI * j) * S::PITCH;
                            const bool ok = ok_of(r, S::PG * r + RPI * j + lrow);
                            if (column) copy16(to, ok ? p : base, ok ? 16 : 0);
                            p += RPI * stride;
                        }
                    }
                };
                if (!partial) all([](int, int) { return true; });
                else all([&](int r, int t) { return ((there >> r) & 1u) && t >= lo && t < hi; });
            } else {
#pragma unroll
                for (int t0 = 0; t0 < STEP; t0 += RPI) {
                    const int t = t0 + lrow;
                    const char* p = base - lrow * stride + __shfl_sync(0xFFFFFFFFu, at[0], t);
                    const bool ok = ((there >> t) & 1u) && t >= lo && t < hi;
                    const uint32_t to = (dst ^ (CH >= 8 ? (t0 & 7) << 4 : 0)) + t0 * S::PITCH;
                    if (column) copy16(to, ok ? p : base, ok ? 16 : 0);
                }
            }
        };
        int seg0 = 0;            // the share's steps before segment ld
        int stage = pw, x = pw;  // of this warp's next step
        uint32_t phase = 0;
#pragma unroll 1
        for (bool more = locate(ld); more;) {
        const int seg_end = seg0 + ld.step_end - ld.step;
        if (x < seg_end) open(ld.step + x - seg0);
#pragma unroll 1
        for (; x < seg_end; x += S::PW) {
            const int st = first_st + ld.step + x - seg0;
            int64_t kat[NG], vat[NG];
            uint32_t there = 0;  // groups, or tokens, whose page is there
#pragma unroll
            for (int r = 0; r < NG; ++r) {
                const int tok = st * STEP + (S::GROUPS ? S::PG * r : lane);
                const int page = S::GROUPS ? __shfl_sync(0xFFFFFFFFu, pid, in_batch * NG + r) : pid;
                const bool in = wanted(tok) && (S::GROUPS || lane < STEP);
                const bool ok = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
                if (in && !ok) record_status(a.status, kDecInvalidArg);
                const int slot = tok - page_of(tok) * a.page_size;
                kat[r] = ok ? page * kps + slot * kss : 0;
                vat[r] = ok ? page * vps + slot * vss : 0;
                if constexpr (S::GROUPS) there |= static_cast<uint32_t>(ok) << r;
                else there = __ballot_sync(0xFFFFFFFFu, ok);
            }
            const int lo = ld.span.first - st * STEP, hi = ld.span.len - st * STEP;
            const bool partial = there != (1u << NG) - 1 || lo > 0 || hi < STEP;
            mbar_wait_warp(empty + 8 * stage, phase ^ 1u, &abort_flag, a.status, a.timeout_ns);
            const uint32_t dst = ring + stage * 2 * S::SLOT + lane_at;
            if (lane == 0) {
                metas[stage] = there;
                mbar_arrive(full_k + 8 * stage);
            }
            copy(dst, kbase, kat, kss, there, lo, hi, partial);
            copies_arrive(full_k + 8 * stage);
            copy(dst + S::SLOT, vbase, vat, vss, there, lo, hi, partial);
            copies_arrive(full_v + 8 * stage);
            if (++in_batch == PB) {
                in_batch = 0;
                pid = pid_next;
                pid_next = fetch_pages(st + (PB + 1) * S::PW);  // the batch after the one from st + PW on
            }
            stage += S::PW;
            if (stage >= NST) stage -= NST, phase ^= 1u;
        }
        seg0 = seg_end;
        more = more_after(ld);
        if (more) ld = after(ld);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }

    // ---- consumers ----
    constexpr int CT = 32 * W;  // their threads
    constexpr int E = (ROWS * DP / 4 + CT - 1) / CT;  // 16-byte pieces of a result per thread
    // ---- parts of an item that several CTAs hold ----
    auto part_of = [&](const Cut& c, int k) {  // part k of the item
        return parts + (2 * (c.c0 + k) + (k == 0 ? 1 : 0)) * attn_part_floats(ROWS, DP);
    };
    // One row of an item from its parts, by one warp: lane k has part k's m and l (of 32 parts at
    // a time), kAtOnce parts' values are under way together.
    constexpr int JV = DP > 128 ? DP / 128 : 1;      // 16-byte pieces of a row per lane
    constexpr int JS = DP < 128 ? 128 / DP : 1;      // parts that a warp reads side by side
    constexpr int kAtOnce = 16 / JV;
    auto join_row = [&](const Cut& c, int row, int k_first, int stride, int count, bool final) {
        const int sub = lane / (32 / JS), l4 = 4 * (lane % (32 / JS));
        float top = -INFINITY, sum = 0.0f;
        float4 acc[JV];
#pragma unroll
        for (int v = 0; v < JV; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int k32 = 0; k32 < count; k32 += 32) {
            const int mine = k32 + lane;
            const float pm = mine < count ? __ldcg(part_of(c, k_first + mine * stride) + row) : -INFINITY;
            const float pl = mine < count ? __ldcg(part_of(c, k_first + mine * stride) + ROWS + row) : 0.0f;
            float f = 0.0f;
#pragma unroll 1
            for (int k0 = 0; k0 < 32 && k32 + k0 < count; k0 += kAtOnce * JS) {
                float4 x[kAtOnce][JV];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                    for (int v = 0; v < JV; ++v) {
                        const int k = k32 + k0 + j * JS + sub, d = l4 + 128 * v;
                        x[j][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (k < count && d < a.head_dim)
                            x[j][v] = __ldcg(reinterpret_cast<const float4*>(part_of(c, k_first + k * stride) + 2 * ROWS + row * DP + d));
                    }
                if (k0 == 0) {  // the new maximum, and what it makes of the sums so far
                    const float now = max_nan(top, warp_max_nan(pm));
                    const float old = top == -INFINITY ? 0.0f : exp2_fast(top - now);
                    top = now;
                    f = pm == -INFINITY ? 0.0f : exp2_fast(pm - now);
                    sum = sum * old + warp_sum(pl * f);
#pragma unroll
                    for (int v = 0; v < JV; ++v) acc[v].x *= old, acc[v].y *= old, acc[v].z *= old, acc[v].w *= old;
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const float fk = __shfl_sync(0xFFFFFFFFu, f, (k0 + j * JS + sub) & 31);
#pragma unroll
                    for (int v = 0; v < JV; ++v) {
                        acc[v].x = fmaf(x[j][v].x, fk, acc[v].x), acc[v].y = fmaf(x[j][v].y, fk, acc[v].y);
                        acc[v].z = fmaf(x[j][v].z, fk, acc[v].z), acc[v].w = fmaf(x[j][v].w, fk, acc[v].w);
                    }
                }
            }
        }
        if constexpr (JS == 2) {
            acc[0].x += __shfl_xor_sync(0xFFFFFFFFu, acc[0].x, 16), acc[0].y += __shfl_xor_sync(0xFFFFFFFFu, acc[0].y, 16);
            acc[0].z += __shfl_xor_sync(0xFFFFFFFFu, acc[0].z, 16), acc[0].w += __shfl_xor_sync(0xFFFFFFFFu, acc[0].w, 16);
        }
        if (!final) {  // a run's result stands where its first part did
            float* to = part_of(c, k_first);
#pragma unroll
            for (int v = 0; v < JV; ++v)
                if (sub == 0) *reinterpret_cast<float4*>(to + 2 * ROWS + row * DP + l4 + 128 * v) = acc[v];
            if (lane == 0) to[row] = top, to[ROWS + row] = sum;
            return;
        }
        const float f = sum == 0.0f ? 0.0f : c.vs / sum;
#pragma unroll
        for (int v = 0; v < JV; ++v)
            if (sub == 0 && l4 + 128 * v < a.head_dim) store_out<S::DT>(a, c.b, c.head0 + row, l4 + 128 * v, acc[v], f);
        if (lane == 0) store_lse(a, c.b, c.head0 + row, top, sum, kShift);
    };
    // Counts the parts written, and joins what they complete, a row per warp.  Over 32 parts are
    // joined in two rounds, runs of 16 first, so that several CTAs read them (one sequence of
    // 131072 tokens with one key-value head, 147 parts: 39.7 us in one round, 25.8 in two).
    auto settle = [&](int n_cuts) {
        auto fan_of = [](const Cut& c) { return c.n <= 32 ? 32 : 16; };
        __threadfence();
        consumers_sync<CT>();
        if (tid < n_cuts) {
            Cut& c = cuts[tid];
            // counters by the CTA of the run's first part.  That CTA may end one item and begin
            // another, so first runs, later runs and second rounds count apart.
            const int fan = fan_of(c), run = c.at / fan;
            int* counter = counters + (run == 0 ? 0 : ctas) + c.c0 + run * fan;
            c.last = atomicAdd(counter, 1) == min(fan, c.n - run * fan) - 1;
            if (c.last) *counter = 0;  // ready for the next call
            __threadfence();
        }
        consumers_sync<CT>();
        bool again = false;
        int nth = 0;
        for (int j = 0; j < n_cuts; ++j) {
            if (!cuts[j].last) continue;
            const Cut c = cuts[j];
            const int fan = fan_of(c), run = c.at / fan;
            again |= c.n > fan;
            for (int row = 0; row < c.rows; ++row)
                if (nth++ % W == warp) join_row(c, row, run * fan, 1, min(fan, c.n - run * fan), c.n <= fan);
        }
        if (!again) return;
        __threadfence();
        consumers_sync<CT>();
        if (tid < n_cuts && cuts[tid].last) {
            Cut& c = cuts[tid];
            const int fan = fan_of(c), runs = (c.n + fan - 1) / fan;
            int* counter = counters + 2 * ctas + c.c0;
            c.last = runs > 1 && atomicAdd(counter, 1) == runs - 1;
            if (c.last) *counter = 0;
            __threadfence();
        }
        consumers_sync<CT>();
        for (int j = 0; j < n_cuts; ++j) {
            if (!cuts[j].last) continue;
            const Cut c = cuts[j];
            for (int row = warp; row < c.rows; row += W) join_row(c, row, 0, fan_of(c), (c.n + 15) / 16, true);
        }
    };

    // ---- addresses of ldmatrix's rows in a slot, for this lane ----
    const int mi = lane >> 3, l7 = lane & 7;
    const uint32_t kfrag = ring_at<CH>((mi & 1) * 8 + l7, mi >> 1);
    const uint32_t vfrag = S::E4M3 ? kfrag : ring_at<CH>((mi >> 1) * 8 + l7, mi & 1);
    // chunk pair c, c + 1 (c even) of group r, from the address of chunk pair 0
    auto pair_at = [](int r, int c) {
        return static_cast<uint32_t>(r * 16 * S::PITCH + (CH >= 8 ? (c & ~7) << 4 : 0));
    };

    if (warp == 0) {
        Segment first{};
        const bool any = locate(first);
        if (lane == 0) segs[0] = first, share_n = any;
    }
    consumers_sync<CT>();
    if (!share_n) return;
    long long begin = share_end - segs[0].rest - kItemCost - segs[0].n_steps;  // of the item in the line
    int taken = 0;             // the share's steps before the segment
    int n_cuts = 0;
    // queries as B fragments: lane (g, i) has four values of row 8 nt + g per MMA step
    uint32_t qf[NT][MS][2];
    auto load_q = [&](const Segment& seg) {
        const int kvh = seg.item / row_tiles, row0 = (seg.item - kvh * row_tiles) * ROWS;
        const int rows = min(ROWS, G - row0), head0 = kvh * G + row0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const uint16_t* q = a.q + seg.b * a.ldq + static_cast<int64_t>(head0 + r) * a.head_dim;
#pragma unroll
            for (int ms = 0; ms < MS; ++ms)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = S::E4M3 ? 16 * ms + 4 * i + 2 * h : 16 * ms + 8 * h + 2 * i;
                    qf[nt][ms][h] = r < rows && col < a.head_dim ? *reinterpret_cast<const uint32_t*>(q + col) : 0;
                }
        }
    };
    bool have_q = false;
    for (int turn = 0;; turn ^= 1) {
        const Segment& cur = segs[turn];
        const bool more = more_after(cur);
        if (more && tid == 0) segs[turn ^ 1] = after(cur);
        const int kvh = cur.item / row_tiles, row0 = (cur.item - kvh * row_tiles) * ROWS;
        const int rows = min(ROWS, G - row0), head0 = kvh * G + row0;
        const Span span = cur.span;

        if (!have_q) load_q(cur);
        have_q = false;
        // With an 8-bit cache the MMA is fp16: bf16 queries are scaled there by a power of
        // two per row that brings the largest to 2^8..2^9, undone in the row's factor (beside an
        // infinity or a NaN, as for the largest finite number).
        float fct[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f = a.scale * 1.4426950408889634f;
            if (S::E4M3 && a.kc.scale) f *= a.kc.scale[kvh];
            if constexpr (S::E4M3 && S::DT == 1) {
                uint32_t top = 0;  // of the magnitudes, as numbers of 15 bits
#pragma unroll
                for (int ms = 0; ms < MS; ++ms)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        top = max(top, max(qf[nt][ms][h] & 0x7FFFu, (qf[nt][ms][h] >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int e = min(static_cast<int>(top >> 7) - 127, 127);
                float up = 1.0f;
                if (e > -119) {
                    up = __uint_as_float(static_cast<uint32_t>(8 - e + 127) << 23);
                    f *= __uint_as_float(static_cast<uint32_t>(e - 8 + 127) << 23);
                }
#pragma unroll
                for (int ms = 0; ms < MS; ++ms)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t v = qf[nt][ms][h];
                        qf[nt][ms][h] = dec_pack2<0>(__uint_as_float(v << 16) * up,
                                                     __uint_as_float(v & 0xFFFF0000u) * up);
                    }
            }
            fct[nt][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * i);      // of rows 2i and 2i + 1
            fct[nt][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * i + 4);
        }

        // ---- the warp's steps ----
        float m[NT][2], ref[NT][2], l[NT][2], o[NT][MS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) m[nt][c] = -INFINITY, ref[nt][c] = 0.0f, l[nt][c] = 0.0f;
#pragma unroll
            for (int s = 0; s < MS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.0f;
        }
        const int st1 = span.first / STEP + cur.step_end;
        // A step's warp follows from its place in the item alone: the sums of a part then do
        // not depend on what the CTA did before.
        int st = span.first / STEP + cur.step + ((warp - cur.step - cur.item) & (W - 1));
        int x = taken + st - span.first / STEP - cur.step;
        int stage = x % NST;
        uint32_t phase = (x / NST) & 1;
        taken += cur.step_end - cur.step;
#pragma unroll 1
        for (; st < st1; st += W) {
            const uint32_t kslot = ring + stage * 2 * S::SLOT, vslot = kslot + S::SLOT;
            mbar_wait_warp(full_k + 8 * stage, phase, &abort_flag, a.status, a.timeout_ns);
            const uint32_t there = metas[stage];
            float s[R][NT][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s2[NT][4];  // two sums at a time: half the MMA's latency
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][nt][e] = s2[nt][e] = 0.0f;
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t k[4];
                    ldmatrix4<false>(k, kslot + (kfrag ^ ((c & 7) << 4)) + pair_at(r, c));
                    if constexpr (S::E4M3) {  // chunks c and c + 1 are a step each
                        const uint32_t a0 = dec_e4m3x2_to_f16x2(k[0]), a1 = dec_e4m3x2_to_f16x2(k[1]);
                        const uint32_t a2 = dec_e4m3x2_to_f16x2(k[0] >> 16), a3 = dec_e4m3x2_to_f16x2(k[1] >> 16);
                        const uint32_t b0 = dec_e4m3x2_to_f16x2(k[2]), b1 = dec_e4m3x2_to_f16x2(k[3]);
                        const uint32_t b2 = dec_e4m3x2_to_f16x2(k[2] >> 16), b3 = dec_e4m3x2_to_f16x2(k[3] >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<S::BF>(s[r][nt], a0, a1, a2, a3, qf[nt][c][0], qf[nt][c][1]);
                            mma16816<S::BF>(s2[nt], b0, b1, b2, b3, qf[nt][c + 1][0], qf[nt][c + 1][1]);
                        }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float(&to)[4] = (c & 2) ? s2[nt] : s[r][nt];
                            mma16816<S::BF>(to, k[0], k[1], k[2], k[3], qf[nt][c / 2][0], qf[nt][c / 2][1]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][nt][e] += s2[nt][e];
            }
            // scores in units of log 2; those of tokens that do not count are -inf
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r][nt][e] *= fct[nt][e & 1];
            if (!S::GROUPS || there != (1u << S::NG) - 1 || st * STEP < span.first || st * STEP + STEP > span.len) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = 16 * r + g + 8 * h, tok = st * STEP + t;
                        const bool ok = ((there >> (S::GROUPS ? (16 * r + 8 * h) / S::PG : t)) & 1u) && tok >= span.first && tok < span.len;
                        if (!ok) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[r][nt][2 * h] = s[r][nt][2 * h + 1] = -INFINITY;
                        }
                    }
            }
            bool passed = false;
            float tops[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < R; ++r) top = max_nan(top, max_nan(s[r][nt][c], s[r][nt][c + 2]));
                    tops[nt][c] = top;
                    passed |= !(top <= m[nt][c] + kLag);
                }
            if (__any_sync(0xFFFFFFFFu, passed)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = max_nan(m[nt][c], tops[nt][c]);
                        top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const float f = top == m[nt][c] ? 1.0f : exp2_fast(m[nt][c] - top);
                        m[nt][c] = top;
                        ref[nt][c] = top == -INFINITY ? 0.0f : top - kShift;
                        l[nt][c] *= f;
#pragma unroll
                        for (int ms = 0; ms < MS; ++ms) {
                            o[nt][ms][c] *= f;
                            o[nt][ms][c + 2] *= f;
                        }
                    }
            }
            // weights, split in 16-bit parts, as B fragments.  fp16 keeps 2^-14 as its
            // smallest full number: its weights are scaled by 2^7 (at most 2^15 with the lag).  What is
            // below 2^-25 of it, 2^-32 of the row's largest weight, is lost.
            uint32_t ph[R][NT][2], pl[R][NT][2];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            p[c] = exp2_fast(s[r][nt][2 * h + c] - ref[nt][c]);
                            l[nt][c] += p[c];
                        }
                        const uint32_t hi = S::E4M3 ? dec_pack2<T>(p[0], p[1]) : pack_below<T>(p[0], p[1]);
                        const float low0 = p[0] - dec_to_f32<T>(static_cast<uint16_t>(hi & 0xFFFFu));
                        const float low1 = p[1] - dec_to_f32<T>(static_cast<uint16_t>(hi >> 16));
                        ph[r][nt][h] = transpose8x8(hi);
                        pl[r][nt][h] = transpose8x8(dec_pack2<T>(low0, low1));
                    }
            mbar_wait_warp(full_v + 8 * stage, phase, &abort_flag, a.status, a.timeout_ns);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t v[4];
                    ldmatrix4<true>(v, vslot + (vfrag ^ ((c & 7) << 4)) + pair_at(r, c));
                    auto accumulate = [&](int ms, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<S::BF>(o[nt][ms], a0, a1, a2, a3, ph[r][nt][0], ph[r][nt][1]);
                            mma16816<S::BF>(o[nt][ms], a0, a1, a2, a3, pl[r][nt][0], pl[r][nt][1]);
                        }
                    };
                    if constexpr (S::E4M3) {
                        // a pair of bytes per token: (d, d + 1) of tokens 2i, 2i + 1 to pairs of tokens
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = __byte_perm(v[2 * h], 0, 0x3120);
                            const uint32_t y = __byte_perm(v[2 * h + 1], 0, 0x3120);
                            accumulate(c + h, dec_e4m3x2_to_f16x2(x), dec_e4m3x2_to_f16x2(x >> 16),
                                       dec_e4m3x2_to_f16x2(y), dec_e4m3x2_to_f16x2(y >> 16));
                        }
                    } else {
                        accumulate(c / 2, v[0], v[1], v[2], v[3]);
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            stage += W;
            if (stage >= NST) stage -= NST, phase ^= 1u;
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
            }
        float4 acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * nt + 2 * i + c;
                if (row >= rows) continue;
                float* dst = so + (warp * ROWS + row) * S::OP;
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) {
                    dst[16 * ms + (S::E4M3 ? 2 * g : g)] = o[nt][ms][c];
                    dst[16 * ms + (S::E4M3 ? 2 * g + 1 : g + 8)] = o[nt][ms][c + 2];
                }
            }
        consumers_sync<CT>();
        if (more) load_q(segs[turn ^ 1]), have_q = true;  // under way meanwhile
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int at = tid + e * CT, row = at / (DP / 4), d = 4 * (at % (DP / 4));
            if (row >= rows) continue;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) top = max_nan(top, sm_m[w][row]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float mw = sm_m[w][row];
                const float f = mw == -INFINITY ? 0.0f : exp2_fast(mw - top);
                const float4 x = *reinterpret_cast<const float4*>(so + (w * ROWS + row) * S::OP + d);
                acc[e].x = fmaf(x.x, f, acc[e].x), acc[e].y = fmaf(x.y, f, acc[e].y);
                acc[e].z = fmaf(x.z, f, acc[e].z), acc[e].w = fmaf(x.w, f, acc[e].w);
            }
        }
        auto row_sum = [&](int row, float& top) {
            top = -INFINITY;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) top = max_nan(top, sm_m[w][row]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float mw = sm_m[w][row];
                sum += mw == -INFINITY ? 0.0f : sm_l[w][row] * exp2_fast(mw - top);
            }
            return sum;
        };
        const bool begins = cur.step == 0, ends = cur.step_end == cur.n_steps;
        const bool whole = begins && ends;
        const float vs = S::E4M3 && a.vc.scale ? a.vc.scale[kvh] : 1.0f;
        float* part = parts + (2 * cta + (begins ? 1 : 0)) * attn_part_floats(ROWS, DP);
        float top;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int at = tid + e * CT, row = at / (DP / 4), d = 4 * (at % (DP / 4));
            if (row >= rows || d >= a.head_dim) continue;
            if (whole) {
                const float sum = row_sum(row, top);
                store_out<S::DT>(a, cur.b, head0 + row, d, acc[e], sum == 0.0f ? 0.0f : vs / sum);
            } else {
                *reinterpret_cast<float4*>(part + 2 * ROWS + row * DP + d) = acc[e];
            }
        }
        if (tid < rows) {
            const float sum = row_sum(tid, top);
            if (whole) store_lse(a, cur.b, head0 + tid, top, sum, kShift);
            else part[tid] = top, part[ROWS + tid] = sum;
        }
        if (!whole) {
            Cut c{0, 0, 0, cur.b, head0, rows, 0, vs};
            if (line.apart) {
                c.at = static_cast<int>(quotient(cur.step, line.share));
                c.c0 = cta - c.at;
                c.n = parts_of(line, cur.n_steps);
            } else {
                c.c0 = static_cast<int>(quotient(begin + kItemCost, line.share));
                c.at = cta - c.c0;
                c.n = static_cast<int>(quotient(begin + kItemCost + cur.n_steps - 1, line.share)) - c.c0 + 1;
            }
            if (tid == 0) cuts[n_cuts] = c;
            ++n_cuts;
        }
        if (!more) break;
        begin += kItemCost + cur.n_steps;
        consumers_sync<CT>();
    }
    if (n_cuts) settle(n_cuts);
}

template <class S>
int launch_attn_shape(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    if (cudaFuncSetAttribute(attn_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) !=
        cudaSuccess)
        return -3;
    return launch_dependent(attn_kernel<S>, dim3(static_cast<unsigned>(ctx.num_sms)),
                            dim3(S::THREADS), S::SMEM, stream, a, power_of_two(a.page_size));
}

template <int DT, bool E4M3, int DP>
int launch_attn_dp(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream) {
    const bool narrow = a.q_heads / a.kv_heads <= 8;
    if (a.page_size % 16 == 0)
        return narrow ? launch_attn_shape<AttnShape<DT, E4M3, DP, 1, 16>>(ctx, a, stream)
                      : launch_attn_shape<AttnShape<DT, E4M3, DP, 2, 16>>(ctx, a, stream);
    if (a.page_size % 8 == 0)
        return narrow ? launch_attn_shape<AttnShape<DT, E4M3, DP, 1, 8>>(ctx, a, stream)
                      : launch_attn_shape<AttnShape<DT, E4M3, DP, 2, 8>>(ctx, a, stream);
    return narrow ? launch_attn_shape<AttnShape<DT, E4M3, DP, 1, 1>>(ctx, a, stream)
                  : launch_attn_shape<AttnShape<DT, E4M3, DP, 2, 1>>(ctx, a, stream);
}

}  // namespace

// One instance per translation unit (attn_*.cu), which compile in parallel.
template <int DT, bool E4M3>
int launch_attn_typed(const DeviceCtx& ctx, const AttnArgs& a, cudaStream_t stream);

}  // namespace w4g
