// Attention of drafted tokens over a paged key-value cache (include/decode.h).
//
// With G query heads per key-value head, n drafted tokens are G n rows that read the same keys and
// values: 2 G n operations per byte of a 16-bit cache, 512 rows for 64 tokens of 8 heads.  The
// kernel reads the cache once per item (up to 256 rows of one sequence and key-value head) and
// multiplies on tcgen05 in tiles of 128 rows:
//   S = Q K^T   128 rows x 128 tokens, fp32 in TMEM; both operands in shared memory, K-major;
//   O += P V    P in TMEM, in the place of S; V in shared memory, its rows as they come from the
//               cache: the MN-major operand.
// (mma.sync, which dec_attn_paged uses for its few rows, would be short from some 40 rows on.)
// P is carried as two 16-bit parts, each multiplied with V (a single rounding to bf16, 2^-8, would
// show in the result as much as the result's own); a block of 16 tokens' S, 16 columns, holds both
// parts of its P.  The softmax's state and all sums are fp32.  So a step of 128 tokens and 128 rows is some 1600
// cycles of the tensor pipe (512 for S, 1024 for P V at the peak), against the 2800 that an SM's share of the
// memory takes for its 64 KB: padding rows cost nothing while the cache streams.
//
// Roles: two warps issue the MMAs, one for each of two streams of (S, O) in TMEM; two softmax warpgroups, one
// for each stream, a thread per row; loaders.  An item of more than 128 rows has a stream per tile of
// 128; one of fewer gives its steps to the streams in turn, whose sums are joined at its end.  While one
// stream's softmax runs the tensor pipe works on the other's products; streams at work together take turns,
// a stream's P V and next S as one, which keeps them half a round apart (a step of both 5.0 thousand cycles
// instead of 5.7).  (Heads of more than 128 values: one stream, whose S alternates between two places; O
// alone takes half of TMEM.)
// All copies and MMAs of a warp are issued by one thread with operands that are known to be the same in all
// lanes; issued by several lanes, or from registers that might differ, each takes several times as long.
//
// Loaders, 16-bit cache: two warps, one has the keys, the other queries and values, as tensor copies (a box is
// up to 128 tokens of a page, one head) into a ring of 128 KB, keys and values in turn.  8-bit cache: a warp
// copies the raw tiles, five convert them to fp16, exactly, into the ring, which takes them some 900 cycles a
// tile and bounds this form (16 sequences of up to 4096, 64 heads on 8, 8 drafted: 48 us, and 43 with the bf16 cache of
// twice the bytes; with the rows' conversions one after another 66 against 45).  Pages that no tensor map
// describes (sizes that no 8 divides, strides of 0) are copied 16 bytes at a time: the same batch takes 43 us
// with bf16 pages of 64, 69 with pages of 5 and of 1; 114 with 8-bit pages of 5.
//
// Softmax.  A running reference m per row: weights are exp2(s - m); only when a score passes m by
// more than 2^8 is O, in TMEM, scaled to a new reference.  Maxima carry NaN, and come with the loads from TMEM.
// Its loops stay loops: the roles' code together has to fit in the instruction cache.
//
// Masks are applied to S by index (words of 32 tokens per row) in the steps that need them: the
// drafted tokens' and those at the window's edges.  Values of such tokens that are infinite or NaN are
// replaced by 0 in shared memory, as 0 times them would reach the rows that do not see them, and
// added at the end to the rows that do.
//
// Work split.  All items of the batch stand in one line, each as long as its steps, weighted, and
// kTreeItemCost, cut in equal shares, one per CTA.  An item that is cut leaves (m, l, O) of each
// part in fp32 in the workspace, and a second kernel joins the parts in their order, 32 rows and columns a
// block (one sequence of 131072, 8 drafted: 106 to 109 us; 112 with 32 rows and all columns a block).
//
// What bounds it.  16 sequences of up to 4096 tokens, 16 drafted, 32 heads on 32, fp16: memory, 546 MB in 106 us, 5.2
// TB/s, and the ends of 512 short items.  32 sequences of up to 8192, 32 drafted, 64 heads on 8: the tensor pipe (59 %
// busy; 154 us: 540 TFLOP/s, 815 with P's two parts), and between its turns the softmax's chain from S to P.
// One tree of 8 over 777 tokens: 16 us of code that runs once.
#pragma once
#include "decode.cuh"

namespace w4g {

// The line's units: a step of an item of one tile, of one of two, and an item by itself.  (32 ragged sequences, trees of
// up to 32: 152 us; 162 with equal steps, and 176 with an item as one of them.  16 sequences with 32 of 32
// heads: 110 us; 114 with an item as two steps, 121 as one.)
constexpr int kTreeStep = 2, kTreeDualStep = 3, kTreeItemCost = 6;
constexpr float kTreeLag = 8.0f;   // scores may pass the reference by 2^8
constexpr int kTreeRows = 128;     // of a tile: the MMA's M

// Of the workspace: a TreePart per CTA, then two parts per CTA (an item begun by an earlier CTA, one left
// to a later) of m[rows], l[rows], O[dp / 4][rows][4], rows being 128 for each stream.
struct TreePart {
    int n;       // parts of the item that this CTA begins and another ends; 0: none
    int row0;    // its first row in q and out is that of token row0 / G, head head0 + row0 % G
    int rows, head0, first;
    float vs;    // the values' scale
    int pad[2];
};
__host__ __device__ constexpr size_t tree_part_floats(int rows, int dp) {
    return static_cast<size_t>(rows) * (dp + 2);
}
constexpr int tree_dp(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
__host__ __device__ constexpr int tree_streams(int dp) { return dp <= 128 ? 2 : 1; }
inline size_t tree_workspace(int ctas, int dp) {
    return sizeof(TreePart) * ctas + 2ull * ctas * tree_part_floats(kTreeRows * tree_streams(dp), dp) * 4;
}

// One side of the cache as a tensor of [page][head][slot][value], in boxes of `box` tokens of one head: with 16-bit
// values 64 columns each, 128-byte swizzled; with 8-bit ones whole rows of dp bytes.  Values from head_dim on and
// pages from num_pages on are outside: zeros.  False if there is no such view.
bool tree_map(CUtensorMap* map, const TreeArgs& a, const KvView& kv, bool e4m3, int dp, int box);
// The queries as [token][head][value], in boxes of 64 columns of a key-value head's heads of `box` tokens.
bool tree_query_map(CUtensorMap* map, const TreeArgs& a, int box);

namespace {

__device__ __forceinline__ float tree_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float tree_max(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// 16 bytes global -> shared, asynchronously; zeros where `bytes` is 0.
__device__ __forceinline__ void tree_copy16(uint32_t dst, const char* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tree_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void tree_wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tree_store16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// The same, and the largest of the 32 values (NaN if one is).
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t (&v)[32], uint32_t& most) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.NaN.f32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(most)
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's loads; names the registers that they fill, which are not to be used before.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :: "memory");
    asm volatile(""
                 : "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :: "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :: "memory");
}
// Waits for the phase of the given parity, by all lanes of a warp; gives up like mbar_wait_warp.  A
// function, as the kernel's loops have to fit in the instruction cache; its first tests read no
// clock, as the global timer's read would add to the latency of every hand-over.
static __device__ __noinline__ void tree_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                   uint64_t limit_ns) {
    for (int n = 0; n < 64; ++n)
        if (mbar_try_wait(bar, parity)) return;
    mbar_wait_bounded(bar, parity, abort_flag, status, limit_ns);
}
__device__ __forceinline__ void tree_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, uint64_t limit_ns) {
    if (!mbar_try_wait(bar, parity)) tree_wait_slow(bar, parity, abort_flag, status, limit_ns);
    __syncwarp();
}
// One lane of a converged warp, always the same: a branch on it is known to be a single thread's.
__device__ __forceinline__ bool tree_elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(p));
    return p != 0;
}
// A value that is the same in all lanes, known to be.
__device__ __forceinline__ uint32_t tree_uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
// D[tmem] (+)= A[smem] . B[smem]^T, kind::f16.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc),
        "r"(idesc), "r"(accumulate)
        : "memory");
}
// The MN-major operand with 128-byte swizzle: atoms of 64 values (M or N) x 8 (K), 1024 bytes
// apart along K and `block` bytes along M or N.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t block) {
    return sw128_desc(saddr & 0x3FFFFu) & ~(0x3FFFull << 16) | static_cast<uint64_t>(block >> 4) << 16;
}
constexpr uint32_t kIdescBMajorMn = 1u << 16;

// Zeros in the place of values that are infinite or NaN; true if there were any.  BF: bf16, else fp16.
template <bool BF>
__device__ __forceinline__ bool tree_scrub(uint4& v) {
    constexpr uint32_t kExp = BF ? 0x7F80u : 0x7C00u;
    uint32_t* w = &v.x;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool lo = (w[e] & kExp) == kExp, hi = (w[e] >> 16 & kExp) == kExp;
        if (lo) w[e] &= 0xFFFF0000u;
        if (hi) w[e] &= 0x0000FFFFu;
        any |= lo | hi;
    }
    return any;
}
// The same of E4M3, whose only such values are NaN, 0x7F and 0xFF.
__device__ __forceinline__ bool tree_scrub_e4m3(uint4& v) {
    uint32_t* w = &v.x;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t nan = __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        w[e] &= ~nan;
        any |= nan != 0;
    }
    return any;
}

// DT: 0 fp16, 1 bf16 (queries, output).  E4M3: 8-bit cache.  DP: head dimension rounded up.
template <int DT_, bool E4M3_, int DP_>
struct TreeShape {
    static constexpr int DT = DT_, DP = DP_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr bool BF = DT == 1 && !E4M3;   // type of the MMA's operands
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int STREAMS = tree_streams(DP);
    static constexpr int STEP = DP <= 128 ? 128 : 64;        // tokens of a step
    static constexpr int ROWS = kTreeRows * STREAMS;         // of an item
    static constexpr int BLOCKS = DP / 64;                   // 64-value blocks of a row
    static constexpr int SLOT = STEP * DP * 2;               // bytes of a step's keys, or values
    static constexpr int QTILE = kTreeRows * DP * 2;
    // Slots of the ring, 128 KB: the steps' keys in the even ones, their values in the odd ones.  A multiple
    // of four: with one stream per step a slot then is always the same stream's.
    static constexpr int NSLOT = DP == 64 ? 8 : 4;
    // 8-bit tiles as they come from the cache, before they are converted into the ring
    static constexpr int RAW = STEP * DP, NRAW = E4M3 ? (DP == 64 ? 4 : 2) : 0;
    static constexpr int SW = 4 * STREAMS;                   // softmax warps
    // A warp for the MMAs of each stream, then the loaders, which with an 8-bit cache convert.
    static constexpr int LW = E4M3 ? 6 : 2;
    static constexpr int LOADERS = 2, SOFTMAX = LOADERS + LW;
    static constexpr int THREADS = 32 * (SOFTMAX + SW);      // 384: 168 registers each; 512: 128
    static constexpr int CH = DP / 8;                        // 16-byte chunks of a row in shared memory
    static constexpr int GROUPS = STEP / 16;                 // of 16 tokens: loader warp w has w, w + LW, ...
    static constexpr int TM_O = 2 * STEP;                    // TMEM columns: S twice, then O of each stream
    // Shared memory: TreeControl, the queries' tiles, the ring.  The tiles' 1024-byte alignment follows
    // from the declared alignment of the dynamic part.
    static constexpr int CONTROL = 3 * 1024;
    static constexpr int SMEM = CONTROL + STREAMS * QTILE + NSLOT * SLOT + NRAW * RAW;
    static_assert(TM_O + STREAMS * DP <= 512, "TMEM");
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(NSLOT % 4 == 0 && SOFTMAX % 4 == 0, "see above; a warp's lanes of TMEM");
    static_assert(THREADS * 8 <= STREAMS * QTILE, "the prefix sums lie in the queries' place");
};

// The line's shares, the same in every CTA.
struct TreeLine {
    long long end, share;
};

template <class S>
struct TreeControl {
    uint64_t bars[2 * S::NSLOT + 13 + 2 * S::NRAW];
    TreeLine line;
    long long scan[S::THREADS / 32];
    uint32_t tmem_base;
    int abort_flag;
    int bad_page;                                   // a page lay outside the cache: masks look again
    int dirty;                                      // infinite values or NaN were replaced by 0
    float2 stats[S::STREAMS][kTreeRows];            // (m, l) of the streams, at the end of an item
    int pages[2][16];                               // of a step's boxes, for the thread that copies them
    int8_t qe[S::STREAMS][kTreeRows];               // exponents of the rows' scaling of the queries
};

// A sequence as the kernel sees it.
struct TreeSeq {
    int first, n, len;     // rows first .. first + n - 1
    int sink_tiles, tile0; // steps: tiles 0 .. sink_tiles - 1, then from tile0 on
    int steps, row_tiles;  // row_tiles: items of a key-value head
    int weight;            // of a step, in units of the line
};
template <class S>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
    TreeSeq s{};
    const int first = a.starts[b], last = a.starts[b + 1], len = a.lens[b];
    if (first == last && first >= 0 && first <= a.T) return s;
    const int n = last - first;
    if (first < 0 || last < first || last > a.T || n > 64 || len < n || len > a.max_pages * a.page_size) {
        if (report) record_status(a.status, kDecInvalidArg);
        return s;
    }
    s.first = first, s.n = n, s.len = len;
    const int lo = a.window > 0 ? max(0, len - n - a.window) : 0;  // a row without bits sees from here
    s.sink_tiles = a.window > 0 ? (min(a.sinks, len) + S::STEP - 1) / S::STEP : 0;
    s.tile0 = lo / S::STEP;
    if (s.sink_tiles >= s.tile0) s.sink_tiles = s.tile0 = 0;
    s.steps = s.sink_tiles + (len + S::STEP - 1) / S::STEP - s.tile0;
    const int rows = n * (a.q_heads / a.kv_heads);
    s.row_tiles = (rows + S::ROWS - 1) / S::ROWS;
    s.weight = S::STREAMS == 2 && rows > kTreeRows ? kTreeDualStep : kTreeStep;
    return s;
}

// Steps [step, step_end) of an item as one CTA takes them.
struct TreeSeg {
    TreeSeq seq;
    int b, item, step, step_end;
    long long rest;   // what the CTA's share holds after this item
};

template <class S>
__device__ __forceinline__ long long tree_items(const TreeArgs& a, const TreeSeq& s) {
    return static_cast<long long>(s.row_tiles) * a.kv_heads;
}
__device__ __forceinline__ long long tree_units(const TreeSeq& s) {  // of an item
    return static_cast<long long>(s.steps) * s.weight + kTreeItemCost;
}

// a / b for numbers >= 0; the long division, out of line, only where 32 bits do not hold them.
static __device__ __noinline__ long long tree_long_quotient(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long tree_quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return tree_long_quotient(a, b);
}

__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {  // bits lo .. hi - 1 of 0 .. 31
    lo = max(lo, 0), hi = min(hi, 32);
    return lo < hi ? (0xFFFFFFFFu >> (32 - (hi - lo))) << lo : 0;
}

// What one row sees of the tokens t0 .. t0 + 31.
struct TreeRow {
    uint64_t word;
    int ctx, from, sinks;
    __device__ __forceinline__ uint32_t seen(int t0) const {
        uint32_t v = 0;
        if (t0 < ctx) v = range_bits(from - t0, ctx - t0) | range_bits(-t0, min(sinks, ctx) - t0);
        const int sh = t0 - ctx;
        if (sh > -32 && sh < 64)
            v |= static_cast<uint32_t>(sh >= 0 ? word >> sh : word << -sh);
        return v;
    }
};

// box_rows: tokens of a box of the cache's tensor maps (a power of two that divides the page size), or 0: it is
// read without them.  q_box: tokens of a tile of queries, in boxes of qmap, or 0.
template <class S>
__global__ void __launch_bounds__(S::THREADS, 1)
tree_kernel(TreeArgs a, int page_shift, int box_rows, int q_box, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
    constexpr int STEP = S::STEP, DP = S::DP, STREAMS = S::STREAMS, NSLOT = S::NSLOT, SW = S::SW, LW = S::LW;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    static_assert(sizeof(TreeControl<S>) <= S::CONTROL, "the control block fits");
    // the tiles begin at a multiple of 1024, the control block lies before or behind them
    TreeControl<S>& ctl = *reinterpret_cast<TreeControl<S>*>(smem_raw);
    TreeLine& line = ctl.line;
    long long* prefix = reinterpret_cast<long long*>(smem_raw + S::CONTROL);  // until the queries come

    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
    const int G = a.q_heads / a.kv_heads;
    const uint32_t base = smem_addr(smem_raw) + S::CONTROL;
    const uint32_t q_smem = base, ring = base + STREAMS * S::QTILE;
    const uint32_t bar0 = smem_addr(ctl.bars);
    const uint32_t full = bar0, empty = full + 8 * NSLOT, q_full = empty + 8 * NSLOT, q_empty = q_full + 8;
    const uint32_t s_full = q_empty + 8, p_full = s_full + 16, o_full = p_full + 16, o_free = o_full + 8;
    const uint32_t pv_done = o_free + 8, fix_full = pv_done + 8, turn = fix_full + 8;
    const uint32_t raw_full = turn + 16, raw_empty = raw_full + 8 * S::NRAW, q_raw = raw_empty + 8 * S::NRAW;
    TreePart* heads = static_cast<TreePart*>(a.workspace);
    float* parts = reinterpret_cast<float*>(heads + ctas);

    // columns past the head dimension are never copied: zero, so that they add nothing
    if (a.head_dim < DP)
        for (uint32_t e = tid; e < (STREAMS * S::QTILE + NSLOT * S::SLOT) / 16; e += S::THREADS)
            tree_store16(base + 16 * e, make_uint4(0, 0, 0, 0));
    if (tid < NSLOT) {
        mbar_init(full + 8 * tid, S::E4M3 || box_rows > 0 ? 1 : LW);  // one thread, or every loader warp
        mbar_init(empty + 8 * tid, STREAMS);
    }
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_raw, 1);
        for (int s = 0; s < 2 * S::NRAW; ++s) mbar_init(raw_full + 8 * s, 1);
        mbar_init(q_empty, STREAMS + SW);
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + 8 * s, 2);  // the MMAs are done; what the producers noted can be seen
            mbar_init(p_full + 8 * s, 4);
            mbar_init(turn + 8 * s, 1);
        }
        mbar_init(o_full, 2 * STREAMS);
        mbar_init(o_free, SW);
        mbar_init(pv_done, 1);
        mbar_init(fix_full, 1);
        fence_mbar_init();
        ctl.abort_flag = ctl.bad_page = ctl.dirty = 0;
    }
    fence_proxy_async_smem();  // the zeros
    if (tid == 32) {
        if (box_rows > 0) {
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        if (q_box > 0) prefetch_tensormap(&qmap);
    }
    grid_dep_wait();
    grid_dep_launch();
    if (warp == 0) {
        tmem_alloc(smem_addr(&ctl.tmem_base), 512);
        tmem_relinquish();
    }

    // ---- the line: prefix[t] is what lies before thread t's sequences ----
    const int per_thread = (a.B + S::THREADS - 1) / S::THREADS;
    {
        const int b_lo = min(a.B, tid * per_thread), b_hi = min(a.B, b_lo + per_thread);
        long long mine = 0;
        int dual = 0;
        for (int b = b_lo; b < b_hi; ++b) {
            const TreeSeq s = tree_seq<S>(a, b, cta == 0);
            mine += tree_items<S>(a, s) * tree_units(s);
            dual |= s.weight == kTreeDualStep;
        }
        long long incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) ctl.scan[warp] = incl;
        dual = __syncthreads_or(dual);
        long long total = 0;
        for (int w = 0; w < S::THREADS / 32; ++w) {
            if (w < warp) incl += ctl.scan[w];
            total += ctl.scan[w];
        }
        prefix[tid] = incl - mine;
        // no share is shorter than a step: each between an item's first and last has one of its steps
        const long long least = dual ? kTreeDualStep : kTreeStep;
        if (tid == 0) line = TreeLine{total, max(tree_quotient(total + ctas - 1, ctas), least)};
    }
    if (tid == 32 * S::SOFTMAX) heads[cta] = TreePart{};
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    const long long share_end = min(line.end, line.share * (cta + 1));

    auto open_item = [&](TreeSeg& s, long long begin, long long from) {  // its steps at or after `from`
        const long long at0 = begin + kTreeItemCost;
        const long long units = static_cast<long long>(s.seq.steps) * s.seq.weight;
        auto steps_before = [&](long long to) {   // a step is whose share its first unit lies in
            const unsigned n = static_cast<unsigned>(min(max(to - at0, 0ll), units));   // (below 2^27)
            return static_cast<int>(s.seq.weight == kTreeStep ? (n + kTreeStep - 1) / kTreeStep : (n + kTreeDualStep - 1) / kTreeDualStep);
        };
        s.step = steps_before(from);
        s.step_end = steps_before(share_end);
        s.rest = share_end - at0 - units;
    };
    // The segment after s; false: there is none.
    auto after = [&](TreeSeg& s) {
        if (s.rest <= kTreeItemCost) return false;
        if (++s.item == tree_items<S>(a, s.seq)) {
            s.item = 0;
            do {
                s.seq = tree_seq<S>(a, ++s.b, false);
            } while (s.seq.steps == 0 && s.b + 1 < a.B);
        }
        open_item(s, share_end - s.rest, 0);
        return s.step < s.step_end;
    };
    // The first segment of the CTA's share; false: there is none.  By all lanes of a warp.
    auto locate = [&](TreeSeg& s) {
        const long long u = line.share * cta;
        if (u >= line.end) return false;
        int t = 0;
        for (int t0 = 0; t0 < S::THREADS && t0 * per_thread < a.B; t0 += 32)
            t += __popc(__ballot_sync(0xFFFFFFFFu, prefix[t0 + lane] <= u));
        --t;
        long long at = prefix[t];
        s.b = t * per_thread;
        s.seq = tree_seq<S>(a, s.b, false);
        while (at + tree_items<S>(a, s.seq) * tree_units(s.seq) <= u && s.b + 1 < a.B) {
            at += tree_items<S>(a, s.seq) * tree_units(s.seq);
            s.seq = tree_seq<S>(a, ++s.b, false);
        }
        const long long per = tree_units(s.seq);
        s.item = static_cast<int>(tree_quotient(u - at, per));
        open_item(s, at + s.item * per, u);
        return s.step < s.step_end || after(s);
    };
    // row / G: by a multiplication where that is exact (rows are below 64 G)
    const uint32_t g_inv = G > 1 && G < 8192 ? 0xFFFFFFFFu / static_cast<uint32_t>(G) + 1 : 0;
    auto token_of_row = [&](int row) {
        return G == 1 ? row : g_inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), g_inv)) : row / G;
    };
    // Row tiles of an item are neighbours in the line, so that they find its tokens in L2.
    auto head_of = [&](const TreeSeg& s) { return s.item / s.seq.row_tiles; };
    auto row0_of = [&](const TreeSeg& s) { return s.item % s.seq.row_tiles * S::ROWS; };
    auto rows_of = [&](const TreeSeg& s) { return min(S::ROWS, s.seq.n * G - row0_of(s)); };
    auto tile_of = [&](const TreeSeq& s, int step) {
        return step < s.sink_tiles ? step : s.tile0 + step - s.sink_tiles;
    };
    auto wait = [&](uint32_t bar, uint32_t phase) { tree_wait(bar, phase, &ctl.abort_flag, a.status, a.timeout_ns); };

    TreeSeg seg{};
    bool more = locate(seg);
    // The prefix sums have been read; where they stood may be zeros that the queries need.  The queries come by
    // copies of the async proxy, which nothing but a fence by every thread orders behind its ordinary accesses.
    if (a.head_dim < DP) {
        __syncthreads();
        for (uint32_t e = tid; e < (S::THREADS * 8 + 15) / 16; e += S::THREADS)
            tree_store16(base + 16 * e, make_uint4(0, 0, 0, 0));
    }
    fence_proxy_async_smem();
    __syncthreads();

    if (warp >= S::LOADERS && warp < S::SOFTMAX) {
        // ================= loaders =================
        // In steps that not all rows see in full, at the ends of what is visible, the values are looked
        // through: zeros for tokens that no row sees, and finite ones where some row does not see a
        // token.  (Keys need no such care: their scores are masked.)
        const int lw = warp - S::LOADERS;
        constexpr int CH = S::CH;
        const int row_chunks = a.head_dim / 8;        // of 16-bit values
        auto page_of = [&](int tok) { return page_shift >= 0 ? tok >> page_shift : tok / a.page_size; };
        // the shared-memory address of chunk c of row r, from a tile of `rows` rows
        auto at_smem = [](int rows, int r, int c) {
            return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        };
        int slot = 0;
        uint32_t phase = 0, q_phase = 0;
        int raw_at = 0;                     // of the 8-bit tiles
        uint32_t raw_phase = 0, fix_phase = 0;
        auto next_slot = [&]() {
            if (++slot == NSLOT) slot = 0, phase ^= 1u;
        };
        auto loaders_sync = [&]() { asm volatile("bar.sync 2, %0;" ::"n"(32 * LW) : "memory"); };
        // what all loaders wrote is there: for the MMAs, which read it through the other proxy
        auto all_there = [&](uint32_t bar) {
            fence_proxy_async_smem();
            loaders_sync();
            if (lw == 0 && lane == 0) mbar_arrive(bar);
        };
        while (more) {
            const TreeSeq& sq = seg.seq;
            const int ctx = sq.len - sq.n, kvh = head_of(seg);
            const int32_t* table = a.block_table + seg.b * a.ld_table;
            // the first token that the row with the fewest bits sees in the window
            int lo = 0;
            if (a.window > 0) {
                int least = 1;
                if (a.mask) {
                    const uint64_t all = sq.n == 64 ? ~0ull : (1ull << sq.n) - 1;
                    least = 64;
                    for (int i = lane; i < sq.n; i += 32) least = min(least, __popcll(a.mask[sq.first + i] & all));
                    least = __reduce_min_sync(0xFFFFFFFFu, least);
                }
                lo = max(0, min(ctx, ctx + least - a.window));
            }
            const int edge = a.window > 0 ? ctx + sq.n - a.window : 0;  // tokens from here on are in every window
            auto clean = [&](int step) {   // all rows see all tokens
                const int tok0 = tile_of(sq, step) * STEP;
                return tok0 + STEP <= ctx && (tok0 >= edge || tok0 + STEP <= a.sinks);
            };
            auto wanted = [&](int tok) { return tok < sq.len && (tok >= lo || tok < a.sinks); };   // some row sees it
            auto some_not = [&](int tok) { return tok >= ctx || (tok < edge && tok >= a.sinks); }; // and some may not
            auto bad = [&]() {
                record_status(a.status, kDecInvalidArg);
                *static_cast<volatile int*>(&ctl.bad_page) = 1;
            };

            // ---- tensor copies: lane g has the page of the step's box g of box_rows tokens; one thread issues
            // them all (copies of different lanes take several times as long), the pages handed to it through
            // shared memory ----
            const int boxes = box_rows > 0 ? STEP / box_rows : 0;
            auto box_page = [&](int step) {  // num_pages, which gives zeros, where nobody sees a token
                const int tok = tile_of(sq, step) * STEP + lane * box_rows;
                return lane < boxes && step < seg.step_end && tok < sq.len && (tok + box_rows > lo || tok < a.sinks)
                           ? table[page_of(tok)] : a.num_pages;
            };
            auto issue = [&](uint32_t dst, uint32_t bar, uint32_t bytes, const CUtensorMap* map, int step, int page) {
                const int tok0 = tile_of(sq, step) * STEP, tok = tok0 + lane * box_rows;
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) {
                    // (num_pages itself may stand in the table)
                    if (page != a.num_pages || (lane < boxes && tok < sq.len && (tok + box_rows > lo || tok < a.sinks))) bad();
                    page = a.num_pages;
                }
                int* pages = ctl.pages[lw & 1];
                if (lane < boxes) pages[lane] = page;
                const uint32_t to = tree_uniform(dst), done = tree_uniform(bar), head = tree_uniform(kvh);
                uint32_t in_page = tree_uniform(tok0 - page_of(tok0) * a.page_size);
                __syncwarp();
                if (tree_elect() && *static_cast<volatile int*>(&ctl.abort_flag) == 0) {
                    mbar_arrive_expect_tx(done, bytes);
#pragma unroll 2
                    for (int g = 0; g < boxes; ++g) {
                        const int from = pages[g];
#pragma unroll
                        for (int block = 0; block < (S::E4M3 ? 1 : S::BLOCKS); ++block)
                            tma_tensor_4d_g2s(to + g * box_rows * (S::E4M3 ? DP : 128) + block * STEP * 128, map, 64 * block,
                                              in_page, head, from, done);
                        in_page += box_rows;
                        if (in_page == static_cast<uint32_t>(a.page_size)) in_page = 0;
                    }
                }
                __syncwarp();
            };

            // ---- by all loaders: lanes 0 .. 15 and 16 .. 31 have the tokens of the warp's first two groups, ----
            // ---- those of its third are in a second set of registers                                      ----
            constexpr int MINE = (S::GROUPS + LW - 1) / LW, SETS = (MINE + 1) / 2;
            int64_t kat[SETS], vat[SETS];   // where their keys and values stand (-1: nowhere)
            uint32_t mixed[SETS];           // tokens that not every row sees
            auto look = [&](int step) {
#pragma unroll
                for (int s = 0; s < SETS; ++s) {
                    const int group = lw + LW * (2 * s + lane / 16);
                    const int tok = tile_of(sq, step) * STEP + group * 16 + lane % 16;
                    const bool want = group < S::GROUPS && wanted(tok);
                    const int in = want ? page_of(tok) : 0, pid = want ? table[in] : 0;
                    const bool ok = want && static_cast<unsigned>(pid) < static_cast<unsigned>(a.num_pages);
                    if (want && !ok) bad();
                    const int64_t in_page = tok - static_cast<int64_t>(in) * a.page_size;
                    kat[s] = ok ? (pid * a.kc.page_stride + in_page * a.kc.slot_stride + kvh * a.kc.head_stride) * S::ES : -1;
                    vat[s] = ok ? (pid * a.vc.page_stride + in_page * a.vc.slot_stride + kvh * a.vc.head_stride) * S::ES : -1;
                    mixed[s] = __ballot_sync(0xFFFFFFFFu, ok && some_not(tok));
                }
            };
            constexpr int FC = DP * S::ES / 16;            // chunks of a row in the cache
            constexpr int LR = 32 / FC;                    // rows of one load of the warp
            const int fc = lane % FC, fsub = lane / FC;
            auto put = [&](uint32_t dst, uint4 v, int r) { // chunk fc of row r, from the cache's type
                if constexpr (S::E4M3) {
                    if (2 * fc >= row_chunks) return;
                    const uint32_t* w = &v.x;
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = dec_e4m3x2_to_f16x2(w[e]);
                        h[2 * e + 1] = dec_e4m3x2_to_f16x2(w[e] >> 16);
                    }
                    // (eight lanes have a row of 128: half of them store their second chunk first, all banks at once)
                    const int swap = DP > 64 ? (fc >> 2) & 1 : 0;
                    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                    tree_store16(dst + at_smem(STEP, r, 2 * fc + swap), swap ? hi : lo);
                    tree_store16(dst + at_smem(STEP, r, 2 * fc + 1 - swap), swap ? lo : hi);
                } else {
                    if (fc < row_chunks) tree_store16(dst + at_smem(STEP, r, fc), v);
                }
            };
            auto finite = [&](uint4& v) {  // zeros for infinite values and NaN, which the end of the item adds
                bool any;
                if constexpr (S::E4M3) any = tree_scrub_e4m3(v);
                else any = tree_scrub<S::BF>(v);
                if (any) *static_cast<volatile int*>(&ctl.dirty) = 1;
                return any;
            };
            auto fill = [&](uint32_t dst, const void* from, const int64_t (&at)[SETS]) {   // values, looked through
                constexpr int LN = 16 / LR;   // loads of a group
#pragma unroll
                for (int n = 0; n < MINE; ++n) {
                    const int group = lw + LW * n;
                    if (group >= S::GROUPS) break;
                    uint4 v[LN];
#pragma unroll
                    for (int x = 0; x < LN; ++x) {
                        const int64_t off = __shfl_sync(0xFFFFFFFFu, at[n / 2], n % 2 * 16 + x * LR + fsub);
                        v[x] = make_uint4(0, 0, 0, 0);
                        if (off >= 0 && fc < row_chunks)
                            v[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(from) + off) + fc);
                    }
#pragma unroll
                    for (int x = 0; x < LN; ++x) {
                        if (mixed[n / 2] >> (n % 2 * 16 + x * LR + fsub) & 1u) finite(v[x]);
                        put(dst, v[x], group * 16 + x * LR + fsub);
                    }
                }
            };
            // Queries: by tensor copies where a tile of rows is whole tokens, else 16 bytes at a time by all loaders but an
            // 8-bit cache's copying one.  Tokens of G heads are G rows, one after another.  Rows behind the
            // sequence's are another's, or zeros: nobody reads what they give.
            constexpr int Q_WARP = 1;
            constexpr bool Q_CONVERT = S::E4M3 && S::DT == 1;
            // |q_scale| belongs to the softmax; a negative or zero one is folded into the queries
            const float q_scale = a.scale * (S::E4M3 && a.kc.scale ? a.kc.scale[kvh] : 1.0f);
            const bool by_copy = q_box > 0 && (Q_CONVERT || q_scale > 0.0f);
            const int q_rows = rows_of(seg), padded = q_rows > kTreeRows ? 2 * kTreeRows : kTreeRows;
            auto ask_queries = [&]() {
                if (!by_copy || lw != Q_WARP) return;
                const uint32_t bar = Q_CONVERT ? q_raw : q_full;
                wait(q_empty, q_phase ^ 1u);
                if (__any_sync(0xFFFFFFFFu, *static_cast<volatile int*>(&ctl.abort_flag) != 0)) return;
                if (lane == 0) mbar_arrive_expect_tx(bar, padded * DP * 2);
                __syncwarp();
                const int tile = lane / S::BLOCKS, block = lane % S::BLOCKS;
                if (tile * kTreeRows < padded)
                    tma_tensor_4d_g2s(q_smem + tile * S::QTILE + block * kTreeRows * 128, &qmap, 64 * block, kvh * G,
                                      sq.first + token_of_row(row0_of(seg)) + tile * q_box, 0, bar);
                __syncwarp();
            };
            auto finish_queries = [&]() {
                constexpr int parts = S::E4M3 ? LW - 1 : LW;
                const int part = lw - (LW - parts);
                const uint32_t phase_now = q_phase;
                q_phase ^= 1u;
                if (part < 0 || (by_copy && !Q_CONVERT)) return;
                constexpr int RPI = 32 / CH;
                const int c = lane % CH, sub = lane / CH;
                if (by_copy) {
                    wait(q_raw, phase_now);
                } else {
                    wait(q_empty, phase_now ^ 1u);
                    const int row0 = row0_of(seg);
                    // (a short loop: it runs once per item, as code that comes from beyond the SM)
#pragma unroll 1
                    for (int n = part * RPI + sub; n < padded; n += parts * RPI) {
                        const int row = row0 + n, i = token_of_row(row);
                        const uint16_t* from = a.q + static_cast<int64_t>(sq.first + i) * a.ldq +
                                               static_cast<int64_t>(kvh * G + row - i * G) * a.head_dim + 8 * c;
                        if (c < row_chunks)
                            tree_copy16(q_smem + n / kTreeRows * S::QTILE + at_smem(kTreeRows, n % kTreeRows, c),
                                        reinterpret_cast<const char*>(n < q_rows ? from : a.q), n < q_rows ? 16 : 0);
                    }
                    tree_commit();
                    tree_wait_copies<0>();
                }
                // bf16 queries against an 8-bit cache, whose MMA is fp16: scaled by a power of two that brings the
                // row's largest to 2^8 .. 2^9.  (The threads go through the chunks that they would have copied.)
                if constexpr (Q_CONVERT) {
#pragma unroll 1
                    for (int n = part * RPI + sub; n < padded; n += parts * RPI) {
                        const int t = n / kTreeRows, r = n % kTreeRows;
                        const uint32_t at = q_smem + t * S::QTILE + at_smem(kTreeRows, r, c);
                        uint4 v = lds_v4(at);
                        uint32_t* w = &v.x;
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
#pragma unroll
                        for (int d = CH / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                        const int e2 = min(static_cast<int>(top >> 7) - 127, 127);
                        const int exponent = e2 > -119 ? e2 - 8 : 0;
                        const float up = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = dec_pack2<0>(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
                        if (c == 0) ctl.qe[t][r] = static_cast<int8_t>(exponent);
                        if (c < row_chunks) tree_store16(at, v);
                    }
                }
                if (!(q_scale > 0.0f) && c < row_chunks) {   // times -1, or 0, which makes NaN of infinite values and NaN
                    constexpr uint32_t kExp = S::BF ? 0x7F80u : 0x7C00u;
#pragma unroll 1
                    for (int n = part * RPI + sub; n < padded; n += parts * RPI) {
                        const uint32_t at = q_smem + n / kTreeRows * S::QTILE + at_smem(kTreeRows, n % kTreeRows, c);
                        uint4 v = lds_v4(at);
                        uint32_t* w = &v.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = q_scale == 0.0f ? ((w[e] & kExp) == kExp ? 0x7FFFu : 0u) | ((w[e] >> 16 & kExp) == kExp ? 0x7FFF0000u : 0u)
                                 : q_scale < 0.0f ? w[e] ^ 0x80008000u : w[e];
                        tree_store16(at, v);
                    }
                }
                if (parts == LW) {
                    all_there(q_full);
                } else {
                    fence_proxy_async_smem();
                    asm volatile("bar.sync 3, %0;" ::"n"(32 * (LW - 1)) : "memory");
                    if (part == 0 && lane == 0) mbar_arrive(q_full);
                }
            };
            if constexpr (S::E4M3) {
                // The first warp copies 8-bit tiles; the others convert them into the ring.
                constexpr int NRAW = S::NRAW, CW = LW - 1;
                const uint32_t raw = ring + NSLOT * S::SLOT;
                if (lw == 0 && box_rows == 0) {
                    // pages that no tensor map describes, 16 bytes at a time; a tile is announced when the next
                    // one's copies are under way
                    int before = -1, page[STEP / 32], ahead[STEP / 32];
                    auto pages_of = [&](int step, int (&to)[STEP / 32]) {   // of tokens 32 x + lane; -1: not wanted
#pragma unroll
                        for (int x = 0; x < STEP / 32; ++x) {
                            const int tok = tile_of(sq, step) * STEP + 32 * x + lane;
                            to[x] = -1;
                            if (step < seg.step_end && wanted(tok)) {
                                to[x] = table[page_of(tok)];
                                if (to[x] == -1) to[x] = a.num_pages;   // (as bad as it)
                            }
                        }
                    };
                    pages_of(seg.step, ahead);
#pragma unroll 1
                    for (int half = 2 * seg.step; half < 2 * seg.step_end; ++half) {
                        wait(raw_empty + 8 * raw_at, raw_phase ^ 1u);
                        if (!(half & 1)) {
#pragma unroll
                            for (int x = 0; x < STEP / 32; ++x) page[x] = ahead[x];
                            pages_of((half >> 1) + 1, ahead);
                        }
                        const KvView& kv = half & 1 ? a.vc : a.kc;
                        const char* from = static_cast<const char*>(kv.p);
#pragma unroll
                        for (int x = 0; x < STEP / 32; ++x) {
                            const int tok = tile_of(sq, half >> 1) * STEP + 32 * x + lane;
                            const bool ok = static_cast<unsigned>(page[x]) < static_cast<unsigned>(a.num_pages);
                            if (page[x] != -1 && !ok) bad();
                            const int64_t at = ok ? page[x] * kv.page_stride +
                                                    (tok - static_cast<int64_t>(page_of(tok)) * a.page_size) * kv.slot_stride +
                                                    kvh * kv.head_stride : -1;
#pragma unroll 4
                            for (int r = fsub; r < 32; r += LR) {
                                const int64_t off = __shfl_sync(0xFFFFFFFFu, at, r);
                                if (16 * fc < a.head_dim)
                                    tree_copy16(raw + raw_at * S::RAW + (32 * x + r) * DP + 16 * fc, off >= 0 ? from + off + 16 * fc : from,
                                                off >= 0 ? 16 : 0);
                            }
                        }
                        tree_commit();
                        if (before >= 0) {
                            tree_wait_copies<1>();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(raw_full + 8 * before);
                        }
                        before = raw_at;
                        if (++raw_at == NRAW) raw_at = 0, raw_phase ^= 1u;
                    }
                    tree_wait_copies<0>();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_full + 8 * before);
                } else if (lw == 0) {
                    int pid = box_page(seg.step), pid1 = box_page(seg.step + 1);
#pragma unroll 1
                    for (int half = 2 * seg.step; half < 2 * seg.step_end; ++half) {
                        wait(raw_empty + 8 * raw_at, raw_phase ^ 1u);
                        issue(raw + raw_at * S::RAW, raw_full + 8 * raw_at, S::RAW, half & 1 ? &vmap : &kmap, half >> 1, pid);
                        if (half & 1) pid = pid1, pid1 = box_page((half + 3) >> 1);
                        if (++raw_at == NRAW) raw_at = 0, raw_phase ^= 1u;
                    }
                } else {
                    ask_queries();
#pragma unroll 1
                    for (int half = 2 * seg.step; half < 2 * seg.step_end; ++half) {
                        wait(empty + 8 * slot, phase ^ 1u);
                        wait(raw_full + 8 * raw_at, raw_phase);
                        const uint32_t from = raw + raw_at * S::RAW, dst = ring + slot * S::SLOT;
                        const int tok0 = tile_of(sq, half >> 1) * STEP;
                        const bool care = (half & 1) && !clean(half >> 1);
                        if (!care) {   // all rows' loads together
                            constexpr int ROWS = (STEP + CW * LR - 1) / (CW * LR);
                            const int r0 = (lw - 1) * LR + fsub;
                            uint4 v[ROWS];
#pragma unroll
                            for (int x = 0; x < ROWS; ++x)
                                if (r0 + x * CW * LR < STEP) v[x] = lds_v4(from + (r0 + x * CW * LR) * DP + 16 * fc);
#pragma unroll
                            for (int x = 0; x < ROWS; ++x)
                                if (r0 + x * CW * LR < STEP) put(dst, v[x], r0 + x * CW * LR);
                        } else {
#pragma unroll 1
                            for (int r = (lw - 1) * LR + fsub; r < STEP; r += CW * LR) {
                                uint4 v = lds_v4(from + r * DP + 16 * fc);
                                if (!wanted(tok0 + r)) v = make_uint4(0, 0, 0, 0);
                                else if (some_not(tok0 + r)) finite(v);
                                put(dst, v, r);
                            }
                        }
                        fence_proxy_async_smem();
                        asm volatile("bar.sync 3, %0;" ::"n"(32 * CW) : "memory");
                        if (lw == 1 && lane == 0) {
                            mbar_arrive(full + 8 * slot);
                            mbar_arrive(raw_empty + 8 * raw_at);
                        }
                        next_slot();
                        if (++raw_at == NRAW) raw_at = 0, raw_phase ^= 1u;
                        if (half == 2 * seg.step) finish_queries();   // behind the first keys
                    }
                }
            } else if (box_rows == 0) {
                // Pages that no tensor map describes: every warp copies its groups of tokens and arrives by itself.
                auto there = [&](uint32_t bar) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                uint32_t under_way[2] = {0, 0};   // barriers of slots whose copies are, the older one first
                auto settle = [&]() {
                    if (under_way[0]) {
                        tree_wait_copies<1>();
                        there(under_way[0]);
                    }
                    if (under_way[1]) {
                        tree_wait_copies<0>();
                        there(under_way[1]);
                    }
                    under_way[0] = under_way[1] = 0;
                };
#pragma unroll 1
                for (int st = seg.step; st < seg.step_end; ++st) {
                    look(st);
                    uint32_t some = 0;
#pragma unroll
                    for (int s = 0; s < SETS; ++s) some |= mixed[s];
#pragma unroll 1
                    for (int side = 0; side < 2; ++side) {
                        const uint32_t dst = ring + slot * S::SLOT, bar = full + 8 * slot;
                        if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(empty + 8 * slot, phase ^ 1u))) {
                            settle();   // what is under way may be what the slot's readers wait for
                            wait(empty + 8 * slot, phase ^ 1u);
                        }
                        if (side && some) {
                            fill(dst, a.vc.p, vat);
                            there(bar);
                        } else {
                            constexpr int RPI = 32 / CH;
                            const int c = lane % CH, sub = lane / CH;
                            const char* from = static_cast<const char*>(side ? a.vc.p : a.kc.p);
#pragma unroll
                            for (int n = 0; n < MINE; ++n) {
                                const int group = lw + LW * n;
                                if (group >= S::GROUPS) break;
                                const int64_t mine = side ? vat[n / 2] : kat[n / 2];
#pragma unroll
                                for (int r0 = 0; r0 < 16; r0 += RPI) {
                                    const int64_t off = __shfl_sync(0xFFFFFFFFu, mine, n % 2 * 16 + r0 + sub);
                                    if (c < row_chunks)
                                        tree_copy16(dst + at_smem(STEP, group * 16 + r0 + sub, c), off >= 0 ? from + off + 16 * c : from,
                                                    off >= 0 ? 16 : 0);
                                }
                            }
                            tree_commit();
                            if (under_way[0]) {
                                tree_wait_copies<2>();
                                there(under_way[0]);
                            }
                            under_way[0] = under_way[1], under_way[1] = bar;
                        }
                        next_slot();
                    }
                    if (st == seg.step) {
                        settle();
                        ask_queries();
                        finish_queries();
                    }
                }
                settle();
            } else {
                // Keys by the first warp, queries and values by the second (or the queries by both, behind the
                // first step, as their place is taken until the item before has its last scores).  Each waits
                // for slots of its own alone.
                if (q_box > 0) {
                    ask_queries();
                    finish_queries();
                }
                int pid = box_page(seg.step), pid1 = box_page(seg.step + 1);
#pragma unroll 1
                for (int st = seg.step; st < seg.step_end; ++st) {
                    const bool as_it_is = clean(st);
                    const int mine = slot + lw;
                    wait(empty + 8 * mine, phase ^ 1u);
                    issue(ring + mine * S::SLOT, lw && !as_it_is ? fix_full : full + 8 * mine, S::SLOT, lw ? &vmap : &kmap, st, pid);
                    pid = pid1;
                    pid1 = box_page(st + 2);
                    if (!as_it_is) {
                        if (lw == 1) {  // the only one to wait for it: the other could not tell its phases apart
                            wait(fix_full, fix_phase);
                            fix_phase ^= 1u;
                        }
                        loaders_sync();
                        const uint32_t tile = ring + (slot + 1) * S::SLOT;
                        const int tok0 = tile_of(sq, st) * STEP;
                        // (behind the window's edges only the drafted tokens and those past the end)
                        const int r_lo = tok0 >= edge ? max(ctx - tok0, 0) & ~(LW * LR - 1) : 0;
#pragma unroll 2
                        for (int r = r_lo + lw * LR + fsub; r < STEP; r += LW * LR) {
                            const uint32_t at = tile + at_smem(STEP, r, fc);
                            if (!wanted(tok0 + r)) {
                                tree_store16(at, make_uint4(0, 0, 0, 0));
                            } else if (some_not(tok0 + r)) {
                                uint4 v = lds_v4(at);
                                if (finite(v)) tree_store16(at, v);
                            }
                        }
                        all_there(full + 8 * (slot + 1));
                    }
                    next_slot();
                    next_slot();
                    if (st == seg.step && q_box == 0) finish_queries();
                }
            }
            more = after(seg);
        }
    } else if (warp < S::LOADERS) {
        // ================= the MMAs =================
        // Each stream's by a warp of its own (one thread issues them), so that neither waits for the
        // other's softmax.  With one stream, which has two places for S, the next S goes ahead of P V.
        constexpr int TYPE = S::BF ? 1 : 0;
        constexpr uint32_t idesc_s = idesc_f16(TYPE, 128, STEP), idesc_o = idesc_f16(TYPE, 128, DP) | kIdescBMajorMn;
        const int stream = warp;
        if (stream >= STREAMS) more = false;
        uint32_t q_phase = 0, free_phase = 0, p_phase = 0;  // p_phase: bit x of place x
        int step0 = 0, turns = 0;                           // the CTA's steps before this item; those of both streams
#pragma unroll 1
        while (more) {
            const bool dual = rows_of(seg) > kTreeRows;
            const int steps = seg.step_end - seg.step;
            // the stream's steps: all, or every other one of the CTA's; those that it has alone it frees for both
            const bool alone = STREAMS == 2 && !dual;
            const int first = alone ? (stream ^ step0) & 1 : 0, stride = alone ? 2 : 1;
            wait(q_full, q_phase);
            q_phase ^= 1u;
            auto scores = [&](int st) {
                const int at = step0 + st, slot = 2 * at % NSLOT, place = STREAMS == 2 ? stream : at & 1;
                wait(full + 8 * slot, (2 * at / NSLOT) & 1);
                tc_fence_after();
                const uint32_t q_at = tree_uniform(q_smem + (dual ? stream * S::QTILE : 0));
                const uint32_t k_at = tree_uniform(ring + slot * S::SLOT), d = tree_uniform(tmem + place * STEP);
                if (tree_elect()) {
                    const uint64_t q = sw128_desc(q_at), k = sw128_desc(k_at);
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c)
                        tc_mma_ss(d, q + (c >> 2) * (kTreeRows * 128 >> 4) + (c & 3) * 2,
                                  k + (c >> 2) * (STEP * 128 >> 4) + (c & 3) * 2, idesc_s, c > 0);
                    tc_commit(s_full + 8 * place);
                    tc_commit(empty + 8 * slot);
                    if (alone) tc_commit(empty + 8 * slot);
                    if (st + stride >= steps) tc_commit(q_empty);
                    mbar_arrive(s_full + 8 * place);
                }
                __syncwarp();
            };
            auto values = [&](int st) {
                const int at = step0 + st, slot = 2 * at % NSLOT + 1, place = STREAMS == 2 ? stream : at & 1;
                if (st == first) {
                    wait(o_free, free_phase ^ 1u);  // the previous item's sums have been read
                    free_phase ^= 1u;
                }
                wait(full + 8 * slot, (2 * at / NSLOT) & 1);
                const uint32_t d = tree_uniform(tmem + S::TM_O + stream * DP);
                const uint32_t p = tree_uniform(tmem + place * STEP), tile = tree_uniform(ring + slot * S::SLOT);
                const uint32_t fresh = st == first;   // it begins the sums
                wait(p_full + 8 * place, (p_phase >> place) & 1u);
                p_phase ^= 1u << place;
                if (dual) wait(turn + 8 * stream, (turns & 1) ^ (stream == 0));
                tc_fence_after();
                if (tree_elect()) {
                    const uint64_t v = sw128_desc_mn(tile, STEP * 128);
#pragma unroll
                    for (int kb = 0; kb < STEP / 16; ++kb) {
                        tc_mma_ts(d, p + 16 * kb, v + 128 * kb, idesc_o, kb > 0 || !fresh);
                        tc_mma_ts(d, p + 16 * kb + 8, v + 128 * kb, idesc_o, 1);
                    }
                    tc_commit(empty + 8 * slot);
                    if (alone) tc_commit(empty + 8 * slot);
                    if (STREAMS == 1) tc_commit(pv_done);
                    if (st + stride >= steps) {
                        tc_commit(o_full);
                        mbar_arrive(o_full);
                    }
                }
                __syncwarp();
            };
            if (first >= steps) {  // the one step is the other stream's
                if (lane == 0) mbar_arrive(q_empty);
                wait(o_free, free_phase ^ 1u);
                free_phase ^= 1u;
                // (only now: o_full's phase before this item's is complete, so that no arrival counts for it)
                if (lane == 0) {
                    mbar_arrive(o_full);
                    mbar_arrive(o_full);
                }
            }
#pragma unroll 1
            for (int st = first - stride; st < steps; st += stride) {
                const bool again = st + stride < steps;
                if (STREAMS == 1 && again) scores(st + stride);
                if (st >= first) {
                    values(st);
                    // With both streams at work their products go in turn, a stream's P V and next S as one: the
                    // streams then are half a round apart, and one's softmax has the cores while the other's
                    // products run.  The turn is not held for keys that are not there yet.
                    if (dual) {
                        const int at = step0 + st + 1, slot = 2 * at % NSLOT;
                        const bool there = again && __all_sync(0xFFFFFFFFu, mbar_test_wait(full + 8 * slot, (2 * at / NSLOT) & 1));
                        if (there) scores(st + 1);
                        if (lane == 0) mbar_arrive(turn + 8 * (stream ^ 1));
                        ++turns;
                        if (again && !there) scores(st + 1);
                        continue;
                    }
                }
                if (STREAMS == 2 && again) scores(st + stride);
            }
            step0 += steps;
            more = after(seg);
        }
    } else {
        // ================= softmax =================
        constexpr float kShift = S::BF ? 0.0f : 7.0f;  // fp16 weights are scaled by 2^7
        const int stream = (warp - S::SOFTMAX) >> 2;
        const int r = tid & (kTreeRows - 1);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's lanes of TMEM
        uint32_t s_phase = 0, o_phase = 0, pv_jobs = 0;
        int step0 = 0;
        while (more) {
            const TreeSeq& sq = seg.seq;
            const int kvh = head_of(seg), row0 = row0_of(seg), rows = rows_of(seg);
            const bool dual = rows > kTreeRows;
            const int steps = seg.step_end - seg.step;
            const int ctx = sq.len - sq.n;
            const int tile = dual ? stream : 0;
            const int in_item = tile * kTreeRows + r;
            const bool live = in_item < rows;
            const int row = row0 + in_item, i = live ? token_of_row(row) : 0, head = kvh * G + (live ? row - i * G : 0);
            const bool any_live = __any_sync(0xFFFFFFFFu, live);
            TreeRow see{0, ctx, 0, a.window > 0 ? a.sinks : 0};
            if (live) {
                const uint64_t all = sq.n == 64 ? ~0ull : (1ull << sq.n) - 1;
                see.word = (a.mask ? a.mask[sq.first + i] : ~0ull >> (63 - i)) & all;
                if (a.window > 0) see.from = max(0, ctx + __popcll(see.word) - a.window);
            }
            const int edge = a.window > 0 ? ctx + sq.n - a.window : 0;
            const int32_t* table = a.block_table + seg.b * a.ld_table;
            const float fabs_scale = fabsf(a.scale * (S::E4M3 && a.kc.scale ? a.kc.scale[kvh] : 1.0f));
            float f = (fabs_scale == 0.0f ? 1.0f : fabs_scale) * 1.4426950408889634f;
            if (fabs_scale < INFINITY) f = fminf(f, 3.4028235e38f);   // so that scores of 0 stay 0
            float m = -INFINITY, ref = 0.0f, l = 0.0f;
            bool first = true;
            const bool alone = STREAMS == 2 && !dual;
            const int first_step = alone ? (stream ^ step0) & 1 : 0;
            if (first_step >= steps) {
                __syncwarp();
                if (lane == 0) mbar_arrive(q_empty);
            }
            for (int st = first_step; st < steps; st += alone ? 2 : 1) {
                const int buf = STREAMS == 2 ? stream : (step0 + st) & 1;
                const int tok0 = tile_of(sq, seg.step + st) * STEP;
                const uint32_t s_at = tmem + lanes + buf * STEP;
                const uint32_t o_at = tmem + lanes + S::TM_O + stream * DP;
                wait(s_full + 8 * buf, (s_phase >> buf) & 1u);
                s_phase ^= 1u << buf;
                tc_fence_after();
                if (first) {
                    if constexpr (S::E4M3 && S::DT == 1) {
                        f *= __uint_as_float(static_cast<uint32_t>(ctl.qe[tile][r] + 127) << 23);
                        // neither 0, which would make NaN of hidden tokens' -infinity, nor infinite: scores are below
                        // 2^26 here, so that next to 0 they stay there
                        if (fabs_scale < INFINITY) f = fminf(fmaxf(f, 0x1p-126f), 3.4028235e38f);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_empty);
                }
                if (!any_live) {  // what these rows of P hold reaches only rows that nobody reads
                    if (lane == 0) mbar_arrive(p_full + 8 * buf);
                    first = false;
                    if constexpr (STREAMS == 1) ++pv_jobs;
                    continue;
                }
                const bool bad = *static_cast<volatile int*>(&ctl.bad_page) != 0;
                const bool masked = bad || tok0 + STEP > ctx ||
                                    (a.window > 0 && tok0 < edge && tok0 + STEP > a.sinks);
                auto seen_of = [&](int t0) {
                    uint32_t v = see.seen(t0);
                    if (bad)
                        for (uint32_t left = v; left; left &= left - 1) {
                            const int bit = __ffs(left) - 1, tok = t0 + bit;
                            if (static_cast<unsigned>(table[page_shift >= 0 ? tok >> page_shift : tok / a.page_size]) >=
                                static_cast<unsigned>(a.num_pages))
                                v &= ~(1u << bit);
                        }
                    return v;
                };
                if (masked) {  // -infinity, in TMEM, for what the row does not see
                    auto hide = [&](uint32_t (&x)[32], int c) {
                        const uint32_t seen = seen_of(tok0 + c);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = (seen >> e) & 1u ? x[e] : 0xFF800000u;
                        tmem_st16(s_at + c, reinterpret_cast<uint32_t(&)[16]>(x[0]));
                        tmem_st16(s_at + c + 16, reinterpret_cast<uint32_t(&)[16]>(x[16]));
                    };
#pragma unroll 1
                    for (int c = 0; c < STEP; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(s_at + c, x);
                        tmem_wait_ld32(x);
                        hide(x, c);
                    }
                    tmem_wait_st();
                }
                // The row's maximum comes with the loads; the last 64 tokens stay in registers, the first come again
                // while those are at work.  In loops: with a whole row's code in one line the roles' code no
                // longer fits in the instruction cache and is fetched anew in every step.
                constexpr int NC = STEP / 32;
                uint32_t xa[32], xb[32], most[4] = {0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u};
                if (NC == 4) {
                    tmem_ld32_max(s_at, xa, most[0]);
                    tmem_ld32_max(s_at + 32, xb, most[1]);
                    tmem_wait_ld32(xa);
                    tmem_wait_ld32(xb);
                    asm volatile("" : "+r"(most[0]), "+r"(most[1]));
                }
                tmem_ld32_max(s_at + STEP - 64, xa, most[2]);
                tmem_ld32_max(s_at + STEP - 32, xb, most[3]);
                tmem_wait_ld32(xa);
                tmem_wait_ld32(xb);
                asm volatile("" : "+r"(most[2]), "+r"(most[3]));
                const float top = f * tree_max(tree_max(__uint_as_float(most[0]), __uint_as_float(most[1])),
                                               tree_max(__uint_as_float(most[2]), __uint_as_float(most[3])));
                if (__any_sync(0xFFFFFFFFu, !(top <= m + kTreeLag))) {
                    const float now = tree_max(m, top);
                    const float scale = now == m ? 1.0f : tree_exp2(m - now);
                    m = now;
                    ref = now == -INFINITY ? 0.0f : now - kShift;
                    l *= scale;
                    if (!first) {
                        if constexpr (STREAMS == 1) wait(pv_done, (pv_jobs - 1) & 1u);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < DP; c += 16) {
                            uint32_t y[16];
                            tmem_ld16(o_at + c, y);
                            tmem_wait_ld16(y);
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * scale);
                            tmem_st16(o_at + c, y);
                        }
                    }
                }
                uint64_t l2[2] = {0, 0};
                const uint64_t f2 = pack_f2(f, f), ref2 = pack_f2(-ref, -ref);
                auto weights = [&](const uint32_t (&x)[32], int h, uint32_t to) {
                    uint32_t y[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const uint32_t* xe = &x[h + e];
                        float p0, p1;
                        unpack_f2(fma_f2(pack_f2(__uint_as_float(xe[0]), __uint_as_float(xe[1])), f2, ref2), p0, p1);
                        p0 = tree_exp2(p0);
                        p1 = tree_exp2(p1);
                        l2[e / 2 & 1] = add_f2(l2[e / 2 & 1], pack_f2(p0, p1));
                        // two parts, both positive over 16-bit caches so that an infinite value gives its infinity
                        uint32_t hi;
                        float low0, low1;
                        if constexpr (S::BF) {
                            // the high part is cut off, not rounded; the rest and 2^-22 of the weight are never 0
                            const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                            hi = __byte_perm(b0, b1, 0x7632);
                            const uint64_t cut = pack_f2(__uint_as_float((b0 & 0xFFFF0000u) ^ 0x80000000u),
                                                         __uint_as_float((b1 & 0xFFFF0000u) ^ 0x80000000u));
                            unpack_f2(fma_f2(pack_f2(p0, p1), pack_f2(1.0f + 0x1p-22f, 1.0f + 0x1p-22f), cut), low0, low1);
                        } else {
                            // likewise, to 10 bits; over 16-bit caches of a weight less 2^-10 of it
                            float c0 = p0, c1 = p1;
                            if constexpr (!S::E4M3)
                                unpack_f2(mul_f2(pack_f2(p0, p1), pack_f2(1.0f - 0x1p-10f, 1.0f - 0x1p-10f)), c0, c1);
                            asm("cvt.rz.relu.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(c1), "f"(c0));
                            const uint64_t cut = pack_f2(__uint_as_float((__float_as_uint(c0) & 0xFFFFE000u) ^ 0x80000000u),
                                                         __uint_as_float((__float_as_uint(c1) & 0xFFFFE000u) ^ 0x80000000u));
                            unpack_f2(add_f2(pack_f2(p0, p1), cut), low0, low1);
                        }
                        // of a block of 16 tokens the high parts in columns 0 .. 7, the low ones in 8 .. 15
                        y[e / 2] = hi;
                        y[e / 2 + 8] = dec_pack2<S::BF ? 1 : 0>(low0, low1);
                    }
                    tmem_st16(to, y);
                };
#pragma unroll 1
                for (int c = NC - 2; c >= 0; c -= 2) {
                    weights(xa, 0, s_at + 32 * c);
                    weights(xa, 16, s_at + 32 * c + 16);
                    if (c > 0) tmem_ld32(s_at, xa);
                    weights(xb, 0, s_at + 32 * c + 32);
                    weights(xb, 16, s_at + 32 * c + 48);
                    if (c > 0) {
                        tmem_ld32(s_at + 32, xb);
                        tmem_wait_ld32(xa);
                        tmem_wait_ld32(xb);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * buf);
                {
                    float s0, s1;
                    unpack_f2(add_f2(l2[0], l2[1]), s0, s1);
                    l += s0 + s1;
                }
                first = false;
                if constexpr (STREAMS == 1) ++pv_jobs;
            }

            // ---- the end of the segment ----
            wait(o_full, o_phase);
            o_phase ^= 1u;
            tc_fence_after();
            const bool begins = seg.step == 0, ends = seg.step_end == sq.steps, whole = begins && ends;
            float* part = parts + (2 * cta + (begins ? 1 : 0)) * tree_part_floats(S::ROWS, DP);
            const float vs = S::E4M3 && a.vc.scale ? a.vc.scale[kvh] : 1.0f;
            // the sums of stream x times fx[x]
            float fx[2] = {1.0f, 1.0f};
            int c0 = 0, c1 = DP;             // columns of this thread
            bool use[2] = {stream == 0 || STREAMS == 1, stream == 1};
            if (STREAMS == 2 && !dual) {     // the streams' sums of the same rows are joined
                // (they have been read before the next item's first P V, which o_free holds back)
                float2 (&st)[STREAMS][kTreeRows] = ctl.stats;
                st[stream][r] = make_float2(m, l);
                asm volatile("bar.sync 1, %0;" ::"n"(32 * SW) : "memory");
                const float2 s0 = st[0][r], s1 = st[STREAMS - 1][r];
                m = tree_max(s0.x, s1.x);
                fx[0] = s0.x == -INFINITY ? 0.0f : tree_exp2(s0.x - m);
                fx[1] = s1.x == -INFINITY ? 0.0f : tree_exp2(s1.x - m);
                l = s0.y * fx[0] + s1.y * fx[1];
                // A stream that had no job has nothing in its place.  (One whose weights vanish beside the other's has: its
                // sums are finite, or infinite and NaN from such values, which 0 times them hands on as NaN.)
                use[0] = steps > 1 || (step0 & 1) == 0;
                use[1] = steps > 1 || (step0 & 1) == 1;
                c0 = stream * (DP / 2), c1 = c0 + DP / 2;
            }
            const int64_t out_row = sq.first + i;
            const float inv = l == 0.0f ? 0.0f : vs / l;
            const bool patch = *static_cast<volatile int*>(&ctl.dirty) != 0;
            // (in short pieces, as code that runs once per item comes from beyond the SM)
#pragma unroll 1
            for (int c = any_live ? c0 : c1; c < c1; c += 16) {
                uint32_t x[STREAMS][16];
                float o[16];
#pragma unroll
                for (int s = 0; s < STREAMS; ++s) tmem_ld16(tmem + lanes + S::TM_O + s * DP + c, x[s]);
#pragma unroll
                for (int s = 0; s < STREAMS; ++s) tmem_wait_ld16(x[s]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    o[e] = use[0] ? __uint_as_float(x[0][e]) * fx[0] : 0.0f;
                    if (STREAMS == 2 && use[1]) o[e] = fmaf(__uint_as_float(x[STREAMS - 1][e]), fx[1], o[e]);
                }
                if (patch && live) {  // infinite values and NaN of tokens that this row sees
#pragma unroll 1
                    for (int st = seg.step; st < seg.step_end; ++st) {
                        const int tok0 = tile_of(sq, st) * STEP;
#pragma unroll 1
                        for (int t0 = tok0; t0 < tok0 + STEP; t0 += 32) {
                            if (t0 + 32 <= ctx && (t0 >= edge || t0 + 32 <= a.sinks)) continue;   // seen by all rows
#pragma unroll 1
                            for (uint32_t left = see.seen(t0); left; left &= left - 1) {
                                const int tok = t0 + __ffs(left) - 1;
                                if (!(tok >= ctx || (tok < edge && tok >= a.sinks))) continue;
                                const int in = page_shift >= 0 ? tok >> page_shift : tok / a.page_size;
                                const int page = table[in];
                                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) continue;
                                const int64_t at = page * a.vc.page_stride + (tok - in * a.page_size) * a.vc.slot_stride +
                                                   kvh * a.vc.head_stride + c;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    if (c + e >= a.head_dim) continue;
                                    float v;
                                    if constexpr (S::E4M3)
                                        v = (static_cast<const uint8_t*>(a.vc.p)[at + e] & 0x7F) == 0x7F ? NAN : 0.0f;
                                    else
                                        v = dec_to_f32<S::DT>(static_cast<const uint16_t*>(a.vc.p)[at + e]);
                                    if (!(fabsf(v) < INFINITY)) o[e] += v;
                                }
                            }
                        }
                    }
                }
                if (!live) continue;
                if (whole) {
                    uint16_t* dst = a.out + out_row * a.ldo + static_cast<int64_t>(head) * a.head_dim + c;
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        if (c + e < a.head_dim)
                            *reinterpret_cast<uint4*>(dst + e) = make_uint4(
                                dec_pack2<S::DT>(o[e] * inv, o[e + 1] * inv), dec_pack2<S::DT>(o[e + 2] * inv, o[e + 3] * inv),
                                dec_pack2<S::DT>(o[e + 4] * inv, o[e + 5] * inv), dec_pack2<S::DT>(o[e + 6] * inv, o[e + 7] * inv));
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + 2 * S::ROWS) + c / 4 * S::ROWS + in_item;
#pragma unroll
                    for (int e = 0; e < 16; e += 4) dst[e / 4 * S::ROWS] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            if (live && c0 == 0) {
                if (!whole) part[in_item] = m, part[S::ROWS + in_item] = l;
                else if (a.lse)
                    a.lse[out_row * a.q_heads + head] =
                        l > 0.0f ? (m - kShift) * 0.69314718055994531f + logf(l) : l == 0.0f ? -INFINITY : m;
            }
            if (begins && !ends && tid == 32 * S::SOFTMAX) {
                const long long last = share_end - seg.rest - sq.weight;  // its last step's place in the line
                heads[cta] = TreePart{static_cast<int>(tree_quotient(last, line.share)) - cta + 1, row0, rows, kvh * G,
                                      sq.first, vs, {0, 0}};
            }
            step0 += steps;
            more = after(seg);
        }
    }
    // every MMA is done before TMEM is given back: the last ones were waited for by the softmax warps;
    // after a wait that ran out a millisecond lets what is under way come to its end
    if (*static_cast<volatile int*>(&ctl.abort_flag) != 0)
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) __nanosleep(1000);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the parts of items that several CTAs hold.  blockIdx.x: the CTA that began the item; blockIdx.y: 32 of its
// rows, a lane each, and 32 columns, four for each warp.
constexpr int kTreeJoinThreads = 256;
template <int DT, int DP, bool SHIFT>
__global__ void __launch_bounds__(kTreeJoinThreads) tree_join_kernel(TreeArgs a, int ctas) {
    constexpr float kShift = SHIFT ? 7.0f : 0.0f;
    constexpr int ROWS = kTreeRows * tree_streams(DP), PIECES = DP / 32;
    constexpr int PITCH = 36;   // of a staged row, so that lanes' 8 bytes fall in different banks
    __shared__ __align__(16) uint16_t staged[32 * PITCH];
    grid_dep_wait();
    const TreePart* heads = static_cast<const TreePart*>(a.workspace);
    const TreePart h = heads[blockIdx.x];
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int row0 = 32 * static_cast<int>(blockIdx.y / PIECES), col0 = 32 * static_cast<int>(blockIdx.y % PIECES);
    const int row = row0 + lane;
    if (h.n <= 0 || row0 >= h.rows || col0 >= a.head_dim) return;
    const int G = a.q_heads / a.kv_heads;
    // Part k: the item's first stands second in its CTA's place, the others first in theirs.  (Rows behind the
    // last hold whatever they held: they are not stored.)
    constexpr size_t PART = tree_part_floats(ROWS, DP);
    const float* parts = reinterpret_cast<const float*>(heads + ctas) + 2 * blockIdx.x * PART + row;
    auto part_of = [&](int k) { return parts + (k == 0 ? PART : 2 * k * PART); };
    float top = -INFINITY;
#pragma unroll 8
    for (int k = 0; k < h.n; ++k) top = tree_max(top, *part_of(k));
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < h.n; ++k) {
        const float* p = part_of(k);
        const float m = p[0], l = p[ROWS];
        const float4 x = *(reinterpret_cast<const float4*>(p - row + 2 * ROWS) + (col0 / 4 + warp) * ROWS + row);
        const float f = m == -INFINITY ? 0.0f : tree_exp2(m - top);
        sum += l * f;
        // (a part whose weights vanish still hands on values that are infinite or NaN, as NaN)
        acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
    }
    const float inv = sum == 0.0f ? 0.0f : h.vs / sum;
    *reinterpret_cast<uint2*>(staged + lane * PITCH + 4 * warp) =
        make_uint2(dec_pack2<DT>(acc.x * inv, acc.y * inv), dec_pack2<DT>(acc.z * inv, acc.w * inv));
    if (warp == 0 && col0 == 0 && row < h.rows && a.lse) {
        const int r = h.row0 + row, i = r / G, head = h.head0 + r - i * G;
        a.lse[static_cast<int64_t>(h.first + i) * a.q_heads + head] =
            sum > 0.0f ? (top - kShift) * 0.69314718055994531f + logf(sum) : sum == 0.0f ? -INFINITY : top;
    }
    __syncthreads();
    const int in = tid >> 2, c = tid & 3;   // four 16-byte chunks of a row
    if (in < 32 && row0 + in < h.rows && col0 + 8 * c < a.head_dim) {
        const int r = h.row0 + row0 + in, i = r / G, head = h.head0 + r - i * G;
        const uint16_t* from = staged + in * PITCH + 8 * c;
        const uint2 lo = *reinterpret_cast<const uint2*>(from), hi = *reinterpret_cast<const uint2*>(from + 4);
        *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(h.first + i) * a.ldo +
                                  static_cast<int64_t>(head) * a.head_dim + col0 + 8 * c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

template <class S>
int launch_tree_shape(const DeviceCtx& ctx, const TreeArgs& a, cudaStream_t stream) {
    if (cudaFuncSetAttribute(tree_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM) != cudaSuccess)
        return -3;
    // Boxes of the largest power of two of tokens that divides the pages: from 8 on, the rows of one
    // swizzle pattern.  Other pages, and heads or slots of stride 0, are read without tensor maps.
    int box = a.page_size & -a.page_size;
    box = box < S::STEP ? box : S::STEP;
    CUtensorMap maps[3] = {};
    if (box < 8 || !tree_map(&maps[0], a, a.kc, S::E4M3, S::DP, box) || !tree_map(&maps[1], a, a.vc, S::E4M3, S::DP, box))
        box = 0;
    // Queries by tensor copies where a tile of rows is whole tokens.
    const int G = a.q_heads / a.kv_heads;
    int q_box = kTreeRows % G == 0 ? kTreeRows / G : 0;
    if (q_box > 0 && !tree_query_map(&maps[2], a, q_box)) q_box = 0;
    const int rc = launch_dependent(tree_kernel<S>, dim3(static_cast<unsigned>(ctx.num_sms)), dim3(S::THREADS),
                                    S::SMEM, stream, a, power_of_two(a.page_size), box, q_box, maps[0], maps[1], maps[2]);
    if (rc != 0) return rc;
    return launch_dependent(tree_join_kernel<S::DT, S::DP, !S::BF>, dim3(static_cast<unsigned>(ctx.num_sms), S::ROWS / 32 * (S::DP / 32)),
                            dim3(kTreeJoinThreads), 0, stream, a, ctx.num_sms);
}

template <int DT, bool E4M3>
int launch_tree_dp(const DeviceCtx& ctx, const TreeArgs& a, cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_tree_shape<TreeShape<DT, E4M3, 64>>(ctx, a, stream);
    if (a.head_dim <= 128) return launch_tree_shape<TreeShape<DT, E4M3, 128>>(ctx, a, stream);
    return launch_tree_shape<TreeShape<DT, E4M3, 256>>(ctx, a, stream);
}

}  // namespace

// One instance per translation unit (tree_*.cu), which compile in parallel.
template <int DT, bool E4M3>
int launch_tree_typed(const DeviceCtx& ctx, const TreeArgs& a, cudaStream_t stream);

}  // namespace w4g
