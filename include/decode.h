/*
 * decode.h -- C ABI of the decoder-layer operators that stand between the 4-bit GEMMs of
 * the library (NVIDIA GB300, sm_103a):
 *
 *   dec_rms_norm, _i8, _mx   root-mean-square norm of x + residual, written as fp16 / bf16,
 *                            as int8 rows with fp32 scales (what w4a8_gemm takes) or as
 *                            E4M3 with E8M0 block scales (what mx_gemm takes)
 *   dec_rope_table           cosines and sines of every position, scaled for long contexts
 *   dec_rope_append          rotary positions on new queries and keys; keys and values
 *                            written to their slots of a paged cache
 *   dec_attn_paged           attention of one new token per sequence over that cache
 *   dec_attn_tree            attention of up to 64 drafted tokens per sequence, in a tree or a chain,
 *                            over that cache; sliding window with first tokens that stay visible
 *   dec_token_logprobs       log probabilities of given tokens, entropy and largest logits
 *   dec_kv_move              cached tokens moved to other slots (the accepted ones of a tree)
 *
 * A decoder layer runs them as  norm -> QKV GEMM -> rope + append -> attention -> output
 * GEMM (residual fused) -> norm -> feed-forward GEMMs.  With drafted tokens the attention is
 * dec_attn_tree; the model's last GEMM is followed by dec_token_logprobs, from which the program
 * chooses the accepted path, and dec_kv_move then closes every layer's cache up.
 *
 * Conventions are those of w4a16.h: device pointers on the current device, caller-owned
 * buffers, `stream` a cudaStream_t passed as void*, asynchronous calls that a CUDA graph
 * can capture, w4a16_status return codes, kernel-detected errors in the device status word
 * read by w4a16_get_device_status().  Every kernel here is launched with programmatic
 * dependent launch and reads and writes memory only after the previous kernel in the
 * stream has finished (of them only the norm of aligned rows lets the next one start before it
 * ends itself).  Strides ("ld...") count elements; 0 stands for packed rows.
 */
#ifndef DECODE_H_
#define DECODE_H_

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- root-mean-square norm -------------------------------------------------------------
 *
 *   h[m, i] = x[m, i] + residual[m, i]                       (fp32; x alone without one)
 *   r[m]    = 1 / sqrt( sum_i h[m, i]^2 / H + eps )          (fp32)
 *   y[m, i] = (h[m, i] * weight[i]) * r[m]                   (fp32)
 *   residual_out[m, i] = RNE_dtype( h[m, i] )
 *
 * The sums take h before it is rounded: y does not depend on residual_out's rounding.  The
 * products are taken in that order, so h^2 and h weight have to stay within fp32's range.
 *   x         device, dtype [M] rows of H, ldx elements apart.
 *   residual  device, dtype [M] rows, ldr apart, or NULL.
 *   weight    device, dtype [H], or NULL (all ones).
 *   M, H      M >= 0 (0 is a no-op), 1 <= H <= 1048576.
 *   dtype     w4a16_dtype of x, residual, weight and residual_out (and of y).
 *   eps       >= 0, finite.  With 0 a zero row gives NaN in 16 bits (0 / 0) and zeros in 8 bits.
 *   residual_out  device output, rows ldr apart, or NULL (not written).  It may be
 *             `residual` itself, or x where ldx == ldr.
 *   ldx, ldr, ldy  row strides in elements, 0 = H; else at least H.
 * Pointers need the alignment of their element type only; rows that are 16-byte aligned
 * (base and stride) with H a multiple of 8 and at most 32768 take the faster path.
 * Errors: INVALID_ARG (null pointer, M < 0, H < 1, eps, stride below H, misaligned),
 * UNSUPPORTED (dtype, H too large), CUDA.
 */

/* y[m, i] rounded to dtype: device output, rows ldy apart; it may be x itself (ldy == ldx). */
int dec_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                 const void* weight, int M, int H, int dtype, float eps, void* residual_out,
                 void* y, int64_t ldy, void* stream);

/*
 * y as int8 rows, the activations that w4a8_gemm takes, from the fp32 values (they are not
 * rounded to dtype in between, unlike dec_rms_norm followed by w4a8_quantize_act):
 *     s_y[m] = max_i |y[m, i]| / 127   (fp32; 1 for a zero row)
 *     y_i8[m, i] = rint(y[m, i] * (127 / max))
 * (the fp32 product with a rounded factor: within 2^-22 of the quotient y / s_y, relative, so that
 * a code differs from the quotient's only where that is as near to a half).
 *   y_i8  device output, int8 [M][H] packed, 8-byte aligned; H a multiple of 8, at most
 *         32768 (w4a8_gemm itself wants a multiple of 128).
 *   s_y   device output, float [M].
 * x, residual, residual_out and weight have to be 16-byte aligned with ldx, ldr multiples
 * of 8 (INVALID_ARG otherwise).  A row whose h holds an infinity or a NaN gives undefined codes, and
 * NaN as its scale.
 */
int dec_rms_norm_i8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                    const void* weight, int M, int H, int dtype, float eps,
                    void* residual_out, int8_t* y_i8, float* s_y, void* stream);

/*
 * y as E4M3 codes with one E8M0 scale per 32 values, the activations that mx_gemm takes:
 *     X = clamp(floor(log2(max |y|)) - 8, -127, 127) over the block (-127 for a zero block)
 *     y_scales = X + 127,  y_codes = RNE_E4M3(y * 2^-X), saturated to +-448
 *   y_codes   device output, uint8 [M][H] packed, 8-byte aligned; H a multiple of 32, at
 *             most 32768 (mx_gemm itself wants a multiple of 128).
 *   y_scales  device output, uint8 [M][H/32] packed.
 * Alignment of the inputs as for dec_rms_norm_i8.  A block that holds an infinity or a NaN
 * gives an undefined scale.
 */
int dec_rms_norm_mx(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                    const void* weight, int M, int H, int dtype, float eps,
                    void* residual_out, uint8_t* y_codes, uint8_t* y_scales, void* stream);

/* ---- the paged key-value cache ----------------------------------------------------------
 *
 * Element d of head h of the key in slot s of page p stands at
 *     k + p * k_page_stride + s * k_slot_stride + h * k_head_stride + d
 * (elements; likewise v), so pages may hold tokens of all heads ([page][slot][head][d]) or
 * heads of all tokens ([page][head][slot][d]).  Offsets are computed in 64 bits.
 */
typedef enum dec_kv_dtype {
    DEC_KV_FP16 = 0,
    DEC_KV_BF16 = 1,
    DEC_KV_E4M3 = 2  /* one byte a value; the value is the E4M3 number times the head's scale */
} dec_kv_dtype;

typedef struct dec_kv_cache {
    void* k;               /* device, 16-byte aligned                                      */
    void* v;
    const float* k_scale;  /* device, float [kv_heads], E4M3 only; NULL = all ones          */
    const float* v_scale;
    int64_t k_page_stride, k_slot_stride, k_head_stride; /* >= 0, multiples of 16 bytes    */
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int num_pages;         /* >= 1                                                         */
    int page_size;         /* slots of a page, >= 1                                        */
    int kv_heads;          /* >= 1                                                         */
    int head_dim;          /* 8..256, a multiple of 8 (E4M3: 16..256, of 16)               */
    int dtype;             /* dec_kv_dtype                                                 */
    int reserved;          /* 0                                                            */
} dec_kv_cache;

/* ---- rotary positions -------------------------------------------------------------------
 *
 * Pair j < rot_dim / 2 of a head turns by angle(pos, j) = pos * f(j):
 *     a' = a cos - b sin,  b' = b cos + a sin,
 * with (a, b) = (x[j], x[j + rot_dim/2]) in the HALF layout and (x[2j], x[2j+1]) in the
 * INTERLEAVED one.  Values from rot_dim on are copied.
 */
typedef enum dec_rope_layout {
    DEC_ROPE_HALF = 0,
    DEC_ROPE_INTERLEAVED = 1
} dec_rope_layout;

/* How the frequencies f(j) = base^(-2j / rot_dim) are scaled for contexts longer than those
 * a model was trained on. */
typedef enum dec_rope_scaling_kind {
    DEC_ROPE_SCALE_NONE = 0,
    DEC_ROPE_SCALE_LINEAR = 1, /* f / factor (positions interpolated)                       */
    DEC_ROPE_SCALE_BASE = 2,   /* base' = base * factor^(rot_dim / (rot_dim - 2))           */
    DEC_ROPE_SCALE_RAMP = 3    /* by the turns t = original_len * f / (2 pi) that a pair makes
                                  over the trained length: w = clamp((t - low) / (high - low),
                                  0, 1), f' = w f + (1 - w) f / factor                      */
} dec_rope_scaling_kind;

typedef struct dec_rope_scaling {
    int kind;            /* dec_rope_scaling_kind                                           */
    float factor;        /* > 0                                                             */
    float low, high;     /* RAMP: turns, low < high                                         */
    float original_len;  /* RAMP: the trained length, > 0                                   */
    float magnitude;     /* cos and sin are multiplied by it; 0 stands for 1                */
} dec_rope_scaling;

/*
 * The table of cosines and sines that dec_rope_append takes, computed in fp64 and rounded
 * once:  table[pos][j] = magnitude * cos(angle(pos, j)),  table[pos][rot_dim/2 + j] =
 * magnitude * sin(angle(pos, j)), for pos < table_len.  Run once per model.
 *   rot_dim    even, 2..256 (BASE scaling: at least 4).
 *   base       > 1, finite.
 *   scaling    NULL = none.
 *   table      device output, float [table_len][rot_dim], 16-byte aligned.
 * Errors: INVALID_ARG, UNSUPPORTED (rot_dim), CUDA.
 */
int dec_rope_table(int rot_dim, double base, const dec_rope_scaling* scaling, float* table,
                   int table_len, void* stream);

typedef struct dec_rope_config {
    int q_heads;         /* >= 0; 0 = no queries                                            */
    int kv_heads;        /* >= 0; 0 = no keys and values                                    */
    int head_dim;        /* 8..256, a multiple of 8                                         */
    int dtype;           /* w4a16_dtype of q, k, v and their outputs                        */
    int rot_dim;         /* even, 0..head_dim                                               */
    int layout;          /* dec_rope_layout                                                 */
    int table_len;       /* positions in the table                                          */
    int reserved;        /* 0                                                               */
    const float* table;  /* device, float [table_len][rot_dim], as by dec_rope_table        */
    int64_t ldq, ldk, ldv;  /* row strides of q, k, v; 0 = heads * head_dim; multiples of 8 */
    int64_t ldqo, ldko;     /* row strides of q_out, k_out                                  */
} dec_rope_config;

/*
 * Rotates the queries and keys of T new tokens and writes keys and values into the cache.
 *   cfg        host struct, read during the call.
 *   cache      host struct, read during the call, or NULL (nothing is cached).  kv_heads and
 *              head_dim as in cfg; dtype cfg's, or E4M3: then keys and values are stored as
 *              RNE_E4M3(value / scale), saturated to +-448, from the fp32 rotation.
 *   q, k, v    device, dtype, T rows of heads * head_dim, 16-byte aligned (they may be slices
 *              of one fused projection's rows).  q is NULL only if cfg->q_heads is 0, k only
 *              if kv_heads is 0; v may be NULL without a cache.
 *   positions  device, int32 [T]: row of the table.
 *   slots      device, int64 [T]: page * page_size + slot of the token in the cache; negative
 *              = the token is not cached (so for padding).  A token's values are written by threads
 *              of their own: a slot that two tokens share holds a mix of both, each of its
 *              values from either.  May be NULL without a cache.
 *   q_out      device output, rows ldqo apart; it may be q itself (ldqo == ldq).
 *   k_out      device output, rows ldko apart, or NULL; it may be k itself.
 *   T          0 is a no-op.
 * A position outside the table or a slot outside the cache writes nothing of that token (a
 * slot: nothing of it to the cache) and records W4A16_ERR_INVALID_ARG in the status word.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, rot_dim, dtype, stride multiples), CUDA.
 */
int dec_rope_append(const dec_rope_config* cfg, const dec_kv_cache* cache, const void* q,
                    const void* k, const void* v, int T, const int32_t* positions,
                    const int64_t* slots, void* q_out, void* k_out, void* stream);

/* ---- attention of one new token ----------------------------------------------------------
 *
 * Sequence b's token, query head h (key-value head g = h / (q_heads / kv_heads)), over the
 * cached tokens j with max(0, lens[b] - window) <= j < lens[b]:
 *     s_j = scale * sum_d q[b, h, d] k_j[g, d]
 *     out[b, h, :] = sum_j exp(s_j) v_j[g, :] / sum_j exp(s_j),   lse[b, h] = log sum_j exp(s_j)
 * The new token's own key and value are cached before the call (dec_rope_append) and lens
 * counts them.  A sequence of length 0 gives out = 0 and lse = -infinity.  What the pages
 * hold outside those tokens is not used, whatever it is.  A score that is NaN gives NaN in the row's
 * out and lse, one of +infinity NaN in out and +infinity in lse.  One of -infinity has the
 * weight 0; a row with no other gives what a length of 0 does.  An infinite value gives that infinity
 * (NaN with one of the other sign) if its token's weight is at least 2^-28 of the row's
 * largest, else that or NaN; a value that is NaN gives NaN.  Otherwise the weights are exact to 2^-15,
 * and with fp16 or 8-bit caches to 2^-32 of the row's largest.
 */
typedef struct dec_attn_config {
    int q_heads;         /* a multiple of the cache's kv_heads                              */
    int dtype;           /* w4a16_dtype of q and out                                        */
    int max_pages;       /* columns of block_table                                          */
    int window;          /* tokens attended to, counted back from the newest; 0 = all       */
    float scale;         /* finite                                                          */
    int reserved;        /* 0                                                               */
    int64_t ldq, ldo;    /* row strides of q and out; 0 = q_heads * head_dim; multiples of 8 */
    int64_t ld_table;    /* row stride of block_table; 0 = max_pages                        */
} dec_attn_config;

/*
 * Bytes of workspace that dec_attn_paged needs on the current device, for any batch and any
 * lengths; 0 for arguments that it refuses.  The caller fills the workspace with zeros once;
 * each call leaves it ready for the next one in stream order.  Calls that may run at the
 * same time (other streams) need workspaces of their own.
 */
size_t dec_attn_workspace_bytes(const dec_attn_config* cfg, const dec_kv_cache* cache);

/*
 *   cfg, cache   host structs, read during the call.  The cache's dtype is cfg's, or E4M3.
 *   q            device, dtype [B] rows of q_heads * head_dim, 16-byte aligned.
 *   block_table  device, int32 [B] rows of max_pages page indexes: token j of sequence b is
 *                in slot j % page_size of page block_table[b][j / page_size].  Columns past
 *                the sequence's length (or before its window) are not read.
 *   lens         device, int32 [B], 0 .. max_pages * page_size; together, times q_heads, below 2^39.
 *   out          device output, dtype, rows ldo apart, 16-byte aligned.
 *   lse          device output, float [B][q_heads], or NULL.
 *   workspace    device, 16-byte aligned, ws_bytes >= dec_attn_workspace_bytes(cfg, cache).
 *   B            0 .. 2^27 - 1 (more: UNSUPPORTED); 0 is a no-op.
 * Results do not depend on how the work is split in time: the partial results are joined in
 * a fixed order, and equal inputs give equal bits.  A length outside its range is cut to it,
 * and a page index outside the cache leaves its tokens out; both record
 * W4A16_ERR_INVALID_ARG in the status word.  A wait inside the kernel that runs out
 * records W4A16_ERR_DEVICE_TIMEOUT; the results are then undefined and the workspace has to be
 * filled with zeros again.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
int dec_attn_paged(const dec_attn_config* cfg, const dec_kv_cache* cache, const void* q,
                   const int32_t* block_table, const int32_t* lens, int B, void* out,
                   float* lse, void* workspace, size_t ws_bytes, void* stream);

/* ---- attention of drafted tokens ---------------------------------------------------------
 *
 * Sequence b has n = starts[b+1] - starts[b] drafted tokens, rows starts[b] .. starts[b+1] - 1 of
 * q and out, whose keys and values are the last n of its lens[b] cached tokens: drafted token j
 * is cached token ctx + j, ctx = lens[b] - n.  (Rotary positions are the caller's: tokens of one
 * depth of the tree have the same.)  With mask word w, row i of the sequence sees
 *     the cached tokens j < ctx with  j < sinks  or  j >= ctx + popcount(w) - window
 *         (all of them with window = 0; popcount over the bits below n), and
 *     the drafted tokens j with bit j of w set: its ancestors in the tree and itself.
 * Without a mask the drafted tokens are a chain: w has the bits 0 .. i.  A row then sees the sinks
 * and the newest `window` tokens of its path (and no fewer than what w names).  Over the tokens it sees
 *     s_j = scale * sum_d q[h, d] k_j[g, d],   g = h / (q_heads / kv_heads)
 *     out[h, :] = sum_j exp(s_j) v_j[g, :] / sum_j exp(s_j),   lse[h] = log sum_j exp(s_j)
 * and a row that sees none gives out = 0 and lse = -infinity.  Nothing that a row does not see
 * changes its result, whatever it holds.  A score that is NaN gives NaN in the row's out and lse,
 * one of +infinity NaN in out and +infinity in lse; one of -infinity has the weight 0.  An
 * infinite value gives that infinity (NaN with one of the other sign) if its token's weight is at
 * least 2^-20 of the row's largest, else that or NaN; a value that is NaN gives NaN.
 *
 * Otherwise a token's weight is exact to 2^-15 of itself over a bf16 cache, 2^-19 over an fp16 one and
 * 2^-20 over an 8-bit one (or to 2^-30 of the row's largest, where that is more); the products q k and all sums are
 * fp32's, and what passes its range is infinite.  bf16 queries meet an 8-bit cache in fp16, each row and head scaled by
 * a power of two: values are exact down to 2^-25 of its largest, smaller ones to 2^-33 of it, and a row
 * whose largest is below 2^-118 counts as zeros.
 */
typedef struct dec_tree_config {
    int q_heads;         /* a multiple of the cache's kv_heads                              */
    int dtype;           /* w4a16_dtype of q and out                                        */
    int max_pages;       /* columns of block_table                                          */
    int window;          /* newest tokens of its path that a row sees; 0 = all              */
    int sinks;           /* first tokens that stay visible outside the window, >= 0         */
    float scale;         /* finite                                                          */
    int64_t ldq, ldo;    /* row strides of q and out; 0 = q_heads * head_dim; multiples of 8 */
    int64_t ld_table;    /* row stride of block_table; 0 = max_pages                        */
} dec_tree_config;

/*
 * Bytes of workspace that dec_attn_tree needs on the current device, for any batch and any
 * lengths; 0 for arguments that it refuses.  Its contents before a call do not matter.  Calls that
 * may run at the same time (other streams) need workspaces of their own.
 */
size_t dec_attn_tree_workspace_bytes(const dec_tree_config* cfg, const dec_kv_cache* cache);

/*
 *   cfg, cache   host structs, read during the call.  The cache's dtype is cfg's, or E4M3.
 *   q            device, dtype [T] rows of q_heads * head_dim, 16-byte aligned.
 *   block_table  device, int32 [B] rows of max_pages page indexes, as for dec_attn_paged.
 *   lens         device, int32 [B], n .. max_pages * page_size; together, times q_heads, below 2^39.
 *   starts       device, int32 [B + 1], ascending, 0 .. T; 0 .. 64 tokens each.  A sequence
 *                without drafted tokens costs nothing (its lens is not read).
 *   mask         device, uint64 [T], or NULL (chains).  Bits from n on are ignored.
 *   B            0 .. 2^24 (more: UNSUPPORTED); 0 is a no-op.
 *   T            rows of q, out, mask and lse; 0 is a no-op.
 *   out          device output, dtype, rows ldo apart, 16-byte aligned.  Rows before
 *                starts[0] and from starts[B] on (padding) are left as they were.
 *   lse          device output, float [T][q_heads], or NULL.
 *   workspace    device, 16-byte aligned, ws_bytes >= dec_attn_tree_workspace_bytes(cfg, cache).
 * Equal inputs give equal bits.  A sequence whose starts or lens are out of range is left out (its
 * rows stay as they were), and a page index outside the cache leaves its tokens out; both record
 * W4A16_ERR_INVALID_ARG in the status word.  A wait inside the kernel that runs out records
 * W4A16_ERR_DEVICE_TIMEOUT; the results are then undefined.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
int dec_attn_tree(const dec_tree_config* cfg, const dec_kv_cache* cache, const void* q,
                  const int32_t* block_table, const int32_t* lens, const int32_t* starts,
                  const uint64_t* mask, int B, int T, void* out, float* lse, void* workspace,
                  size_t ws_bytes, void* stream);

/* ---- log probabilities --------------------------------------------------------------------
 *
 * For row t of logits x, with z[t, i] = factor[t] * x[t, i]:
 *     lse[t]          = log sum_i exp(z[t, i])
 *     logprobs[t, c]  = z[t, ids[t, c]] - lse[t]
 *     entropy[t]      = lse[t] - sum_i p_i z[t, i],   p_i = exp(z[t, i] - lse[t])
 *     top_ids[t, 0 .. top-1]   the tokens of the row's largest logits x, in descending order, the
 *                              lowest index first among equals (-0 equals 0)
 *     top_logprobs[t, c]       = z[t, top_ids[t, c]] - lse[t]
 * all in fp32 or more.  A logit of -infinity (a token that is masked out) has probability 0 and adds
 * nothing; in a row of nothing else lse and all log probabilities are -infinity and the entropy
 * is 0.  With a logit of +infinity lse is +infinity, finite logits' log probabilities are -infinity and
 * the infinite ones' and the entropy NaN; with a NaN all three are NaN.  Among the largest logits NaN
 * counts as larger than any number.
 */
typedef enum dec_logits_dtype {
    DEC_LOGITS_FP16 = 0,
    DEC_LOGITS_BF16 = 1,
    DEC_LOGITS_FP32 = 2
} dec_logits_dtype;

typedef struct dec_logprob_config {
    int vocab;           /* logits of a row, 1 .. 2^24                                      */
    int dtype;           /* dec_logits_dtype                                                */
    int n_ids;           /* given tokens of a row, 0 .. 65536                               */
    int top;             /* largest logits of a row, 0 .. min(32, vocab)                    */
    int64_t ld;          /* row stride of the logits in elements; 0 = vocab, else at least that */
} dec_logprob_config;

/*
 *   cfg           host struct, read during the call.
 *   logits        device, T rows, aligned to their element.  Any stride and length; rows whose
 *                 first elements are 16-byte aligned alike take no slow beginning.
 *   factor        device, float [T], 1 / temperature, or NULL (all 1).  One that is not positive, or
 *                 above 2^127, gives NaN in the row's lse, entropy and log probabilities.
 *   ids           device, int32 [T][n_ids]; NULL only if n_ids is 0.  A negative one stands for no
 *                 token: its log probability is written as 0.  One of vocab or more gives NaN and
 *                 records W4A16_ERR_INVALID_ARG in the status word.
 *   T             0 is a no-op.
 *   logprobs      device output, float [T][n_ids]; NULL only if n_ids is 0.
 *   lse, entropy  device output, float [T], or NULL.
 *   top_ids       device output, int32 [T][top]; NULL only if top is 0.
 *   top_logprobs  device output, float [T][top], or NULL.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype, vocab, n_ids, top), CUDA.
 */
int dec_token_logprobs(const dec_logprob_config* cfg, const void* logits, const float* factor,
                       const int32_t* ids, int T, float* logprobs, float* lse, float* entropy,
                       int32_t* top_ids, float* top_logprobs, void* stream);

/* ---- cached tokens to other slots ------------------------------------------------------------
 *
 * Copies the keys and values of all heads in slot src[i] to slot dst[i] (slots numbered page *
 * page_size + slot, as in dec_rope_append) for the moves i of group b, starts[b] <= i <
 * starts[b+1], one after another in their order: a slot that an earlier move of the group wrote
 * is read as written, and of two moves to one slot the later stands.  Groups (one per sequence)
 * run at the same time and may not touch one another's slots.  To keep the path i0 < i1 < ... of
 * a tree cached from slot(ctx) on, move slot(ctx + ij) to slot(ctx + j) for every j.
 *   cache     host struct, read during the call.  No two pages, slots or heads of it, nor keys and
 *             values, may share memory; a stride of 0 where there are several is INVALID_ARG.
 *   src, dst  device, int64 [N].  A negative one stands for no move; one outside the cache moves
 *             nothing and records W4A16_ERR_INVALID_ARG in the status word.
 *   starts    device, int32 [B + 1], ascending, 0 .. N; a group that is out of range moves nothing
 *             and records W4A16_ERR_INVALID_ARG.
 *   B         groups, 0 is a no-op.
 *   N         0 is a no-op.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
int dec_kv_move(const dec_kv_cache* cache, const int64_t* src, const int64_t* dst,
                const int32_t* starts, int B, int N, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_H_ */
