/*
 * bqd.h -- C ABI of libbqd: the decode-time low-bit quantized matrix-vector
 * product (QMV), its prefill matrix product (QMM), the speculative-decoding
 * verification kernel, a paged 8-bit KV cache (append, attention over it, page
 * operations) and what a step with a tree of drafts needs beside them (norm and
 * rotation of queries and keys, attention and verification of a tree, acceptance
 * in the cache, log probabilities), on GB300 (sm_103a).
 *
 * Page defining the operations: "oMLX Bonsai 自定义内核:Qwen 系列快速 QMV 路径
 * 完整解析" (oMLX Bonsai custom kernels: the fast QMV path for the Qwen
 * family), cnnetsun.cn/a/4328761.  Section numbers (§二.1 ...) are that page's.
 *
 * The product (§二.1, §二.2):
 *     y[m, n] = sum_k x[m, k] * (scale[n, k/gs] * q[n, k] + bias[n, k/gs])
 * for m < M activation rows, n < N weight rows (output features), k < K input
 * features, group size gs in {64, 128}, G = K / gs groups per row.
 *
 * Data layout (all tensors dense, row-major, no strides):
 *   x       fp16 [M, K]
 *   scales  fp16 [N, G]
 *   biases  fp16 [N, G], or NULL ("sym": bias = -ratio * scale, not read)
 *   out     fp16 [M, N]   (fp32 accumulation, rounded to nearest even)
 *   w_packed, row n at byte offset n * bqd_packed_bytes(format, 1, K, gs):
 *     BQD_FMT_AFFINE1: uint32 [N, K/32]; code k = 32j+i is bit i of word j
 *     BQD_FMT_AFFINE2: uint32 [N, K/16]; code k = 16j+i is bits 2i..2i+1
 *     BQD_FMT_T5     : uint8  [N, G*ceil(gs/5)]; trits {0,1,2}; byte p of a
 *                      group holds weights 5p..5p+4 of it as sum_i t_i 3^i
 *                      (first weight least significant); 13 bytes per
 *                      64-group, 26 per 128-group (§二.3); the unused high
 *                      trits of a group's last byte are 0
 *   Words are little-endian.
 *
 * Conventions for every entry point:
 *  - Pointers named d_* or documented as device pointers are device memory of
 *    the current CUDA device; the caller allocates, owns and frees them.  The
 *    library allocates no device memory per call.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and return the status of argument validation plus kernel
 *    launch.  Errors found in the DATA (a bad t5 byte, a 2-bit code 3 where a
 *    ternary code is needed) are written to a caller-provided device counter,
 *    which the caller reads back after synchronising.  Kernels never trap.
 *  - Validation happens on the host before anything is enqueued: on an error
 *    nothing is launched and no output is touched.
 *  - Thread-safe and reentrant; calls on one stream run in order.
 */
#ifndef BQD_H
#define BQD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BQD_ABI_VERSION 1

/* status codes */
enum {
    BQD_OK = 0,
    BQD_ERR_INVALID_ARG = 1, /* null pointer, bad size, bad format/group size */
    BQD_ERR_UNSUPPORTED = 2, /* valid request this build does not serve      */
    BQD_ERR_ALIGNMENT = 3,   /* pointer alignment below what is documented   */
    BQD_ERR_BAD_T5_BYTE = 4, /* (for callers mapping a validate count)       */
    BQD_ERR_NOT_TERNARY = 5, /* (for callers mapping a repack count)         */
    BQD_ERR_CUDA = 6,        /* a CUDA runtime call or a launch failed       */
    BQD_ERR_TIMEOUT = 7,     /* a bounded device-side wait ran out           */
    BQD_ERR_ABI = 8          /* header / library ABI mismatch                */
};

/* weight formats */
enum { BQD_FMT_AFFINE1 = 1, BQD_FMT_AFFINE2 = 2, BQD_FMT_T5 = 3 };

/* element types: F16 and F32 for bqd_spec_decode_verify's logits, all three for
 * those of bqd_spec_tree_verify and bqd_token_logprobs, F16 and BF16 for the
 * tensors of the KV cache's entry points and of bqd_qk_norm_rope */
enum { BQD_DTYPE_F16 = 1, BQD_DTYPE_F32 = 2, BQD_DTYPE_BF16 = 3 };

/* code types of the KV cache */
enum { BQD_KV_INT8 = 1, BQD_KV_E4M3 = 2 };

/* tokens that share one scale of the KV cache */
#define BQD_KV_BLOCK 16

/* opaque CUDA stream (binary-compatible with cudaStream_t / CUstream) */
typedef struct CUstream_st *bqd_stream_t;

/*
 * ABI probe (§三: the extension is probed before use).  Returns
 * BQD_ABI_VERSION of the built library; a caller compiled against another
 * header version must not call the rest.  Host-only, never fails.
 */
int bqd_abi_version(void);

/* Static, human-readable text for a status code.  Host-only. */
const char *bqd_status_string(int status);

/*
 * Bytes of the packed weight matrix for (format, N, K, group_size): N*K/8 for
 * 1-bit, N*K/4 for 2-bit, N*(K/gs)*ceil(gs/5) for t5 (13 or 26 bytes per
 * group, §二.3).  Returns 0 for an invalid request (K not a multiple of gs,
 * gs not 64/128, unknown format, negative sizes).  Host-only.
 */
size_t bqd_packed_bytes(int format, int64_t N, int64_t K, int group_size);

/*
 * Quantized matrix-vector / matrix product, §二.1 (M = 1, qmv_fast),
 * §二.2 (M = 2..5, qmv_wide: each packed weight byte is read once for all M
 * rows; sym variant with biases == NULL reads no bias tensor), §二.3 (t5
 * decode, and the fused unpack + tensor-core matrix product for prefill).
 * Any M >= 0 is accepted; the library picks the kernel (decode kernels for
 * small M, the fused product once M is large enough for it on the layer's
 * shape -- beyond 10 to 64 rows depending on format and N).
 *   x        device fp16 [M, K], 16-byte aligned
 *   w_packed device, layout above, 16-byte aligned
 *   scales   device fp16 [N, G], 2-byte aligned
 *   biases   device fp16 [N, G] or NULL.  NULL means the sym identity I-B of
 *            §二.2 with the format's default ratio: 0.5 (1-bit), 1.5 (2-bit),
 *            1.0 (t5: w = scale*t - scale); bias = fp16(-ratio * scale)
 *   out      device fp16 [M, N], 16-byte aligned; fully overwritten
 * M >= 0, N >= 0, K >= 0 with K % group_size == 0.  M == 0 or N == 0 is a
 * no-op; K == 0 writes zeros.  Returns BQD_OK, BQD_ERR_INVALID_ARG,
 * BQD_ERR_ALIGNMENT or BQD_ERR_CUDA.
 */
int bqd_qmv(const void *x, const void *w_packed, const void *scales,
            const void *biases, int64_t M, int64_t N, int64_t K, int format,
            int group_size, void *out, bqd_stream_t stream);

/*
 * Sym variant with an explicit ratio (§二.2 identity I-B: bias =
 * -scale * ratio; the bias tensor does not exist and is not read).  The bias
 * is rebuilt as fp16_rne(float(-ratio) * float(scale)).  Arguments and errors
 * as bqd_qmv; ratio must be finite.
 */
int bqd_qmv_sym(const void *x, const void *w_packed, const void *scales,
                float ratio, int64_t M, int64_t N, int64_t K, int format,
                int group_size, void *out, bqd_stream_t stream);

/*
 * Pack codes into the format's layout (the layout above; §二.1, §二.3).
 *   codes    device uint8 [N, K]; values must be < 2 (1-bit), < 4 (2-bit),
 *            < 3 (t5); larger values are masked (1/2-bit) or taken as 0 (t5)
 *   w_packed device output, bqd_packed_bytes(format, N, K, gs) bytes
 * Returns BQD_OK, BQD_ERR_INVALID_ARG or BQD_ERR_CUDA.
 */
int bqd_pack(const uint8_t *codes, int64_t N, int64_t K, int format,
             int group_size, void *w_packed, bqd_stream_t stream);

/* Inverse of bqd_pack: w_packed (device) -> codes uint8 [N, K] (device). */
int bqd_unpack(const void *w_packed, int64_t N, int64_t K, int format,
               int group_size, uint8_t *codes, bqd_stream_t stream);

/*
 * Repack a 2-bit matrix whose codes are ternary {0,1,2} into t5 (§二.3: the
 * repack_ternary_t5 tool).  The scales are unchanged; the caller's 2-bit
 * biases must equal -scale (t5 has no bias tensor) for the product to be
 * unchanged.
 *   w2       device, 2-bit layout [N, K/16] uint32
 *   w_t5     device output, bqd_packed_bytes(BQD_FMT_T5, N, K, gs) bytes
 *   d_status device int32: receives the number of 2-bit codes equal to 3
 *            (0 = success; otherwise the affected t5 bytes are unspecified).
 *            Reset to 0 by this call before counting.
 */
int bqd_repack_2bit_to_t5(const void *w2, int64_t N, int64_t K, int group_size,
                          uint8_t *w_t5, int *d_status, bqd_stream_t stream);

/*
 * Validate a t5 matrix (§二.3 load path accepting uint8 t5 weights).
 *   d_status device int32: receives the number of invalid bytes (>= 243, or a
 *            group's last byte with non-zero padding trits); reset to 0 by
 *            this call before counting.  The QMV/QMM kernels do not check
 *            bytes; their output for an invalid byte is unspecified.
 */
int bqd_validate_t5(const uint8_t *w_t5, int64_t N, int64_t K, int group_size,
                    int *d_status, bqd_stream_t stream);

/*
 * Load-time detection of identity I-B (§二.2): counts the (n, g) for which
 * biases[n,g] != fp16_rne(float(-ratio) * float(scales[n,g])), comparing
 * bit patterns.  A count of 0 means the bias tensor can be dropped and the
 * sym path used.
 *   scales, biases device fp16 [N, G];  d_mismatches device int32 (reset to 0
 *   by this call before counting).
 */
int bqd_detect_sym(const void *scales, const void *biases, int64_t N, int64_t G,
                   float ratio, int *d_mismatches, bqd_stream_t stream);

/*
 * Speculative-decoding verification in one kernel (§三: spec_decode_verify
 * fuses "compare the draft tokens -> count the accepted length -> produce the
 * correction token").  The page gives no formula; greedy reading:
 *   t[b, i]       = argmax over v of logits[b, i, v], i = 0 .. D (ties: the
 *                   smallest v; NaN entries are never chosen; a row of NaNs
 *                   gives -1)
 *   accepted[b]   = the largest a in [0, D] with draft[b, i] == t[b, i] for
 *                   every i < a (a -1 from a row of NaNs matches nothing)
 *   next_token[b] = t[b, accepted[b]]: the target's token where the draft was
 *                   first rejected, or the bonus token after D accepted drafts
 * Arguments (device pointers):
 *   logits      [B, D+1, V] of `dtype` (BQD_DTYPE_F16 or BQD_DTYPE_F32),
 *               aligned to its element size; row (b, i) scores the token
 *               that follows the prefix and draft[b, 0 .. i-1]
 *   draft       int32 [B, D] (may be NULL when D == 0); ids outside [0, V)
 *               never match
 *   accepted, next_token  int32 [B]
 *   argmax_out  int32 [B, D+1], or NULL: t[b, i] of every row
 * Sizes: 0 <= B <= 2^26, 0 <= D <= 4095, 1 <= V <= 2^31 - 1024.  B == 0
 * launches nothing.  Every logit is read once (the call is bound by HBM
 * bandwidth); one thread-block cluster of min(D+1, 16) CTAs per sequence.
 */
int bqd_spec_decode_verify(const void *logits, int dtype, const int32_t *draft, int64_t B, int64_t D,
                           int64_t V, int32_t *accepted, int32_t *next_token, int32_t *argmax_out,
                           bqd_stream_t stream);

/*
 * A tree of drafts for each of `rows` sequences.  Row r's nodes are tokens
 * starts[r] .. starts[r+1]-1 of a ragged batch; parents[i] is the row's own index
 * of node i's parent, which comes before it: any value outside [0, i) makes node
 * i a root.  Nodes of no row are left as they are.
 *   parents    device int32 [tokens];  starts  device int32 [rows + 1]
 *   words      64-bit words of a node's mask, 1 .. BQD_TREE_MAX_WORDS
 *   mask       device [tokens, words] or NULL: bit j of node i's mask (bit j % 64 of
 *              word j / 64) is set where node j of the row is an ancestor of node i
 *              or i itself; nodes past 64 words have no bit
 *   depth      device int32 [tokens] or NULL: ancestors of the node
 *   base       device int32 [rows], or NULL without positions
 *   positions  device int32 [tokens] or NULL: base[r] + depth
 */
#define BQD_TREE_MAX_WORDS 16
int bqd_tree_mask(const int32_t *parents, const int32_t *starts, int64_t rows, int64_t tokens, int words,
                  const int32_t *base, uint64_t *mask, int32_t *depth, int32_t *positions, bqd_stream_t stream);

/*
 * Greedy verification of such trees.  With t[i] = argmax over v of logits[i, v]
 * (ties: the smallest v; NaN entries are never chosen; a row of NaNs gives -1), the
 * walk starts at the row's node 0, which is taken as it is, and goes on from a node
 * i to its lowest child whose drafted token is t[i], as long as there is one.
 *   logits      device [tokens, V] of `dtype` (F16, BF16 or F32), rows row_stride
 *               elements apart, aligned to its element size; row i scores the token
 *               that follows node i
 *   drafted     device int32 [tokens]: the nodes' tokens; ids outside [0, V) never
 *               match
 *   max_path    nodes of a path at most, >= 1: the walk ends there
 *   accepted    device int32 [rows]: nodes of the path without node 0 (0 for a row
 *               without nodes)
 *   next_token  device int32 [rows]: t of the path's last node (-1 for a row without
 *               nodes)
 *   path        device int32 [rows, max_path]: the path's nodes, then -1
 *   argmax_out  device int32 [tokens]: t, of every node (also the call's scratch)
 * tokens <= 2^28, 1 <= V <= 2^31 - 1024.  rows == 0 launches nothing.
 */
int bqd_spec_tree_verify(const void *logits, int dtype, int64_t row_stride, int64_t V, const int32_t *drafted,
                         const int32_t *parents, const int32_t *starts, int64_t rows, int64_t tokens, int max_path,
                         int32_t *accepted, int32_t *next_token, int32_t *path, int32_t *argmax_out,
                         bqd_stream_t stream);

/*
 * Log probabilities under softmax(logits[r, :]), for each row r:
 *   logprob[r]   of tokens[r]; -infinity for an id outside [0, V)
 *   entropy[r]   -sum p log p (natural logarithm)
 *   rank[r]      entries before tokens[r]: larger, or equal with a lower index; -1 for
 *                an id outside [0, V)
 *   top_ids, top_logprobs [r, k], k < top: the largest entries in this order
 * NaN counts as -infinity, which has probability 0: it is never listed (the list
 * ends with ids of -1 at -infinity), and a row of nothing else gives -infinity and an
 * entropy of 0.  A row with +infinity has no distribution: its log probabilities
 * and entropy are NaN, its ids and rank hold.  Sums are fp32.
 *   logits  device [rows, V] of `dtype` (F16, BF16 or F32), rows row_stride elements
 *           apart, aligned to its element size
 *   tokens  device int32 [rows]; NULL without logprob and rank
 *   top     0 .. BQD_MAX_TOP
 *   logprob, entropy, rank [rows], top_ids, top_logprobs [rows, top]: device fp32 and
 *           int32, each may be NULL
 */
#define BQD_MAX_TOP 32
int bqd_token_logprobs(const void *logits, int dtype, int64_t row_stride, int64_t rows, int64_t V, const int32_t *tokens,
                       int top, float *logprob, float *entropy, int32_t *rank, int32_t *top_ids, float *top_logprobs,
                       bqd_stream_t stream);

/*
 * Norm of each query and key head and the rotation by position, in one pass:
 *   y = x w / sqrt(mean(x^2) + eps) over the head's head_dim values (norm != 0),
 * then the pairs j < rotary_dim / 2 of y, (j, j + rotary_dim / 2) or (2 j, 2 j + 1)
 * (interleaved != 0), become amplitude (a cos t - b sin t, a sin t + b cos t) with t =
 * positions[token] * inv_freq[j].  Values past rotary_dim are not rotated.  All of
 * it in fp32 (squares sum to less than 2^128), rounded once.
 *   q_weight, k_weight  device [head_dim] of weight_dtype (the tensors' type, or F32),
 *                       or NULL: ones
 *   freqs       device [rotary_dim / 2]: inv_freq[j] / (2 pi) * 2^64, rounded, modulo
 *               2^64, so that a product with a position is the angle modulo a turn
 *   head_dim    64, 128 or 256;  rotary_dim  a multiple of 16 up to head_dim; 0: none
 */
typedef struct bqd_qk_rope {
    const void *q_weight, *k_weight;
    const uint64_t *freqs;
    int32_t head_dim, rotary_dim, weight_dtype, interleaved, norm, reserved; /* reserved: 0 */
    float eps, amplitude; /* eps > 0 (with norm), amplitude finite */
} bqd_qk_rope;

/*
 * q, k, q_out, k_out: device [tokens, heads, head_dim] of `dtype` (F16 or BF16),
 * each with strides of token and head in elements; head_dim is contiguous, and no two
 * heads of an output share memory.  16-byte aligned bases with strides of multiples
 * of 8 take 16-byte accesses, others element accesses.  An output may be its input
 * (the same base and strides); any other overlap is not allowed.  k_heads == 0 (or
 * q_heads == 0): no k (no q).
 *   positions   device int32 [tokens], of any value; NULL with rotary_dim == 0
 */
int bqd_qk_norm_rope(const bqd_qk_rope *plan, const void *q, int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                     const void *k, int64_t k_token_stride, int64_t k_head_stride, int k_heads, int dtype,
                     const int32_t *positions, int64_t tokens, void *q_out, int64_t q_out_token_stride,
                     int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                     bqd_stream_t stream);

/*
 * Paged 8-bit KV cache.  The page this library follows stops at the linear
 * layers and the verification step; the cache below is what a decode step
 * reads and writes between the k/v projections and the o projection.
 *
 * A stored value is code * scale, with an 8-bit code (BQD_KV_INT8: -127..127;
 * BQD_KV_E4M3: finite e4m3) and one fp32 scale for each block of BQD_KV_BLOCK
 * tokens and head (K and V apart).  Rows (sequences) list their pages in
 * `table`: token p of row r is token p % page_tokens of page
 * table[r, p / page_tokens].  All layers share the table.  The struct holds
 * device pointers and sizes; the caller owns everything it points to:
 *   k_codes, v_codes    [layers, pages, kv_heads, page_tokens, head_dim], 1
 *                       byte a code, 16-byte aligned
 *   k_scales, v_scales  fp32 [layers, pages, kv_heads, page_tokens / 16]
 *   table               int32 [rows, row_pages]; entries past a row's last
 *                       page are not read (the library writes -1 there)
 *   lens                int32 [rows]: tokens of each row (0: an empty row)
 *   refs                int32 [pages]: table entries (and pins of the caller)
 *                       that name the page; 0 = free
 * head_dim is 64, 128 or 256; page_tokens 16, 32, 64, 128 or 256; rows <=
 * 65535; row_pages * page_tokens < 2^30; pages < 2^30.  Page ids and lengths
 * are device data and are not checked on the host: an id outside [0, pages)
 * is read as page 0 (written: skipped) and a length is cut to the table's
 * capacity, so that no access leaves the pools.
 */
typedef struct bqd_kv_cache {
    void *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int32_t *table;
    int32_t *lens;
    int32_t *refs;
    int64_t pages;
    int32_t layers, kv_heads, head_dim, page_tokens;
    int32_t rows, row_pages;
    int32_t format; /* BQD_KV_INT8 or BQD_KV_E4M3 */
    int32_t reserved; /* 0 */
} bqd_kv_cache;

/*
 * Quantise new keys and values into the cache of one layer.  Row r's new
 * tokens are starts[r] .. starts[r+1]-1 of k and v (starts == NULL: token r,
 * one for each row) and go to positions base[r], base[r]+1, ... (base[r] < 0:
 * the row is skipped); bqd_kv_reserve gives base and the pages.
 * A block that gets new values takes the scale
 *     s' = max(s, fp32(max(amax, 2^-80) * fp32(1 / top))),  top = 127 or 448,
 * amax over the finite new values of the block and head, s the block's scale
 * if it holds tokens before base[r] and 0 otherwise.  With r = fp32(1 / s'),
 * new codes are rnd(fp32(x * r)) and, where s' > s, the earlier tokens' codes
 * become rnd(fp32(fp32(code * s) * r)): round to nearest even, infinities and
 * larger values clamped to +-top, NaN stored as 0.  Appending the same tokens
 * twice gives the same bytes as appending them once.
 *   k, v    device [tokens, kv_heads, head_dim] of `dtype` (F16 or BF16), each
 *           with its own strides of token and head, in elements; head_dim is
 *           contiguous.  16-byte aligned bases with strides of multiples of 8
 *           take 16-byte loads, others element loads
 *   base    device int32 [rows];  starts device int32 [rows + 1] or NULL
 *   tokens  rows of k and v (== rows when starts is NULL)
 *   max_new an upper bound of starts[r+1] - starts[r] (later tokens of a row
 *           are not stored), cut to `tokens`
 * A page that two rows list must not be appended to through either
 * (bqd_kv_reserve replaces it).  Returns BQD_OK, BQD_ERR_INVALID_ARG,
 * BQD_ERR_ALIGNMENT or BQD_ERR_CUDA.
 */
int bqd_kv_append(const bqd_kv_cache *cache, int layer, const void *k, int64_t k_token_stride,
                  int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, int dtype,
                  const int32_t *base, const int32_t *starts, int64_t tokens, int64_t max_new,
                  bqd_stream_t stream);

/*
 * Attention over the cache of one layer.  Row r's queries are starts[r] ..
 * starts[r+1]-1 of q (starts == NULL: query r, one for each row), n of them,
 * at positions lens[r] - n + i: the cache already holds their own tokens.
 * Query i sees the keys j <= p = lens[r] - n + i (and j > p - window where
 * window > 0); head h reads KV head h / (q_heads / kv_heads):
 *     out = sum_j softmax_j(scale * q . K_j) V_j,
 *     lse = log sum_j exp(scale * q . K_j)   (natural logarithm)
 * A query that sees no key (an empty row, or p < 0) gives 0 and -infinity.
 * Scores, softmax sums and outputs accumulate in fp32; the weights that meet
 * V are rounded to fp16 after a power-of-two scaling that keeps the largest
 * near 1.  bf16 queries are taken in fp16, scaled by a power of two: elements
 * below 2^-16 of a query's largest lose bits, 2^-25 of that largest at most.
 * A weight times its block's V scale that is below 2^-126 of the row's largest
 * such product counts as 0, in out and lse: blocks of zeros (their V scale is
 * near 2^-87) stay in the sum beside values of V up to 4e6 where their weight is
 * above 2^-24 of the largest.
 *   q       device [tokens, q_heads, head_dim] of `dtype` (F16 or BF16), strides
 *           of token and head in elements, head_dim contiguous
 *   out     device [tokens, q_heads, head_dim] of `dtype`, dense, 16-byte
 *           aligned; rows of q outside every row's range are left as they are
 *   lse     device fp32 [tokens, q_heads] or NULL
 *   max_new an upper bound of starts[r+1] - starts[r].  A row's later queries,
 *           and those past `tokens`, are not computed; the others keep the
 *           positions that the row's true count n gives them.  It also decides
 *           between the kernels for few and for many queries and plans the
 *           scratch, so a loose bound costs time
 *   max_len a bound of lens that the launch is planned for (0: the table's
 *           capacity); longer rows stay correct
 *   scale   finite;  window >= 0 (0: none)
 *   work    device scratch, 16-byte aligned, of work_bytes bytes, or NULL with
 *           0.  bqd_kv_attend_workspace (host-only) gives the bytes that a
 *           call with the same sizes takes to share its keys evenly between
 *           CTAs, and with many queries to convert each row's codes once
 *           instead of once for each tile of queries; with less, work is not
 *           used.  The answer is correct either way, and nothing is kept in it.
 * Returns BQD_OK, BQD_ERR_INVALID_ARG, BQD_ERR_ALIGNMENT or BQD_ERR_CUDA;
 * bqd_kv_attend_workspace returns 0 where no scratch is of use or the
 * arguments are invalid.
 */
int64_t bqd_kv_attend_workspace(const bqd_kv_cache *cache, int q_heads, int64_t tokens, int64_t max_new,
                                int64_t max_len, int64_t window);
int bqd_kv_attend(const bqd_kv_cache *cache, int layer, const void *q, int64_t q_token_stride,
                  int64_t q_head_stride, int dtype, int q_heads, const int32_t *starts, int64_t tokens,
                  int64_t max_new, int64_t max_len, float scale, int64_t window, void *out, float *lse,
                  void *work, int64_t work_bytes, bqd_stream_t stream);

/*
 * The same for a tree of drafted tokens, or any other mask over a row's last tokens.
 * With n = starts[r+1] - starts[r] (1 without starts), every query of row r sees the
 * tokens before the row's last n, j < lens[r] - n, and of those the ones whose bit is
 * set in its mask: token lens[r] - n + j where bit j % 64 of word j / 64 is set (itself
 * only where its own bit is; bits at or past n are not read, and tokens past 64 words
 * are seen by none; with lens[r] < n the first n - lens[r] tokens are absent).  A query
 * without any key gives 0 and -infinity.
 *   mask    device [tokens, words], words 1 .. BQD_TREE_MAX_WORDS (bqd_tree_mask)
 *   depth   device int32 [tokens]: with a window, query i is at position p = lens[r] - n
 *           + depth[i] (cut to [0, n)) and sees of the tokens before the last n only
 *           j > p - window; the mask alone decides on the last n.  NULL without one
 * bqd_kv_attend_masked_workspace gives the bytes of scratch that such a call is better
 * with, as bqd_kv_attend_workspace does.
 */
int64_t bqd_kv_attend_masked_workspace(const bqd_kv_cache *cache, int q_heads, int64_t tokens, int64_t max_new,
                                       int64_t max_len, int64_t window);
int bqd_kv_attend_masked(const bqd_kv_cache *cache, int layer, const void *q, int64_t q_token_stride,
                         int64_t q_head_stride, int dtype, int q_heads, const int32_t *starts, int64_t tokens,
                         int64_t max_new, int64_t max_len, float scale, int64_t window, const uint64_t *mask, int words,
                         const int32_t *depth, void *out, float *lse, void *work, int64_t work_bytes,
                         bqd_stream_t stream);

/*
 * Room for counts[r] more tokens in each row (counts == NULL: one for each
 * row that is not empty).  lens grows, table gets the new pages (free pages,
 * lowest index first, in the order of the rows and of their tokens) and refs
 * follows.  A partly filled last page that other table entries name too is
 * first replaced by a copy (all layers, K, V and scales); where all its
 * references are rows of this call that end in it, the first of them keeps it.
 *   base    device int32 [rows]: length before the call, or -1 where the call
 *           failed
 *   copies  device int32 [rows, 2]: (source, copy) of a row's replaced page,
 *           or (-1, -1)
 *   status  device int32 [2]: pages that were missing, and rows that the table
 *           has no room for.  (0, 0) is success; otherwise nothing changes.
 * counts device int32 [rows], >= 0.  rows <= 4096.
 */
int bqd_kv_reserve(const bqd_kv_cache *cache, const int32_t *counts, int32_t *base, int32_t *copies,
                   int32_t *status, bqd_stream_t stream);

/*
 * New rows from old ones: row i of `to` lists the pages of the first
 * min(keep[i], lens[parents[i]]) tokens of row parents[i] of `from` (keep ==
 * NULL: all; a parent outside [0, rows): an empty row), and to->refs = from->
 * refs minus what from's rows name plus what to's rows name.  This forks
 * (beams), reorders, cuts back (rejected draft tokens) and frees rows.
 * `from` and `to` share pools and sizes but for rows; table, lens and refs of
 * `to` are other memory than those of `from`, and every page is shared: no
 * K or V moves.  parents, keep: device int32 [to->rows].
 */
int bqd_kv_fork(const bqd_kv_cache *from, const bqd_kv_cache *to, const int32_t *parents, const int32_t *keep,
                bqd_stream_t stream);

/*
 * Acceptance of a path through each row's last tokens.  Row r's last n = starts[r+1]
 * - starts[r] tokens (starts == NULL: its last one) are nodes; it keeps those that its
 * path names, in every layer: the token at position lens[r] - n + path[r, k] moves to
 * lens[r] - n + k.  `to` gets the table, lens and refs that follow, as from
 * bqd_kv_fork: rows end behind what they keep, and pages that no row lists any more
 * are free.  Rows without nodes stay as they are.
 * A row with fewer tokens than starts gives it nodes has n = lens[r], and nodes 0 .. n -
 * 1 are its tokens from the first on.  (bqd_kv_attend_masked counts such a row's nodes
 * from its end, like the positions of its queries: its tokens are there the last lens[r]
 * nodes.)
 * A 16-token block that gets tokens takes s', the largest scale of the tokens that it
 * then holds; codes of another scale s become rnd(fp32(fp32(code * s) * fp32(1 / s'))),
 * the others keep their bits.
 *   path    device int32 [rows, width]: nodes in rising order, as bqd_spec_tree_verify
 *           gives them; a path ends before the first entry that does not rise or is
 *           outside [0, n)
 * The blocks are changed in place: as for bqd_kv_append, no other row (of `from`, or
 * of a cache that shares the pools) may list a page that gets tokens.  `from` and `to`
 * as for bqd_kv_fork, with the same number of rows.
 */
int bqd_kv_accept(const bqd_kv_cache *from, const bqd_kv_cache *to, const int32_t *path, int width,
                  const int32_t *starts, bqd_stream_t stream);

/*
 * Compaction: with L live pages (refs > 0), the k-th live page at an index >=
 * L moves to the k-th free index below L, in every layer; `to` gets the table,
 * lens and refs that follow (other memory than those of `from`; pools and
 * sizes are the same).  The bytes of a page that moved away stay as they are.
 * Pages that only a pin of the caller holds move too.
 *   work    device int32 [2 * pages]: scratch in the first half; work[pages + q]
 *           is the new index of page q (q where it stayed), for what the caller
 *           knows by its index
 *   moved   device int32 [1]: pages moved
 */
int bqd_kv_compact(const bqd_kv_cache *from, const bqd_kv_cache *to, int32_t *work, int32_t *moved,
                   bqd_stream_t stream);

/*
 * Copy page src[i] to page dst[i], i < n, in every layer (K, V and scales).
 * src and dst: device int32 [n]; no page may be in both, nor twice in dst.
 * Ids outside [0, pages) are skipped.
 */
int bqd_kv_copy_pages(const bqd_kv_cache *cache, const int32_t *src, const int32_t *dst, int64_t n,
                      bqd_stream_t stream);

/*
 * Device-side failure report.  Kernels that wait on asynchronous copies
 * (mbarrier waits) bound every wait; a wait that runs out makes that CTA skip
 * its work and bumps a library-owned device counter instead of hanging.  This
 * call synchronises `stream`, reads and clears that counter, and returns
 * BQD_ERR_TIMEOUT if any wait expired since the previous call (the outputs of
 * the affected calls are then unspecified), BQD_ERR_CUDA if the
 * synchronisation failed, else BQD_OK.  Host + device, blocking.
 */
int bqd_device_status(bqd_stream_t stream);

/*
 * Process-wide options: a control for tests and measurements, with no
 * counterpart on the page.  Host-only; a change applies to calls made after
 * it (calls already enqueued keep what they were launched with).
 *   BQD_OPT_KERNEL         BQD_KERNEL_AUTO (the dispatcher picks) or one
 *                          kernel family forced for every QMV call; a forced
 *                          family that cannot serve a request makes that call
 *                          return BQD_ERR_UNSUPPORTED instead of falling back
 *   BQD_OPT_T5_STAGES      0, or 1 / 2: the ring depth of the register-
 *                          streaming t5 kernel (0 = the planner's choice)
 *   BQD_OPT_WAIT_LIMIT_NS  time, in ns of %globaltimer, after which a pipeline
 *                          wait of the ring kernels gives up (see
 *                          bqd_device_status); 0 restores the default of 1 s.
 *                          The waits that let a CTA's own copies land before
 *                          it exits always keep the default limit
 *   BQD_OPT_DEBUG_PLAN     non-zero: print each launch plan to stderr
 * The environment gives the first values, read once on first use:
 * BQD_FORCE_KERNEL=generic|mma|tma|qmm, BQD_T5_STAGES=1|2, BQD_DEBUG_PLAN.
 * bqd_set_option returns BQD_OK or BQD_ERR_INVALID_ARG (unknown option or
 * value out of range); bqd_get_option returns the value, or -1 for an
 * unknown option.
 */
enum { BQD_OPT_KERNEL = 1, BQD_OPT_T5_STAGES = 2, BQD_OPT_WAIT_LIMIT_NS = 3, BQD_OPT_DEBUG_PLAN = 4 };
enum {
    BQD_KERNEL_AUTO = 0,    /* the dispatcher's choice                       */
    BQD_KERNEL_GENERIC = 1, /* CUDA-core kernel, any shape                   */
    BQD_KERNEL_MMA = 2,     /* register-streaming tensor-core decode kernels */
    BQD_KERNEL_TMA = 3,     /* TMA-ring decode kernels                       */
    BQD_KERNEL_QMM = 4      /* tcgen05 prefill product                       */
};
int bqd_set_option(int option, int64_t value);
int64_t bqd_get_option(int option);

#ifdef __cplusplus
}
#endif
#endif /* BQD_H */
