/*
 * kvq8attn.h -- C ABI of the Q8_0 GQA verify / prompt attention library (GB300, sm_103a).
 *
 * The operation: multi-row causal attention of fp32 (verify) or fp16 (prompt) query rows
 * over a grouped-query KV cache stored in the Q8_0 format -- int8 codes plus one fp16
 * scale per 32-value block.  Sources (titles and sections of the pages):
 *   - "perf(gfx1100): share Q8 KV scans across verifier rows", Summary: one wave owns
 *     four or eight Q8 attention query rows and shares each K/V scan across them; the
 *     partials layout and reducer stay as they are; the route is limited to Q8 KV,
 *     head_dim 128 or 256 and sequential (non-tree) windows of 4-32 rows.
 *   - "gfx12 WMMA kernel for the int8-KV QSA prompt attention", How: int8-KV prompt
 *     attention with online softmax and the V scale folded into p; the heads that
 *     share one KV head fill the rows of the tensor-core tile.
 *   - "Engine perf(hip): MTP draft, shared expert, verify/sampler head", Summary
 *     item 4: the warp-per-block Q8_0 quantiser, bitwise equal to its CPU reference.
 *
 * Layout of the cache (all device memory, owned by the caller):
 *   codes  int8   [n_kv_heads][capacity][head_dim]        one row of head_dim codes per token
 *   scales uint16 [n_kv_heads][capacity][head_dim / 32]   fp16 bit patterns, one per 32-code block
 * The dequantised value of element j of token n is codes[h][n][j] * fp16(scales[h][n][j/32]).
 *
 * Conventions shared by every entry point:
 *   - Query head h reads KV head h / (n_q_heads / n_kv_heads).
 *   - Query row i of a call sees keys n with n <= q_pos0 + i and n < kv_len.  A verify
 *     window of T rows after ctx cached tokens uses q_pos0 = ctx, kv_len = ctx + T; a
 *     prompt chunk of n_q rows ending the context uses q_pos0 = kv_len - n_q.
 *   - All pointers are device pointers (cudaMalloc / torch), 16-byte aligned, caller-owned.
 *     The library never allocates, frees or synchronises and keeps no state between
 *     calls; work is enqueued on `stream` (NULL = the legacy default stream).
 *   - Every call validates its arguments on the host first and, on any error, returns a
 *     nonzero status and launches nothing ("fail closed": there is no fallback route).
 *     A CUDA launch error is returned as KVQ8_ERR_CUDA.
 */
#ifndef KVQ8ATTN_H
#define KVQ8ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st* kvq8_stream_t;

enum kvq8_status {
    KVQ8_OK = 0,
    KVQ8_ERR_INVALID_ARG = 1,   /* null pointer, negative or inconsistent size          */
    KVQ8_ERR_UNSUPPORTED = 2,   /* head_dim, group or row count outside what is built   */
    KVQ8_ERR_MISALIGNED = 3,    /* a pointer is not 16-byte aligned                     */
    KVQ8_ERR_WORKSPACE = 4,     /* workspace missing or smaller than required           */
    KVQ8_ERR_CUDA = 5           /* a CUDA call or kernel launch failed                  */
};

/* The caller's cache planes.  head_dim is 128 or 256; capacity >= kv_len of any call. */
typedef struct {
    const int8_t* k_codes;
    const uint16_t* k_scales;
    const int8_t* v_codes;
    const uint16_t* v_scales;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t capacity;
} kvq8_cache;

/* A K8V4 KV pool: K as Q8_0 planes (as kvq8_cache), V as 4-bit blocks: v_codes holds
 * [n_kv_heads][capacity][head_dim / 2] bytes, element 2m in the low nibble of byte m stored
 * as code + 8 (code in [-7, 7]), v_scales one fp16 scale per 32 values as for Q8_0.
 * The pages run such a pool without stating its V format; the reading is the Q8_0 rule with
 * 7 in place of 127 ("gfx12 WMMA kernel for the int8-KV QSA prompt attention", Gating). */
typedef struct {
    const int8_t* k_codes;
    const uint16_t* k_scales;
    const uint8_t* v_codes;
    const uint16_t* v_scales;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t capacity;
} kvk8v4_cache;

/* An fp16 KV pool: K and V as IEEE binary16 bits, [n_kv_heads][capacity][head_dim] each,
 * device memory owned by the caller.  The pool format the pages keep on their older kernel
 * ("gfx12 WMMA kernel for the int8-KV QSA prompt attention", Gating and Limits). */
typedef struct {
    const uint16_t* k;
    const uint16_t* v;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t capacity;
} kvf16_cache;

/* Element types of the calls that take more than one. */
enum kvq8_dtype { KVQ8_F32 = 0, KVQ8_F16 = 1, KVQ8_BF16 = 2 };

/* A paged Q8_0 cache: codes [n_pages][n_kv_heads][page_size][head_dim], scales
 * [n_pages][n_kv_heads][page_size][head_dim / 32] (fp16 bits), so a page holds page_size
 * consecutive rows of every KV head.  head_dim 128 or 256; page_size a power of two, 16 .. 1024.
 * Token slot s is row s % page_size of page s / page_size.  A request's page table lists its pages
 * in order of position.  Slots and element offsets are 64-bit; n_pages * n_kv_heads * page_size, the
 * rows of a plane, is at most 2^31 - 1 (UNSUPPORTED otherwise). */
typedef struct {
    const int8_t* k_codes;
    const uint16_t* k_scales;
    const int8_t* v_codes;
    const uint16_t* v_scales;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t page_size;
    int32_t n_pages;
} kvq8_paged_cache;

/*
 * kvq8_quantize -- append n_tok tokens of K (or V) values to one plane pair.
 *   x      : fp32 [n_tok][n_kv_heads][head_dim]
 *   codes  : int8 plane [n_kv_heads][capacity][head_dim]; tokens land at [pos0, pos0 + n_tok)
 *   scales : uint16 plane [n_kv_heads][capacity][head_dim / 32]
 * Per 32-value block: amax = max |x|; d32 = amax / 127 (IEEE fp32 division); the stored
 * scale is fp16(d32) rounded to nearest even; code = clamp(round-half-away-from-zero(x / d32),
 * -127, 127) with an IEEE fp32 division; a block with d32 == 0 stores scale 0 and zero codes.
 * Results are bit-exact with that definition.  Inputs must be finite; for amax > 65504 * 127
 * the stored scale is +inf.  head_dim must be a multiple of 32.
 * Source: "Engine perf(hip): ...", Summary item 4 (warp-per-block Q8_0 quantiser).
 */
int kvq8_quantize(const float* x, int n_tok, int n_kv_heads, int head_dim,
                  int8_t* codes, uint16_t* scales, int capacity, int pos0, kvq8_stream_t stream);

/*
 * kvq8_append -- append n_tok tokens of K and V to both planes of a cache in one launch.
 *   k, v : fp32 [n_tok][kv->n_kv_heads][kv->head_dim], device memory; tokens land at
 *          positions [pos0, pos0 + n_tok) of every KV head.
 * Each plane is quantised exactly as kvq8_quantize would (bit-exact with it); the cache's
 * plane pointers are written through although the struct declares them const.
 * Errors: INVALID_ARG for null pointers, negative n_tok or pos0, or pos0 + n_tok > capacity;
 * UNSUPPORTED when head_dim is not a multiple of 32; MISALIGNED unless every pointer is
 * 16-byte aligned.
 * Source: "Engine perf(hip): ...", Summary item 4 (warp-per-block Q8_0 quantiser).
 */
int kvq8_append(const float* k, const float* v, int n_tok, const kvq8_cache* kv, int pos0,
                kvq8_stream_t stream);

/* Bytes of workspace attn_verify_q8 needs for this shape (n_split 0 = the automatic choice). */
size_t attn_verify_q8_workspace_bytes(int n_rows, int n_q_heads, int head_dim, int kv_len,
                                      int n_kv_heads, int n_split);

/*
 * attn_verify_q8 -- speculative-decode verify attention over a Q8_0 cache.
 *   q        : fp32 [n_rows][n_q_heads][head_dim], 1 <= n_rows <= 32
 *   kv       : the cache (head_dim 128 or 256; n_q_heads / n_kv_heads integral, <= 64)
 *   kv_len   : tokens of the cache to attend over; q_pos0: position of row 0 (see above)
 *   out      : fp32 [n_rows][n_q_heads][head_dim], normalised attention output
 *   workspace: device scratch of at least attn_verify_q8_workspace_bytes(...) bytes,
 *              caller-owned; holds the split-context partials between the two kernels
 *   n_split  : context slices per KV head (0 = automatic; otherwise 1..1024)
 * One thread block per (KV head, context slice) reads each K/V block of its slice from
 * HBM once for all n_rows x group query rows; the per-slice (o, m, l) partials are then
 * merged by log-sum-exp.  fp32 result; q and p enter the tensor cores as fp16 hi + lo
 * pairs, so the result stays within 1e-4 of the fp64 oracle (max |err| / max |out|).
 * Source: "perf(gfx1100): share Q8 KV scans across verifier rows", Summary.
 */
int attn_verify_q8(const float* q, int n_rows, int n_q_heads, const kvq8_cache* kv, int kv_len,
                   int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                   int n_split, kvq8_stream_t stream);

/* Partials attn_verify_q8_partials writes for this shape (its resolved n_split; 0 = invalid). */
int attn_verify_q8_partials_count(int n_rows, int n_q_heads, int head_dim, int kv_len, int n_kv_heads,
                                  int n_split);

/*
 * attn_verify_q8_partials -- the split-context scan of attn_verify_q8 without the merge: the
 * per-slice partials of the window rows over cache positions [0, kv_len).
 *   q_pos0   : position of row 0 in this cache's coordinates; row i sees positions <= q_pos0 + i.
 *              It may be negative (down to -2^30): a rank holding a later context slice in a
 *              cache of its own passes q_pos0 - (its slice's first key), and rows that see
 *              none of its keys get empty partials.
 *   part_o   : fp32 [n][n_rows * n_q_heads][head_dim], n = attn_verify_q8_partials_count(...)
 *   part_ml  : fp32 [n][n_rows * n_q_heads][2]
 *   The layout attn_combine takes: per slice and row, o = sum exp(s_n - m) v_n (unnormalised),
 *   m = max s_n in natural-log units (-inf when the row sees no key of the slice, o = 0 and
 *   l = 0 then) and l = sum exp(s_n - m).
 * Concatenating the partials of several calls (other ranks' slices of one context, in any
 * order) and passing them to attn_combine gives the attention over the union of the
 * slices.  Other arguments and errors as for attn_verify_q8; no workspace is used.
 * Source: "perf(gfx1100): share Q8 KV scans across verifier rows", Summary: the partials
 * layout and the reducer are kept; here they are the exchange of a context-sharded verify.
 */
int attn_verify_q8_partials(const float* q, int n_rows, int n_q_heads, const kvq8_cache* kv, int kv_len,
                            int q_pos0, float softmax_scale, float* part_o, float* part_ml, int n_split,
                            kvq8_stream_t stream);

/* Bytes of workspace attn_verify_append_q8 needs (kv_len = q_pos0 + n_rows; n_split as there). */
size_t attn_verify_append_q8_workspace_bytes(int n_rows, int n_q_heads, int head_dim, int q_pos0,
                                             int n_kv_heads, int n_split);

/*
 * attn_verify_append_q8 -- kvq8_append of the window's K and V, then attn_verify_q8 over
 * kv_len = q_pos0 + n_rows, as one call.
 *   k_new, v_new : fp32 [n_rows][kv->n_kv_heads][kv->head_dim], device, 16-byte aligned:
 *                  the window tokens' keys and values, quantised into positions
 *                  [q_pos0, q_pos0 + n_rows) of the cache (bit-exact with kvq8_append).
 *   n_split      : context slices over the keys below q_pos0 (0 = automatic); the window
 *                  keys get one more slice of their own.
 * Two launches, as attn_verify_q8: the verify grid gets one more slice per KV head holding
 * the window keys alone, and that slice's blocks quantise k_new / v_new themselves (into
 * their tiles and into the cache) while every other block scans the old keys.  The cache
 * bytes equal kvq8_append's; the result equals kvq8_append followed by attn_verify_q8 up to
 * rounding order (the slices differ).
 * Errors: as for kvq8_append and attn_verify_q8; INVALID_ARG also when k_new or v_new is
 * null or q_pos0 + n_rows > capacity.
 * No counterpart on the pages: the verify rows of "perf(gfx1100): share Q8 KV scans across
 * verifier rows" (Summary) attend to the window's own keys, so those keys must be in the
 * cache first; this entry point fuses that write (the quantiser of "Engine perf(hip): ...",
 * Summary item 4) with the scan so the two overlap.
 */
int attn_verify_append_q8(const float* q, const float* k_new, const float* v_new, int n_rows,
                          int n_q_heads, const kvq8_cache* kv, int q_pos0, float softmax_scale,
                          float* out, void* workspace, size_t workspace_bytes, int n_split,
                          kvq8_stream_t stream);

/* Device scratch attn_verify_append_q8_host needs (inputs, output and the verify workspace). */
size_t attn_verify_append_q8_host_scratch_bytes(int n_rows, int n_q_heads, int head_dim, int q_pos0,
                                                int n_kv_heads, int n_split);

/*
 * attn_verify_append_q8_host -- attn_verify_append_q8 from and to HOST buffers: the one entry
 * point that touches host memory.
 *   h_in   : host fp32, q [n_rows][n_q_heads][head_dim] followed by k_new and v_new
 *            [n_rows][n_kv_heads][head_dim] each (pinned memory keeps the copy asynchronous)
 *   h_out  : host fp32 [n_rows][n_q_heads][head_dim]
 *   d_scratch : device, 16-byte aligned, attn_verify_append_q8_host_scratch_bytes(...) bytes
 * Pinned host buffers (mapped into the device address space, as every pinned allocation is
 * on unified-addressing systems): a copy kernel reads h_in once over the host link into the
 * scratch, the two kernels of attn_verify_append_q8 run, and the merge writes h_out in place.
 * Pageable buffers: a host-to-device copy-engine transfer, the two kernels, a device-to-host
 * transfer.  All queued on `stream`; h_out is valid once the stream has reached the end (the
 * call itself does not synchronise).  Errors as for attn_verify_append_q8, WORKSPACE for a
 * short scratch; nothing is queued on error.
 */
int attn_verify_append_q8_host(const float* h_in, int n_rows, int n_q_heads, const kvq8_cache* kv,
                               int q_pos0, float softmax_scale, float* h_out, void* d_scratch,
                               size_t scratch_bytes, int n_split, kvq8_stream_t stream);

/*
 * kvk8v4_append -- append n_tok tokens of K (to Q8_0) and V (to 4-bit blocks) into a K8V4
 * pool at positions [pos0, pos0 + n_tok), one launch.  k, v: fp32 [n_tok][n_kv_heads][head_dim]
 * on the device.  The K bytes equal kvq8_append's.  Errors as for kvq8_append.
 */
int kvk8v4_append(const float* k, const float* v, int n_tok, const kvk8v4_cache* kv, int pos0,
                  kvq8_stream_t stream);

/*
 * attn_verify_k8v4 -- attn_verify_q8 over a K8V4 pool: the same window semantics, shapes,
 * workspace (attn_verify_q8_workspace_bytes), precision bound and errors; the V codes are
 * expanded from their nibbles in registers.
 */
int attn_verify_k8v4(const float* q, int n_rows, int n_q_heads, const kvk8v4_cache* kv, int kv_len,
                     int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                     int n_split, kvq8_stream_t stream);

/*
 * attn_prompt_k8v4 -- attn_prompt_q8 over a K8V4 pool (the same shapes, routes, workspace
 * from attn_prompt_q8_workspace_bytes, precision bound and errors); the dequantisers expand
 * the 4-bit V blocks (value (nibble - 8) * scale, rounded once to fp16) into the V tiles or,
 * on the two-pass route, into the fp16 copy.
 */
int attn_prompt_k8v4(const uint16_t* q, int n_q, int n_q_heads, const kvk8v4_cache* kv, int kv_len,
                     int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                     kvq8_stream_t stream);

/*
 * Bytes of workspace attn_prompt_f16 needs for this shape: the partials only (an fp16 pool has
 * no copy to make).  Never more than attn_prompt_q8_workspace_bytes for the same shape.
 */
size_t attn_prompt_f16_workspace_bytes(int n_q, int n_q_heads, int head_dim, int kv_len, int q_pos0,
                                       int n_kv_heads);

/*
 * attn_prompt_f16 -- attn_prompt_q8 over an fp16 pool (the same shapes, precision bound and
 * errors; workspace from attn_prompt_f16_workspace_bytes).  The K and V tiles are loaded
 * straight into the tensor-core operand layout by tensor copies over (head_dim, kv_len,
 * n_kv_heads), so keys at or past kv_len read as zeros; the caller's pool needs no padding.
 */
int attn_prompt_f16(const uint16_t* q, int n_q, int n_q_heads, const kvf16_cache* kv, int kv_len,
                    int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                    kvq8_stream_t stream);

/*
 * kvf16_append -- round n_tok tokens of K and V (fp32 [n_tok][n_kv_heads][head_dim], device)
 * to fp16 (nearest even) into both planes of an fp16 pool at positions [pos0, pos0 + n_tok).
 * Errors: INVALID_ARG for null pointers, negative sizes or pos0 + n_tok > capacity;
 * UNSUPPORTED when head_dim is not a multiple of 4; MISALIGNED unless every pointer is
 * 16-byte aligned.  The pool's plane pointers are written through.
 */
int kvf16_append(const float* k, const float* v, int n_tok, const kvf16_cache* kv, int pos0,
                 kvq8_stream_t stream);

/* Bytes of workspace attn_verify_f16 needs for this shape (n_split 0 = the automatic choice). */
size_t attn_verify_f16_workspace_bytes(int n_rows, int n_q_heads, int head_dim, int kv_len,
                                       int n_kv_heads, int n_split);

/*
 * attn_verify_f16 -- attn_verify_q8 over an fp16 KV pool: the same window semantics, shapes
 * (head_dim 128 or 256, 1 <= n_rows <= 32), split-context partials, merge, precision bound
 * (q and p as fp16 hi + lo, fp32 accumulation; within 1e-4 of the fp64 oracle) and errors.
 * The K and V values enter the tensor cores as they are stored; there are no block scales.
 * Source: "perf(gfx1100): share Q8 KV scans across verifier rows", Summary, for the
 * multi-row scan; the fp16 pool of "gfx12 WMMA kernel for the int8-KV QSA prompt
 * attention", Gating and Limits.
 */
int attn_verify_f16(const float* q, int n_rows, int n_q_heads, const kvf16_cache* kv, int kv_len,
                    int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                    int n_split, kvq8_stream_t stream);

/*
 * attn_verify_tree_q8 -- attn_verify_q8 for a tree-shaped verify window.
 *   window_mask : device uint32 [n_rows], 4-byte aligned: row i sees every key n < q_pos0
 *                 and the window key q_pos0 + j (j < 32, q_pos0 + j < kv_len) exactly when
 *                 bit j of window_mask[i] is set.  The sequential window of attn_verify_q8
 *                 is window_mask[i] = 2^(i+1) - 1; a tree of drafted tokens sets the bits
 *                 of a row's ancestors and of itself.  A row that sees no key gets zeros.
 * Everything else (shapes, workspace from attn_verify_q8_workspace_bytes, n_split,
 * precision, errors) is as for attn_verify_q8; a null window_mask is INVALID_ARG and a
 * misaligned one MISALIGNED.
 * The pages admit only sequential windows on the multi-row route and send trees to the
 * fallback ("perf(gfx1100): share Q8 KV scans across verifier rows", Summary: route
 * conditions); here a tree costs the same K/V scan as a chain.
 */
int attn_verify_tree_q8(const float* q, int n_rows, int n_q_heads, const kvq8_cache* kv, int kv_len,
                        int q_pos0, const uint32_t* window_mask, float softmax_scale, float* out,
                        void* workspace, size_t workspace_bytes, int n_split, kvq8_stream_t stream);

/*
 * argmax_rows_top_prob -- verify-head acceptance: per row of fp32 logits [n_rows][vocab]
 * (device, 4-byte aligned), argmax[i] (int32) = the first index of the row's maximum and
 * top_prob[i] (fp32) = softmax(row)[argmax[i]] = 1 / sum_j exp(x_j - max).
 * Special values: a row holding NaN gives the index of its first NaN and probability NaN;
 * +inf entries share the probability mass equally (argmax = the first +inf); a row of -inf
 * only gives index 0 and probability 1 / vocab; otherwise -inf entries carry probability 0.
 * argmax is exact; top_prob is within 1e-5 (relative) of its fp64 value.
 * workspace: device scratch of argmax_rows_top_prob_workspace_bytes(n_rows, vocab) bytes,
 * 16-byte aligned.  1 <= n_rows <= 65535, vocab >= 1.  Errors: INVALID_ARG, WORKSPACE,
 * MISALIGNED.  Two kernel launches; asynchronous on `stream`.
 * Source: "Engine perf(hip): MTP draft, shared expert, verify/sampler head", Summary item 1
 * and "Verification & Parity Evidence" (argmax_rows, row_top_prob over T x 248,320 logits).
 */
size_t argmax_rows_top_prob_workspace_bytes(int n_rows, int vocab);
int argmax_rows_top_prob(const float* logits, int n_rows, int vocab, int32_t* argmax, float* top_prob,
                         void* workspace, size_t workspace_bytes, kvq8_stream_t stream);

/*
 * attn_combine -- merge split-context partials (log-sum-exp reducer).
 *   part_o  : fp32 [n_split][rows][head_dim]  unnormalised o_s = sum_n exp(s_n - m_s) v_n
 *   part_ml : fp32 [n_split][rows][2]         (m_s, l_s): m_s = max s_n over the slice in natural-log
 *             units (-inf for an empty slice), l_s = sum_n exp(s_n - m_s)
 *   out     : fp32 [rows][head_dim] = sum_s o_s e^(m_s - m*) / sum_s l_s e^(m_s - m*), m* = max_s m_s;
 *             a row whose every slice is empty is written as zeros
 * head_dim is a multiple of 4, <= 1024; 1 <= n_split <= 4096.
 * Source: "perf(gfx1100): share Q8 KV scans across verifier rows", Summary (partials + reducer).
 */
int attn_combine(const float* part_o, const float* part_ml, int n_split, int rows, int head_dim,
                 float* out, kvq8_stream_t stream);

/*
 * Bytes of workspace attn_prompt_q8 (and attn_prompt_k8v4 / attn_prompt_f16) needs for this
 * shape (on the current device): the partials, plus, for chunks of 24 or more 128-row tiles
 * per KV head, room for the fp16 copy of both planes (2 * n_kv_heads * min(kv_len, q_pos0 +
 * n_q) * head_dim * 2 bytes) that the two-pass route writes.  fp16 pools never use that room
 * (attn_prompt_f16_workspace_bytes gives their smaller size).
 */
size_t attn_prompt_q8_workspace_bytes(int n_q, int n_q_heads, int head_dim, int kv_len, int q_pos0,
                                      int n_kv_heads);

/*
 * attn_prompt_q8 -- prompt-chunk attention: many query rows over a long Q8_0 context.
 *   q        : fp16 bits [n_q][n_q_heads][head_dim], head_dim 128 or 256
 *   kv       : the cache (the same head_dim, any n_kv_heads dividing n_q_heads)
 *   out      : fp32 [n_q][n_q_heads][head_dim]
 *   workspace: device scratch of at least attn_prompt_q8_workspace_bytes(...) bytes,
 *              caller-owned; holds the per-slice partials merged by the last kernel and,
 *              on the two-pass route, the fp16 copy of the planes
 *   softmax_scale must be > 0.
 * Row i sees keys n <= q_pos0 + i, n < kv_len.  K and V are dequantised to fp16 (code *
 * scale, one rounding) and contracted on the tcgen05 tensor cores with fp32 accumulation in
 * tensor memory; p enters the PV product as fp16.  Short chunks (fewer than 24 row tiles per
 * KV head) dequantise each tile on chip, once per row tile that sees it.  Longer chunks take
 * the two-pass route: one pass writes the fp16 planes of keys < min(kv_len, q_pos0 + n_q)
 * into the workspace, and the kernel of attn_prompt_f16 runs over that copy; the operands, and
 * so the results, are the same on both routes.  The work -- key tiles
 * (64 keys at head_dim 256, 128 at 128) of 128-row tiles of (query, head) pairs of every
 * KV head -- is cut into one equal
 * contiguous share per SM (a persistent grid); each share writes partials that the
 * log-sum-exp combine merges into `out`.  Tiles past a row tile's causal bound are
 * skipped.  Within 2e-3 of the fp64 oracle (max |err| / max |out|) for values inside the
 * fp16 range.  Every internal wait is bounded; a timeout sets the flag that
 * kvq8_device_error reports (the output is then undefined).
 * Source: "gfx12 WMMA kernel for the int8-KV QSA prompt attention", How and Measurements.
 */
int attn_prompt_q8(const uint16_t* q, int n_q, int n_q_heads, const kvq8_cache* kv, int kv_len,
                   int q_pos0, float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                   kvq8_stream_t stream);

/*
 * attn_verify_q8_noalloc -- attn_verify_q8 for callers that cannot allocate device memory.
 *
 * No counterpart on the pages: this is a library convenience.  Some callers cannot call
 * cudaMalloc at the point where they run attention: a runtime that hands all device memory
 * out of its own fixed arena and forbids other allocations, code running inside a custom
 * allocator's callback (where allocating again would re-enter the allocator), or a plug-in
 * that is not allowed to touch the process allocator at all.  This entry point takes the same
 * arguments as attn_verify_q8 minus the workspace: the split-context partials live in one
 * static device array of KVQ8_NOALLOC_SCRATCH_BYTES bytes built into the library, which
 * every GPU that loads the library holds until the process exits.
 *   - It never calls cudaMalloc, cudaFree or any allocating library routine.
 *   - The first call on each device looks up the array's device address (with that device
 *     current); make that first call before any stream capture.
 *   - All calls share the one array: calls that overlap on the GPU (different streams, or
 *     several host threads) race on it and must be serialised by the caller.
 *   - With n_split = 0 the automatic plan is used: each KV head and row chunk (up to 24
 *     row x q-head pairs) gets at most SM count / (KV heads x chunks) context slices, so the
 *     partials take at most about SM count x 24 x (head_dim + 2) x 4 bytes (3.8 MB at
 *     head_dim 256 on 152 SMs).  When there are more KV heads x chunks than SMs every chunk
 *     gets one slice, n_rows * n_q_heads * (head_dim + 2) * 4 bytes in all.  A plan, automatic
 *     or from an explicit n_split, whose partials exceed the array returns KVQ8_ERR_WORKSPACE
 *     and launches nothing.
 */
#define KVQ8_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
int attn_verify_q8_noalloc(const float* q, int n_rows, int n_q_heads, const kvq8_cache* kv, int kv_len,
                           int q_pos0, float softmax_scale, float* out, int n_split, kvq8_stream_t stream);

/*
 * ---- Serving a batch over a paged cache --------------------------------------------------------
 * One step for n_seqs requests of different lengths, all lengths on the device:
 *   kvq8_paged_tables (pages and slots of the new tokens), kvq8_paged_append (their K and V into the
 *   pages), attn_verify_paged_q8 (every request's window over its pages), logits_adjust (penalties,
 *   biases and grammars on the window's logits), argmax_rows_top_prob; token_counts keeps what the
 *   penalties read.
 * The new tokens of all requests are the rows of one batch: request b owns rows row_starts[b] ..
 * row_starts[b + 1] - 1 (int32, device, n_seqs + 1 entries, ascending), its window of T rows.  No call
 * synchronises or reads a length on the host, so a step can be captured into a graph and replayed
 * as the lengths change.  n_seqs is at most 4096.
 */

/*
 * kvq8_paged_tables -- block tables and slots from request lengths.
 *   lens, n_new : int32 [n_seqs]: tokens each request holds after the step, and how many of them are
 *                 new (0 <= n_new <= lens); lens = 0 ends a request
 *   held        : int32 [n_seqs]: pages each request holds now
 *   page_table  : int32 [n_seqs][max_pages], updated: entries [held, need) of a request that grows to
 *                 need = ceil(lens / page_size) pages are filled; other entries are left alone
 *   free_ring   : int32 [n_pages], updated: the free pages, ring_state = int32 {head, count}; entry
 *                 (head + i) % n_pages, i < count, is the i-th free page
 *   held_out, ring_out : held and ring_state after the step; may be the inputs themselves
 *   row_starts  : int32 [n_seqs + 1]: exclusive sums of n_new (output)
 *   slots, positions : int64 / int32 [n_rows]: cache slot and position of every new token, in request
 *                 order; -1 in the rows behind the last
 *   status      : int32 [1]: 0; 1 = too few free pages; 2 = malformed (a length below 0, n_new > lens,
 *                 lens > max_pages * page_size, held outside [0, max_pages], more than n_rows new
 *                 tokens, a ring_state outside its range, or more pages free and given back than
 *                 n_pages; pages that stay held are not counted)
 * Pages are taken from the ring's head and given back behind its tail in order of request, then of
 * position; a page given back in a call is not taken in the same call.  All or nothing: with a
 * nonzero status held_out and ring_out repeat the inputs, page_table and free_ring are unchanged,
 * every slot is -1 and every row start 0, so the step's other calls then do nothing.
 * Page ids are passed through as they stand in the ring; the calls that use them check their range.
 * Errors: INVALID_ARG, UNSUPPORTED (n_seqs > 4096, page_size, n_pages or n_rows > 2^30), MISALIGNED
 * (4 bytes; slots 8).  One launch.
 */
int kvq8_paged_tables(const int32_t* lens, const int32_t* n_new, const int32_t* held, int n_seqs, int page_size,
                      int32_t* page_table, int max_pages, int32_t* free_ring, int n_pages,
                      const int32_t* ring_state, int32_t* held_out, int32_t* ring_out, int32_t* row_starts,
                      int64_t* slots, int32_t* positions, int n_rows, int32_t* status, kvq8_stream_t stream);

/*
 * kvq8_paged_append -- quantise n_tok tokens of K and V into the cache at their slots, one launch.
 *   k, v   : [n_tok][n_kv_heads][head_dim] of `dtype` (KVQ8_F32, KVQ8_F16, KVQ8_BF16), device;
 *            k_stride / v_stride elements between tokens (>= n_kv_heads * head_dim; a multiple of
 *            16 bytes), the heads of a token contiguous
 *   slots  : int64 [n_tok], device; a token whose slot lies outside [0, n_pages * page_size) is
 *            skipped.  No two tokens of a call may have the same slot: its contents would be a
 *            mixture of theirs.
 * The bytes are those of kvq8_append for the same values (in fp32), also of values that are not finite: a NaN has code -127 beside
 * numbers, and 32 of them the scale NaN.  The planes are written through.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, page_size), MISALIGNED (16 bytes; slots 8).
 */
int kvq8_paged_append(const void* k, const void* v, int dtype, int n_tok, int64_t k_stride, int64_t v_stride,
                      const kvq8_paged_cache* kv, const int64_t* slots, kvq8_stream_t stream);

/*
 * kvq8_paged_read -- the values code * scale of n_tok slots, rounded once to `dtype`, one launch.
 *   k, v : [token][head][head_dim] of `dtype`; k_strides / v_strides (host, 2 entries): elements
 *          between tokens and between heads, each >= head_dim and a multiple of 16 bytes; no two
 *          rows of a plane may overlap.  Strides {head_dim, capacity * head_dim} write the planes of a
 *          kvf16_cache, over which attn_prompt_f16 then runs: a prompt chunk behind a paged context.
 *   slots : int64 [n_tok], device, repeats allowed; a slot outside the cache gives zeros.
 * Errors: as for kvq8_paged_append; INVALID_ARG for overlapping rows.
 */
int kvq8_paged_read(const kvq8_paged_cache* kv, const int64_t* slots, int n_tok, int dtype, void* k, void* v,
                    const int64_t* k_strides, const int64_t* v_strides, kvq8_stream_t stream);

/* Bytes of workspace attn_verify_paged_q8 needs on the current device (0: unsupported shape). */
size_t attn_verify_paged_q8_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim, int max_rows);

/*
 * attn_verify_paged_q8 -- verify attention of every request's window over the paged cache: chains
 * and trees of drafted tokens, and plain decoding (windows of one row).
 *   q        : fp16 or bf16 (`dtype`) [n_rows][n_q_heads][head_dim], q_stride elements between rows
 *              (a multiple of 16 bytes); out: the same type, [n_rows][n_q_heads][head_dim], contiguous
 *   page_table : int32 [n_seqs][max_pages]; lens: int32 [n_seqs], tokens of each request in the cache,
 *              the window's own included
 *   max_rows : the longest window of the batch, 1 .. 64
 *   window_mask : uint64 [n_rows] or null.  A row sees every key before the window (n < lens - T), and
 *              the window key lens - T + j exactly when bit j < T of its word is set; null: j <= its
 *              place in the window.  A row that sees no key gets zeros.
 *   workspace : attn_verify_paged_q8_workspace_bytes(...) bytes; calls that may overlap need one each
 * Rows of no request (behind row_starts[n_seqs]) and the rows of a malformed request (T > max_rows,
 * T > lens, lens > max_pages * page_size, rows outside [0, n_rows)) are left as they were.  Keys on a
 * page id outside [0, n_pages) are left out, as if masked.  Masked and unused cache rows may hold any
 * codes, but their scales must be finite where they stand before lens.
 * K, V and p enter the tensor cores in fp16 (code * scale rounded once), bf16 q as fp16 times a power
 * of two (one for the rows that a thread block holds); scores, softmax statistics and sums are fp32.
 * That is 4e-4 of an fp16 output (2-norm, half of it the output's own rounding) and nothing beside the
 * rounding of a bf16 one; attn_verify_tree_q8 over a contiguous cache is nearer (1.6e-5).  Values of the
 * cache must stay inside the fp16 range, and scores scale * q . k below 2^24 in size: references are fp32,
 * and a row far above that may come out as NaN.  Rows of one window whose bf16 queries are more
 * than 2^25 apart in size lose the small ones.  A query that is not a number gives a row of NaN; one that
 * is not finite changes no other row.  The same call gives the same bits.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, page_size, n_q_heads / n_kv_heads > 64, max_rows > 64,
 * n_seqs > 4096, n_rows > 2^24, a cache of too many rows), WORKSPACE, MISALIGNED (16 bytes; the code planes 32: a block is one load; int32 arrays 4, window_mask 8).  Two launches.
 */
int attn_verify_paged_q8(const void* q, int dtype, int64_t q_stride, int n_rows, int n_q_heads,
                         const kvq8_paged_cache* kv, const int32_t* page_table, int max_pages, const int32_t* lens,
                         const int32_t* row_starts, int n_seqs, int max_rows, const uint64_t* window_mask,
                         float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                         kvq8_stream_t stream);

/*
 * logits_adjust -- penalties for repeated tokens, biases and grammar masks on a window's logits.
 *   logits  : [n_rows][vocab] of `dtype`, logits_stride elements between rows
 *   out     : fp32 [n_rows][vocab], out_stride elements between rows; may be `logits` itself (fp32,
 *             equal strides); rows of it that share bytes with rows of `logits` in any other way are refused
 *   penalties : fp32 [n_seqs][3] repetition, frequency, presence, or null (none; then counts and
 *             window_tokens must be null)
 *   counts  : uint32 [n_states][vocab] as token_counts keeps them, or null; state_of: int32 [n_seqs],
 *             the counts row of each request (null: b; outside [0, n_states): nothing counted)
 *   window_tokens : int32 [n_rows] or null: the drafted tokens; row r also counts those of its own
 *             path, the tokens of window places j whose bit is set in window_mask[r] (uint64 [n_rows];
 *             null: j <= its place)
 *   bias_starts : int32 [n_seqs + 1] or null: request b adds bias_values[i] to bias_tokens[i] for i in
 *             [bias_starts[b], bias_starts[b + 1]) (n_bias entries in all); of several entries of one
 *             token the last holds
 *   grammar : uint32 [n_grammar][ceil(vocab / 32)] or null, bit v % 32 of word v / 32 = value v is
 *             allowed; grammar_of: int32 [n_rows], the mask of each row (null: r; outside
 *             [0, n_grammar): everything is allowed)
 * With c = times v was generated, seen = c > 0 or v in the prompt, in fp32 and in this order (each
 * operation rounded once, the quotient within one unit of its last place):
 *   seen: x = x > 0 ? x / repetition : x * repetition;
 *   x += bias - (frequency * c + (c > 0 ? presence : 0));  not allowed: x = -inf (whatever x was).
 * Tokens outside [0, vocab) are ignored.  Rows of no request, and of a request with more than 64 rows
 * where window_tokens is given, are left as they were.
 * Errors: INVALID_ARG (an overlap as well), UNSUPPORTED (n_seqs > 4096, vocab > 2^30, n_rows > 262140), MISALIGNED (element
 * size; window_mask 8).  One launch.
 */
int logits_adjust(const void* logits, int dtype, int64_t logits_stride, int n_rows, int vocab,
                  const int32_t* row_starts, int n_seqs, const float* penalties, const uint32_t* counts,
                  int n_states, const int32_t* state_of, const int32_t* window_tokens, const uint64_t* window_mask,
                  const int32_t* bias_starts, const int32_t* bias_tokens, const float* bias_values, int n_bias,
                  const uint32_t* grammar, int n_grammar, const int32_t* grammar_of, float* out, int64_t out_stride,
                  kvq8_stream_t stream);

/*
 * token_counts -- count tokens into counts rows: bit 31 of a value's word = it stands in the prompt,
 * bits 0 .. 30 = times generated.
 *   tokens  : int32 [n_tokens]; list i is [token_starts[i], token_starts[i + 1]) (int32 [n_lists + 1]),
 *             its first prompt_lens[i] tokens (int32 [n_lists]; null: none) the prompt, the rest generated
 *   state_of : int32 [n_lists], the counts row of each list (null: i; outside [0, n_states): skipped);
 *             several lists may have the same row
 *   clear   : nonzero: the lists' rows start from zero, else the tokens are added to what they hold
 * Tokens outside [0, vocab) and lists outside [0, n_tokens] are ignored.  Integer sums: the result does
 * not depend on the order of execution.  Errors: INVALID_ARG, UNSUPPORTED (n_lists > 4096, sizes above
 * 2^30), MISALIGNED (4 bytes).
 */
int token_counts(const int32_t* tokens, const int32_t* token_starts, int n_lists, int n_tokens,
                 const int32_t* prompt_lens, const int32_t* state_of, int clear, uint32_t* counts, int n_states,
                 int vocab, kvq8_stream_t stream);

/*
 * ---- Beams, trees and rotary positions ---------------------------------------------------------
 * What stands around the calls above in a step that rotates its keys, searches with beams or verifies trees:
 *   kvq8_paged_append_rope (in place of kvq8_paged_append, and of the rotation before it); behind the logits beam_select, then
 *   token_counts_fork and kvq8_paged_fork let the beams' counts and pages follow, and kvq8_paged_copy copies, in every layer's
 *   cache, the pages that could not be shared; kvq8_paged_compact moves the accepted path of a tree together.
 * A sequence is what has a row of a page table: a request, or one of its beams.  Like the calls above these neither
 * synchronise nor read a length on the host, and can be captured into graphs; and what they read must not be written while they run.
 */

/* Bytes of workspace beam_select needs (0: unsupported sizes). */
size_t beam_select_workspace_bytes(int n_rows, int vocab, int n_seqs, int n_out);

/*
 * beam_select -- the n_out best continuations of every request, over all of its beams and the vocabulary.
 *   logits  : [n_rows][vocab] of `dtype`, logits_stride elements between rows: a row a beam; request b has the rows
 *             row_starts[b] .. row_starts[b + 1] - 1 (int32 [n_seqs + 1], ascending), 64 at most
 *   scores  : fp32 [n_rows] or null (zeros): the beams' totals so far
 *   weights : fp32 [n_rows] or null (ones): positive factors by which totals are compared, 1 / length^a for instance
 *   ended   : int32 [n_rows] or null: a row with ended[r] >= 0 has come to its end; its logits are not read, and its only
 *             continuation is itself, with the token ended[r] and the total scores[r]
 *   n_out   : 1 .. 64
 *   parents, tokens, totals : int32, int32, fp32 [n_seqs][n_out], best first: row, token and total of each; where a request has
 *             fewer, -1, -1 and -inf
 *   workspace : beam_select_workspace_bytes(...) bytes, 16-byte aligned; calls that may overlap need one each
 * total = scores[r] + (x - log sum exp x) over the row's logits x: the sum in 32 bits, its log off by less than 3e-6 + 2e-13 vocab (3e-7 at
 * most as measured) whatever the logits' size, the rest in 64 bits, totals rounded to fp32 at the end.  Continuations are ordered by
 * weight * total in 64 bits; of different rows' ones that are nearer to each other than the sums are exact either may come first.  Equal
 * ones of different rows are ordered by row, those of a row by logit, then by token (-0 equals 0).
 * A logit of -inf is no continuation.  A row with a NaN or +inf among its logits, a score that is not finite or a weight that is
 * not positive and finite has none.  Requests without rows, with more than 64 or outside [0, n_rows) get -1; rows of no request are
 * not read for any.  The same call gives the same bits.
 * Errors: INVALID_ARG (an output over an input, the workspace or another output as well), UNSUPPORTED (n_rows > 65535, vocab > 2^30,
 * n_seqs > 4096, n_out > 64), WORKSPACE, MISALIGNED (element size; workspace 16).  One launch for up to 2048 values, and for some hundreds of
 * rows of up to some ten thousand; else two.
 */
int beam_select(const void* logits, int dtype, int64_t logits_stride, int n_rows, int vocab, const int32_t* row_starts,
                int n_seqs, const float* scores, const float* weights, const int32_t* ended, int n_out, int32_t* parents,
                int32_t* tokens, float* totals, void* workspace, size_t workspace_bytes, kvq8_stream_t stream);

/* Bytes of workspace token_counts_fork needs (0: unsupported sizes). */
size_t token_counts_fork_workspace_bytes(int n_children);

/*
 * token_counts_fork -- the counts rows of n_children sequences that go on from n_seqs ones.
 *   parents  : int32 [n_children]: the sequence that child i goes on from; < 0: there is no child i
 *   state_of : int32 [n_seqs] or null (row q): the counts row of each sequence; outside [0, n_states): none, and its children
 *              have none
 *   state_of_out : int32 [n_children]: the children's rows (-1: none); may be state_of
 *   status   : int32 [1]: 0; 1 = too few rows; 2 = malformed (a parent >= n_seqs, or two sequences of one row that both have
 *              children)
 * The first child of a sequence, the one of the lowest number, keeps its row; the others get copies of it, in the order of their
 * numbers in the lowest rows that no first child keeps.  So every row of `counts` belongs to one of the call's sequences or to
 * nobody: a row of a sequence that is not in the call would be written over.  With a nonzero status no row changes and every
 * state_of_out is -1 (in place: the rows are then known to the caller alone).  (token_counts then adds the children's tokens.)
 * Errors: INVALID_ARG (an output, counts among them, over an input, the workspace or another output as well, but for state_of_out that is
 * state_of), UNSUPPORTED (n_children or n_seqs > 4096, n_states > 65536, vocab > 2^30), WORKSPACE, MISALIGNED (4 bytes; workspace 16).
 * Two launches.
 */
int token_counts_fork(const int32_t* parents, int n_children, const int32_t* state_of, int n_seqs, uint32_t* counts,
                      int n_states, int vocab, int32_t* state_of_out, int32_t* status, void* workspace,
                      size_t workspace_bytes, kvq8_stream_t stream);

/* Bytes of workspace kvq8_paged_fork needs (0: unsupported sizes). */
size_t kvq8_paged_fork_workspace_bytes(int n_seqs, int n_children, int n_pages);

/*
 * kvq8_paged_fork -- the pages of n_children sequences that go on from n_seqs ones: forks, reorders, cuts short and ends.
 *   parents  : int32 [n_children]: the sequence that child i goes on from; < 0: there is no child i.  A sequence without
 *              children ends.
 *   lens, held : int32 [n_seqs]: the tokens of each sequence that its children take over, and the pages it holds
 *   page_table : int32 [n_seqs][max_pages]; shares: int32 [n_pages], how many sequences hold a page beyond the first (0 where
 *              one holds it, and where nobody does); free_ring, ring_state as in kvq8_paged_tables
 *   page_table_out : int32 [n_children][max_pages]: entries before held_out are filled, others left alone
 *   lens_out, held_out : int32 [n_children], ceil(lens_out / page_size) pages; 0 where there is no child
 *   shares_out, ring_out : after the call; may be shares and ring_state themselves
 *   copy_src, copy_dst, copy_rows : int32 [n_children], for kvq8_paged_copy: pages to copy from and to and how many of their
 *              rows; -1, -1, 0 where a child copies nothing
 *   status   : int32 [1]: 0; 1 = too few free pages; 2 = malformed (a parent >= n_seqs, held outside [0, max_pages], a parent's lens
 *              outside [0, held * page_size], a ring_state outside its range)
 * Children share their parent's full pages.  A last page that is not full goes to the first child (of the lowest number) if no other
 * sequence holds it; every other child takes a free page, in the order of their numbers from the ring's head, and a place in the
 * copy list.  Pages that nobody holds any more go back behind the ring's tail, ascending; one given back in a call is not taken in it,
 * so the copies may be made until the next call of kvq8_paged_tables or kvq8_paged_fork.
 * With a nonzero status nothing changes: held_out and lens_out are 0, the copy list is empty, ring_out and shares_out repeat their inputs.
 * Page ids outside [0, n_pages) are passed on and not counted.  A shares or a ring that does not agree with the tables is not
 * noticed; the results then are no better, but nothing outside the arrays is touched.
 * kvq8_paged_tables takes pages for growing sequences as before (a fresh page's share is 0, and a sequence grows only in pages of its
 * own).  It gives pages back whoever shares them: sequences with shared pages are cut short and ended by this call.
 * Errors: INVALID_ARG (outputs over inputs or one another as well, but for the two that may be updated in place; free_ring counts as an
 * output), UNSUPPORTED (n_seqs or n_children > 4096, page_size, n_pages > 2^30, max_pages > 2^24), WORKSPACE, MISALIGNED (4 bytes;
 * workspace 16).  One launch for small tables, else three.
 */
int kvq8_paged_fork(const int32_t* parents, int n_children, const int32_t* lens, const int32_t* held, int n_seqs,
                    int page_size, const int32_t* page_table, int max_pages, const int32_t* shares, int32_t* free_ring,
                    int n_pages, const int32_t* ring_state, int32_t* page_table_out, int32_t* lens_out, int32_t* held_out,
                    int32_t* shares_out, int32_t* ring_out, int32_t* copy_src, int32_t* copy_dst, int32_t* copy_rows,
                    int32_t* status, void* workspace, size_t workspace_bytes, kvq8_stream_t stream);

/*
 * kvq8_paged_copy -- the first rows[i] rows (null: all) of every head of page src_pages[i] to page dst_pages[i], K and V, codes
 * and scales, for i < n; one launch.  int32 [n], device.  An entry with a page outside [0, n_pages), or the same page twice, does
 * nothing.  No page may be written by one entry and read or written by another.
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED (the cache as for kvq8_paged_append; lists 4 bytes).
 */
int kvq8_paged_copy(const kvq8_paged_cache* kv, const int32_t* src_pages, const int32_t* dst_pages, const int32_t* rows,
                    int n, kvq8_stream_t stream);

/*
 * kvq8_paged_compact -- keep some rows of every request's window and move them together, in their order, to its first places:
 * the accepted path of a tree, whose tokens a step appended behind the context.  One launch.
 *   page_table, lens, row_starts as in attn_verify_paged_q8: request b's window of T <= 64 rows are its last T tokens
 *   kept     : uint64 [n_seqs], bit j = place j of the window is kept (bits from T on are ignored; a row's window_mask word is
 *              its path)
 *   lens_out : int32 [n_seqs] or null: lens - T + rows kept; over lens or another input it is refused
 * Places behind the kept ones hold what they held or a moved row's old copy.  Rows from or to a page outside [0, n_pages) do not move.
 * A malformed request (T outside [0, 64], T > lens, lens > max_pages * page_size) is left as it is.  The pages of a window belong
 * to one request.
 * Errors: INVALID_ARG, UNSUPPORTED (n_seqs > 4096, the cache), MISALIGNED (4 bytes; kept 8).
 */
int kvq8_paged_compact(const kvq8_paged_cache* kv, const int32_t* page_table, int max_pages, const int32_t* lens,
                       const int32_t* row_starts, int n_seqs, const uint64_t* kept, int32_t* lens_out, kvq8_stream_t stream);

/*
 * kvq8_paged_append_rope -- kvq8_paged_append of keys that are rotated on the way, and the queries rotated with them, one launch.
 *   q, k, v  : [n_tok][n_q_heads or n_kv_heads][head_dim] of `dtype`, strides as for kvq8_paged_append (elements between tokens, a
 *              multiple of 16 bytes)
 *   positions : int32 [n_axes][n_tok], n_axes 1 .. 4 (time, height and width of an image's patches, for instance)
 *   turns    : uint64 [rot_dim / 2]: pair i's frequency, in 2^-64 turns a position: frequency / (2 pi) * 2^64 modulo 2^64
 *   axis_of  : int32 [rot_dim / 2] or null (axis 0): the axis whose position turns pair i; outside [0, n_axes) it does not turn
 *   rot_dim  : the first rot_dim dims of a head are rotated, a multiple of 64; the others pass as they are
 *   pairs    : 0: pair i is dims i and i + rot_dim / 2; else 2 i and 2 i + 1.  (a, b) becomes (a cos - b sin, b cos + a sin)
 *   slots    : int64 [n_tok] as for kvq8_paged_append; a token whose slot lies outside the cache is left alone, its row of q_out too
 *   q_out    : as q, out_stride elements between tokens; may be q itself (equal strides).  Rows of it that share bytes with rows of
 *              q in any other way, or of k or v, or with positions, turns, axis_of or slots, are refused
 * Angles are exact modulo a turn to about 2^-28 of it at any position (an int32), their sines and cosines fp32 (3e-7), products and sums fp32; q_out
 * is rounded once, and the rotated keys are quantised from fp32, as kvq8_append would, without a rounding in between.
 * Errors: INVALID_ARG, UNSUPPORTED (the cache, rot_dim, n_axes > 4, n_q_heads > 65536), MISALIGNED (16 bytes; slots and turns 8,
 * positions and axis_of 4).
 */
int kvq8_paged_append_rope(const void* q, const void* k, const void* v, int dtype, int n_tok, int n_q_heads,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* positions, int n_axes,
                           const uint64_t* turns, const int32_t* axis_of, int rot_dim, int pairs, const kvq8_paged_cache* kv,
                           const int64_t* slots, void* q_out, int64_t out_stride, kvq8_stream_t stream);

/*
 * kvq8_selftest_convert -- a self-test hook: runs the code -> fp16 conversions that the verify
 * and prompt kernels use, unchanged, on caller data, so that a test can check them exhaustively.
 *   kind 0: in[i] = 4 int8 codes; out[2i], out[2i+1] = fp16 pairs of codes (0, 1) and (2, 3)
 *           (the K operand of the verify scans, the prompt dequantisers).  out: 2n words.
 *   kind 1: in[2i], in[2i+1] = words w0, w1 of 4 codes each (two key rows); out[4i + m] = the fp16
 *           pair (w0 byte m, w1 byte m) through the byte interleave of the PV operands.  n even;
 *           out: 2n words.
 *   kind 2: in[i] = two 16-bit halves of 4 nibbles each (stored code + 8); out[4i .. 4i+3] = the
 *           pairs of nibbles (0, 4), (1, 5), (2, 6), (3, 7), one from each half (the 4-bit PV
 *           operands).  out: 4n words.
 *   kind 3: in[i] = 4 bytes of nibble pairs; out[4i + m] = the pair (low, high) of byte m as
 *           codes (the 4-bit prompt dequantiser).  out: 4n words.
 * Each fp16 value must equal the code exactly.  in, out: device, 4-byte aligned.  Errors:
 * INVALID_ARG (kind, n, null pointers), MISALIGNED.  One launch on `stream`.
 * Source: "gfx12 WMMA kernel for the int8-KV QSA prompt attention", How: the exact int8 -> fp16
 * conversion, checked over all byte pairs.
 */
int kvq8_selftest_convert(int kind, const uint32_t* in, uint32_t* out, int n, kvq8_stream_t stream);

/*
 * kvq8_selftest_wait_timeout -- a self-test hook for the kernels' failure path: one launch whose
 * thread waits on an mbarrier that nothing arrives on, with the bounded wait every pipeline
 * kernel of the library uses, limited to `polls` polls.  The wait gives up, the kernel sets the
 * library's device error flag (read with kvq8_device_error) and returns; the context stays
 * usable.  polls: 1 .. 1 << 20.  Errors: INVALID_ARG (polls out of range), CUDA (no device
 * flag).  One launch on `stream`.
 */
int kvq8_selftest_wait_timeout(int polls, kvq8_stream_t stream);

/*
 * kvq8_device_error -- read (and with reset != 0, clear) the library's device error flag.
 * Nonzero means a kernel gave up on an internal wait after its bounded poll count and
 * returned early.  Returns the flag, or -1 if it could not be read.  Unlike every other
 * entry point this one synchronises: it copies the flag from the current device.
 */
int kvq8_device_error(int reset);

/* Human-readable name of a status code (static string). */
const char* kvq8_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* KVQ8ATTN_H */
