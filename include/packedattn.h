/*
 * packedattn.h -- C ABI of libpackedattn, forward attention over flat-packed
 * variable-length sequences on NVIDIA GB300 (sm_103a).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor argument is a DEVICE pointer to caller-owned memory.  The
 *   library never allocates, frees or keeps a reference to caller memory;
 *   outputs are written asynchronously on `stream` and are valid once the
 *   stream has reached that point.
 * - Attention tensors are bf16, token-major and contiguous: element
 *   (token t, head h, dim d) sits at offset (t * H + h) * D + d.
 * - Sequence boundaries are int32 "cu_seqlens" arrays of batch + 1 entries:
 *   cu[0] = 0, non-decreasing, sequence b owns rows [cu[b], cu[b+1]).
 * - Every call returns a pa_status.  Arguments are checked on the host before
 *   anything is launched; a failed check launches nothing.  Nothing blocks
 *   the host, synchronizes the device or copies device -> host, except
 *   pa_get_device_status.  Nothing aborts, traps or throws.
 * - Checks that need the contents of device arrays (cu_seqlens monotone and
 *   consistent with the totals, lengths within max_q / max_k) run inside the
 *   kernels: a violation records an error code in a per-device status word
 *   (read with pa_get_device_status) and the offending work is skipped.
 * - Every kernel wait on the GPU is bounded; a wait that runs out records
 *   PA_DEVICE_ERR_TIMEOUT in the status word and the kernel returns.
 * - `stream` is a cudaStream_t (NULL = the legacy default stream).
 */
#ifndef PACKEDATTN_H
#define PACKEDATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *pa_stream_t; /* identical to cudaStream_t */

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,  /* null pointer, negative or zero size, non-finite scale */
  PA_ERR_UNSUPPORTED = 2,  /* valid but not implemented: D not 64/128, too many sequences */
  PA_ERR_MISALIGNED = 3,   /* a pointer or row pitch breaks the 16-byte rule */
  PA_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed (launch, tensor map) */
  PA_ERR_DEVICE = 5        /* pa_get_device_status found a recorded device error */
} pa_status;

/* Device-side error codes recorded in the status word (first error wins). */
#define PA_DEVICE_OK 0
#define PA_DEVICE_ERR_CU_SEQLENS 1   /* cu[0] != 0, decreasing, or cu[batch] != total */
#define PA_DEVICE_ERR_MAX_LEN 2      /* a sequence longer than max_q / max_k / s_max */
#define PA_DEVICE_ERR_TIMEOUT 3      /* a bounded pipeline wait ran out */
#define PA_DEVICE_ERR_LENGTH 4       /* a negative length, or a sum above INT32_MAX, in
                                        pa_cu_seqlens_from_lengths */
#define PA_DEVICE_ERR_CAPACITY 5     /* pa_varlen_work_order: more items than capacity */
#define PA_DEVICE_ERR_SMEM_ALIGN 6   /* dynamic shared memory not 1024-byte aligned (kernel skipped) */
#define PA_DEVICE_ERR_SEGMENT 7      /* pa_cfg_combine: bad sequence index, image offset or
                                        mismatched positive/negative image spans */
#define PA_DEVICE_ERR_PAGE 8         /* a page index outside [0, num_pages) in a page table */

/* Largest batch (number of packed sequences) the attention kernels accept. */
#define PA_MAX_BATCH 1024

/* What a paged K/V cache holds: bf16 rows, or e4m3 rows with an exponent byte each. */
#define PA_CACHE_BF16 0
#define PA_CACHE_E4M3 1

/* Activations of the linear layers with an epilogue: x; max(x, 0); x s(x) with the
 * logistic function s; x (1 + erf(x / sqrt 2)) / 2; and its approximation
 * x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2. */
#define PA_ACT_NONE 0
#define PA_ACT_RELU 1
#define PA_ACT_SILU 2
#define PA_ACT_GELU 3
#define PA_ACT_GELU_TANH 4

/* Query rows per work item of pa_varlen_attn_fwd (two 128-row tensor-core tiles). */
#define PA_VARLEN_TILE_M 256

/*
 * pa_varlen_attn_fwd -- non-causal softmax attention over a flat packed batch.
 *
 * Defined by the flat varlen attention path of "[Perf][Diffusion][Qwen-Image]
 * Replace per-bucket varlen loop with flat varlen attention for mixfusion"
 * (Key changes: AttentionMetadata with q_cu_seqlens / kv_cu_seqlens /
 * max_q_len / max_kv_len, packed [total_tokens, heads, head_dim] Q/K/V, no
 * attention mask, no padded tokens) and "feat: Support dynamic batching for
 * heterogeneous diffusion requests" (AttentionMetadata: tokens of one request
 * never attend to another's).  For sequence b, head h and query row i of b:
 *   out[i,h,:] = sum_j softmax_j(scale * <q[i,h,:], k[j,h,:]>) * v[j,h,:]
 * over the key rows j of the same sequence only.  A sequence with queries but
 * no keys gets all-zero output rows.
 *
 * q     [total_q, H, D] bf16      k, v [total_k, H, D] bf16
 * out   [total_q, H, D] bf16, written only at rows that belong to a sequence
 *       (rows >= cu_seqlens_q[batch] are left untouched)
 * cu_seqlens_q / cu_seqlens_k: device int32 [batch + 1]
 * batch in [1, PA_MAX_BATCH]; total_q/total_k >= cu[batch] (extra rows are
 * padding that belongs to no sequence and is never written); max_q / max_k
 * bound every sequence length; H >= 1; D in {64, 128}; scale finite
 * (1/sqrt(D) is usual).
 * Rows outside a sequence never change its result, whatever their bits
 * (NaN and Inf included): the last 128-row key tile of a sequence is loaded
 * whole, so up to 127 rows after the sequence end (the next sequence's rows
 * or trailing padding, within total_k) are read into shared memory, but
 * their scores are masked and their value rows are cleared before use.
 * q, k, v, out must be 16-byte aligned.
 * Deterministic: every output row is computed by one CTA in a fixed order, so
 * a sequence's result does not depend on which other sequences share the
 * batch (bit-identical to running it alone).
 */
pa_status pa_varlen_attn_fwd(const void *q, const void *k, const void *v, void *out,
                             const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                             int32_t batch, int32_t total_q, int32_t total_k,
                             int32_t max_q, int32_t max_k, int32_t H, int32_t D,
                             float scale, pa_stream_t stream);

/*
 * pa_prompt_attn_fwd -- softmax attention of packed prompts, causal and with
 * grouped heads, over K and V rows that are packed too (a prompt before it is
 * in a cache, or behind a prefix that pa_kv_cache_read returned).
 *
 * Sequence b has L_b queries (from cu_seqlens_q) and K_b keys (cu_seqlens_k).
 * With causal != 0 its queries are the last L_b of K_b positions: query i sees
 * key j iff j <= K_b - L_b + i (K_b = L_b: the tokens up to its own); with
 * causal = 0 it sees every key.  Query head h reads K/V head h / (Hq / Hkv).
 *   out[i,h,:] = sum_j softmax_j(scale * <q[i,h,:], k[j,h',:]>) * v[j,h',:]
 * A query that sees no key gets zeros.  Scores, maxima, sums and the output's
 * accumulation are fp32; softmax weights are rounded to bf16 for the product
 * with V (the tensor cores take both factors of V's type), and the output once to
 * bf16.  Weights of a causal call are held 2^-24 of their size until the end, so an
 * output may be off by some 2^-124 in absolute terms (n 2^-124 at most, of n keys):
 * values of V below 2^-112 in size lose digits there, others do not.
 *
 * q [total_q, Hq, D], k, v [total_k, Hkv, D] bf16, with q_stride, k_stride,
 * v_stride elements from one token to the next (>= heads * D, multiples of 8:
 * the rows may be slices of a fused projection's output); out [total_q, Hq, D]
 * bf16 contiguous, written at the rows that belong to a sequence only, and not
 * overlapping q, k or v.  cu_seqlens_q / cu_seqlens_k device int32 [batch + 1],
 * batch in [1, PA_MAX_BATCH]; total_q, total_k >= cu[batch] and at most 2^30
 * (total_q = 0 or max_q = 0 does nothing; q and out, k and v may be NULL where
 * their total is 0); max_q / max_k bound every length; Hq a multiple of Hkv
 * and at most 65535, Hq / Hkv <= 128; (total_q * Hq / 128 + batch * Hkv at most
 * 2^30); D in {64, 128}; scale and scale * log2(e) finite, and scores of at most
 * 2^29 in size once scaled by it (the rounding of a larger one can leave the
 * exponent's range).
 * Rows outside a sequence never reach its result, whatever their bits.  A key
 * that causal order hides from a query has weight zero there; a NaN or infinity
 * in its V row can still reach that query as 0 * NaN (in its K row it cannot).
 * A sequence with bad boundaries (PA_DEVICE_ERR_CU_SEQLENS) or longer than
 * max_q / max_k (PA_DEVICE_ERR_MAX_LEN) is skipped, its rows left untouched.
 * Deterministic, and independent of the batch around a sequence.
 */
pa_status pa_prompt_attn_fwd(const void *q, const void *k, const void *v, void *out,
                             const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                             int32_t batch, int32_t total_q, int32_t total_k,
                             int32_t max_q, int32_t max_k, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, int32_t Hq, int32_t Hkv,
                             int32_t D, int32_t causal, float scale, pa_stream_t stream);

/*
 * pa_block_window_attn_fwd -- block-local attention of the Token2Wav DiT.
 *
 * Defined by "[Perf][Model] Use block-sparse attention in Qwen2.5-Omni
 * Token2Wav DiT" (Purpose; Change: the same result as dense attention under
 * the block-difference mask).  Frames are grouped in blocks of `block`; query
 * i attends to key j iff j < n and
 *   -look_back <= floor(j / block) - floor(i / block) <= look_ahead
 * (look_back blocks before, look_ahead blocks after).  Whether any masking is
 * needed is decided from these integers on the host; nothing is read back
 * from the device.
 *
 * q, k, v, out [batch, n, H, D] bf16 contiguous (token-major per batch entry).
 * batch >= 1, n >= 1, block >= 1, look_back >= 0, look_ahead >= 0, H >= 1,
 * D in {64, 128}, scale finite; pointers 16-byte aligned.
 */
pa_status pa_block_window_attn_fwd(const void *q, const void *k, const void *v, void *out,
                                   int32_t batch, int32_t n, int32_t block,
                                   int32_t look_back, int32_t look_ahead,
                                   int32_t H, int32_t D, float scale, pa_stream_t stream);

/*
 * pa_block_window_attn_fwd_f32 -- the same block-local attention in fp32.
 *
 * The Token2Wav DiT runs in fp32 with classifier-free guidance as batch 2
 * ("[Perf][Model] Use block-sparse attention in Qwen2.5-Omni Token2Wav DiT",
 * Purpose), and its block-local result stayed within 6e-6 of the dense masked
 * SDPA (Test Result).  The window rule and the argument rules are those of
 * pa_block_window_attn_fwd; q, k, v, out are fp32 [batch, n, H, D]
 * contiguous, 16-byte aligned, caller-owned; out must not overlap q, k or v.
 * Every product and sum is IEEE fp32 (no tensor-core tf32); the softmax runs
 * in base 2 on the hardware exp2 with scale * log2(e) folded into q, so the
 * result is within a few fp32 roundings of the exact one.  Rows are staged
 * with TMA tensor copies (strides H * D * 4 and n * H * D * 4 bytes, so the
 * 16-byte alignment above is what they need); a wait that runs out records
 * PA_DEVICE_ERR_TIMEOUT in the device status word.
 */
pa_status pa_block_window_attn_fwd_f32(const float *q, const float *k, const float *v,
                                       float *out, int32_t batch, int32_t n, int32_t block,
                                       int32_t look_back, int32_t look_ahead, int32_t H,
                                       int32_t D, float scale, pa_stream_t stream);

/*
 * pa_cu_seqlens_from_lengths -- cu[0] = 0, cu[b+1] = cu[b] + lengths[b].
 *
 * The flat path's boundaries come from each request's real token count
 * ("[Perf][Diffusion][Qwen-Image] Replace per-bucket varlen loop with flat
 * varlen attention for mixfusion", Key changes: cu_seqlens built from real
 * text lengths via mask.sum).  lengths: device int32 [batch]; cu: device int32
 * [batch + 1].  batch >= 1.  A negative length records
 * PA_DEVICE_ERR_LENGTH and is treated as 0.
 */
pa_status pa_cu_seqlens_from_lengths(const int32_t *lengths, int32_t *cu, int32_t batch,
                                     pa_stream_t stream);

/*
 * pa_pack -- copy the real rows of a padded batch into the flat layout.
 *
 * Only real tokens enter the packed tensor ("feat: Support dynamic batching
 * for heterogeneous diffusion requests", How batching works).  padded is
 * [batch, s_max, row_bytes] bytes, flat is [total, row_bytes]; row r of
 * sequence b (r < cu[b+1] - cu[b]) goes from padded[b, r] to flat[cu[b] + r].
 * Flat rows >= cu[batch] are not touched.  cu: device int32 [batch + 1].
 * batch >= 1, s_max >= 0, total >= 0, row_bytes > 0 and a multiple of 16;
 * pointers 16-byte aligned.  A sequence longer than s_max records
 * PA_DEVICE_ERR_MAX_LEN, boundaries outside [0, total] or decreasing record
 * PA_DEVICE_ERR_CU_SEQLENS; such a sequence is skipped.
 */
pa_status pa_pack(const void *padded, void *flat, const int32_t *cu, int32_t batch,
                  int32_t s_max, int32_t total, int64_t row_bytes, pa_stream_t stream);

/*
 * pa_unpack -- the inverse scatter: flat[cu[b] + r] -> padded[b, r] for
 * r < cu[b+1] - cu[b]; padding rows of `padded` are left untouched (output
 * unpacked by cu_seqlens, same page as pa_cu_seqlens_from_lengths).
 * Same argument rules as pa_pack.
 */
pa_status pa_unpack(const void *flat, void *padded, const int32_t *cu, int32_t batch,
                    int32_t s_max, int32_t total, int64_t row_bytes, pa_stream_t stream);

/*
 * pa_rope_packed -- rotary position embedding on packed q and k, in place,
 * with request-local positions.
 *
 * The dynamic path rebuilds RoPE per request from request-local state and
 * never infers positions from packed global offsets, so a request gets the
 * same RoPE alone or inside a mixed batch ("feat: Support dynamic batching
 * for heterogeneous diffusion requests", Correctness model).  The pages give
 * no formula; this is the rotary embedding of Su et al. (RoFormer) on
 * interleaved pairs: token j of sequence b sits at position
 * p = pos_offset[b] + j and every head's pair (x_2i, x_2i+1) is rotated by the
 * angle p * base^(-2i/D).  Angles are reduced exactly (double-precision
 * fraction of a turn), sin/cos and the rotation in fp32, output bf16.
 *
 * q [total_q, H, D] and k [total_k, H, D] bf16 are updated in place at the
 * rows of their sequences (rows past cu[batch] are left untouched).
 * cu_seqlens_q / cu_seqlens_k: device int32 [batch + 1]; pos_offset: device
 * int32 [batch] or NULL (all zero).  batch in [1, 65535], H >= 1, D even,
 * a multiple of 8 and at most 512, base finite and > 0; q, k 16-byte
 * aligned.  Bad boundaries record PA_DEVICE_ERR_CU_SEQLENS; the sequence is
 * skipped.
 */
pa_status pa_rope_packed(void *q, void *k, const int32_t *cu_seqlens_q,
                         const int32_t *cu_seqlens_k, const int32_t *pos_offset,
                         int32_t batch, int32_t total_q, int32_t total_k, int32_t H,
                         int32_t D, float base, pa_stream_t stream);

/*
 * pa_rope_axes -- rotary positions with several axes (time, height, width of
 * image and video tokens), on packed q and k.
 *
 * Pair i of a head's rotated width R = sum of axis_dims, i in [0, R / 2), belongs
 * to the axis whose stretch of axis_dims[a] / 2 pairs holds it, the axes in order.
 * Its two elements, 2i and 2i + 1 or (halves != 0) i and i + R / 2, are turned by
 * the angle positions[a, t] * theta_i: (x, y) -> (x cos - y sin, x sin + y cos).
 * theta_i = base^(-2 j / axis_dims[a]) with j the pair's place on its axis, or
 * (shared != 0: one spectrum over all axes) base^(-2 i / R).  Elements past R
 * are copied.  theta_i is off by 2^-52 at most (base >= 1), the angle by that times
 * the position and not more; sin, cos and the rotation are fp32, the output is rounded
 * once.
 *
 * q, q_out [total, Hq, D], k, k_out [total, Hkv, D] bf16 with their strides in
 * elements from one token to the next (>= heads * D, multiples of 8); q_out = q
 * and k_out = k (with the same stride) turn in place, else outputs must not
 * overlap inputs; Hkv = 0: no k.  positions: device int32 [axes, total],
 * any values.  num_tokens: device int32, or NULL: only rows below it are
 * turned, the others left untouched (cu_seqlens + batch, for buffers with rows
 * behind the last sequence).  axis_dims: HOST int32 [axes], even, >= 2; axes
 * in [1, 8]; R a multiple of 8 and at most D; D a multiple of 8 and at most
 * 256; heads at most 2^20 each; total * heads at most 2^30; base finite and
 * > 0.  total = 0 does nothing (pointers may then be NULL).
 */
pa_status pa_rope_axes(const void *q, const void *k, void *q_out, void *k_out,
                       const int32_t *positions, const int32_t *num_tokens,
                       const int32_t *axis_dims, int32_t axes, int32_t total,
                       int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                       int64_t k_out_stride, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t halves, int32_t shared, float base, pa_stream_t stream);

/*
 * Paged K/V caches
 * ----------------
 * A program that answers token by token, or takes a long input in chunks,
 * keeps K and V between calls.  The cache is a pool of pages that any
 * sequence may hold, in any order:
 *
 *   k_cache, v_cache  [num_pages, page_size, Hkv, D], each page contiguous;
 *                     page g starts page_stride elements after page g - 1
 *                     (page_size * Hkv * D, or more where pages of K and V
 *                     alternate in one buffer)
 *   page_table        device int32 [batch, table_pages]: position p of
 *                     sequence b is row p % page_size of page
 *                     page_table[b, p / page_size].  Entries past a
 *                     sequence's last position may hold anything.
 *   format            PA_CACHE_BF16: bf16 rows; k_exp and v_exp are ignored.
 *                     PA_CACHE_E4M3: 8-bit rows.  A row (one token and head)
 *                     x[0..D) is held as e4m3 values y and one exponent e
 *                     with x ~ y * 2^e: e is the smallest integer with
 *                     max |x| * 2^-e <= 448, kept within [-100, 7], and
 *                     y = x * 2^-e rounded to nearest even, saturating at
 *                     +-448 (so magnitudes above 57344, infinities among
 *                     them, read back as 57344).  e + 127 is the row's byte in
 *   k_exp, v_exp      [num_pages, Hkv, page_size], contiguous.  Byte 255: the
 *                     row held a NaN and reads back as NaN throughout.
 *                     (A cache filled by other means holds bytes 27 to 134,
 *                     or 255; an e4m3 NaN in it is a NaN wherever it is read.)
 *
 * page_size a power of two in [16, 256], D in {64, 128}, Hkv in [1, 4096],
 * num_pages and table_pages >= 1; page_stride * element size a multiple of 16
 * bytes; k_cache, v_cache, k_exp, v_exp 16-byte aligned.  A page index
 * outside [0, num_pages) records PA_DEVICE_ERR_PAGE: its tokens are not
 * written, and read as zeros.
 */

/*
 * pa_kv_cache_write -- packed new rows into a paged cache, quantised as they
 * are written where the cache holds 8-bit rows.
 *
 * Row j of packed sequence b goes to position pos_offset[b] + j (NULL: j),
 * the position pa_rope_packed rotated it by.  k, v: bf16 [total, Hkv, D] with
 * k_stride / v_stride elements from one token to the next (>= Hkv * D,
 * multiples of 8: the rows may be slices of a fused projection's output).
 * cu_seqlens device int32 [batch + 1]; pos_offset device int32 [batch].
 * batch in [1, 65535]; total >= cu_seqlens[batch], later rows are ignored
 * (total = 0 does nothing, and k, v may then be NULL).
 * Everything of the cache that no row goes to is left as it was.  Two rows of
 * one call must not share a place: which of them is kept, or a mixture, is
 * not defined.  k, v must not overlap the cache.  Bad boundaries record
 * PA_DEVICE_ERR_CU_SEQLENS; a negative offset or a position beyond
 * table_pages * page_size records PA_DEVICE_ERR_MAX_LEN; such a sequence is
 * skipped.
 */
pa_status pa_kv_cache_write(const void *k, const void *v, void *k_cache, void *v_cache,
                            uint8_t *k_exp, uint8_t *v_exp, const int32_t *cu_seqlens,
                            const int32_t *pos_offset, const int32_t *page_table,
                            int32_t batch, int32_t total, int64_t k_stride, int64_t v_stride,
                            int32_t num_pages, int32_t page_size, int32_t table_pages,
                            int64_t page_stride, int32_t Hkv, int32_t D, int32_t format,
                            pa_stream_t stream);

/*
 * pa_kv_cache_read -- cached rows back as packed bf16 rows, the inverse
 * gather: positions [pos_offset[b], pos_offset[b] + L_b) of sequence b, with
 * L_b = cu_seqlens[b+1] - cu_seqlens[b], become rows [cu_seqlens[b],
 * cu_seqlens[b+1]) of k and v, bf16 [total, Hkv, D] contiguous.  Rows of 8-bit
 * caches come back as y * 2^e, which bf16 holds exactly.  Rows of k and v
 * past cu_seqlens[batch] are left as they were.  The other rules are
 * pa_kv_cache_write's.
 */
pa_status pa_kv_cache_read(const void *k_cache, const void *v_cache, const uint8_t *k_exp,
                           const uint8_t *v_exp, void *k, void *v, const int32_t *cu_seqlens,
                           const int32_t *pos_offset, const int32_t *page_table,
                           int32_t batch, int32_t total, int32_t num_pages, int32_t page_size,
                           int32_t table_pages, int64_t page_stride, int32_t Hkv, int32_t D,
                           int32_t format, pa_stream_t stream);

/*
 * pa_paged_attn_fwd -- softmax attention of packed new tokens over a paged
 * K/V cache: a step of single tokens, chunks of long inputs, both in one
 * batch, or (causal = 0) tokens over cached states of another length.
 *
 * Sequence b has L_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] queries and
 * seq_lens[b] cached keys.  With causal != 0 its queries are the last L_b of
 * those positions (their own K and V written before the call): query i sees
 * key j iff j <= seq_lens[b] - L_b + i; with causal = 0 it sees every key.
 * Query head h reads K/V head h / (Hq / Hkv).
 *   out[i,h,:] = sum_j softmax_j(scale * <q[i,h,:], k[j,h',:]>) * v[j,h',:]
 * A query that sees no key gets zeros.  8-bit rows enter the products as the
 * bf16 values that pa_kv_cache_read returns.  Scores, maxima, sums and the
 * output's accumulation are fp32; softmax weights are rounded to bf16 for the
 * product with V, and the output once to bf16.  Few queries (L_b * Hq / Hkv
 * <= 32) over an 8-bit cache: w * 2^e, weight times the exponent of the V row,
 * is rounded to f16 instead, in full down to 2^-28 of the largest that the
 * query and head sees and in steps of at most 2^-38 of that below; and so are
 * q's elements, against the largest of their row.
 *
 * q [total_q, Hq, D] bf16, q_stride elements from one token to the next
 * (>= Hq * D, a multiple of 8); out [total_q, Hq, D] bf16 contiguous, written
 * at the rows that belong to a sequence only, and not overlapping q or the
 * cache.  cu_seqlens_q device int32 [batch + 1], seq_lens device int32
 * [batch], batch in [1, PA_MAX_BATCH]; total_q >= cu_seqlens_q[batch]
 * (total_q = 0 or max_q = 0 does nothing; with total_q = 0 q and out may be
 * NULL); max_q / max_k bound every L_b and seq_lens[b]; total_q, max_q and
 * max_k at most 2^30; Hq a multiple of Hkv, Hq / Hkv <= 128; scale and
 * scale * log2(e) finite, and scale * <q, k> below 2^29 in magnitude (beyond, where
 * fp32 scores lie 32 and more apart, a result may be NaN).
 * Rows of a page past a sequence's last position never reach a result,
 * whatever their bits.  A key that causal order hides from a query has weight
 * zero there; a NaN or infinity in its V row can still reach that query as
 * 0 * NaN (in its K row it cannot).
 *
 * workspace: device memory of at least pa_paged_attn_workspace_bytes() bytes,
 * 16-byte aligned, for the partial results of keys that are split over
 * several CTAs, and for the 8-bit rows of long sequences as bf16 where these
 * take at most 1 GB (NULL where that is 0).  Its contents need not be kept or
 * cleared; two calls that may run at the same time need one each.  The bytes
 * follow from the bounds: with 32 heads on 8 of 128 and max_k = 16,384 a
 * sequence of one token takes 1 MB, one of 64 tokens up to 23 MB.  They are never
 * more than 2 GB: a call whose batch could need more asks for that and takes its
 * sequences in turns, each with launches of its own, and in fewer where
 * workspace_bytes is larger.
 *
 * A sequence with bad boundaries (PA_DEVICE_ERR_CU_SEQLENS), a negative
 * seq_lens (PA_DEVICE_ERR_LENGTH), or a length beyond max_q, max_k or
 * table_pages * page_size (PA_DEVICE_ERR_MAX_LEN) is skipped, its rows left
 * untouched; where bad boundaries make sequences overlap, others may be too.
 * Deterministic, and independent of the batch around a sequence:
 * how its keys are split depends on its own lengths alone.
 */
pa_status pa_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache,
                            const uint8_t *k_exp, const uint8_t *v_exp, void *out,
                            const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                            const int32_t *page_table, int32_t batch, int32_t total_q,
                            int32_t max_q, int32_t max_k, int64_t q_stride,
                            int32_t num_pages, int32_t page_size, int32_t table_pages,
                            int64_t page_stride, int32_t Hq, int32_t Hkv, int32_t D,
                            int32_t format, int32_t causal, float scale, void *workspace,
                            int64_t workspace_bytes, pa_stream_t stream);

/* Workspace of a pa_paged_attn_fwd call with these arguments, in bytes (host
 * arithmetic alone); -1 where that call would be refused.  A workspace serves
 * every call that needs no more than it has.  (Over a bf16 cache that is every
 * call of smaller bounds; over an 8-bit one such a call may widen rows that the larger
 * bounds leave no room for, and need more.) */
int64_t pa_paged_attn_workspace_bytes(int32_t batch, int32_t total_q, int32_t max_q,
                                      int32_t max_k, int32_t Hq, int32_t Hkv, int32_t D,
                                      int32_t format);

/*
 * pa_linear_bf16 -- batch-invariant packed-M linear layer.
 *
 *   y[m, n] = sum_k x[m, k] * w[n, k] + bias[n]
 *
 * The packed path runs its projections on the flat [total_tokens, C]
 * activations of all requests at once, and batched and serial outputs are
 * bit-identical because these GEMMs give each row the same result whatever
 * the packed M is ("feat: Support dynamic batching for heterogeneous
 * diffusion requests", packed varlen step batching: Setup, Determinism;
 * Notes, item 1).  Here every M runs one tile shape with a fixed K order and
 * no split-K, so row m of y depends only on row m of x, w and bias: rows
 * computed packed, alone or at any row offset are equal bit for bit.
 *
 * x [M, K], w [N, K] (out_features x in_features), y [M, N]: bf16 row-major
 * contiguous, device, caller-owned; bias: bf16 [N] or NULL.  Accumulation
 * in fp32, bias added in fp32, one round to bf16 (nearest even).  M >= 0
 * (M = 0 does nothing and x, y may then be NULL), N >= 1, K >= 1; K and N
 * multiples of 8 and every pointer 16-byte aligned, else PA_ERR_MISALIGNED.
 * y must not overlap x, w or bias.
 */
pa_status pa_linear_bf16(const void *x, const void *w, const void *bias, void *y, int32_t M,
                         int32_t N, int32_t K, pa_stream_t stream);

/*
 * pa_linear_act_bf16 -- the packed-M linear layer with bias, activation and
 * residual in its epilogue.
 *
 *   y[m, n] = residual[m, n] + act(sum_k x[m, k] * w[n, k] + bias[n])
 *
 * x [M, K], residual, y [M, N] bf16 with their strides in elements from one row
 * to the next (>= K or N, multiples of 8); w [N, K] bf16 contiguous; bias bf16
 * [N] or NULL; residual or NULL (its stride is then ignored); act one of
 * PA_ACT_*.  y may be residual itself (in place, with the same stride), and must
 * not overlap x, w, bias or the residual otherwise.  Accumulation, activation
 * and sums are fp32, rounded to bf16 once.  A row depends on its own x and
 * residual row, w and bias alone: packed, alone or at any row offset its bits
 * agree.  M >= 0 (0 does nothing; x and y may then be NULL), N >= 1, K in
 * [1, 2^26]; K and N multiples of 8; every pointer 16-byte aligned.
 */
pa_status pa_linear_act_bf16(const void *x, const void *w, const void *bias,
                             const void *residual, void *y, int32_t M, int32_t N, int32_t K,
                             int64_t x_stride, int64_t residual_stride, int64_t y_stride,
                             int32_t act, pa_stream_t stream);

/*
 * pa_linear_gated_bf16 -- the first half of a gated feed-forward block: two
 * projections, the activation of one and their product.
 *
 *   y[m, n] = act(sum_k x[m, k] * w_gate[n, k]) * (sum_k x[m, k] * w_up[n, k])
 *
 * w_gate, w_up [N, K] bf16, contiguous each (two tensors, or the halves of one).
 * Neither product is rounded before the last step.  The other rules are
 * pa_linear_act_bf16's.
 */
pa_status pa_linear_gated_bf16(const void *x, const void *w_gate, const void *w_up, void *y,
                               int32_t M, int32_t N, int32_t K, int64_t x_stride,
                               int64_t y_stride, int32_t act, pa_stream_t stream);

/*
 * pa_cfg_combine -- segment-aware unpack of each request's image span with
 * the per-request classifier-free-guidance combine.
 *
 * Defined by "feat: Support dynamic batching for heterogeneous diffusion
 * requests" (AttentionSegment: text / image / negative-text spans used to
 * scatter outputs back to request-local state; CFG behavior: after the
 * per-request split, out = negative + true_cfg_scale * (positive - negative),
 * with true_cfg_scale and cfg_normalize per request).  Request r's positive
 * pass is packed sequence pos_seq[r], its negative pass sequence neg_seq[r]
 * (< 0: no CFG, the positive image rows are copied).  The image span of
 * sequence b is rows [cu[b] + img_off[b], cu[b+1]) of `flat`.  With
 * cfg_normalize[r] != 0 each combined row is rescaled to the L2 norm of its
 * positive row (rows whose combined norm is 0 are written as 0).
 *
 * flat [total, row_elems] bf16; out [requests, img_max, row_elems] bf16:
 * rows [0, n_img(r)) of slot r are written, the others left untouched.
 * cu device int32 [batch + 1]; img_off device int32 [batch]; pos_seq,
 * neg_seq, cfg_normalize device int32 [requests]; cfg_scale device float
 * [requests].  Arithmetic in fp32, output rounded to bf16.
 * batch in [1, 65535], requests in [1, 65535], total >= 0, img_max >= 0,
 * row_elems a positive multiple of 8; flat and out 16-byte aligned.
 * A request with an out-of-range sequence or image offset, positive and
 * negative image spans of different lengths, or more than img_max image
 * rows records PA_DEVICE_ERR_SEGMENT and is skipped.
 */
pa_status pa_cfg_combine(const void *flat, void *out, const int32_t *cu,
                         const int32_t *img_off, const int32_t *pos_seq,
                         const int32_t *neg_seq, const float *cfg_scale,
                         const int32_t *cfg_normalize, int32_t batch, int32_t requests,
                         int32_t total, int32_t img_max, int32_t row_elems,
                         pa_stream_t stream);

/*
 * pa_varlen_num_work_items -- host-side count of attention work items,
 * sum_b H * ceil(Lq[b] / tile_m), from HOST copies of cu_seqlens_q.
 * Returns -1 on invalid arguments.
 */
int64_t pa_varlen_num_work_items(const int32_t *cu_seqlens_q_host, int32_t batch,
                                 int32_t H, int32_t tile_m);

/*
 * pa_varlen_work_order -- the order in which the attention kernel visits its
 * work items, written by the same device code the kernel schedules with.
 *
 * Sequences are taken longest key length first (equal lengths: lower index
 * first); within a sequence heads in order, within a head query tiles of
 * tile_m rows in order.  The largest request dominates a mixed batch and the
 * old per-bucket loop left bubbles ("[Perf][Diffusion][Qwen-Image] Replace
 * per-bucket varlen loop ...", Purpose), so the longest work starts first.
 * items: device int32 [capacity, 3] receiving (sequence, head, q_tile) for
 * item 0, 1, ...; when there are more items than capacity, the first
 * `capacity` are written and PA_DEVICE_ERR_CAPACITY is recorded.  Boundaries
 * are checked as in pa_varlen_attn_fwd (without totals or maxima); a bad
 * sequence gets no items.  batch in [1, PA_MAX_BATCH], H >= 1, tile_m >= 1.
 * PA_VARLEN_TILE_M is the tile the attention kernel uses.
 */
pa_status pa_varlen_work_order(const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                               int32_t batch, int32_t H, int32_t tile_m,
                               int32_t *items, int64_t capacity, pa_stream_t stream);

/*
 * pa_get_device_status -- synchronize the current device, then read and
 * clear its status word.  *code receives PA_DEVICE_OK or the first
 * PA_DEVICE_ERR_* recorded since the last call.  Returns PA_ERR_DEVICE when
 * an error was recorded, PA_ERR_CUDA when the synchronize fails.  For tests
 * and debugging: it blocks the host.
 */
pa_status pa_get_device_status(int32_t *code);

/*
 * pa_selftest_wait_timeout -- exercises the bounded-wait path the pipelined
 * kernels use: one CTA waits on an mbarrier that nothing ever arrives at,
 * gives up after about `timeout_us` microseconds (1 .. 10,000,000), records
 * PA_DEVICE_ERR_TIMEOUT in the status word and returns, leaving the context
 * usable.  No counterpart on the pages; it tests this library's own failure
 * handling without faulting the GPU.
 */
pa_status pa_selftest_wait_timeout(int32_t timeout_us, pa_stream_t stream);

/* Name of the last CUDA error this thread met inside the library, the cause
 * behind a PA_ERR_CUDA (static string, never NULL; "cudaSuccess" if none). */
const char *pa_last_cuda_error(void);

/* Human-readable name of a status code (static string, never NULL). */
const char *pa_status_string(pa_status status);

#ifdef __cplusplus
}
#endif

#endif /* PACKEDATTN_H */
