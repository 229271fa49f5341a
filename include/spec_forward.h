/*
 * spec_forward.h -- C ABI of the operators that a verify forward needs on either side of
 * its model, on MI355X (gfx950): the paged KV cache (write and attention) and the
 * adjustment of the logits that spec_verify (spec_verify.h) then reads.
 *
 * The verify forward of batch row b consumes R = k + 1 tokens, the pending token and the
 * k drafts ("Speculative Decoding: The Physics of Stolen Time", section 1 stage 3);
 * R = 1 is the ordinary decoding of single tokens. Their keys and values stand at
 * positions kv_len[b]..kv_len[b] + R - 1 of the sequence (spec_kv_append), each of them
 * attends to the whole sequence up to itself (spec_attention), and the logits pass the
 * request's penalties, biases and grammar masks (spec_adjust) before spec_verify and
 * spec_commit, which advances kv_len by what was accepted.
 *
 * Common rules, those of spec_verify.h: every pointer argument is a DEVICE pointer on the
 * current HIP device, owned by the caller; the calls only enqueue work on `stream` (a
 * hipStream_t; NULL = the null stream), allocate nothing and never synchronise the host.
 * Errors are synchronous negative codes (SPEC_ERR_* of spec_verify.h; nothing enqueued);
 * spec_forward_last_error() then describes the last one of the calling thread. Bad data
 * on the device (a length, a page or an index out of its range) never leads to an access
 * out of range; what it does to its own batch row is stated at each call. Results are
 * bitwise reproducible for the same arguments on the same device.
 *
 * Ragged drafts: draft_len [B] int32 (NULL: every row has k drafts) holds k_b in [0, k];
 * then only the first k_b + 1 of a batch row's R tokens are in use.
 *
 * Paged cache: page_table [B, max_pages] int32; position t of batch row b is token
 * t % page_size of page page_table[b, t / page_size]. page_size is a power of two up to
 * 65536, and max_pages * page_size at most 2^30. k_cache and v_cache hold `pages` pages; element (page, h, token, j) of cache
 * head h is at page * stride[0] + h * stride[1] + token * stride[2] + j (strides in
 * elements, j < D contiguous), so both the [pages, Hkv, page_size, D] and the
 * [pages, page_size, Hkv, D] order are served. Base pointers are 16-byte aligned and
 * strides multiples of 16 bytes, tokens at most 2^27 bytes apart. Offsets are 64-bit. The cache holds bfloat16 or float16
 * (the type of the new keys, values and queries), or e4m3 (OCP, finite range +-448) with
 * one positive float32 scale per cache head: value = code * scale[h].
 */
#ifndef SPEC_FORWARD_H
#define SPEC_FORWARD_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_DTYPE_F16 2
#define SPEC_DTYPE_E4M3 3

#define SPEC_MAX_PAGE 65536

/*
 * Write the keys and values of R new tokens per batch row into the cache, at positions
 * kv_len[b]..kv_len[b] + R - 1 (or as many of them as draft_len says are in use).
 *   k, v: [B, R, Hkv, D], dtype bfloat16 or float16; element (b, i, h, j) at
 *     b * stride[0] + i * stride[1] + h * stride[2] + j (elements; 16-byte aligned base,
 *     strides multiples of 8), e.g. slices of a fused projection's output.
 *   cache_dtype: dtype, or SPEC_DTYPE_E4M3 with k_scale, v_scale [Hkv] float32 (NULL
 *     otherwise): code = e4m3(x / scale[h]), the quotient in float32, then nearest with
 *     ties to even, saturating at +-448; NaN stays NaN.
 * A batch row whose kv_len is negative, whose draft_len is outside [0, R - 1] or whose
 * tokens do not fit max_pages * page_size positions is not written; a token whose page is
 * outside [0, pages) is not written. Distinct tokens of a call must go to distinct cache
 * places (where two share one, either may end up in it). The cache must not overlap k, v.
 * 1 <= B <= 2^21, 1 <= R <= 2^20, 1 <= Hkv <= 1024, D in {64, 128, 256}.
 * Enqueues one kernel. Errors: SPEC_ERR_SHAPE, SPEC_ERR_DTYPE, SPEC_ERR_NULL,
 * SPEC_ERR_ALIGN, SPEC_ERR_HIP.
 */
int spec_kv_append(const void* k, const int64_t* k_stride, const void* v, const int64_t* v_stride, int dtype,
                   int32_t B, int32_t R, int32_t Hkv, int32_t D, void* k_cache, const int64_t* k_cache_stride,
                   void* v_cache, const int64_t* v_cache_stride, int cache_dtype, int64_t pages,
                   int32_t page_size, const int32_t* page_table, int32_t max_pages, const int32_t* kv_len,
                   const int32_t* draft_len, const float* k_scale, const float* v_scale, void* stream);

/*
 * Attention of the R new tokens of every batch row over its paged cache, which already
 * holds their keys and values. Query head h of Hq reads cache head h / (Hq / Hkv). For
 * token i, at position p = kv_len[b] + i:
 *   s_t = cap(scale * q . k_t) + slope[h] * (t - p),  p - window < t <= p  (t >= 0)
 *   out = sum_t exp(s_t) v_t / sum_t exp(s_t)
 *   cap(x) = softcap * tanh(x / softcap), or x when softcap is 0; slopes NULL: no bias;
 *   window 0: no lower bound.
 *   q: [B, R, Hq, D], dtype bfloat16 or float16, with strides as k of spec_kv_append.
 *   out: [B, R, Hq, D] dense, of q's dtype, 16-byte aligned, fully overwritten, not
 *     overlapping q or the cache: tokens behind draft_len's get zeros; a batch row with a
 *     bad kv_len or draft_len (as in spec_kv_append) or a page outside [0, pages) among
 *     those it needs gets NaN.
 * Only cache places that a used token sees are used: pages before every window and behind
 * the last token may be unmapped, and NaN or infinities there change nothing.
 * Products of q and k are summed in float32, the softmax and the sums are float32; the
 * weights exp(s - m) are rounded once to q's dtype for the product with v. (m is at
 * or below the true maximum, so their magnitude is at most 2^8, or 2^15 in float16, where
 * the maximum's is at least 2^7.)
 * The length is split over workgroups, whose partial results are joined by a second
 * kernel; how it is split depends on the lengths on the device, not on the host.
 * Workspace: at least spec_attention_workspace_size() bytes, 256-byte aligned, no
 * initialisation needed, one call at a time. 1 <= R <= SPEC_MAX_K + 1,
 * 1 <= Hkv <= 1024, Hq a multiple of Hkv up to 1024, otherwise the limits of
 * spec_kv_append. Errors: as there, plus SPEC_ERR_VALUE (scale not finite, softcap
 * negative, not finite or below 1e-30 |scale| without being 0, window negative) and
 * SPEC_ERR_WORKSPACE.
 */
int spec_attention(const void* q, const int64_t* q_stride, int dtype, int32_t B, int32_t R, int32_t Hq, int32_t Hkv,
                   int32_t D, const void* k_cache, const int64_t* k_cache_stride, const void* v_cache,
                   const int64_t* v_cache_stride, int cache_dtype, int64_t pages, int32_t page_size,
                   const int32_t* page_table, int32_t max_pages, const int32_t* kv_len, const int32_t* draft_len,
                   float scale, float softcap, int32_t window, const float* slopes, const float* k_scale,
                   const float* v_scale, void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace spec_attention needs (0 if the sizes are invalid). Host-only. */
size_t spec_attention_workspace_size(int32_t B, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int cache_dtype,
                                     int32_t page_size, int32_t max_pages);

/*
 * Penalties for repeated tokens, biases and grammar masks on the logits of a verify step.
 *   logits [B, R, V] float32 or bfloat16 (dtype), out [B, R, V] of out_dtype: float32, or
 *     bfloat16 for bfloat16 logits. out may be logits itself (same dtype), else it must
 *     not overlap it. R = k + 1 (target rows) or R = k (draft rows).
 * Row i of batch row b follows the request's history and its drafts 0..i-1:
 *   history [B, H] int32, hist_len [B] int32 in [0, H]: the committed tokens;
 *   prompt_len [B] int32 in [0, hist_len] (NULL: 0): how many of them were the prompt;
 *   draft_tokens [B, k] int32. Tokens outside [0, V) count for nothing.
 * With seen(v) = v is in the history or among those drafts, count(v) = how often v is in
 * the history behind the prompt and among those drafts, in float32 and in this order:
 *   x = seen(v) ? (x > 0 ? x / repetition[b] : x * repetition[b]) : x
 *   x = x - frequency[b] * count(v), x = x - presence[b] if count(v) > 0
 *   x = x + the values of every j with bias_tokens[b, j] = v, summed in the order of j
 *   x = -inf if v is not admitted by row admit_row[b, i] of admit
 * and one rounding to out_dtype. repetition, frequency, presence [B] float32: NULL means
 * 1, 0, 0. bias_tokens [B, n_bias] int32, bias_values [B, n_bias] float32: entries whose
 * token is outside [0, V) (padding) are skipped. admit [n_admit, (V + 31) / 32] uint32: bit
 * (v & 31) of word v >> 5 admits token v (spec_gate's layout); admit_row [B, R] int32:
 * -1 = everything is admitted; NULL: row b * R + i (n_admit must then be B * R). A token
 * that is not admitted becomes -inf whatever its logit was, NaN included.
 * A batch row whose hist_len or prompt_len is out of range, whose repetition is not finite
 * and positive, or whose frequency or presence is not finite gets NaN in all its rows (so
 * spec_verify reports it as invalid); so does a row whose admit_row is outside
 * [-1, n_admit). With draft_len, rows behind the ones in use (the first k_b + 1 target
 * rows or k_b draft rows; a batch row whose draft_len is outside [0, k]: all) are left as
 * they were.
 * 1 <= B <= 2^21, 0 <= k <= SPEC_MAX_K, R >= 1, 1 <= V <= 2^29, 0 <= H < 2^29 (0: no
 * history), 0 <= n_bias <= 65536. Enqueues one kernel, no workspace. Errors:
 * SPEC_ERR_SHAPE, SPEC_ERR_DTYPE, SPEC_ERR_NULL, SPEC_ERR_ALIGN, SPEC_ERR_HIP.
 */
int spec_adjust(const void* logits, int32_t B, int32_t R, int32_t V, int dtype, const int32_t* draft_tokens, int32_t k,
                const int32_t* draft_len, const int32_t* history, int32_t H, const int32_t* hist_len,
                const int32_t* prompt_len, const float* repetition, const float* frequency, const float* presence,
                const int32_t* bias_tokens, const float* bias_values, int32_t n_bias, const uint32_t* admit,
                int32_t n_admit, const int32_t* admit_row, void* out, int out_dtype, void* stream);

/* Thread-local description of the last non-zero return of these functions. */
const char* spec_forward_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_FORWARD_H */
