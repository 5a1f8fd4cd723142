/*
 * qlora_decoder.h - C ABI of the operators of a decoder block around the
 * frozen-NF4 linears of qlora_nf4.h: the residual update with its norms,
 * rotary positions, and decoding from a paged key-value cache.
 *
 * The conventions are those of qlora_nf4.h: caller-owned device buffers,
 * 16-byte aligned (int32 arrays and lse: 4-byte aligned); work is only enqueued, on `stream`; arguments are checked
 * on the host before anything is enqueued; a negative qlora_status and
 * qlora_last_error() on failure; no state between calls.  Buffers of one
 * call must not overlap unless the entry point says so.  The current HIP
 * device must be the one `stream` belongs to.
 */
#ifndef QLORA_DECODER_H
#define QLORA_DECODER_H

#include <stdint.h>

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row of the residual update. */
#define QLORA_NORM_MAX_WIDTH 16384

/* ------------------------------------------------ norm, gate and residual */

/*
 * qlora_norm_residual_fwd - the step between two branches of a block.  For
 * every row t of D elements, with rms(z) = sqrt(mean(z^2) + eps):
 *     u  = h / rms(h) * w_post     (u = h when w_post is NULL)
 *     xo = x + alpha * gate * u    (gate = 1 when NULL; xo = x when h is NULL)
 *     n  = xo / rms(xo) * w_pre
 *
 *   x, xo     [T, D], x_dtype: the residual stream before and after.  xo may
 *             be x itself.  With h NULL nothing is added: xo may then be NULL
 *             (not written).
 *   h, n      [T, D], h_dtype: the output of the last branch (NULL: none) and
 *             the input of the next one (NULL: not written, w_pre unused).
 *   w_post, gate, w_pre   fp32 [D] or NULL (w_pre is required with n).
 *   x_dtype, h_dtype      F32 and F32, F32 and BF16, or BF16 and BF16.
 *   T >= 0 (0 enqueues nothing); 1 <= D <= QLORA_NORM_MAX_WIDTH; eps >= 0.
 * fp32 throughout, each output rounded once (n is formed from xo before it is
 * rounded).  xo or n must be given.  A row whose sum of squares passes fp32's range
 * (values beyond 10^17) counts as one of infinite rms.
 */
int qlora_norm_residual_fwd(const void* x, int32_t x_dtype, const void* h, int32_t h_dtype, int64_t T, int64_t D,
                            const float* w_post, const float* gate, float alpha, const float* w_pre, float eps,
                            void* xo, void* n, void* stream);

/*
 * qlora_norm_residual_bwd - gradients of qlora_norm_residual_fwd for the
 * upstream gradients dxo of xo and dn of n:
 *     r  = 1 / rms(xo),  a = dn * w_pre
 *     dx = dxo + r * (a - xo * r^2 * mean(a * xo))
 *     y  = h / rms(h),  b = alpha * gate * dx       (y = h without w_post)
 *     dh = (b * w_post - y * mean(b * w_post * y)) / rms(h)   (dh = b without)
 *     dw_pre = sum_t dn * xo * r,  dw_post = sum_t b * y,
 *     dgate  = sum_t alpha * dx * y * w_post
 *
 *   dxo, xo   [T, D], x_dtype (dxo NULL: zero).  xo is what the forward wrote
 *             (x, when the forward had no h).
 *   dn, h     [T, D], h_dtype.  dn NULL: zero (w_pre unused).  h may be NULL
 *             when neither w_post nor dgate is given.
 *   dx        [T, D], x_dtype; may be dxo itself.
 *   dh        [T, D], h_dtype, or NULL; may be dn itself.
 *   dw_post, dgate, dw_pre   fp32 [D] or NULL (not wanted); written, never
 *             added to.  dw_post needs w_post, dw_pre needs dn.
 *   ws        device workspace of at least the bytes
 *             qlora_norm_residual_bwd_workspace gives with sums = how many of
 *             the three are wanted (0 bytes for none: ws may then be NULL).
 * With T = 0 the wanted sums are set to zero.  Sums over tokens are fp32 in an
 * order that depends on T and D alone, so results repeat bit for bit.
 */
int qlora_norm_residual_bwd_workspace(int64_t T, int64_t D, int32_t x_dtype, int32_t h_dtype, int32_t sums,
                                      int64_t* ws_bytes);
int qlora_norm_residual_bwd(const void* dxo, const void* xo, int32_t x_dtype, const void* dn, const void* h,
                            int32_t h_dtype, int64_t T, int64_t D, const float* w_post, const float* gate,
                            float alpha, const float* w_pre, float eps, void* dx, void* dh, float* dw_post,
                            float* dgate, float* dw_pre, void* ws, int64_t ws_bytes, void* stream);

/* -------------------------------------------------------- rotary positions */

/* How the frequencies are stretched for contexts longer than the trained one,
 * from f_i = base^(-2i / rot_dim):
 *   NONE    f_i
 *   LINEAR  f_i / factor (positions interpolated)
 *   NTK     f_i of the base base * factor^(rot_dim / (rot_dim - 2))
 *   YARN    f_i / factor * (1 - g_i) + f_i * g_i, g_i = clamp((t_i - beta_slow)
 *           / (beta_fast - beta_slow), 0, 1) with t_i = original_len * f_i /
 *           2 pi the turns over the trained length, and every rotated value
 *           multiplied by 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient
 *           Context Window Extension of Large Language Models",
 *           arXiv 2309.00071, sections 3.2 and 3.4). */
typedef enum {
  QLORA_ROPE_NONE = 0,
  QLORA_ROPE_LINEAR = 1,
  QLORA_ROPE_NTK = 2,
  QLORA_ROPE_YARN = 3
} qlora_rope_scaling;

/* Host only.  Writes the rotary table: turns[i] = f_i / 2 pi for i <
 * rot_dim / 2 (host array; the device entry points take a device copy) and
 * the factor of the rotated values to *mscale.  rot_dim even, 2 .. 1024 (4 at
 * least with NTK); base > 1; factor >= 1; original_len, beta_fast and
 * beta_slow count for YARN only (original_len >= 1, beta_fast > beta_slow
 * >= 0). */
int qlora_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, double original_len,
                           double beta_fast, double beta_slow, double* turns, float* mscale);

/*
 * qlora_rope - rotary positions on the queries and keys of T tokens.  The
 * first rot_dim elements of each head are pairs (a_i, b_i), i < rot_dim / 2;
 * pair i of a token at position p becomes
 *     mscale * (a_i cos t - b_i sin t, a_i sin t + b_i cos t),
 *     t = 2 pi p turns[i],
 * and the rest of the head is copied.  With inverse = 1, t counts backwards:
 * that is the gradient of the forward (both are mscale times an orthogonal
 * map).
 *
 *   q, qo     [T, q_heads, head_dim], dtype; the heads of a token are dense,
 *             tokens are q_stride and qo_stride elements apart.  qo may be q
 *             (with the same stride).  q_heads = 0: no queries.
 *   k, ko     likewise with kv_heads (0: no keys).
 *   positions int32 [T], any value.
 *   turns     device fp64 [rot_dim / 2]; may be NULL when rot_dim = 0.
 *   interleaved  0: a_i = element i, b_i = element i + rot_dim / 2;
 *             1: a_i = element 2i, b_i = element 2i + 1.
 *   1 <= head_dim <= 1024; rot_dim even, 0 <= rot_dim <= head_dim; strides at
 *   least heads * head_dim; T < 2^24.
 * The angle, its cosine and its sine are fp64; they and mscale's product are
 * rounded to fp32 once, the rotation is fp32, rounded once.
 */
int qlora_rope(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride, const void* k,
               int64_t k_stride, int32_t kv_heads, void* ko, int64_t ko_stride, int64_t T, int32_t head_dim,
               int32_t rot_dim, int32_t dtype, const int32_t* positions, const double* turns, float mscale,
               int32_t interleaved, int32_t inverse, void* stream);

/* -------------------------------------------------- paged key-value cache */

/*
 * The cache of one layer is two bf16 buffers [num_pages, kv_heads, page_size,
 * head_dim], keys (rotated) and values.  Token slot s is row s % page_size of
 * page s / page_size.  A sequence's tokens are in the pages of its row of the
 * block table, token i in page table[i / page_size].
 */

/*
 * qlora_rope_cache_write - qlora_rope for tokens entering the cache: queries
 * are rotated into qo, keys are rotated into their slots of k_cache and the
 * values copied into the same slots of v_cache.
 *
 *   q, qo, k, positions, turns, mscale, interleaved, sizes: as for qlora_rope
 *             (bf16; q_heads = 0: no queries; kv_heads >= 1).
 *   v         [T, kv_heads, head_dim], tokens v_stride elements apart.
 *   slots     int32 [T]; a token whose slot is negative or not below num_pages
 *             * page_size is not stored (its query is still rotated).  No two
 *             tokens may have the same slot (else either is stored, possibly
 *             mixed).
 *   page_size 1 .. 1024, a power of two; num_pages * page_size < 2^31.
 * Slots that no token names keep their contents.
 */
int qlora_rope_cache_write(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t kv_heads,
                           int64_t T, int32_t head_dim, int32_t rot_dim, const int32_t* positions,
                           const double* turns, float mscale, int32_t interleaved, const int32_t* slots,
                           void* k_cache, void* v_cache, int64_t num_pages, int32_t page_size, void* stream);

/* Most sequences of one qlora_paged_plan call. */
#define QLORA_PLAN_MAX_SEQS 4096

/*
 * qlora_paged_plan - pages, slots and positions of a batch in which sequence
 * s, with cached_lens[s] tokens in the cache, gets new_lens[s] more.
 *
 *   cached_lens, new_lens   int32 [S]; negative values count as 0.  S <=
 *             QLORA_PLAN_MAX_SEQS; sums beyond 2^31 - 1 (all new tokens, or
 *             cached + new of a sequence) count as 2^31 - 1.
 *   free_pages int32 [n_free]: pages not in use.  The sequences take the pages
 *             they need from its front, in order of s and of position.
 *   table     int32 [S, table_cols]: the block table.  The pages that cached
 *             tokens occupy must be there; the pages taken are written behind
 *             them, every other entry is left as it is.  Where the free list
 *             has run out the entry becomes -1; no page is taken that the
 *             table has no column for.
 *   total_lens int32 [S]: cached + new; not cached_lens or new_lens themselves.
 *   starts    int32 [S + 1]: the first row of each sequence's new tokens, and
 *             the number of new tokens.
 *   slots, positions  int32 [T]: for the new tokens in order of s, the slot
 *             (-1 without a page) and the position in the sequence; rows
 *             behind the last new token get slot -1 and position 0, rows that
 *             T does not hold are left out.
 *   pages_needed  int32 [1]: pages the batch takes; more than n_free means that
 *             some tokens got no slot (as do tokens beyond table_cols pages).
 *   page_size >= 1.
 * One launch; integers only, so the result does not depend on the launch.
 */
int qlora_paged_plan(const int32_t* cached_lens, const int32_t* new_lens, int64_t S, int32_t page_size,
                     const int32_t* free_pages, int64_t n_free, int32_t* table, int64_t table_cols, int64_t T,
                     int32_t* total_lens, int32_t* starts, int32_t* slots, int32_t* positions,
                     int32_t* pages_needed, void* stream);

/*
 * qlora_paged_attention - attention of one new token per sequence over its
 * cached tokens (its own among them): for sequence s and query head h, with
 * kv head j = h / (q_heads / kv_heads) and n = lengths[s],
 *     out = sum_i p_i v_i,  p = softmax_i(scale * q . k_i),  i < n.
 *
 *   q         bf16 [S, q_heads, head_dim], sequences q_stride elements apart.
 *   k_cache, v_cache, num_pages, page_size   the cache; page_size a power of
 *             two, 16 .. 1024.
 *   table     int32 [S, table_cols]: the block table.  Tokens of a page that is
 *             negative or not below num_pages take no part.
 *   lengths   int32 [S], cut to 0 .. table_cols * page_size.  What the cache
 *             holds behind them is never used, whatever it is.
 *   scale     of the scores (finite).
 *   out       bf16 [S, q_heads, head_dim], dense; zeros for a sequence in
 *             which no token takes part.
 *   lse       fp32 [S, q_heads] or NULL: ln sum_i exp(scale * q . k_i),
 *             -inf for no token.
 *   head_dim  a multiple of 8, 8 .. 256; q_heads a multiple of kv_heads.
 *   ws        workspace of at least qlora_paged_attention_workspace bytes (may
 *             be 0: ws may then be NULL).
 * Long sequences are split over workgroups and joined by a second kernel in a
 * fixed order; scores, weights, their sums and the products with V are fp32 (a
 * weight enters as the sum of three bf16 numbers), the output is rounded once.
 * Results repeat bit for bit.
 */
int qlora_paged_attention_workspace(int64_t S, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                    int64_t table_cols, int32_t page_size, int64_t* ws_bytes);
int qlora_paged_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const void* k_cache, const void* v_cache, int64_t num_pages,
                          int32_t page_size, const int32_t* table, int64_t table_cols, const int32_t* lengths,
                          float scale, void* out, float* lse, void* ws, int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_DECODER_H */
