/*
 * qlora_kvcache.h - C ABI of the further forms of the paged key-value cache of
 * qlora_decoder.h: rows held in 8 bits with a scale each, and a prefix that the
 * sequences of a batch share.
 *
 * The conventions are those of qlora_decoder.h: caller-owned device buffers,
 * 16-byte aligned (int32 arrays and lse: 4-byte aligned); work is only
 * enqueued, on `stream`; arguments are checked on the host before anything is
 * enqueued; a negative qlora_status and qlora_last_error() on failure; no state
 * between calls.  Buffers of one call must not overlap unless the entry point
 * says so.  The current HIP device must be the one `stream` belongs to.
 */
#ifndef QLORA_KVCACHE_H
#define QLORA_KVCACHE_H

#include <stdint.h>

#include "qlora_decoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a row (the keys or the values of one token and kv head) is held.  BF16:
 * the numbers themselves.  INT8 and E4M3: a code of 8 bits per element, a whole
 * number in two's complement or an OCP E4M3FN number, and an fp32 scale per
 * row; an element stands for code * scale. */
typedef enum {
  QLORA_CACHE_BF16 = 0,
  QLORA_CACHE_INT8 = 1,
  QLORA_CACHE_E4M3 = 2
} qlora_cache_type;

/*
 * Descriptor of the cache of one layer.  Plain data: the caller fills it and
 * owns every buffer it points to.
 *
 *   k, v       [num_pages, kv_heads, page_size, head_dim]: rotated keys and
 *              values, bf16 or codes.  Token slot s is row s % page_size of page
 *              s / page_size.
 *   k_scale, v_scale   fp32 [num_pages, kv_heads, page_size]: the rows' scales
 *              (NULL for BF16), finite; qlora_kv_write makes none below 0, but any
 *              may be.  NaN marks a row that cannot be held: it reads as NaN
 *              throughout.
 *   page_size  a power of two, 1 .. 1024 (16 .. 1024 for the attention);
 *              num_pages * page_size < 2^31.
 *   head_dim   up to 256, a multiple of 16 (of 8 for BF16).
 *   type       qlora_cache_type.
 */
typedef struct qlora_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t type;
} qlora_kv_cache;

/*
 * qlora_kv_write - qlora_rope_cache_write for a cache of any type: queries are
 * rotated into qo, keys are rotated and stored with the values in their slots.
 * For the 8-bit types a row z (the fp32 rotated keys, or the values) of largest
 * size a is stored as
 *     scale = a / M rounded to fp32,  M = 127 (INT8) or 448 (E4M3),
 *     code  = the one nearest to z / scale (that quotient exactly, ties to the
 *             even code), at most M in size;
 * a row of zeros has scale 0 and codes 0 (as has one whose scale rounds to 0), a row
 * that holds a NaN or an infinity scale NaN and codes 0.
 *
 *   q, qo, k, v, positions, turns, mscale, interleaved, slots, strides: as for
 *              qlora_rope_cache_write (bf16).  No two tokens may have the same
 *              slot (else either is stored, possibly mixed).
 * Slots that no token names keep their contents.
 */
int qlora_kv_write(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int32_t rot_dim,
                   const int32_t* positions, const double* turns, float mscale, int32_t interleaved,
                   const int32_t* slots, const qlora_kv_cache* cache, void* stream);

/*
 * qlora_kv_read - rows of the cache as numbers: for every t < T the keys and
 * values in slots[t], code * scale in fp32, rounded once to dtype.
 *
 *   slots      int32 [T], in any order, any of them several times; a slot that is
 *              negative or not below num_pages * page_size gives zeros.
 *   k, v       [T, kv_heads, head_dim], dtype (QLORA_DTYPE_F32 or _BF16), dense;
 *              either may be NULL.
 *   T < 2^24.
 */
int qlora_kv_read(const qlora_kv_cache* cache, const int32_t* slots, int64_t T, int32_t dtype, void* k, void* v,
                  void* stream);

/*
 * qlora_kv_attention - qlora_paged_attention for a cache of any type: attention
 * of one new token per sequence over the numbers that its cached rows stand for.
 * The arguments are those of qlora_paged_attention.  Codes enter the products
 * as they are (bf16 holds them exactly), a key's scale is put on its score, a
 * value's on its weight, in fp32, and the weight enters the product with V with all
 * of its 24 bits, whatever the sizes of the call (with less where it is under 2^-109,
 * so where a value's scale is under 2^-100 or so).  Weights are exp of the score less
 * the row's largest, at most 1; the sum of the values they weigh has to stay in the
 * range of fp32 before it is divided by theirs.
 */
int qlora_kv_attention_workspace(const qlora_kv_cache* cache, int64_t S, int32_t q_heads, int64_t table_cols,
                                 int64_t* ws_bytes);
int qlora_kv_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, const qlora_kv_cache* cache,
                       const int32_t* table, int64_t table_cols, const int32_t* lengths, float scale, void* out,
                       float* lse, void* ws, int64_t ws_bytes, void* stream);

/*
 * qlora_prefix_attention - attention of one new token per sequence for a batch
 * that shares a prefix: sequence s attends to the prefix's tokens and, behind
 * them, to its own,
 *     out = sum_i p_i v_i,  p = softmax_i(scale * q . k_i),
 * i over the first *prefix_len tokens of prefix_table and the first lengths[s]
 * of row s of the block table.  The prefix's keys and values are read once for
 * a tile of query rows, not once per sequence.
 *
 *   prefix_table  int32 [prefix_cols]: the pages of the prefix; prefix_len int32
 *              [1] (device), cut to 0 .. prefix_cols * page_size.  Any length:
 *              the last page need not be full.  prefix_cols * page_size at most
 *              2^31 - 4097.
 *   table, lengths   the sequences' own tokens, as for qlora_paged_attention (a
 *              length of 0: the prefix alone); table_cols may be 0.
 *   the rest   as for qlora_paged_attention.  S * q_heads < 2^26.
 * Tokens of a page that is negative or not below num_pages take no part; a
 * sequence in which no token takes part gives zeros (lse -inf).  Results repeat
 * bit for bit.
 */
int qlora_prefix_attention_workspace(const qlora_kv_cache* cache, int64_t S, int32_t q_heads, int64_t prefix_cols,
                                     int64_t table_cols, int64_t* ws_bytes);
int qlora_prefix_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, const qlora_kv_cache* cache,
                           const int32_t* prefix_table, int64_t prefix_cols, const int32_t* prefix_len,
                           const int32_t* table, int64_t table_cols, const int32_t* lengths, float scale, void* out,
                           float* lse, void* ws, int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_KVCACHE_H */
