// C ABI of the 8-bit and the shared key-value cache: argument validation (host
// only, before any launch), workspace sizes and dispatch.  See
// include/qlora_kvcache.h for the contract of each entry point.
#include <hip/hip_runtime.h>
#include <math.h>

#include "abi_checks.h"
#include "kvcache.h"
#include "qlora_kvcache.h"

using namespace qlora;

namespace {

// The descriptor's sizes; its buffers are looked at when there is work.
int check_descriptor(const qlora_kv_cache* c, const char* fn) {
  if (!c) return fail(QLORA_ERR_INVALID_ARG, "%s: cache is NULL", fn);
  if (c->type < QLORA_CACHE_BF16 || c->type > QLORA_CACHE_E4M3)
    return fail(QLORA_ERR_UNSUPPORTED_DTYPE, "%s: the cache's type must be one of the qlora_cache_type values", fn);
  const int unit = c->type == QLORA_CACHE_BF16 ? 8 : 16;
  if (c->head_dim < unit || c->head_dim > 256 || c->head_dim % unit)
    return fail(QLORA_ERR_INVALID_ARG, "%s: head_dim must be a multiple of %d in [%d, 256]", fn, unit, unit);
  if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
    return fail(QLORA_ERR_INVALID_ARG, "%s: kv_heads must be in [1, %d]", fn, kMaxHeads);
  if (shift_of(c->page_size) < 0)
    return fail(QLORA_ERR_INVALID_ARG, "%s: page_size must be a power of two in [1, 1024]", fn);
  if (c->num_pages < 1 || c->num_pages > kMaxRows || c->num_pages * c->page_size > kMaxRows)
    return fail(QLORA_ERR_INVALID_ARG, "%s: need num_pages >= 1 and num_pages * page_size < 2^31", fn);
  if (c->num_pages * c->page_size > kMaxNumel / ((int64_t)c->kv_heads * c->head_dim))
    return fail(QLORA_ERR_INVALID_ARG, "%s: the cache must be below 2^37 elements", fn);
  return QLORA_OK;
}

int check_buffers(const qlora_kv_cache* c, const char* fn) {
  int st;
  if ((st = check_ptr(c->k, "cache.k", fn)) || (st = check_ptr(c->v, "cache.v", fn))) return st;
  if (c->type == QLORA_CACHE_BF16) {
    if (c->k_scale || c->v_scale) return fail(QLORA_ERR_INVALID_ARG, "%s: a BF16 cache has no scales", fn);
    return QLORA_OK;
  }
  if ((st = check_ptr(c->k_scale, "cache.k_scale", fn))) return st;
  return check_ptr(c->v_scale, "cache.v_scale", fn);
}

KvCache rows_of(const qlora_kv_cache* c) {
  return {c->k, c->v, c->k_scale, c->v_scale, c->num_pages, c->kv_heads, c->head_dim, shift_of(c->page_size), c->type};
}

int check_attention(const qlora_kv_cache* c, int64_t S, int32_t q_heads, int64_t prefix_cols, int64_t table_cols,
                    const char* fn) {
  int st;
  if ((st = check_descriptor(c, fn))) return st;
  if (S < 0 || S > 65535) return fail(QLORA_ERR_INVALID_ARG, "%s: S must be in [0, 65535]", fn);
  if (q_heads < 1 || q_heads > kMaxHeads || q_heads % c->kv_heads)
    return fail(QLORA_ERR_INVALID_ARG, "%s: q_heads must be a multiple of kv_heads in [1, %d]", fn, kMaxHeads);
  if (shift_of(c->page_size) < 4)
    return fail(QLORA_ERR_INVALID_ARG, "%s: page_size must be a power of two in [16, 1024]", fn);
  for (int64_t cols : {prefix_cols, table_cols})
    if (cols < 0 || cols > kMaxRows || cols * c->page_size > kMaxRows)
      return fail(QLORA_ERR_INVALID_ARG, "%s: columns * page_size of a table must be in [0, 2^31)", fn);
  // positions in the prefix are counted a step or two ahead in 32 bits
  if (prefix_cols * c->page_size > kMaxRows - 4096)
    return fail(QLORA_ERR_INVALID_ARG, "%s: prefix_cols * page_size must be at most 2^31 - 4097", fn);
  // a wave per row joins the parts: a grid holds 2^32 - 1 threads
  if (prefix_cols && S * q_heads >= (1 << 26))
    return fail(QLORA_ERR_INVALID_ARG, "%s: S * q_heads must be below 2^26 with a prefix", fn);
  return QLORA_OK;
}

int64_t attention_ws(const qlora_kv_cache* c, int64_t S, int32_t q_heads, const KvParts& p) {
  const int64_t parts = p.own + p.prefix;
  return parts > 1 ? S * q_heads * parts * (int64_t)(c->head_dim + 2) * 4 : 0;
}

// The call after its sizes were checked.  prefix_len NULL: no shared prefix.
int attend(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, const qlora_kv_cache* cache,
           const int32_t* prefix_table, int64_t prefix_cols, const int32_t* prefix_len, const int32_t* table,
           int64_t table_cols, const int32_t* lengths, float scale, void* out, float* lse, void* ws, int64_t ws_bytes,
           void* stream, const char* fn) {
  int st;
  if (!isfinite(scale)) return fail(QLORA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
  if (q_stride < (int64_t)q_heads * cache->head_dim || q_stride % 8 || (S && q_stride > kMaxNumel / S))
    return fail(QLORA_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 8, at least q_heads * head_dim", fn);
  if (S == 0) return QLORA_OK;
  if ((st = check_buffers(cache, fn)) || (st = check_ptr(q, "q", fn)) || (st = check_ptr(out, "out", fn)) ||
      (st = check_ptr(lengths, "lengths", fn, 4)) || (table_cols && (st = check_ptr(table, "table", fn, 4))) ||
      (lse && (st = check_ptr(lse, "lse", fn, 4))))
    return st;
  KvAttnArgs a = {};
  a.c = rows_of(cache);
  const KvParts p = kv_parts(a.c, S, q_heads, table_cols, prefix_cols);
  a.splits = p.own, a.psplits = p.prefix;
  const int64_t need = attention_ws(cache, S, q_heads, p);
  if (need) {
    if (ws_bytes < need)
      return fail(QLORA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %lld bytes", fn, (long long)need);
    if ((st = check_ptr(ws, "ws", fn))) return st;
    a.part_o = (float*)ws, a.part_ml = (float*)ws + S * q_heads * (p.own + p.prefix) * (int64_t)cache->head_dim;
  }
  a.q = (const uint16_t*)q, a.table = table, a.lengths = lengths;
  a.prefix_table = prefix_table, a.prefix_len = prefix_len;
  a.out = (uint16_t*)out, a.lse = lse;
  a.q_stride = q_stride, a.S = S, a.table_cols = table_cols, a.prefix_cols = prefix_cols;
  a.q_heads = q_heads, a.scale = scale;
  return finish(launch_kv_attention(a, (hipStream_t)stream), fn);
}

}  // namespace

extern "C" {

int qlora_kv_write(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int32_t rot_dim,
                   const int32_t* positions, const double* turns, float mscale, int32_t interleaved,
                   const int32_t* slots, const qlora_kv_cache* cache, void* stream) {
  static const char* fn = "qlora_kv_write";
  int st;
  if ((st = check_descriptor(cache, fn))) return st;
  if (cache->type == QLORA_CACHE_BF16) {
    if (T > 0 && (st = check_buffers(cache, fn))) return st;
    return qlora_rope_cache_write(q, q_stride, q_heads, qo, qo_stride, k, k_stride, v, v_stride, cache->kv_heads, T,
                                  cache->head_dim, rot_dim, positions, turns, mscale, interleaved, slots, cache->k,
                                  cache->v, cache->num_pages, cache->page_size, stream);
  }
  if ((st = check_rope(q_stride, q_heads, qo_stride, k_stride < v_stride ? k_stride : v_stride, cache->kv_heads, T,
                       cache->head_dim, rot_dim, interleaved, 0, fn)))
    return st;
  if (T && (k_stride > kMaxNumel / T || v_stride > kMaxNumel / T))
    return fail(QLORA_ERR_INVALID_ARG, "%s: T * stride must be below 2^37", fn);
  if (T == 0) return QLORA_OK;
  if ((st = check_buffers(cache, fn))) return st;
  if (q_heads && ((st = check_ptr(q, "q", fn)) || (st = check_ptr(qo, "qo", fn)))) return st;
  if ((st = check_ptr(k, "k", fn)) || (st = check_ptr(v, "v", fn)) || (st = check_ptr(slots, "slots", fn, 4)))
    return st;
  if (rot_dim && ((st = check_ptr(positions, "positions", fn, 4)) || (st = check_ptr(turns, "turns", fn)))) return st;
  if (q_heads && q == qo && q_stride != qo_stride)
    return fail(QLORA_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  RopeArgs a = {};
  if (q_heads) a.q = q, a.qo = qo, a.q_stride = q_stride, a.qo_stride = qo_stride, a.q_heads = q_heads;
  a.k = k, a.k_stride = k_stride, a.v = v, a.v_stride = v_stride, a.kv_heads = cache->kv_heads;
  a.positions = positions, a.turns = turns, a.slots = slots, a.T = T;
  a.k_cache = cache->k, a.v_cache = cache->v, a.num_slots = cache->num_pages * cache->page_size;
  a.page_shift = shift_of(cache->page_size);
  a.head_dim = cache->head_dim, a.rot_dim = rot_dim, a.mscale = mscale;
  a.interleaved = interleaved != 0;
  return finish(launch_kv_write(a, cache->k_scale, cache->v_scale, cache->type, (hipStream_t)stream), fn);
}

int qlora_kv_read(const qlora_kv_cache* cache, const int32_t* slots, int64_t T, int32_t dtype, void* k, void* v,
                  void* stream) {
  static const char* fn = "qlora_kv_read";
  int st;
  if ((st = check_descriptor(cache, fn))) return st;
  if (dtype != QLORA_DTYPE_F32 && dtype != QLORA_DTYPE_BF16)
    return fail(QLORA_ERR_UNSUPPORTED_DTYPE, "%s: dtype must be F32 or BF16", fn);
  if (T < 0 || T >= (1 << 24)) return fail(QLORA_ERR_INVALID_ARG, "%s: T must be in [0, 2^24)", fn);
  if (T > kMaxNumel / ((int64_t)cache->kv_heads * cache->head_dim))
    return fail(QLORA_ERR_INVALID_ARG, "%s: T rows must be below 2^37 elements", fn);
  if (T == 0 || (!k && !v)) return QLORA_OK;
  if ((st = check_buffers(cache, fn)) || (st = check_ptr(slots, "slots", fn, 4)) || (st = check_opt(k, "k", fn)) ||
      (st = check_opt(v, "v", fn)))
    return st;
  KvReadArgs a = {};
  a.c = rows_of(cache);
  a.slots = slots, a.k = k, a.v = v, a.T = T, a.num_slots = cache->num_pages * cache->page_size;
  return finish(launch_kv_read(a, dtype == QLORA_DTYPE_F32, (hipStream_t)stream), fn);
}

int qlora_kv_attention_workspace(const qlora_kv_cache* cache, int64_t S, int32_t q_heads, int64_t table_cols,
                                 int64_t* ws_bytes) {
  static const char* fn = "qlora_kv_attention_workspace";
  int st;
  if ((st = check_attention(cache, S, q_heads, 0, table_cols, fn))) return st;
  if (!ws_bytes) return fail(QLORA_ERR_INVALID_ARG, "%s: ws_bytes is NULL", fn);
  *ws_bytes = attention_ws(cache, S, q_heads, kv_parts(rows_of(cache), S, q_heads, table_cols, 0));
  return QLORA_OK;
}

int qlora_kv_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, const qlora_kv_cache* cache,
                       const int32_t* table, int64_t table_cols, const int32_t* lengths, float scale, void* out,
                       float* lse, void* ws, int64_t ws_bytes, void* stream) {
  static const char* fn = "qlora_kv_attention";
  int st;
  if ((st = check_attention(cache, S, q_heads, 0, table_cols, fn))) return st;
  return attend(q, q_stride, S, q_heads, cache, nullptr, 0, nullptr, table, table_cols, lengths, scale, out, lse, ws,
                ws_bytes, stream, fn);
}

int qlora_prefix_attention_workspace(const qlora_kv_cache* cache, int64_t S, int32_t q_heads, int64_t prefix_cols,
                                     int64_t table_cols, int64_t* ws_bytes) {
  static const char* fn = "qlora_prefix_attention_workspace";
  int st;
  if ((st = check_attention(cache, S, q_heads, prefix_cols, table_cols, fn))) return st;
  if (!ws_bytes) return fail(QLORA_ERR_INVALID_ARG, "%s: ws_bytes is NULL", fn);
  *ws_bytes = attention_ws(cache, S, q_heads, kv_parts(rows_of(cache), S, q_heads, table_cols, prefix_cols));
  return QLORA_OK;
}

int qlora_prefix_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, const qlora_kv_cache* cache,
                           const int32_t* prefix_table, int64_t prefix_cols, const int32_t* prefix_len,
                           const int32_t* table, int64_t table_cols, const int32_t* lengths, float scale, void* out,
                           float* lse, void* ws, int64_t ws_bytes, void* stream) {
  static const char* fn = "qlora_prefix_attention";
  int st;
  if ((st = check_attention(cache, S, q_heads, prefix_cols, table_cols, fn))) return st;
  if (S && ((st = check_ptr(prefix_len, "prefix_len", fn, 4)) ||
            (prefix_cols && (st = check_ptr(prefix_table, "prefix_table", fn, 4)))))
    return st;
  return attend(q, q_stride, S, q_heads, cache, prefix_table, prefix_cols, prefix_len, table, table_cols, lengths,
                scale, out, lse, ws, ws_bytes, stream, fn);
}

}  // extern "C"
