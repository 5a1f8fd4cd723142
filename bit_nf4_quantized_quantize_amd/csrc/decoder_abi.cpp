// C ABI of the decoder-block operators: argument validation (host only,
// before any launch), workspace sizes and dispatch.  See
// include/qlora_decoder.h for the contract of each entry point.
#include "qlora_decoder.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "abi_checks.h"
#include "decoder.h"

using namespace qlora;

namespace {

int check_dtypes(int32_t x, int32_t h, const char* fn) {
  const bool fx = x == QLORA_DTYPE_F32, bx = x == QLORA_DTYPE_BF16;
  const bool fh = h == QLORA_DTYPE_F32, bh = h == QLORA_DTYPE_BF16;
  if ((fx && (fh || bh)) || (bx && bh)) return QLORA_OK;
  return fail(QLORA_ERR_UNSUPPORTED_DTYPE, "%s: x_dtype and h_dtype must be F32 and F32, F32 and BF16, or BF16 and "
              "BF16", fn);
}

int check_rows(int64_t T, int64_t D, float eps, const char* fn) {
  if (T < 0 || T > kMaxRows) return fail(QLORA_ERR_INVALID_ARG, "%s: T must be in [0, 2^31)", fn);
  if (D < 1 || D > QLORA_NORM_MAX_WIDTH)
    return fail(QLORA_ERR_INVALID_ARG, "%s: D must be in [1, %d]", fn, QLORA_NORM_MAX_WIDTH);
  if (T > kMaxNumel / D) return fail(QLORA_ERR_INVALID_ARG, "%s: T * D must be below 2^37", fn);
  if (!(eps >= 0.0f) || isinf(eps)) return fail(QLORA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  return QLORA_OK;
}

int64_t norm_ws(int64_t T, int64_t D) { return T == 0 ? 0 : 2 * norm_bwd_parts(T, D) * D * 4; }

int check_cache(const void* k_cache, const void* v_cache, int64_t num_pages, int32_t page_size, int32_t kv_heads,
                int32_t head_dim, const char* fn) {
  if (num_pages < 1 || num_pages > kMaxRows || num_pages * page_size > kMaxRows)
    return fail(QLORA_ERR_INVALID_ARG, "%s: need num_pages >= 1 and num_pages * page_size < 2^31", fn);
  if (num_pages * page_size > kMaxNumel / ((int64_t)kv_heads * head_dim))
    return fail(QLORA_ERR_INVALID_ARG, "%s: the cache must be below 2^37 elements", fn);
  int st;
  if ((st = check_ptr(k_cache, "k_cache", fn)) || (st = check_ptr(v_cache, "v_cache", fn))) return st;
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_norm_residual_fwd(const void* x, int32_t x_dtype, const void* h, int32_t h_dtype, int64_t T, int64_t D,
                            const float* w_post, const float* gate, float alpha, const float* w_pre, float eps,
                            void* xo, void* n, void* stream) {
  static const char* fn = "qlora_norm_residual_fwd";
  int st;
  if ((st = check_dtypes(x_dtype, h_dtype, fn)) || (st = check_rows(T, D, eps, fn))) return st;
  if (T == 0) return QLORA_OK;
  if (!xo && !n) return fail(QLORA_ERR_INVALID_ARG, "%s: xo or n must be given", fn);
  if (n && !w_pre) return fail(QLORA_ERR_INVALID_ARG, "%s: n needs w_pre", fn);
  if (!h && (w_post || gate)) return fail(QLORA_ERR_INVALID_ARG, "%s: w_post and gate need h", fn);
  if ((st = check_ptr(x, "x", fn)) || (st = check_opt(h, "h", fn)) || (st = check_opt(w_post, "w_post", fn)) ||
      (st = check_opt(gate, "gate", fn)) || (st = check_opt(w_pre, "w_pre", fn)) || (st = check_opt(xo, "xo", fn)) ||
      (st = check_opt(n, "n", fn)))
    return st;
  NormArgs a = {};
  a.x = x, a.h = h, a.xo = xo, a.n = n;
  a.w_post = w_post, a.gate = gate, a.w_pre = w_pre;
  a.T = T, a.D = (int)D, a.alpha = alpha, a.eps = eps;
  return finish(launch_norm_fwd(a, x_dtype == QLORA_DTYPE_F32, h_dtype == QLORA_DTYPE_F32, (hipStream_t)stream), fn);
}

int qlora_norm_residual_bwd_workspace(int64_t T, int64_t D, int32_t x_dtype, int32_t h_dtype, int32_t sums,
                                      int64_t* ws_bytes) {
  static const char* fn = "qlora_norm_residual_bwd_workspace";
  int st;
  if ((st = check_dtypes(x_dtype, h_dtype, fn)) || (st = check_rows(T, D, 0.0f, fn))) return st;
  if (sums < 0 || sums > 3) return fail(QLORA_ERR_INVALID_ARG, "%s: sums must be in [0, 3]", fn);
  if (!ws_bytes) return fail(QLORA_ERR_INVALID_ARG, "%s: ws_bytes is NULL", fn);
  *ws_bytes = sums ? norm_ws(T, D) : 0;
  return QLORA_OK;
}

int qlora_norm_residual_bwd(const void* dxo, const void* xo, int32_t x_dtype, const void* dn, const void* h,
                            int32_t h_dtype, int64_t T, int64_t D, const float* w_post, const float* gate,
                            float alpha, const float* w_pre, float eps, void* dx, void* dh, float* dw_post,
                            float* dgate, float* dw_pre, void* ws, int64_t ws_bytes, void* stream) {
  static const char* fn = "qlora_norm_residual_bwd";
  int st;
  if ((st = check_dtypes(x_dtype, h_dtype, fn)) || (st = check_rows(T, D, eps, fn))) return st;
  if (dw_post && !w_post) return fail(QLORA_ERR_INVALID_ARG, "%s: dw_post needs w_post", fn);
  if (T > 0 && dw_pre && !dn) return fail(QLORA_ERR_INVALID_ARG, "%s: dw_pre needs dn", fn);
  if (T > 0 && dn && !w_pre) return fail(QLORA_ERR_INVALID_ARG, "%s: dn needs w_pre", fn);
  if (T > 0 && !h && (w_post || dgate)) return fail(QLORA_ERR_INVALID_ARG, "%s: w_post and dgate need h", fn);
  const bool sums = dw_post || dgate || dw_pre;
  if ((st = check_opt(dw_post, "dw_post", fn)) || (st = check_opt(dgate, "dgate", fn)) ||
      (st = check_opt(dw_pre, "dw_pre", fn)))
    return st;
  if (T == 0 && !sums) return QLORA_OK;
  NormArgs a = {};
  if (T > 0) {
    if ((st = check_ptr(xo, "xo", fn)) || (st = check_ptr(dx, "dx", fn)) || (st = check_opt(dxo, "dxo", fn)) ||
        (st = check_opt(dn, "dn", fn)) || (st = check_opt(h, "h", fn)) || (st = check_opt(dh, "dh", fn)) ||
        (st = check_opt(w_post, "w_post", fn)) || (st = check_opt(gate, "gate", fn)) ||
        (st = check_opt(w_pre, "w_pre", fn)))
      return st;
    if (sums) {
      const int64_t need = norm_ws(T, D);
      if (ws_bytes < need)
        return fail(QLORA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %lld bytes", fn, (long long)need);
      if ((st = check_ptr(ws, "ws", fn))) return st;
    }
  }
  a.x = xo, a.h = h, a.dxo = dxo, a.dn = dn, a.xo = dx, a.n = dh;
  a.w_post = w_post, a.gate = gate, a.w_pre = w_pre;
  a.part = (float*)ws, a.dw_post = dw_post, a.dgate = dgate, a.dw_pre = dw_pre;
  a.T = T, a.D = (int)D, a.alpha = alpha, a.eps = eps;
  return finish(launch_norm_bwd(a, x_dtype == QLORA_DTYPE_F32, h_dtype == QLORA_DTYPE_F32, (hipStream_t)stream), fn);
}

int qlora_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, double original_len,
                           double beta_fast, double beta_slow, double* turns, float* mscale) {
  static const char* fn = "qlora_rope_frequencies";
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2)
    return fail(QLORA_ERR_INVALID_ARG, "%s: rot_dim must be even and in [2, 1024]", fn);
  if (!(base > 1.0) || isinf(base)) return fail(QLORA_ERR_INVALID_ARG, "%s: base must be finite and > 1", fn);
  if (scaling < QLORA_ROPE_NONE || scaling > QLORA_ROPE_YARN)
    return fail(QLORA_ERR_INVALID_ARG, "%s: scaling must be one of the qlora_rope_scaling values", fn);
  if (!(factor >= 1.0) || isinf(factor))
    return fail(QLORA_ERR_INVALID_ARG, "%s: factor must be finite and >= 1", fn);
  if (scaling == QLORA_ROPE_NTK && rot_dim < 4)
    return fail(QLORA_ERR_INVALID_ARG, "%s: NTK scaling needs rot_dim >= 4", fn);
  if (scaling == QLORA_ROPE_YARN &&
      (!(original_len >= 1.0) || isinf(original_len) || !(beta_slow >= 0.0) || !(beta_fast > beta_slow) ||
       isinf(beta_fast)))
    return fail(QLORA_ERR_INVALID_ARG, "%s: YARN scaling needs original_len >= 1 and beta_fast > beta_slow >= 0", fn);
  if (!turns || !mscale) return fail(QLORA_ERR_INVALID_ARG, "%s: turns and mscale must be given", fn);
  const double two_pi = 6.283185307179586476925;
  if (scaling == QLORA_ROPE_NTK) base *= pow(factor, rot_dim / (rot_dim - 2.0));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == QLORA_ROPE_LINEAR) f /= factor;
    if (scaling == QLORA_ROPE_YARN) {
      double g = (original_len * f / two_pi - beta_slow) / (beta_fast - beta_slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = f / factor * (1.0 - g) + f * g;
    }
    turns[i] = f / two_pi;
  }
  *mscale = scaling == QLORA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return QLORA_OK;
}

int qlora_rope(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride, const void* k,
               int64_t k_stride, int32_t kv_heads, void* ko, int64_t ko_stride, int64_t T, int32_t head_dim,
               int32_t rot_dim, int32_t dtype, const int32_t* positions, const double* turns, float mscale,
               int32_t interleaved, int32_t inverse, void* stream) {
  static const char* fn = "qlora_rope";
  int st;
  if (dtype != QLORA_DTYPE_F32 && dtype != QLORA_DTYPE_BF16)
    return fail(QLORA_ERR_UNSUPPORTED_DTYPE, "%s: dtype must be F32 or BF16", fn);
  if ((st = check_rope(q_stride, q_heads, qo_stride, k_stride < ko_stride ? k_stride : ko_stride, kv_heads, T,
                       head_dim, rot_dim, interleaved, inverse, fn)))
    return st;
  if (T && kv_heads && (k_stride > kMaxNumel / T || ko_stride > kMaxNumel / T))
    return fail(QLORA_ERR_INVALID_ARG, "%s: T * stride must be below 2^37", fn);
  if (T == 0 || q_heads + kv_heads == 0) return QLORA_OK;
  if (q_heads && ((st = check_ptr(q, "q", fn)) || (st = check_ptr(qo, "qo", fn)))) return st;
  if (kv_heads && ((st = check_ptr(k, "k", fn)) || (st = check_ptr(ko, "ko", fn)))) return st;
  if (rot_dim && ((st = check_ptr(positions, "positions", fn, 4)) || (st = check_ptr(turns, "turns", fn)))) return st;
  if ((q_heads && q == qo && q_stride != qo_stride) || (kv_heads && k == ko && k_stride != ko_stride))
    return fail(QLORA_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  RopeArgs a = {};
  if (q_heads) a.q = q, a.qo = qo, a.q_stride = q_stride, a.qo_stride = qo_stride, a.q_heads = q_heads;
  if (kv_heads) a.k = k, a.ko = ko, a.k_stride = k_stride, a.ko_stride = ko_stride, a.kv_heads = kv_heads;
  a.positions = positions, a.turns = turns, a.T = T;
  a.head_dim = head_dim, a.rot_dim = rot_dim, a.mscale = mscale;
  a.interleaved = interleaved != 0, a.inverse = inverse != 0;
  return finish(launch_rope(a, dtype == QLORA_DTYPE_F32, (hipStream_t)stream), fn);
}

int qlora_rope_cache_write(const void* q, int64_t q_stride, int32_t q_heads, void* qo, int64_t qo_stride,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t kv_heads,
                           int64_t T, int32_t head_dim, int32_t rot_dim, const int32_t* positions,
                           const double* turns, float mscale, int32_t interleaved, const int32_t* slots,
                           void* k_cache, void* v_cache, int64_t num_pages, int32_t page_size, void* stream) {
  static const char* fn = "qlora_rope_cache_write";
  int st;
  if ((st = check_rope(q_stride, q_heads, qo_stride, k_stride < v_stride ? k_stride : v_stride, kv_heads, T, head_dim,
                       rot_dim, interleaved, 0, fn)))
    return st;
  if (kv_heads < 1) return fail(QLORA_ERR_INVALID_ARG, "%s: kv_heads must be at least 1", fn);
  if (T && (k_stride > kMaxNumel / T || v_stride > kMaxNumel / T))
    return fail(QLORA_ERR_INVALID_ARG, "%s: T * stride must be below 2^37", fn);
  const int shift = shift_of(page_size);
  if (shift < 0) return fail(QLORA_ERR_INVALID_ARG, "%s: page_size must be a power of two in [1, 1024]", fn);
  if (T == 0) return QLORA_OK;
  if ((st = check_cache(k_cache, v_cache, num_pages, page_size, kv_heads, head_dim, fn))) return st;
  if (q_heads && ((st = check_ptr(q, "q", fn)) || (st = check_ptr(qo, "qo", fn)))) return st;
  if ((st = check_ptr(k, "k", fn)) || (st = check_ptr(v, "v", fn)) || (st = check_ptr(slots, "slots", fn, 4)))
    return st;
  if (rot_dim && ((st = check_ptr(positions, "positions", fn, 4)) || (st = check_ptr(turns, "turns", fn)))) return st;
  if (q_heads && q == qo && q_stride != qo_stride)
    return fail(QLORA_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  RopeArgs a = {};
  if (q_heads) a.q = q, a.qo = qo, a.q_stride = q_stride, a.qo_stride = qo_stride, a.q_heads = q_heads;
  a.k = k, a.k_stride = k_stride, a.v = v, a.v_stride = v_stride, a.kv_heads = kv_heads;
  a.positions = positions, a.turns = turns, a.slots = slots, a.T = T;
  a.k_cache = k_cache, a.v_cache = v_cache, a.num_slots = num_pages * page_size, a.page_shift = shift;
  a.head_dim = head_dim, a.rot_dim = rot_dim, a.mscale = mscale;
  a.interleaved = interleaved != 0;
  return finish(launch_rope(a, false, (hipStream_t)stream), fn);
}

int qlora_paged_plan(const int32_t* cached_lens, const int32_t* new_lens, int64_t S, int32_t page_size,
                     const int32_t* free_pages, int64_t n_free, int32_t* table, int64_t table_cols, int64_t T,
                     int32_t* total_lens, int32_t* starts, int32_t* slots, int32_t* positions, int32_t* pages_needed,
                     void* stream) {
  static const char* fn = "qlora_paged_plan";
  int st;
  if (S < 0 || S > QLORA_PLAN_MAX_SEQS)
    return fail(QLORA_ERR_INVALID_ARG, "%s: S must be in [0, %d]", fn, QLORA_PLAN_MAX_SEQS);
  if (page_size < 1) return fail(QLORA_ERR_INVALID_ARG, "%s: page_size must be at least 1", fn);
  if (n_free < 0 || n_free > kMaxRows || table_cols < 0 || table_cols > kMaxRows || T < 0 || T > kMaxRows)
    return fail(QLORA_ERR_INVALID_ARG, "%s: n_free, table_cols and T must be in [0, 2^31)", fn);
  if ((st = check_ptr(starts, "starts", fn, 4)) || (st = check_ptr(pages_needed, "pages_needed", fn, 4))) return st;
  if (S && ((st = check_ptr(cached_lens, "cached_lens", fn, 4)) || (st = check_ptr(new_lens, "new_lens", fn, 4)) ||
            (st = check_ptr(total_lens, "total_lens", fn, 4))))
    return st;
  if (S && table_cols && (st = check_ptr(table, "table", fn, 4))) return st;
  if (n_free && (st = check_ptr(free_pages, "free_pages", fn, 4))) return st;
  if (S && (total_lens == cached_lens || total_lens == new_lens))
    return fail(QLORA_ERR_INVALID_ARG, "%s: total_lens must not be cached_lens or new_lens", fn);
  if (T && ((st = check_ptr(slots, "slots", fn, 4)) || (st = check_ptr(positions, "positions", fn, 4)))) return st;
  PlanArgs a = {};
  a.cached = cached_lens, a.fresh = new_lens, a.free_pages = free_pages, a.table = table;
  a.total = total_lens, a.starts = starts, a.slots = slots, a.positions = positions, a.pages_needed = pages_needed;
  a.n_free = n_free, a.table_cols = table_cols, a.T = T, a.S = (int)S, a.page_size = page_size;
  return finish(launch_paged_plan(a, (hipStream_t)stream), fn);
}

static int check_attention(int64_t S, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t table_cols,
                           int32_t page_size, const char* fn) {
  if (S < 0 || S > 65535) return fail(QLORA_ERR_INVALID_ARG, "%s: S must be in [0, 65535]", fn);
  if (kv_heads < 1 || q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads)
    return fail(QLORA_ERR_INVALID_ARG, "%s: q_heads must be a multiple of kv_heads in [1, %d]", fn, kMaxHeads);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(QLORA_ERR_INVALID_ARG, "%s: head_dim must be a multiple of 8 in [8, 256]", fn);
  if (shift_of(page_size) < 4)
    return fail(QLORA_ERR_INVALID_ARG, "%s: page_size must be a power of two in [16, 1024]", fn);
  if (table_cols < 0 || table_cols > kMaxRows || table_cols * page_size > kMaxRows)
    return fail(QLORA_ERR_INVALID_ARG, "%s: table_cols * page_size must be in [0, 2^31)", fn);
  return QLORA_OK;
}

int qlora_paged_attention_workspace(int64_t S, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                    int64_t table_cols, int32_t page_size, int64_t* ws_bytes) {
  static const char* fn = "qlora_paged_attention_workspace";
  int st;
  if ((st = check_attention(S, q_heads, kv_heads, head_dim, table_cols, page_size, fn))) return st;
  if (!ws_bytes) return fail(QLORA_ERR_INVALID_ARG, "%s: ws_bytes is NULL", fn);
  const int splits = paged_splits(S, q_heads, kv_heads, head_dim, table_cols * page_size);
  *ws_bytes = splits > 1 ? S * q_heads * splits * (int64_t)(head_dim + 2) * 4 : 0;
  return QLORA_OK;
}

int qlora_paged_attention(const void* q, int64_t q_stride, int64_t S, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const void* k_cache, const void* v_cache, int64_t num_pages,
                          int32_t page_size, const int32_t* table, int64_t table_cols, const int32_t* lengths,
                          float scale, void* out, float* lse, void* ws, int64_t ws_bytes, void* stream) {
  static const char* fn = "qlora_paged_attention";
  int st;
  if ((st = check_attention(S, q_heads, kv_heads, head_dim, table_cols, page_size, fn))) return st;
  if (!isfinite(scale)) return fail(QLORA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
  if (q_stride < (int64_t)q_heads * head_dim || q_stride % 8 || (S && q_stride > kMaxNumel / S))
    return fail(QLORA_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 8, at least q_heads * head_dim", fn);
  if (S == 0) return QLORA_OK;
  if ((st = check_cache(k_cache, v_cache, num_pages, page_size, kv_heads, head_dim, fn))) return st;
  if ((st = check_ptr(q, "q", fn)) || (st = check_ptr(out, "out", fn)) ||
      (st = check_ptr(lengths, "lengths", fn, 4)) || (table_cols && (st = check_ptr(table, "table", fn, 4))) ||
      (lse && (st = check_ptr(lse, "lse", fn, 4))))
    return st;
  AttnArgs a = {};
  a.splits = paged_splits(S, q_heads, kv_heads, head_dim, table_cols * page_size);
  if (a.splits > 1) {
    const int64_t rows = S * q_heads * a.splits, need = rows * (int64_t)(head_dim + 2) * 4;
    if (ws_bytes < need)
      return fail(QLORA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %lld bytes", fn, (long long)need);
    if ((st = check_ptr(ws, "ws", fn))) return st;
    a.part_o = (float*)ws, a.part_ml = (float*)ws + rows * head_dim;
  }
  a.q = (const uint16_t*)q, a.k_cache = (const uint16_t*)k_cache, a.v_cache = (const uint16_t*)v_cache;
  a.table = table, a.lengths = lengths, a.out = (uint16_t*)out, a.lse = lse;
  a.q_stride = q_stride, a.S = S, a.num_pages = num_pages, a.table_cols = table_cols;
  a.q_heads = q_heads, a.kv_heads = kv_heads, a.head_dim = head_dim, a.page_shift = shift_of(page_size);
  a.scale = scale;
  return finish(launch_paged_attention(a, (hipStream_t)stream), fn);
}

}  // extern "C"
