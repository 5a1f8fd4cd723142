// Argument checks that the ABI files of the decoder operators share (host only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "launch.h"
#include "qlora_nf4.h"

namespace qlora {

inline int fail(int status, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return record_failure(status, msg);
}

inline int finish(hipError_t e, const char* fn) {
  return e == hipSuccess ? QLORA_OK : fail(QLORA_ERR_HIP, "%s: %s", fn, hipGetErrorString(e));
}

constexpr int64_t kMaxNumel = (int64_t)1 << 37;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int kMaxHeads = 4096;

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// A tensor pointer that must be there, on a 16-byte boundary; the int32 arrays
// need no more than their own.
inline int check_ptr(const void* p, const char* name, const char* fn, uintptr_t to = 16) {
  if (!p) return fail(QLORA_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  if (!aligned(p, to)) return fail(QLORA_ERR_MISALIGNED, "%s: %s not %d-byte aligned", fn, name, (int)to);
  return QLORA_OK;
}
inline int check_opt(const void* p, const char* name, const char* fn) {
  return p ? check_ptr(p, name, fn) : QLORA_OK;
}

// Sizes and strides of a rotary call.
inline int check_rope(int64_t q_stride, int32_t q_heads, int64_t qo_stride, int64_t k_stride, int32_t kv_heads, int64_t T,
               int32_t head_dim, int32_t rot_dim, int32_t interleaved, int32_t inverse, const char* fn) {
  // a workgroup of 256 threads per token at most: a grid holds 2^32 - 1 threads
  if (T < 0 || T >= (1 << 24)) return fail(QLORA_ERR_INVALID_ARG, "%s: T must be in [0, 2^24)", fn);
  if (head_dim < 1 || head_dim > 1024) return fail(QLORA_ERR_INVALID_ARG, "%s: head_dim must be in [1, 1024]", fn);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2)
    return fail(QLORA_ERR_INVALID_ARG, "%s: rot_dim must be even and in [0, head_dim]", fn);
  if (q_heads < 0 || q_heads > kMaxHeads || kv_heads < 0 || kv_heads > kMaxHeads)
    return fail(QLORA_ERR_INVALID_ARG, "%s: head counts must be in [0, %d]", fn, kMaxHeads);
  if (interleaved != 0 && interleaved != 1)
    return fail(QLORA_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", fn);
  if (inverse != 0 && inverse != 1) return fail(QLORA_ERR_INVALID_ARG, "%s: inverse must be 0 or 1", fn);
  const int64_t qw = (int64_t)q_heads * head_dim, kw = (int64_t)kv_heads * head_dim;
  if (q_heads && (q_stride < qw || qo_stride < qw))
    return fail(QLORA_ERR_INVALID_ARG, "%s: q strides must be at least q_heads * head_dim", fn);
  if (kv_heads && k_stride < kw)
    return fail(QLORA_ERR_INVALID_ARG, "%s: k strides must be at least kv_heads * head_dim", fn);
  const int64_t most = q_heads ? (q_stride > qo_stride ? q_stride : qo_stride) : 0;
  if (T && (most > kMaxNumel / T || (kv_heads && k_stride > kMaxNumel / T)))
    return fail(QLORA_ERR_INVALID_ARG, "%s: T * stride must be below 2^37", fn);
  return QLORA_OK;
}

// Floor of log2 of a power of two, or -1.
inline int shift_of(int32_t v) {
  for (int s = 0; s <= 10; ++s)
    if (v == 1 << s) return s;
  return -1;
}

}  // namespace qlora
