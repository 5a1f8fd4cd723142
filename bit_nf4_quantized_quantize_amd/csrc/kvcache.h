// Internal launchers of the 8-bit and the shared key-value cache
// (kv_write.hip, kv_attention.hip, kv_prefix.hip), shared with kv_abi.cpp.
// Every launcher only enqueues on `stream` and returns the launch status;
// arguments were checked before.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder.h"

namespace qlora {

// The cache's rows; type as in include/qlora_kvcache.h.
struct KvCache {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t num_pages;
  int kv_heads, head_dim, page_shift, type;
};
enum { kCacheBf16 = 0, kCacheInt8 = 1, kCacheE4m3 = 2 };

// Tokens entering an 8-bit cache: a.k_cache and a.v_cache are codes.
hipError_t launch_kv_write(const RopeArgs& a, float* k_scale, float* v_scale, int type, hipStream_t stream);

struct KvReadArgs {
  KvCache c;
  const int32_t* slots;
  void* k;  // or NULL
  void* v;  // or NULL
  int64_t T, num_slots;
};
hipError_t launch_kv_read(const KvReadArgs& a, bool f32, hipStream_t stream);

// Attention of one token per sequence: over its own tokens in at most `splits`
// parts, and over the tokens that all sequences share in at most `psplits`
// (0: there are none).  With more than one part in all, parts go to part_o and
// part_ml (the shared ones first) and are joined.
struct KvAttnArgs {
  KvCache c;
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* prefix_table;
  const int32_t* prefix_len;
  uint16_t* out;
  float* lse;
  float* part_o;   // [S][q_heads][psplits + splits][head_dim]
  float* part_ml;  // [S][q_heads][psplits + splits][2]: maximum (base-2 scores) and sum
  int64_t q_stride, S, table_cols, prefix_cols;
  int q_heads, splits, psplits;
  int waves, pwaves;  // per workgroup, set by the launcher
  int wide;           // rows of a wide workgroup for the prefix, 0: narrow ones; set by the launcher
  bool joined;        // the own tokens' workgroups join the prefix's parts; set by the launcher
  float scale;
};
// The parts of a call without and with a shared prefix.
struct KvParts {
  int own, prefix;
};
KvParts kv_parts(const KvCache& c, int64_t S, int q_heads, int64_t table_cols, int64_t prefix_cols);
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream);
// The prefix's part for many rows, called by it.
hipError_t launch_kv_prefix(const KvAttnArgs& a, hipStream_t stream);

}  // namespace qlora
