// The host logic of the 8-bit and the shared key-value cache on the CPU: the
// launchers are stand-ins that check the workspace regions they are handed.
// Driven over ordinary and extreme sizes; prints "ok" and the number of launches
// seen.
#include <stdio.h>

#include <string>

#include "kvcache.h"
#include "qlora_kvcache.h"

static int g_launches = 0, g_bad = 0;
static uintptr_t g_lo = 0, g_hi = 0;
static std::string g_err;

static void inside(const void* p, int64_t bytes, const char* what) {
  if ((uintptr_t)p < g_lo || (uintptr_t)p + (uintptr_t)bytes > g_hi) {
    ++g_bad;
    fprintf(stderr, "%s leaves the workspace\n", what);
  }
}

namespace qlora {
int record_failure(int status, const char* msg) {
  g_err = msg;
  return status;
}
int64_t norm_bwd_parts(int64_t T, int64_t) { return T; }
int paged_splits(int64_t, int, int, int, int64_t) { return 1; }
hipError_t launch_norm_fwd(const NormArgs&, bool, bool, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_bwd(const NormArgs&, bool, bool, hipStream_t) { return hipSuccess; }
hipError_t launch_rope(const RopeArgs&, bool, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_paged_plan(const PlanArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_paged_attention(const AttnArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_write(const RopeArgs& a, float* ks, float* vs, int type, hipStream_t) {
  ++g_launches;
  if (a.T <= 0 || a.T >= 1 << 24 || a.head_dim % 16 || a.head_dim > 256 || a.rot_dim > a.head_dim || !ks || !vs ||
      (type != kCacheInt8 && type != kCacheE4m3))
    ++g_bad;
  return hipSuccess;
}
hipError_t launch_kv_read(const KvReadArgs& a, bool, hipStream_t) {
  ++g_launches;
  if (a.T <= 0 || a.T >= 1 << 24 || (!a.k && !a.v) || a.num_slots <= 0 || a.num_slots > INT32_MAX) ++g_bad;
  return hipSuccess;
}
KvParts kv_parts(const KvCache& c, int64_t S, int q_heads, int64_t table_cols, int64_t prefix_cols) {
  if (c.head_dim < 1 || c.kv_heads < 1 || q_heads % c.kv_heads || table_cols < 0 || prefix_cols < 0) ++g_bad;
  return {S && table_cols > 32 ? 7 : 1, S && prefix_cols ? 128 : 0};
}
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t) {
  ++g_launches;
  const int64_t parts = a.splits + a.psplits, rows = a.S * a.q_heads * parts;
  if (parts > 1) inside(a.part_o, rows * a.c.head_dim * 4, "partial outputs"), inside(a.part_ml, rows * 8, "partial sums");
  if (a.psplits && (!a.prefix_table || !a.prefix_len)) ++g_bad;
  return hipSuccess;
}
}  // namespace qlora

int main() {
  char* P = (char*)0x100000;  // never dereferenced
  const int64_t big[] = {-1, 0, 1, 2, 63, 64, 4096, 65535, 65536, (1ll << 24) - 1, 1ll << 24, (1ll << 31) - 1,
                         1ll << 31, 1ll << 37, 1ll << 62, INT64_MAX, INT64_MIN};
  const int32_t some[] = {INT32_MIN, -1, 0, 1, 2, 8, 16, 64, 80, 256, 272, 4096, 4097, INT32_MAX};
  for (int32_t type : {-1, 0, 1, 2, 3})
    for (int64_t pages : big)
      for (int32_t page : {0, 1, 8, 16, 1024, 2048})
        for (int32_t KV : some)
          for (int32_t d : some) {
            qlora_kv_cache c = {P, P, (float*)P, (float*)P, pages, page, KV, d, type};
            if (type == 0) c.k_scale = c.v_scale = nullptr;
            for (int64_t T : {(int64_t)0, (int64_t)1, (int64_t)4096, (int64_t)(1 << 24) - 1, (int64_t)INT64_MAX}) {
              const int64_t st = (int64_t)KV * d;
              qlora_kv_write(P, st, KV, P, st, P, st, P, st, T, 0, nullptr, nullptr, 1, 0, (int32_t*)P, &c, nullptr);
              qlora_kv_write(nullptr, 0, 0, nullptr, 0, P, T, P, T, T, d, (int32_t*)P, (double*)P, 1, 1, (int32_t*)P, &c,
                             nullptr);
              qlora_kv_read(&c, (int32_t*)P, T, 0, P, nullptr, nullptr);
            }
          }
  for (int32_t type : {0, 1, 2})
    for (int64_t S : big)
      for (int64_t cols : big)
        for (int64_t pcols : big)
          for (int32_t H : some)
            for (int32_t KV : {1, 8, 4096})
              for (int32_t d : {16, 64, 256}) {
                qlora_kv_cache c = {P, P, (float*)P, (float*)P, 1024, 16, KV, d, type};
                if (type == 0) c.k_scale = c.v_scale = nullptr;
                int64_t n = -1;
                if (qlora_prefix_attention_workspace(&c, S, H, pcols, cols, &n)) n = 0;
                if (n < 0) ++g_bad;
                g_lo = 0x40000000, g_hi = g_lo + (uintptr_t)n;
                qlora_prefix_attention(P, (int64_t)H * d, S, H, &c, (int32_t*)P, pcols, (int32_t*)P, (int32_t*)P, cols,
                                       (int32_t*)P, 1, P, (float*)P, (void*)g_lo, n, nullptr);
                if (qlora_kv_attention_workspace(&c, S, H, cols, &n)) n = 0;
                g_hi = g_lo + (uintptr_t)n;
                qlora_kv_attention(P, (int64_t)H * d, S, H, &c, (int32_t*)P, cols, (int32_t*)P, 1, P, (float*)P,
                                   (void*)g_lo, n, nullptr);
              }
  if (g_bad) return 1;
  printf("ok %d\n", g_launches);
  return 0;
}
