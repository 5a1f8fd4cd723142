// The decoder-block entry points' host logic on the CPU: abi.cpp is replaced by
// its one function used here, the launchers by stand-ins that check the
// workspace regions they are handed.  Driven over ordinary and extreme sizes;
// prints "ok" and the number of launches seen.
#include <stdio.h>
#include <string.h>

#include <string>

#include "decoder.h"
#include "qlora_decoder.h"

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
int64_t norm_bwd_parts(int64_t T, int64_t) { return T < 512 ? T : 512; }
int paged_splits(int64_t S, int, int kv, int, int64_t len) { return S > 0 && len > 512 && S * kv < 256 ? (int)(256 / (S * kv)) : 1; }
hipError_t launch_norm_fwd(const NormArgs&, bool, bool, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_norm_bwd(const NormArgs& a, bool, bool, hipStream_t) {
  ++g_launches;
  if (a.T && (a.dw_post || a.dgate || a.dw_pre)) inside(a.part, 2 * norm_bwd_parts(a.T, a.D) * a.D * 4, "norm partials");
  return hipSuccess;
}
hipError_t launch_rope(const RopeArgs& a, bool, hipStream_t) {
  ++g_launches;
  if (a.T <= 0 || a.q_heads + a.kv_heads <= 0 || a.rot_dim > a.head_dim) ++g_bad;
  return hipSuccess;
}
hipError_t launch_paged_plan(const PlanArgs&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t) {
  ++g_launches;
  const int64_t rows = a.S * a.q_heads * a.splits;
  if (a.splits > 1) inside(a.part_o, rows * a.head_dim * 4, "partial outputs"), inside(a.part_ml, rows * 8, "partial sums");
  return hipSuccess;
}
}  // namespace qlora

int main() {
  char* P = (char*)0x100000;  // never dereferenced
  const int64_t big[] = {-1, 0, 1, 2, 3, 63, 64, 4096, 8192, 16384, 16385, 65535, 65536, (1ll << 24) - 1, 1ll << 24,
                         (1ll << 31) - 1, 1ll << 31, 1ll << 37, 1ll << 62, INT64_MAX, INT64_MIN};
  const int32_t some[] = {INT32_MIN, -1, 0, 1, 2, 7, 8, 16, 64, 80, 128, 256, 264, 1024, 4096, 4097, INT32_MAX};
  for (int64_t T : big)
    for (int64_t D : big)
      for (int sums = 0; sums <= 3; ++sums) {
        int64_t n = -1;
        if (qlora_norm_residual_bwd_workspace(T, D, 0, 1, sums, &n)) n = 0;
        if (n < 0) ++g_bad;
        g_lo = 0x40000000, g_hi = g_lo + (uintptr_t)n;
        qlora_norm_residual_bwd(P, P, 0, P, P, 1, T, D, (float*)P, (float*)P, 1, (float*)P, 1e-6f, P, P,
                                sums > 0 ? (float*)P : nullptr, sums > 1 ? (float*)P : nullptr,
                                sums > 2 ? (float*)P : nullptr, (void*)g_lo, n, nullptr);
        qlora_norm_residual_fwd(P, 0, P, 1, T, D, nullptr, nullptr, 1, (float*)P, 1e-6f, P, P, nullptr);
      }
  for (int64_t T : big)
    for (int64_t st : big)
      for (int32_t h : some)
        for (int32_t d : some) {
          qlora_rope(P, st, h, P, st, P, st, h, P, st, T, d, d, 1, (int32_t*)P, (double*)P, 1, 0, 0, nullptr);
          qlora_rope_cache_write(P, st, h, P, st, P, st, P, st, h, T, d, 0, nullptr, nullptr, 1, 0, (int32_t*)P, P, P, T,
                                 d, nullptr);
        }
  for (int64_t S : big)
    for (int64_t n : big)
      for (int32_t p : some)
        qlora_paged_plan((int32_t*)P, (int32_t*)P, S, p, (int32_t*)P, n, (int32_t*)P, n, n, (int32_t*)(P + 4096),
                         (int32_t*)P, (int32_t*)P, (int32_t*)P, (int32_t*)P, nullptr);
  for (int64_t S : big)
    for (int64_t cols : big)
      for (int32_t H : some)
        for (int32_t KV : some)
          for (int32_t d : some)
            for (int32_t page : {0, 8, 16, 1024}) {
              int64_t n = -1;
              if (qlora_paged_attention_workspace(S, H, KV, d, cols, page, &n)) n = 0;
              if (n < 0) ++g_bad;
              g_lo = 0x40000000, g_hi = g_lo + (uintptr_t)n;
              qlora_paged_attention(P, (int64_t)H * d, S, H, KV, d, P, P, cols, page, (int32_t*)P, cols, (int32_t*)P, 1,
                                    P, nullptr, (void*)g_lo, n, nullptr);
            }
  if (g_bad) return 1;
  printf("ok %d\n", g_launches);
  return 0;
}
