// Internal launchers of the decoder-block operators (norm.hip, rope.hip,
// paged.hip), shared with decoder_abi.cpp.  Every launcher only enqueues on
// `stream` and returns the launch status; arguments were checked before.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// n / d for n < 2^31 by one multiplication (Granlund and Montgomery, "Division
// by invariant integers using multiplication", PLDI 1994).
struct Div {
  uint32_t mul, d;
  int shift;
};
inline Div div_by(uint32_t d) {
  Div v = {0, d, 0};
  while (((uint64_t)1 << v.shift) < d) ++v.shift;
  v.mul = (uint32_t)(((((uint64_t)1 << v.shift) - d) << 32) / d + 1);
  return v;
}
#ifdef __HIPCC__
__device__ __forceinline__ int operator/(int n, const Div& v) {
  return (int)((__umulhi((uint32_t)n, v.mul) + (uint32_t)n) >> v.shift);
}
#endif

// Residual update (include/qlora_decoder.h, qlora_norm_residual_*).
struct NormArgs {
  const void* x;   // forward: the stream before; backward: xo, the stream after
  const void* h;
  const void* dxo;
  const void* dn;
  void* xo;        // forward: the stream after; backward: dx
  void* n;         // forward: the next input; backward: dh
  const float* w_post;
  const float* gate;
  const float* w_pre;
  float* part;     // backward: [2][norm_bwd_parts][D] partial sums (dx y and dn xo r), or NULL
  float* dw_post;
  float* dgate;
  float* dw_pre;
  int64_t T;
  int D;
  float alpha, eps;
};
hipError_t launch_norm_fwd(const NormArgs& a, bool x_f32, bool h_f32, hipStream_t stream);
// Rows of partial sums the backward writes per wanted sum (T > 0).
int64_t norm_bwd_parts(int64_t T, int64_t D);
hipError_t launch_norm_bwd(const NormArgs& a, bool x_f32, bool h_f32, hipStream_t stream);

// Rotary positions, with the keys and values going to a paged cache when
// `slots` is given.  Strides in elements.
struct RopeArgs {
  const void* q;
  void* qo;
  const void* k;
  void* ko;         // keys in place of a tensor (slots == NULL)
  const void* v;    // only with slots
  const int32_t* positions;
  const double* turns;
  const int32_t* slots;
  void* k_cache;
  void* v_cache;
  int64_t q_stride, qo_stride, k_stride, ko_stride, v_stride, T;
  int64_t num_slots;
  int q_heads, kv_heads, head_dim, rot_dim;
  int page_shift;
  float mscale;
  bool interleaved, inverse;
};
hipError_t launch_rope(const RopeArgs& a, bool f32, hipStream_t stream);

struct PlanArgs {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* total;
  int32_t* starts;
  int32_t* slots;
  int32_t* positions;
  int32_t* pages_needed;
  int64_t n_free, table_cols, T;
  int S, page_size;
};
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream);

// Attention over the paged cache.  paged_splits: how many parts a sequence's
// tokens are cut into at most (1: no workspace, no joining kernel).
struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  float* lse;
  float* part_o;   // [S][q_heads][splits][head_dim]
  float* part_ml;  // [S][q_heads][splits][2]: maximum (base-2 scores) and sum
  int64_t q_stride, S, num_pages, table_cols;
  int q_heads, kv_heads, head_dim, page_shift, splits;
  int waves;       // per workgroup, set by the launcher
  float scale;
};
int paged_splits(int64_t S, int q_heads, int kv_heads, int head_dim, int64_t max_len);
hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream);

}  // namespace qlora
