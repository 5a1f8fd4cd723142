// What the attention kernels over a paged cache share: how a length is cut into
// parts, and the weights as bfloat16 numbers.
#pragma once

#include "device.h"

namespace qlora {

constexpr int kTile = 32;     // tokens per wave and step
constexpr int kMinTiles = 2;  // per wave, before a sequence is cut further

// How a sequence of n tokens is cut: `parts` ranges of `per` tiles (the last
// may be shorter).
struct Cut {
  int64_t tiles, per, parts;
};
__device__ __forceinline__ Cut cut_of(int64_t n, int splits, int waves) {
  Cut c;
  c.tiles = (n + kTile - 1) / kTile;
  int64_t most = (c.tiles + waves * kMinTiles - 1) / (waves * kMinTiles);
  if (most > splits) most = splits;
  if (most < 1) most = 1;
  c.per = (c.tiles + most - 1) / most;
  c.parts = c.per ? (c.tiles + c.per - 1) / c.per : 0;
  return c;
}

// The same where tiles are counted in 32 bits (n < 2^31), a fraction of the
// instructions.
struct Cut32 {
  uint32_t tiles, per, parts;
};
__device__ __forceinline__ Cut32 cut32_of(uint32_t n, int splits, int waves) {
  Cut32 c;
  c.tiles = (n + kTile - 1) / kTile;
  uint32_t most = (c.tiles + waves * kMinTiles - 1) / (uint32_t)(waves * kMinTiles);
  if (most > (uint32_t)splits) most = splits;
  if (most < 1) most = 1;
  c.per = (c.tiles + most - 1) / most;
  c.parts = c.per ? (c.tiles + c.per - 1) / c.per : 0;
  return c;
}

// Keeps a wave's LDS accesses before and after it in program order for the
// compiler; the LDS itself serves a wave's accesses in order.
__device__ __forceinline__ void lds_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The upper halves of eight words: bfloat16 numbers, where the lower ones are 0.
__device__ __forceinline__ bf16x8 upper(const uint32_t (&w)[8]) {
  uint4 v;
  v.x = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
  v.y = __builtin_amdgcn_perm(w[3], w[2], 0x07060302u);
  v.z = __builtin_amdgcn_perm(w[5], w[4], 0x07060302u);
  v.w = __builtin_amdgcn_perm(w[7], w[6], 0x07060302u);
  return __builtin_bit_cast(bf16x8, v);
}

// Weights p as sums of three bfloat16 numbers each, exactly: cut off after 8 bits,
// and what is left again, for weights of either sign (codes with a scale of -0 or
// below).  INF: for weights not below 0 and values that may be infinities.  A part is then
// the bfloat16 number next below what is left, so a remainder is never zero: 16
// bits at most are left after the first and 8 after the second, or the one bit that
// was between neighbours.  All parts are positive (zero for a weight of zero), so
// an infinity of V stays what it is in all three products.
template <bool INF>
__device__ __forceinline__ void split(const float (&p)[8], bf16x8 (&part)[3]) {
  uint32_t w[8];
  float left[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) left[j] = p[j];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = __float_as_uint(left[j]);
      if (INF) w[j] = __builtin_elementwise_sub_sat(w[j], 1u);
      w[j] &= 0xFFFF0000u;
      left[j] -= __uint_as_float(w[j]);
    }
    part[k] = upper(w);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(left[j]);
  part[2] = upper(w);
}

}  // namespace qlora
