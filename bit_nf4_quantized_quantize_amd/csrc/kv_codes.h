// Codes of the 8-bit key-value cache as operands of the matrix products.
#pragma once

#include "device.h"
#include "kvcache.h"

namespace qlora {

// Eight codes as bfloat16 numbers, exactly.
template <int CT>
__device__ __forceinline__ uint4 numbers(uint32_t lo, uint32_t hi) {
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = h ? hi : lo;
    if constexpr (CT == kCacheE4m3) {
      w[2 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
      w[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
    } else {
      // whole numbers of 8 bits: the upper half of their fp32 form holds them
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(c >> (8 * j));
      w[2 * h] = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302u);
      w[2 * h + 1] = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace qlora
