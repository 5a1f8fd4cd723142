// The cosines and sines of rotary positions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// cos and sin of 2 pi pos turns, times mscale.  The product is off by up to half
// an fp64 step of the whole turns (3 u = 3 * 2^-24 radians at 2^31 positions of
// 1 radian), so its remainder is put back once those are off; then the angle is
// exact to 2^-53 turns.  The functions are fp64 too, rounded once: they are few
// beside the elements (fp32 functions take as long, 104.2 us at 8191 tokens of 72
// heads, 103.5 with these).
__device__ __forceinline__ void rotary_angle(int32_t pos, double turns, float mscale, bool inverse, float* c,
                                             float* s) {
  double x = (double)pos * turns;
  const double rest = fma((double)pos, turns, -x);
  x = (x - rint(x)) + rest;
  double sn, cs;
  sincospi(2.0 * x, &sn, &cs);
  *c = (float)(cs * mscale);
  *s = (float)((inverse ? -sn : sn) * mscale);
}

}  // namespace qlora
