// Rotary positions on queries and keys, gfx950, with the rotated keys and the
// values going to a paged cache in the serving form (formulas in
// include/qlora_decoder.h).
//
// Bound by HBM: every element is read once and written once.  The angles of a
// token are the same for all of its heads, so a workgroup first puts the
// cosines and sines of its NT tokens into LDS (one per token and pair; the
// angle is position times turns in fp64, less its whole turns, so far
// positions lose nothing) and then streams the heads of those tokens, 16
// bytes per thread and access.
#include "decoder.h"
#include "device.h"

namespace qlora {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<uint16_t>(uint16_t v) { return bf2f(v); }
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float v) { return f2bf(v); }
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }

// EV elements moved at once (16 bytes, or one element where rows do not
// allow it).
template <typename T, int EV>
struct alignas(EV * sizeof(T)) Piece {
  T e[EV];
};

template <typename T, int EV>
__device__ __forceinline__ Piece<T, EV> ld(const T* p) { return *reinterpret_cast<const Piece<T, EV>*>(p); }
template <typename T, int EV>
__device__ __forceinline__ void st(T* p, const Piece<T, EV>& v) { *reinterpret_cast<Piece<T, EV>*>(p) = v; }

// cos and sin of 2 pi pos turns, times mscale.  The remainder that fp32 drops
// from the reduced angle is put back to first order.
__device__ __forceinline__ void angle(int32_t pos, double turns, float mscale, bool inverse, float* c, float* s) {
  double x = (double)pos * turns;
  x -= rint(x);
  if (inverse) x = -x;
  const float f = (float)x;
  const float d = 6.2831853071795865f * (float)(x - (double)f);
  float sn, cs;
  sincospif(2.0f * f, &sn, &cs);
  *c = (cs - sn * d) * mscale;
  *s = (sn + cs * d) * mscale;
}

// Where a head's row goes.
template <typename T>
__device__ __forceinline__ T* cache_row(void* cache, int32_t slot, int head, const RopeArgs& a) {
  const int64_t page = slot >> a.page_shift;
  const int off = slot & ((1 << a.page_shift) - 1);
  return (T*)cache + (((page * a.kv_heads + head) << a.page_shift) + off) * (int64_t)a.head_dim;
}

// The heads of a token are cut into units: rotated units (a piece of each
// half of the pairs, or a piece of whole pairs when interleaved), then pieces
// of the rest of the head.  blockIdx.y takes a share of a token's units.
template <typename T, int EV, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int nt) {
  extern __shared__ float trig[];  // [nt][half] cosines, then as many sines
  const int half = a.rot_dim / 2;
  const int64_t t0 = (int64_t)blockIdx.x * nt;
  const int n = (int)(a.T - t0 < nt ? a.T - t0 : nt);
  float* cs = trig;
  float* sn = trig + nt * half;
  for (int i = threadIdx.x; i < n * half; i += kThreads)
    angle(a.positions[t0 + i / half], a.turns[i % half], a.mscale, a.inverse, cs + i, sn + i);
  __syncthreads();

  constexpr int PE = INTER ? (EV > 1 ? EV / 2 : 1) : EV;  // pairs per rotated unit
  const int ru = half / PE, tu = (a.head_dim - a.rot_dim) / EV, hu = ru + tu;
  const int vu = a.v ? a.head_dim / EV : 0;
  const int qk = (a.q_heads + a.kv_heads) * hu;
  const int units = qk + a.kv_heads * vu;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < n * units; i += gridDim.y * kThreads) {
    const int tk = i / units, u = i - tk * units;
    const int64_t t = t0 + tk;
    int32_t slot = 0;
    if (a.slots) slot = a.slots[t];
    const bool stored = slot >= 0 && slot < a.num_slots;
    if (u >= qk) {  // values
      const int head = (u - qk) / vu, e = (u - qk - head * vu) * EV;
      if (stored)
        st<T, EV>(cache_row<T>(a.v_cache, slot, head, a) + e,
                  ld<T, EV>((const T*)a.v + t * a.v_stride + (int64_t)head * a.head_dim + e));
      continue;
    }
    int head = u / hu;
    const int w = u - head * hu;
    const T* src;
    T* dst;
    if (head < a.q_heads) {
      src = (const T*)a.q + t * a.q_stride + (int64_t)head * a.head_dim;
      dst = (T*)a.qo + t * a.qo_stride + (int64_t)head * a.head_dim;
    } else {
      head -= a.q_heads;
      src = (const T*)a.k + t * a.k_stride + (int64_t)head * a.head_dim;
      if (a.slots) {
        if (!stored) continue;
        dst = cache_row<T>(a.k_cache, slot, head, a);
      } else {
        dst = (T*)a.ko + t * a.ko_stride + (int64_t)head * a.head_dim;
      }
    }
    if (w >= ru) {  // the part of the head without rotation
      const int e = a.rot_dim + (w - ru) * EV;
      st<T, EV>(dst + e, ld<T, EV>(src + e));
      continue;
    }
    const float* c = cs + tk * half + w * PE;
    const float* s = sn + tk * half + w * PE;
    if (INTER && EV > 1) {
      Piece<T, EV> v = ld<T, EV>(src + w * EV);
#pragma unroll
      for (int j = 0; j < EV / 2; ++j) {
        const float x = to_f<T>(v.e[2 * j]), y = to_f<T>(v.e[2 * j + 1]);
        v.e[2 * j] = from_f<T>(x * c[j] - y * s[j]);
        v.e[2 * j + 1] = from_f<T>(x * s[j] + y * c[j]);
      }
      st<T, EV>(dst + w * EV, v);
    } else {
      const int ea = INTER ? 2 * w : w * EV, eb = INTER ? 2 * w + 1 : half + w * EV;
      Piece<T, EV> x = ld<T, EV>(src + ea), y = ld<T, EV>(src + eb);
#pragma unroll
      for (int j = 0; j < EV; ++j) {
        const float p = to_f<T>(x.e[j]), q = to_f<T>(y.e[j]);
        x.e[j] = from_f<T>(p * c[j] - q * s[j]);
        y.e[j] = from_f<T>(p * s[j] + q * c[j]);
      }
      st<T, EV>(dst + ea, x);
      st<T, EV>(dst + eb, y);
    }
  }
}

template <typename T, int EV>
hipError_t rope_as(const RopeArgs& a, hipStream_t stream) {
  // Few tokens: one token per workgroup and its units over several; many: four
  // tokens share a workgroup.
  const int nt = a.T >= 1024 ? 4 : 1;
  const int64_t gx = (a.T + nt - 1) / nt;
  const unsigned gy = gx >= 512 ? 1 : 4;
  const size_t lds = (size_t)nt * a.rot_dim * sizeof(float);
  if (a.interleaved)
    hipLaunchKernelGGL((rope_kernel<T, EV, true>), dim3((unsigned)gx, gy), dim3(kThreads), lds, stream, a, nt);
  else
    hipLaunchKernelGGL((rope_kernel<T, EV, false>), dim3((unsigned)gx, gy), dim3(kThreads), lds, stream, a, nt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, bool f32, hipStream_t stream) {
  // 16-byte pieces need every row, the two halves of the pairs and the rest of
  // the head to be whole pieces.
  const int ev = f32 ? 4 : 8;
  const bool vec = a.head_dim % ev == 0 && (a.interleaved ? a.rot_dim : a.rot_dim / 2) % ev == 0 &&
                   a.rot_dim % ev == 0 && a.q_stride % ev == 0 && a.qo_stride % ev == 0 && a.k_stride % ev == 0 &&
                   a.ko_stride % ev == 0 && a.v_stride % ev == 0;
  if (f32) return vec ? rope_as<float, 4>(a, stream) : rope_as<float, 1>(a, stream);
  return vec ? rope_as<uint16_t, 8>(a, stream) : rope_as<uint16_t, 1>(a, stream);
}

}  // namespace qlora
