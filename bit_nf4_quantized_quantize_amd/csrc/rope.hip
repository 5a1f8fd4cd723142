// Rotary positions on queries and keys, gfx950, with the rotated keys and the
// values going to a paged cache in the serving form (formulas in
// include/qlora_decoder.h).
//
// Bound by HBM: every element is read once and written once.  The angles of a
// token are the same for all of its heads, so a workgroup first puts the
// cosines and sines of its NT tokens into LDS (one per token and pair; the
// angle is position times turns in fp64, less its whole turns, so far positions
// lose nothing beside the rounding of the table) and then streams the heads of
// those tokens, 16 bytes per thread and access.  Measured: 4096 tokens of 32 + 32 heads of 128
// in bfloat16 21 us (6.3 TB/s, part of the output staying in the Infinity
// Cache), 8191 tokens of 64 + 8 heads in fp32 104 us (5.8 TB/s), 8192 tokens of
// 32 heads into the cache 78 us (5.2 TB/s), 16 tokens 3.4 us.
#include "decoder.h"
#include "device.h"
#include "rotary.h"

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

// EV elements moved at once: 16 bytes, or 8 or one element where rows do not
// allow it.
template <typename T, int EV>
struct alignas(EV * sizeof(T)) Piece {
  T e[EV];
};

template <typename T, int EV>
__device__ __forceinline__ Piece<T, EV> ld(const T* p) { return *reinterpret_cast<const Piece<T, EV>*>(p); }
// PAST: 16-byte stores that do not stay in the L2.
template <typename T, int EV, bool PAST>
__device__ __forceinline__ void st(T* p, const Piece<T, EV>& v) {
  if constexpr (PAST && EV * sizeof(T) == 16) {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(words, v), reinterpret_cast<words*>(p));
  } else {
    *reinterpret_cast<Piece<T, EV>*>(p) = v;
  }
}

// Where a head's row goes.
template <typename T>
__device__ __forceinline__ T* cache_row(void* cache, int32_t slot, int head, const RopeArgs& a) {
  const int64_t page = slot >> a.page_shift;
  const int off = slot & ((1 << a.page_shift) - 1);
  return (T*)cache + (((page * a.kv_heads + head) << a.page_shift) + off) * (int64_t)a.head_dim;
}

// One piece of work: 16 bytes of one head (of each half of its pairs).
template <typename T, int EV>
struct Unit {
  Piece<T, EV> x, y;
  T* dst;        // NULL: nothing to do
  int a, b;      // elements of the head that x and y are (b < 0: x alone)
  int trig;      // index into the cosines, or -1: copied
};

// The heads of a token are cut into units: rotated units (a piece of each
// half of the pairs, or a piece of whole pairs when interleaved), then pieces
// of the rest of the head; the values' heads are pieces throughout.
struct Cuts {
  Div units, hu, vu, half;  // per token, per head of q and k, per head of v; pairs of a head
};

template <typename T, int EV, bool INTER>
__device__ __forceinline__ void load_unit(Unit<T, EV>& w, const RopeArgs& a, const Cuts& by, int64_t t0, int i) {
  constexpr int PE = INTER ? (EV > 1 ? EV / 2 : 1) : EV;  // pairs per rotated unit
  const int half = a.rot_dim / 2, hu = by.hu.d, ru = half / PE, qk = (a.q_heads + a.kv_heads) * hu;
  const int tk = i / by.units, u = i - tk * (int)by.units.d;
  const int64_t t = t0 + tk;
  int32_t slot = 0;
  if (a.slots) slot = a.slots[t];
  const bool stored = slot >= 0 && slot < a.num_slots;
  const T* src;
  w.trig = w.b = -1;
  if (u >= qk) {  // values
    if (!stored) return;
    const int head = (u - qk) / by.vu;
    w.a = (u - qk - head * (int)by.vu.d) * EV;
    src = (const T*)a.v + t * a.v_stride + (int64_t)head * a.head_dim;
    w.dst = cache_row<T>(a.v_cache, slot, head, a);
  } else {
    int head = u / by.hu;
    const int r = u - head * hu;
    if (head < a.q_heads) {
      src = (const T*)a.q + t * a.q_stride + (int64_t)head * a.head_dim;
      w.dst = (T*)a.qo + t * a.qo_stride + (int64_t)head * a.head_dim;
    } else {
      head -= a.q_heads;
      if (a.slots && !stored) return;
      src = (const T*)a.k + t * a.k_stride + (int64_t)head * a.head_dim;
      w.dst = a.slots ? cache_row<T>(a.k_cache, slot, head, a)
                      : (T*)a.ko + t * a.ko_stride + (int64_t)head * a.head_dim;
    }
    if (r < ru) {
      w.trig = tk * half + r * PE;
      w.a = INTER ? 2 * r * PE : r * PE;
      if (!INTER) w.b = half + r * PE;
      else if (EV == 1) w.b = 2 * r + 1;
    } else {
      w.a = a.rot_dim + (r - ru) * EV;
    }
  }
  w.x = ld<T, EV>(src + w.a);
  if (w.b >= 0) w.y = ld<T, EV>(src + w.b);
}

template <typename T, int EV, bool INTER, bool PAST>
__device__ __forceinline__ void store_unit(Unit<T, EV>& w, const float* cs, const float* sn) {
  if (!w.dst) return;
  if (w.trig >= 0) {
    const float* c = cs + w.trig;
    const float* s = sn + w.trig;
    if (INTER && EV > 1) {
#pragma unroll
      for (int k = 0; k < EV / 2; ++k) {
        const float x = to_f<T>(w.x.e[2 * k]), y = to_f<T>(w.x.e[2 * k + 1]);
        w.x.e[2 * k] = from_f<T>(x * c[k] - y * s[k]);
        w.x.e[2 * k + 1] = from_f<T>(x * s[k] + y * c[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < EV; ++k) {
        const float x = to_f<T>(w.x.e[k]), y = to_f<T>(w.y.e[k]);
        w.x.e[k] = from_f<T>(x * c[k] - y * s[k]);
        w.y.e[k] = from_f<T>(x * s[k] + y * c[k]);
      }
    }
  }
  st<T, EV, PAST>(w.dst + w.a, w.x);
  if (w.b >= 0) st<T, EV, PAST>(w.dst + w.b, w.y);
}

// blockIdx.x takes nt tokens, blockIdx.y a share of their units.  A thread
// loads UN units before it stores the first, the first UN before the cosines
// are formed.
template <typename T, int EV, bool INTER, bool PAST, int UN>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int nt, Cuts by) {
  extern __shared__ float trig[];  // [nt][half] cosines, then as many sines
  const int half = a.rot_dim / 2;
  const int64_t t0 = (int64_t)blockIdx.x * nt;
  const int n = (int)(a.T - t0 < nt ? a.T - t0 : nt);
  float* cs = trig;
  float* sn = trig + nt * half;
  const int total = n * (int)by.units.d, step = gridDim.y * kThreads;
  int i0 = blockIdx.y * kThreads + threadIdx.x;
  Unit<T, EV> w[UN];
  auto load = [&] {
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      w[j].dst = nullptr;
      if (i0 + j * step < total) load_unit<T, EV, INTER>(w[j], a, by, t0, i0 + j * step);
    }
  };
  load();
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int tk = i / by.half;
    rotary_angle(a.positions[t0 + tk], a.turns[i - tk * half], a.mscale, a.inverse, cs + i, sn + i);
  }
  __syncthreads();
  while (i0 < total) {
#pragma unroll
    for (int j = 0; j < UN; ++j) store_unit<T, EV, INTER, PAST>(w[j], cs, sn);
    i0 += UN * step;
    load();
  }
}

template <typename T, int EV, bool INTER>
hipError_t rope_as(const RopeArgs& a, hipStream_t stream) {
  const int half = a.rot_dim / 2, pe = INTER ? (EV > 1 ? EV / 2 : 1) : EV;
  const int hu = half / pe + (a.head_dim - a.rot_dim) / EV, vu = a.head_dim / EV;
  const int units = (a.q_heads + a.kv_heads) * hu + (a.v ? a.kv_heads * vu : 0);
  // Tokens per workgroup: about 2048 units, up to 4 tokens (8191 tokens of 72
  // heads of 128 in fp32, 2304 units each: 113 us with one token, 127 with two,
  // 149 with four; 4096 tokens of 64 heads in bf16, 512 units each: 24.3, 22.5,
  // 23.5).  Few tokens: the units of one token over four workgroups.
  int nt = 2048 / units;
  nt = a.T < 1024 || nt < 1 ? 1 : nt > 4 ? 4 : nt;
  const int64_t gx = (a.T + nt - 1) / nt;
  const unsigned gy = gx >= 512 ? 1 : 4;
  const size_t lds = (size_t)nt * a.rot_dim * sizeof(float);
  // More than the L2 holds goes past it (8192 tokens of 32 heads to the cache:
  // 79 us against 85; 4096 rotated: 21.9 and 23.5).
  const int64_t bytes = a.T * ((int64_t)a.q_heads + (a.v ? 2 : 1) * a.kv_heads) * a.head_dim * (int64_t)sizeof(T);
  const auto kernel =
      bytes > ((int64_t)32 << 20) ? rope_kernel<T, EV, INTER, true, 4> : rope_kernel<T, EV, INTER, false, 4>;
  const Cuts by = {div_by(units), div_by(hu), div_by(vu), div_by(half ? half : 1)};
  hipLaunchKernelGGL(kernel, dim3((unsigned)gx, gy), dim3(kThreads), lds, stream, a, nt, by);
  return hipGetLastError();
}

}  // namespace

// Whether pieces of ev elements fit: every row, the two halves of the pairs and
// the rest of the head have to be whole pieces.
static bool pieces_fit(const RopeArgs& a, int ev) {
  return a.head_dim % ev == 0 && (a.interleaved ? a.rot_dim : a.rot_dim / 2) % ev == 0 && a.rot_dim % ev == 0 &&
         a.q_stride % ev == 0 && a.qo_stride % ev == 0 && a.k_stride % ev == 0 && a.ko_stride % ev == 0 &&
         a.v_stride % ev == 0;
}

template <typename T>
static hipError_t rope_of(const RopeArgs& a, hipStream_t stream) {
  constexpr int WIDE = 16 / sizeof(T);
  if (pieces_fit(a, WIDE))
    return a.interleaved ? rope_as<T, WIDE, true>(a, stream) : rope_as<T, WIDE, false>(a, stream);
  if (pieces_fit(a, WIDE / 2))
    return a.interleaved ? rope_as<T, WIDE / 2, true>(a, stream) : rope_as<T, WIDE / 2, false>(a, stream);
  return a.interleaved ? rope_as<T, 1, true>(a, stream) : rope_as<T, 1, false>(a, stream);
}

hipError_t launch_rope(const RopeArgs& a, bool f32, hipStream_t stream) {
  return f32 ? rope_of<float>(a, stream) : rope_of<uint16_t>(a, stream);
}

}  // namespace qlora
