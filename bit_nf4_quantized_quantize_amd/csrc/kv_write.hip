// The 8-bit key-value cache, gfx950: rows quantised as they enter it, with the
// rotary positions, and rows read back (definitions in include/qlora_kvcache.h).
//
// Both are bound by HBM.  A row lies with 1 to 16 neighbouring lanes, 16 elements
// each, so it is loaded, rotated, measured (its largest size over those lanes) and
// coded in registers: every element is read once and leaves as one byte.
// Measured: 8192 tokens of 32 heads of 128 and as many of queries written as E4M3
// in 79 us (337 MB, 4.3 TB/s; a copy reaches 4.95), the codes of 32768 tokens of
// 32 heads read back as bfloat16 in 168 us (4.8 TB/s), 16 tokens written in 5.2
// us.  One row per lane group in flight: with two 86 us, with four 107.
#include "device.h"
#include "kvcache.h"
#include "rotary.h"

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;  // elements of a row per lane

// ----------------------------------------------------------------- codes

// A row's scale and what its lanes need to code elements.  A scale below 2^-100
// is taken 2^64 times larger with its elements, so that nothing in between
// leaves the normal numbers.
struct Scale {
  float stored, s, inv, up;
  bool zero;  // codes are 0
};
template <int CT>
__device__ __forceinline__ Scale scale_of(uint32_t top) {  // top: the largest size, as bits
  constexpr float M = CT == kCacheInt8 ? 127.0f : 448.0f;
  Scale r;
  const bool finite = top < 0x7F800000u;
  r.stored = finite ? __uint_as_float(top) / M : __uint_as_float(0x7FC00000u);
  r.zero = !finite || r.stored == 0.0f;
  r.up = r.stored < 0x1p-100f ? 0x1p64f : 1.0f;
  r.s = r.zero ? 1.0f : r.stored * r.up;
  r.inv = 1.0f / r.s;
  return r;
}

// n is the whole number next to x / s as far as fp32 tells (x and s not
// negative); made the nearest one exactly, ties to the even: the remainder x - n
// s has no rounding (a multiple of half the last place of s, of at most about s
// / 2), so it tells on which side of the middle the quotient lies.
__device__ __forceinline__ int nearest(float x, float s, float n) {
  const float r = fmaf(-n, s, x), two = 2.0f * fabsf(r);
  int i = (int)n;
  if (two > s || (two == s && (i & 1))) i += r > 0.0f ? 1 : -1;
  return i;
}

template <int CT>
__device__ __forceinline__ uint32_t exact_code(float x, const Scale& k) {
  const float a = fabsf(x) * k.up, y = a * k.inv;
  const uint32_t sign = __float_as_uint(x) >> 31;
  int c;
  if (CT == kCacheInt8) {
    c = nearest(a, k.s, rintf(y));
    c = c > 127 ? 127 : c;
    if (sign) c = -c;
  } else {
    // y lies in [2^e, 2^(e+1)), or below 2^-6: codes are 2^(e-3) apart there
    int e = (int)(__float_as_uint(y) >> 23);
    e = e < 121 ? 121 : e;
    const float step = __uint_as_float((uint32_t)(e - 3) << 23), per = __uint_as_float((uint32_t)(257 - e) << 23);
    c = (e - 121) * 8 + nearest(a, k.s * step, rintf(y * per));
    c = c > 126 ? 126 : c;
    c |= (int)sign << 7;
  }
  return k.zero ? 0u : (uint32_t)c & 0xFFu;
}

// The codes of sixteen elements, in four words.  The quotient x * (1 / s) is off
// by less than two steps of fp32, so its rounding is the nearest code unless it
// lies that near to the middle of two; a lane's elements are done over if one is there
// (or under the smallest normal E4M3 number, whose middles lie elsewhere: zeros are).
// That is one element in 10^4 of ordinary rows, so a wave in ten, of 1024 elements,
// takes the longer way; all of them took 91 us where this takes 78 (8192 tokens of
// 32 heads of 128; with one zero in 50 elements 80).
template <int CT>
__device__ __forceinline__ void codes_of(const float (&x)[16], const Scale& k, uint32_t (&w)[4]) {
  bool near = k.zero | (k.up != 1.0f);
  if constexpr (CT == kCacheInt8) {
    constexpr float M = 12582912.0f;  // 1.5 * 2^23: a sum with it has the whole number in its low bits
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y = x[4 * i + j] * k.inv, n = y + M;
        near |= fabsf(y - (n - M)) > 0.5f - 0x1p-14f;
        t[j] = __float_as_uint(n);
      }
      w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t[3], t[2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u), 0x05040100u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = x[4 * i + j] * k.inv;
        near |= ((__float_as_uint(y[j]) + 0x80008u) & 0xFFFFFu) <= 0x10u || fabsf(y[j]) < 0x1p-6f;
      }
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w[i], true);
    }
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = exact_code<CT>(x[4 * i], k) | exact_code<CT>(x[4 * i + 1], k) << 8 | exact_code<CT>(x[4 * i + 2], k) << 16 |
             exact_code<CT>(x[4 * i + 3], k) << 24;
  }
}

// ---------------------------------------------------------------- writing

// Where the 16 elements of lane u lie in a row: two pieces of eight.
struct Pieces {
  int a, b;
  int pair;  // first pair of the rotary table, or -1: not rotated
};

// WIDE: pieces of eight elements in 16-byte accesses (rows, strides and the
// rotated part are whole pieces); else single elements.
template <int CT, bool INTER, bool WIDE>
__device__ __forceinline__ Pieces pieces_of(const RopeArgs& a, int u, bool turned) {
  Pieces p = {kPer * u, kPer * u + 8, -1};
  if (turned && kPer * u < a.rot_dim) {
    p.pair = 8 * u;
    if (WIDE && !INTER) p.a = 8 * u, p.b = a.rot_dim / 2 + 8 * u;
  } else if (WIDE && !turned) {  // neighbouring lanes take neighbouring pieces
    p.a = 8 * u, p.b = a.head_dim / 2 + 8 * u;
  }
  return p;
}

struct Row {
  const uint16_t* src;
  uint16_t* qo;     // queries
  uint8_t* codes;   // keys and values, with
  float* scale;
  int tk;           // token of the workgroup
  bool turned, live;
};

__device__ __forceinline__ Row row_of(const RopeArgs& a, float* k_scale, float* v_scale, int64_t t0, int i, int total,
                                      Div rows) {
  Row r = {};
  r.live = i < total;
  if (!r.live) return r;
  r.tk = i / rows;
  int h = i - r.tk * (int)rows.d;
  const int64_t t = t0 + r.tk;
  if (h < a.q_heads) {
    r.src = (const uint16_t*)a.q + t * a.q_stride + (int64_t)h * a.head_dim;
    r.qo = (uint16_t*)a.qo + t * a.qo_stride + (int64_t)h * a.head_dim;
    r.turned = true;
    return r;
  }
  h -= a.q_heads;
  const int32_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) {
    r.live = false;
    return r;
  }
  const bool value = h >= a.kv_heads;
  if (value) h -= a.kv_heads;
  r.src = value ? (const uint16_t*)a.v + t * a.v_stride : (const uint16_t*)a.k + t * a.k_stride;
  r.src += (int64_t)h * a.head_dim;
  r.turned = !value;
  const int64_t page = slot >> a.page_shift;
  const int64_t at = ((page * a.kv_heads + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
  r.codes = (uint8_t*)(value ? a.v_cache : a.k_cache) + at * a.head_dim;
  r.scale = (value ? v_scale : k_scale) + at;
  return r;
}

// The row's elements of lane u: x[0..7] and x[8..15] are its pieces.
template <bool INTER, bool WIDE>
__device__ __forceinline__ void load_row(const RopeArgs& a, const Row& r, const Pieces& p, uint32_t (&raw)[8],
                                         uint32_t (&other)[8]) {
  if (WIDE) {
    const uint4 x = *reinterpret_cast<const uint4*>(r.src + p.a), y = *reinterpret_cast<const uint4*>(r.src + p.b);
    raw[0] = x.x, raw[1] = x.y, raw[2] = x.z, raw[3] = x.w;
    raw[4] = y.x, raw[5] = y.y, raw[6] = y.z, raw[7] = y.w;
    return;
  }
  const int half = a.rot_dim / 2;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = p.a + j;
    int o = e;  // the other element of the pair
    if (r.turned && e < a.rot_dim) o = INTER ? e ^ 1 : e < half ? e + half : e - half;
    const uint32_t x = r.src[e], y = r.src[o];
    raw[j >> 1] = (j & 1) ? raw[j >> 1] | x << 16 : x;
    other[j >> 1] = (j & 1) ? other[j >> 1] | y << 16 : y;
  }
}

__device__ __forceinline__ float half_of(const uint32_t (&w)[8], int j) {
  return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
}

template <bool INTER, bool WIDE>
__device__ __forceinline__ void turn(const RopeArgs& a, const Row& r, const Pieces& p, const uint32_t (&raw)[8],
                                     const uint32_t (&other)[8], const float* cs, const float* sn, float (&x)[kPer]) {
  const int half = a.rot_dim / 2;
#pragma unroll
  for (int j = 0; j < kPer; ++j) x[j] = half_of(raw, j);
  if (p.pair < 0) return;
  const float* c = cs + r.tk * half;
  const float* s = sn + r.tk * half;
  if (WIDE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int lo = INTER ? 2 * j : j, hi = INTER ? 2 * j + 1 : j + 8;
      const float u = x[lo], v = x[hi], cc = c[p.pair + j], ss = s[p.pair + j];
      x[lo] = u * cc - v * ss;
      x[hi] = u * ss + v * cc;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = p.a + j;
      if (e >= a.rot_dim) continue;
      const bool second = INTER ? (e & 1) : e >= half;
      const int i = INTER ? e >> 1 : second ? e - half : e;
      const float u = x[j], v = half_of(other, j);
      x[j] = second ? v * s[i] + u * c[i] : u * c[i] - v * s[i];
    }
  }
}

// Stores of 16 and 8 bytes; PAST: they do not stay in the L2.
template <bool PAST, typename V>
__device__ __forceinline__ void put_past(void* p, V v) {
  typedef uint32_t words __attribute__((ext_vector_type(sizeof(V) / 4)));
  if constexpr (PAST) __builtin_nontemporal_store(__builtin_bit_cast(words, v), reinterpret_cast<words*>(p));
  else *reinterpret_cast<V*>(p) = v;
}

// blockIdx.x takes nt tokens, blockIdx.y a share of their rows; `group` lanes
// (a power of two) hold a row, those behind its end nothing.  The first row is
// loaded before the cosines are formed.
template <int CT, bool INTER, bool WIDE, bool PAST>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(RopeArgs a, float* k_scale, float* v_scale, int nt,
                                                            int group, Div rows, Div by_half) {
  extern __shared__ float trig[];  // [nt][half] cosines, then as many sines
  const int half = a.rot_dim / 2;
  const int64_t t0 = (int64_t)blockIdx.x * nt;
  const int n = (int)(a.T - t0 < nt ? a.T - t0 : nt);
  float* cs = trig;
  float* sn = trig + nt * half;
  const int total = n * (int)rows.d, per = kThreads / group, step = gridDim.y * per;
  const int u = threadIdx.x & (group - 1), mine = threadIdx.x / group;
  const bool in_row = kPer * u < a.head_dim;
  Row r;
  Pieces p;
  uint32_t raw[8], other[8];
  auto load = [&](int i) {
    r = row_of(a, k_scale, v_scale, t0, i, total, rows);
    p = pieces_of<CT, INTER, WIDE>(a, u, r.turned);
    if (r.live && in_row) load_row<INTER, WIDE>(a, r, p, raw, other);
  };
  load(blockIdx.y * per + mine);
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int tk = i / by_half;
    rotary_angle(a.positions[t0 + tk], a.turns[i - tk * half], a.mscale, false, cs + i, sn + i);
  }
  __syncthreads();
  // every lane of the workgroup makes the same turns, so the exchanges below
  // have all their lanes
  for (int i0 = blockIdx.y * per; i0 < total; i0 += step) {
    const bool live = r.live && in_row;
    float x[kPer];
    uint32_t top = 0;
    if (live) {
      turn<INTER, WIDE>(a, r, p, raw, other, cs, sn, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
      }
    }
    for (int o = 1; o < group; o <<= 1) {
      const uint32_t b = __shfl_xor(top, o, 64);
      top = b > top ? b : top;
    }
    if (live && r.qo) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack_bf2(x[2 * e], x[2 * e + 1]);
      if (WIDE) {
        put_past<PAST>(r.qo + p.a, make_uint4(w[0], w[1], w[2], w[3]));
        put_past<PAST>(r.qo + p.b, make_uint4(w[4], w[5], w[6], w[7]));
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) r.qo[p.a + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    } else if (live) {
      const Scale sc = scale_of<CT>(top);
      uint32_t w[4];
      codes_of<CT>(x, sc, w);
      if (u == 0) *r.scale = sc.stored;
      // rows of codes are whole pieces of 16 bytes whatever the tensors' strides
      put_past<PAST>(r.codes + p.a, make_uint2(w[0], w[1]));
      put_past<PAST>(r.codes + p.b, make_uint2(w[2], w[3]));
    }
    load(i0 + step + mine);
  }
}

template <int CT>
hipError_t write_as(const RopeArgs& a, float* k_scale, float* v_scale, hipStream_t stream) {
  const int rows = a.q_heads + 2 * a.kv_heads, half = a.rot_dim / 2;
  int group = 1;
  while (group * kPer < a.head_dim) group *= 2;
  const bool wide = a.rot_dim % 16 == 0 && a.q_stride % 8 == 0 && a.qo_stride % 8 == 0 && a.k_stride % 8 == 0 &&
                    a.v_stride % 8 == 0;
  const int per = kThreads / group;
  // Tokens per workgroup: a row for every lane group, up to 8 (8192 tokens of 96
  // rows, 32 groups: 80 us with one token, 83 with two).
  int nt = per / rows;
  nt = a.T < 1024 || nt < 1 ? 1 : nt > 8 ? 8 : nt;
  const int64_t gx = (a.T + nt - 1) / nt;
  const unsigned gy = gx >= 512 ? 1 : 4;
  const size_t lds = (size_t)nt * a.rot_dim * sizeof(float);
  // More than the L2 holds goes past it (8192 tokens of 32 heads, written and read
  // back: 121.1 us against 123.6).
  const bool past = a.T * ((int64_t)a.q_heads + a.kv_heads) * a.head_dim * 2 > ((int64_t)32 << 20);
  const auto kernel =
      wide ? (a.interleaved ? (past ? kv_write_kernel<CT, true, true, true> : kv_write_kernel<CT, true, true, false>)
                            : (past ? kv_write_kernel<CT, false, true, true> : kv_write_kernel<CT, false, true, false>))
           : (a.interleaved ? kv_write_kernel<CT, true, false, false> : kv_write_kernel<CT, false, false, false>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)gx, gy), dim3(kThreads), lds, stream, a, k_scale, v_scale, nt, group,
                     div_by(rows), div_by(half ? half : 1));
  return hipGetLastError();
}

// ---------------------------------------------------------------- reading

// EV elements in 16 bytes of the output.
template <int CT, int EV>
__device__ __forceinline__ void decode(const void* cache, int64_t at, float scale, float (&x)[EV]) {
  if constexpr (CT == kCacheBf16) {
    uint32_t w[EV / 2];
    if constexpr (EV == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>((const uint16_t*)cache + at);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>((const uint16_t*)cache + at);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int j = 0; j < EV; ++j) x[j] = __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  } else {
    uint32_t w[EV / 4];
    if constexpr (EV == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>((const uint8_t*)cache + at);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>((const uint8_t*)cache + at);
    }
#pragma unroll
    for (int j = 0; j < EV; ++j) {
      const uint32_t b = w[j >> 2] >> (8 * (j & 3));
      x[j] = (CT == kCacheInt8 ? (float)(int8_t)b : e4m3_decode(b & 0xFFu)) * scale;
    }
  }
}

template <typename T, int EV>
__device__ __forceinline__ void put(T* dst, const float (&x)[EV]) {
  uint4 v;
  if constexpr (EV == 8) {
    v = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
  } else {
    v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  *reinterpret_cast<uint4*>(dst) = v;
}

// blockIdx.x takes nt tokens, blockIdx.y a share of their pieces, blockIdx.z
// the keys or the values.
template <int CT, typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a, int nt, Div units, Div per_row) {
  constexpr int EV = 16 / sizeof(T), UN = 4;
  const KvCache& c = a.c;
  const bool value = blockIdx.z + (a.k == nullptr);
  const void* cache = value ? c.v : c.k;
  const float* scales = value ? c.v_scale : c.k_scale;
  T* out = (T*)(value ? a.v : a.k);
  const int64_t t0 = (int64_t)blockIdx.x * nt;
  const int n = (int)(a.T - t0 < nt ? a.T - t0 : nt);
  const int total = n * (int)units.d, step = gridDim.y * kThreads;
  for (int i0 = blockIdx.y * kThreads + threadIdx.x; i0 < total; i0 += UN * step) {
    float x[UN][EV];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int i = i0 + j * step;
#pragma unroll
      for (int e = 0; e < EV; ++e) x[j][e] = 0.0f;
      if (i >= total) continue;
      const int tk = i / units, w = i - tk * (int)units.d, head = w / per_row;
      const int32_t slot = a.slots[t0 + tk];
      if (slot < 0 || slot >= a.num_slots) continue;
      const int64_t row = ((((int64_t)(slot >> c.page_shift)) * c.kv_heads + head) << c.page_shift) +
                          (slot & ((1 << c.page_shift) - 1));
      decode<CT, EV>(cache, row * c.head_dim + (w - head * (int)per_row.d) * EV, CT == kCacheBf16 ? 1.0f : scales[row],
                     x[j]);
    }
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int i = i0 + j * step;
      if (i < total) put<T, EV>(out + (t0 * units.d + i) * EV, x[j]);
    }
  }
}

template <int CT, typename T>
hipError_t read_as(const KvReadArgs& a, hipStream_t stream) {
  constexpr int EV = 16 / sizeof(T);
  const int per_row = a.c.head_dim / EV, units = a.c.kv_heads * per_row;
  int nt = 1024 / units;  // a turn of every thread, up to 8 tokens
  nt = nt < 1 || a.T < 1024 ? 1 : nt > 8 ? 8 : nt;
  const int64_t gx = (a.T + nt - 1) / nt;
  const unsigned gy = gx >= 512 || units <= kThreads ? 1 : units <= 2 * kThreads ? 2 : 4;
  hipLaunchKernelGGL((kv_read_kernel<CT, T>), dim3((unsigned)gx, gy, a.k && a.v ? 2 : 1), dim3(kThreads), 0, stream, a,
                     nt, div_by(units), div_by(per_row));
  return hipGetLastError();
}

template <int CT>
hipError_t read_to(const KvReadArgs& a, bool f32, hipStream_t stream) {
  return f32 ? read_as<CT, float>(a, stream) : read_as<CT, uint16_t>(a, stream);
}

}  // namespace

hipError_t launch_kv_write(const RopeArgs& a, float* k_scale, float* v_scale, int type, hipStream_t stream) {
  return type == kCacheInt8 ? write_as<kCacheInt8>(a, k_scale, v_scale, stream)
                            : write_as<kCacheE4m3>(a, k_scale, v_scale, stream);
}

hipError_t launch_kv_read(const KvReadArgs& a, bool f32, hipStream_t stream) {
  if (a.c.type == kCacheInt8) return read_to<kCacheInt8>(a, f32, stream);
  if (a.c.type == kCacheE4m3) return read_to<kCacheE4m3>(a, f32, stream);
  return read_to<kCacheBf16>(a, f32, stream);
}

}  // namespace qlora
