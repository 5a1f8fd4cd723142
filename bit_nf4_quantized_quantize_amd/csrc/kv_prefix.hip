// Attention over a shared prefix for many query rows, gfx950: the prefix's part
// of qlora_prefix_attention (include/qlora_kvcache.h) when the rows of a kv head
// (sequences times heads that share it) are more than a narrow workgroup takes.
#include <type_traits>

#include "device.h"
#include "kvcache.h"
#include "kv_codes.h"
#include "paged_device.h"

namespace qlora {

namespace {

// A workgroup takes 32 WQ rows and a part of the prefix: WQ waves with 32 rows
// each, WT of them for each row, which share the tokens of a step.
//   scores^T [32 tokens x 32 rows] = K Q^T,  out^T [d x 32 rows] += V^T P
// with K and V of a step as bfloat16 in LDS.
template <int DP, int CT, int WQ, int WT, int SUB>
struct Wide {
  static constexpr int THREADS = 64 * WQ * WT;
  static constexpr int TT = 32 * WT * SUB;             // tokens of a step
  static constexpr int KP = DP + 8, VP = DP + 16;      // pitches
  static constexpr int EV = CT == kCacheBf16 ? 8 : 16; // elements in 16 bytes
  static constexpr int CH = DP / EV;                   // 16-byte pieces of a padded row
  static constexpr int PER = (TT * CH + THREADS - 1) / THREADS;
  static constexpr int OP = DP + 4;
  struct Step {
    __bf16 k[TT * KP];
    __bf16 v[TT * VP];
    float ks[TT], vs[TT], bias[TT];
    int ok[TT / 16];
  };
  static constexpr int BYTES0 = 2 * sizeof(Step);
  static constexpr int JOIN = WT > 1 ? (WT - 1) * WQ * 32 * (OP + 2) * 4 : 0;
  static constexpr int BYTES = BYTES0 > JOIN ? BYTES0 : JOIN;
};

// What a thread brings in of a step.
template <class W>
struct Load {
  uint4 k[W::PER], v[W::PER];
  bool ok[W::PER];
  float ks, vs;
  bool in;
};

template <int DP, int CT, int WQ, int WT, int SUB>
__global__ __launch_bounds__(64 * WQ * WT) void kv_prefix_kernel(KvAttnArgs a, int row_tiles) {
  using W = Wide<DP, CT, WQ, WT, SUB>;
  typedef typename std::conditional<CT == kCacheBf16, uint16_t, uint8_t>::type Elem;
  constexpr bool CODED = CT != kCacheBf16;
  __shared__ __attribute__((aligned(16))) char lds[W::BYTES];
  typename W::Step* steps = reinterpret_cast<typename W::Step*>(lds);

  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % WQ, wt = wave / WQ, hi = lane >> 5, d = c.head_dim;
  const int group = a.q_heads / c.kv_heads, parts = a.psplits + a.splits;
  int id = blockIdx.x;
  const int z = id % a.psplits;
  id /= a.psplits;
  const int kv = id % c.kv_heads, rt = id / c.kv_heads;
  const int64_t rows = a.S * group, row = (int64_t)rt * 32 * WQ + 32 * wq + (lane & 31);
  const bool busy = (int64_t)rt * 32 * WQ + 32 * wq < rows;  // the wave has rows
  const int64_t cap = a.prefix_cols << c.page_shift;
  int64_t n = *a.prefix_len;
  n = n < 0 ? 0 : n > cap ? cap : n;
  const Cut cut = cut_of(n, a.psplits, a.pwaves);
  if (z >= cut.parts) return;
  const int64_t first = z * cut.per * kTile;
  int64_t last = first + cut.per * kTile;
  if (last > n) last = n;

  // Q^T: column lane % 32 (a row), reduction elements 16 i + 8 (lane / 32) ..
  bf16x8 q[DP / 16];
  int64_t seq = 0;
  int head = 0;
  if (row < rows) seq = row / group, head = kv * group + (int)(row % group);
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) {
    const int e = 16 * i + 8 * hi;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows && e < d) v = *reinterpret_cast<const uint4*>(a.q + seq * a.q_stride + (int64_t)head * d + e);
    q[i] = __builtin_bit_cast(bf16x8, v);
  }
  const float scale2 = a.scale * 1.44269504088896340736f;  // scores in base 2
  float m = -INFINITY, l = 0.0f;
  floatx16 acc[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[t][j] = 0.0f;

  Load<W> ld;
  auto load = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < W::PER; ++i) {
      const int idx = i * W::THREADS + tid, r = idx / W::CH, e = idx % W::CH * W::EV;
      const int64_t tok = t0 + r;
      ld.ok[i] = false;
      ld.k[i] = ld.v[i] = make_uint4(0, 0, 0, 0);
      if (r >= W::TT || tok >= last) continue;
      const int32_t page = a.prefix_table[tok >> c.page_shift];
      ld.ok[i] = page >= 0 && page < c.num_pages;
      if (!ld.ok[i] || e >= d) continue;
      const int64_t at = ((((int64_t)page * c.kv_heads + kv) << c.page_shift) + (tok & ((1 << c.page_shift) - 1))) * d + e;
      ld.k[i] = *reinterpret_cast<const uint4*>((const Elem*)c.k + at);
      ld.v[i] = *reinterpret_cast<const uint4*>((const Elem*)c.v + at);
    }
    if (tid < W::TT) {
      const int64_t tok = t0 + tid;
      ld.ks = 0.0f, ld.vs = 0.0f, ld.in = false;
      if (tok < last) {
        const int32_t page = a.prefix_table[tok >> c.page_shift];
        ld.in = page >= 0 && page < c.num_pages;
        if (CODED && ld.in) {
          const int64_t at = (((int64_t)page * c.kv_heads + kv) << c.page_shift) + (tok & ((1 << c.page_shift) - 1));
          ld.ks = c.k_scale[at], ld.vs = c.v_scale[at];
        }
      }
    }
  };
  auto store = [&](typename W::Step& s) {
#pragma unroll
    for (int i = 0; i < W::PER; ++i) {
      const int idx = i * W::THREADS + tid, r = idx / W::CH, e = idx % W::CH * W::EV;
      if (r >= W::TT) continue;
      uint4* k = reinterpret_cast<uint4*>(s.k + r * W::KP + e);
      uint4* v = reinterpret_cast<uint4*>(s.v + r * W::VP + e);
      if constexpr (CODED) {
        k[0] = numbers<CT>(ld.k[i].x, ld.k[i].y), k[1] = numbers<CT>(ld.k[i].z, ld.k[i].w);
        v[0] = numbers<CT>(ld.v[i].x, ld.v[i].y), v[1] = numbers<CT>(ld.v[i].z, ld.v[i].w);
      } else {
        k[0] = ld.k[i], v[0] = ld.v[i];
      }
    }
    if (tid < W::TT) {
      s.ks[tid] = ld.ks * scale2, s.vs[tid] = ld.vs, s.bias[tid] = ld.in ? 0.0f : -INFINITY;
      // the last token of sixteen is there: so are the others of its page
      if ((tid & 15) == 15) s.ok[tid >> 4] = ld.in;
    }
  };

  load(first);
  store(steps[0]);
  __syncthreads();
  int buf = 0;
  for (int64_t t0 = first; t0 < last; t0 += W::TT, buf ^= 1) {
    const bool more = t0 + W::TT < last;
    if (more) load(t0 + W::TT);
    const typename W::Step& s = steps[buf];
    if (busy) {
      bool full = true;
#pragma unroll
      for (int i = 0; i < W::TT / 16; ++i) full &= s.ok[i] != 0;
      full = __builtin_amdgcn_readfirstlane(full);
      float p[SUB][16];
      const int base = 32 * SUB * wt;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        floatx16 sc;
#pragma unroll
        for (int j = 0; j < 16; ++j) sc[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) sc = mfma32(frag_kc(s.k, W::KP, base + 32 * u, 16 * i, lane), q[i], sc);
#pragma unroll
        for (int j = 0; j < 16; ++j) p[u][j] = sc[j];
        if constexpr (CODED) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const floatx4 ks = *reinterpret_cast<const floatx4*>(s.ks + base + 32 * u + 8 * b + 4 * hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[u][4 * b + j] *= ks[j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) p[u][j] *= scale2;
        }
        if (!full) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const floatx4 bias = *reinterpret_cast<const floatx4*>(s.bias + base + 32 * u + 8 * b + 4 * hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[u][4 * b + j] = bias[j] != 0.0f ? bias[j] : p[u][4 * b + j];
          }
        }
      }
      float mt = m;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) mt = fmaxf(mt, p[u][j]);
      mt = fmaxf(mt, __shfl_xor(mt, 32, 64));
      if (__ballot(mt > m)) {
        const float old = __builtin_amdgcn_exp2f(m - (mt == -INFINITY ? 0.0f : mt));
        l *= old;
#pragma unroll
        for (int t = 0; t < DP / 32; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[t][j] *= old;
        m = mt;
      }
      const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          p[u][j] = __builtin_amdgcn_exp2f(p[u][j] - mu);
          l += p[u][j];
        }
        if constexpr (CODED) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const floatx4 vs = *reinterpret_cast<const floatx4*>(s.vs + base + 32 * u + 8 * b + 4 * hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[u][4 * b + j] *= vs[j];
          }
        }
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          float w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = p[u][8 * k2 + j];
          bf16x8 part[2];
          split2(w, part);
          const int g = lane >> 4, x = lane & 15;
          // reduction slot e of a lane is token 8 (e / 4) + 4 hi + e % 4, as the scores have them
          const __bf16* src = s.v + (base + 32 * u + 16 * k2 + 4 * hi + (x >> 2)) * W::VP + 16 * (g & 1) + 4 * (x & 3);
#pragma unroll
          for (int t = 0; t < DP / 32; ++t) {
            const short4_t v0 = ds_read_tr16(src + 32 * t), v1 = ds_read_tr16(src + 32 * t + 8 * W::VP);
            const short8_t v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int k = 0; k < 2; ++k) acc[t] = mfma32(__builtin_bit_cast(bf16x8, v), part[k], acc[t]);
          }
        }
      }
    }
    if (more) store(steps[buf ^ 1]);
    __syncthreads();
  }

  l += __shfl_xor(l, 32, 64);
  if constexpr (WT > 1) {  // the waves of the same rows join, in order
    float* all = reinterpret_cast<float*>(lds);
    constexpr int ROW = W::OP + 2;
    if (wt > 0) {
      float* o = all + (((wt - 1) * WQ + wq) * 32 + (lane & 31)) * ROW;
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[32 * t + acc_row32(j, lane)] = acc[t][j];
      if (hi == 0) o[W::OP] = m, o[W::OP + 1] = l;
    }
    __syncthreads();
    if (wt > 0) return;
#pragma unroll
    for (int w = 1; w < WT; ++w) {
      const float* o = all + (((w - 1) * WQ + wq) * 32 + (lane & 31)) * ROW;
      const float om = o[W::OP], mx = fmaxf(m, om), mu = mx == -INFINITY ? 0.0f : mx;
      const float f0 = __builtin_amdgcn_exp2f(m - mu), f1 = __builtin_amdgcn_exp2f(om - mu);
      m = mx, l = l * f0 + o[W::OP + 1] * f1;
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[t][j] = acc[t][j] * f0 + o[32 * t + acc_row32(j, lane)] * f1;
    }
  }
  if (row >= rows) return;
  const int64_t at = (seq * a.q_heads + head) * parts + z;
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int e = 32 * t + 8 * b + 4 * hi;
      if (e < d)
        *reinterpret_cast<floatx4*>(a.part_o + at * d + e) =
            (floatx4){acc[t][4 * b], acc[t][4 * b + 1], acc[t][4 * b + 2], acc[t][4 * b + 3]};
    }
  if (hi == 0) a.part_ml[at * 2] = m, a.part_ml[at * 2 + 1] = l;
}

template <int DP, int CT, int WQ, int WT, int SUB>
hipError_t prefix_as(const KvAttnArgs& a, hipStream_t stream) {
  using W = Wide<DP, CT, WQ, WT, SUB>;
  static_assert(W::BYTES <= 160 * 1024, "LDS of a CU");
  const auto kernel = kv_prefix_kernel<DP, CT, WQ, WT, SUB>;
  const int64_t rows = a.S * (a.q_heads / a.c.kv_heads), tiles = (rows + 32 * WQ - 1) / (32 * WQ);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * a.c.kv_heads * a.psplits)), dim3(W::THREADS), 0, stream, a,
                     (int)tiles);
  return hipGetLastError();
}

template <int CT>
hipError_t prefix_of(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.head_dim <= 64) return prefix_as<64, CT, 4, 2, 1>(a, stream);
  if (a.c.head_dim <= 96) return prefix_as<96, CT, 4, 2, 1>(a, stream);
  if (a.c.head_dim <= 128) return prefix_as<128, CT, 4, 2, 1>(a, stream);
  return prefix_as<256, CT, 4, 2, 1>(a, stream);
}

}  // namespace

hipError_t launch_kv_prefix(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.type == kCacheInt8) return prefix_of<kCacheInt8>(a, stream);
  if (a.c.type == kCacheE4m3) return prefix_of<kCacheE4m3>(a, stream);
  return prefix_of<kCacheBf16>(a, stream);
}

}  // namespace qlora
