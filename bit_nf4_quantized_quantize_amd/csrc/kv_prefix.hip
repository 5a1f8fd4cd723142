// Attention over a shared prefix for many query rows, gfx950: the prefix's part
// of qlora_prefix_attention (include/qlora_kvcache.h) when the rows of a kv head
// (sequences times heads that share it) and the prefix's tokens are many.
#include <type_traits>

#include "device.h"
#include "kvcache.h"
#include "kv_codes.h"
#include "paged_device.h"

namespace qlora {

namespace {

// A workgroup takes 32 WQ rows, 32 to a wave, and a part of the prefix in steps
// of TT = 32 WT NS tokens, of which WT waves of the same rows take 32 NS each:
//   scores^T [32 tokens x 32 rows] = K Q^T,  out^T [d x 32 rows] += V^T P
// with K and V of a step as bfloat16 in LDS.
//
// A matrix instruction keeps its unit busy for 32 cycles and the issue for 4, and
// the softmax of a tile has about six vector instructions for each of its matrix
// ones, so a wave has to issue both kinds in turn.  Tile i (32 tokens) is taken
// in three blocks: its scores are formed in block i - 1, its weights in block i,
// its part of the output in block i + 1; within a block nothing depends on
// anything but the last ones' results.
//
// A weight enters the product with V as three bfloat16 parts, with all of its 24
// bits, as in the narrow workgroups: a row's result does not depend on which of them
// take it.  Two parts (64 sequences behind 16384 tokens, as below: 64 us where three
// take 77) left 0.45 % of the results not the nearest bfloat16 number, three 0.04 %.
//
// Bound by the products and the softmax between them: 64 sequences of 8 heads each
// on 8 kv heads of 128 behind 16384 tokens in int8 77 us, 68.7 GFLOP with all
// parts, 0.9 PFLOP/s (a large library product reaches 1.19).  1024 rows behind 2000
// tokens, 32 on 8 heads, E4M3: 31 us.
// The rest was measured with two parts.  Of 64 us the matrix instructions alone took
// 25, the launch, first loads and the 33 MB of parts 10, LDS reads 5, exponentials
// and parts 6, codes to bfloat16 1 to 6, maxima and missing tokens 4.  Scores,
// weights and output of a tile in one block: 73 us.  256 rows per workgroup (K and V
// made bfloat16 and read from memory half as often): 66 us where 128 took 73, but
// twice the parts to join (10.8 us, 7.1); up to 256 rows workgroups of 128, two
// waves of which share a row's tokens.
template <int DP, int CT, int WQ, int WT, int NS>
struct Wide {
  static constexpr int THREADS = 64 * WQ * WT;
  static constexpr int TT = 32 * WT * NS;              // tokens of a step
  static constexpr int KP = DP + 8, VP = DP + 16;      // pitches
  static constexpr int EV = CT == kCacheBf16 ? 8 : 16; // elements in 16 bytes
  static constexpr int CH = DP / EV;                   // 16-byte pieces of a padded row
  static constexpr int PER = (TT * CH + THREADS - 1) / THREADS;
  // Between two barriers the waves are within NS blocks of each other: they read
  // keys of one step, values of up to two or of the one three before that which
  // is written.
  static constexpr int NK = 2, NV = NS == 1 ? 4 : 3;
  struct Lds {
    __bf16 k[NK][TT * KP];
    __bf16 v[NV][TT * VP];
    float ks[NK][TT], vs[NV][TT], bias[NK][TT];
    int ok[NK][TT / 16];
  };
  static constexpr int OP = DP + 6;  // of what a wave leaves for another: outputs, maximum and sum
  static constexpr int JOIN = (WT - 1) * WQ * 32 * OP * 4;
  static constexpr int BYTES = (int)sizeof(Lds) > JOIN ? (int)sizeof(Lds) : JOIN;
};

// What a thread brings in of a step, and the pages (-1: none) it will do so from
// in the next one.
template <class W>
struct Load {
  uint4 k[W::PER], v[W::PER];
  bool ok[W::PER];
  float ks, vs;
  bool in;
  int32_t page[W::PER], row_page;
};

__device__ __forceinline__ int64_t prefix_of(const KvAttnArgs& a) {
  const int64_t n = *a.prefix_len, cap = a.prefix_cols << a.c.page_shift;
  return n < 0 ? 0 : n > cap ? cap : n;
}

template <int DP, int CT, int WQ, int WT, int NS>
__global__ __launch_bounds__(64 * WQ * WT) void kv_prefix_kernel(KvAttnArgs a) {
  using W = Wide<DP, CT, WQ, WT, NS>;
  typedef typename std::conditional<CT == kCacheBf16, uint16_t, uint8_t>::type Elem;
  constexpr bool CODED = CT != kCacheBf16;
  __shared__ __attribute__((aligned(16))) char bytes[W::BYTES];
  typename W::Lds& lds = *reinterpret_cast<typename W::Lds*>(bytes);

  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % WQ, wt = wave / WQ, hi = lane >> 5, d = c.head_dim;
  const int mine = 32 * NS * wt;  // of the tokens of a step
  const int group = a.q_heads / c.kv_heads, parts = a.psplits + a.splits;
  uint32_t id = blockIdx.x;
  const int z = id % (uint32_t)a.psplits;
  id /= (uint32_t)a.psplits;
  const int kv = id % (uint32_t)c.kv_heads, rt = id / (uint32_t)c.kv_heads;
  const int rows = (int)a.S * group, row = (rt * WQ + wq) * 32 + (lane & 31);  // under 65536 * 4096
  const int n = (int)prefix_of(a);
  const Cut32 cut = cut32_of(n, a.psplits, a.pwaves);
  if ((uint32_t)z >= cut.parts) return;
  const int first = z * (int)cut.per * kTile, last = n - first < (int)cut.per * kTile ? n : first + (int)cut.per * kTile;

  Load<W> ld;
  const int in_page = (1 << c.page_shift) - 1;
  const uint32_t page_rows = (uint32_t)c.kv_heads << c.page_shift;
  const int64_t kv_row = (int64_t)kv << c.page_shift;
  // The page of a token, as the table has it; whether it is one is asked when it
  // is used, a step later, so that nothing waits for it here.
  auto entry = [&](int tok) { return a.prefix_table[(tok < last ? tok : last - 1) >> c.page_shift]; };
  auto there = [&](int32_t page, int tok) { return tok < last && page >= 0 && page < c.num_pages; };
  auto look_up = [&](int t0) {
#pragma unroll
    for (int i = 0; i < W::PER; ++i) ld.page[i] = entry(t0 + (i * W::THREADS + tid) / W::CH);
    if (tid < W::TT) ld.row_page = entry(t0 + tid);
  };
  // Rows that are not there are read from the cache's first ones and put as zeros.
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < W::PER; ++i) {
      const int idx = i * W::THREADS + tid, r = idx / W::CH, e = idx % W::CH * W::EV;
      ld.ok[i] = e < d && there(ld.page[i], t0 + r);
      const int64_t at = ((int64_t)ld.page[i] * page_rows + kv_row + ((t0 + r) & in_page)) * d + e;
      ld.k[i] = *reinterpret_cast<const uint4*>((const Elem*)c.k + (ld.ok[i] ? at : 0));
      ld.v[i] = *reinterpret_cast<const uint4*>((const Elem*)c.v + (ld.ok[i] ? at : 0));
    }
    ld.in = tid < W::TT && there(ld.row_page, t0 + tid);
    if (CODED && tid < W::TT) {
      const int64_t at = ld.in ? (int64_t)ld.row_page * page_rows + kv_row + ((t0 + tid) & in_page) : 0;
      ld.ks = c.k_scale[at], ld.vs = c.v_scale[at];
    }
  };
  const float scale2 = a.scale * 1.44269504088896340736f;  // scores in base 2
  auto store = [&](int nk, int nv) {
#pragma unroll
    for (int i = 0; i < W::PER; ++i) {
      const int idx = i * W::THREADS + tid, r = idx / W::CH, e = idx % W::CH * W::EV;
      if (W::TT * W::CH % W::THREADS && r >= W::TT) continue;
      uint4* k = reinterpret_cast<uint4*>(lds.k[nk] + r * W::KP + e);
      uint4* v = reinterpret_cast<uint4*>(lds.v[nv] + r * W::VP + e);
      uint4 kk = ld.k[i], vv = ld.v[i];
      if (!ld.ok[i]) kk = vv = make_uint4(0, 0, 0, 0);
      if constexpr (CODED) {
        k[0] = numbers<CT>(kk.x, kk.y), k[1] = numbers<CT>(kk.z, kk.w);
        v[0] = numbers<CT>(vv.x, vv.y), v[1] = numbers<CT>(vv.z, vv.w);
      } else {
        k[0] = kk, v[0] = vv;
      }
    }
    if (tid < W::TT) {
      lds.ks[nk][tid] = CODED ? (ld.in ? ld.ks * scale2 : 0.0f) : scale2;
      lds.vs[nv][tid] = ld.in ? ld.vs : 0.0f;
      lds.bias[nk][tid] = ld.in ? 0.0f : -INFINITY;
      // the last token of sixteen is there: so are the others of its page
      if ((tid & 15) == 15) lds.ok[nk][tid >> 4] = ld.in;
    }
  };

  look_up(first);
  // Q^T: column lane % 32 (a row), reduction elements 16 i + 8 (lane / 32) ..
  bf16x8 q[DP / 16];
  int64_t seq = 0;
  int head = 0;
  if (row < rows) seq = (uint32_t)row / (uint32_t)group, head = kv * group + (int)((uint32_t)row % (uint32_t)group);
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) {
    const int e = 16 * i + 8 * hi;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows && e < d) v = *reinterpret_cast<const uint4*>(a.q + seq * a.q_stride + (int64_t)head * d + e);
    q[i] = __builtin_bit_cast(bf16x8, v);
  }
  // the values of the step before the first are zeros, with weights of zero
  for (int i = tid; i < W::TT * W::VP / 8; i += W::THREADS)
    reinterpret_cast<uint4*>(lds.v[W::NV - 1])[i] = make_uint4(0, 0, 0, 0);
  load(first);
  look_up(first + W::TT);
  store(0, 0);
  load(first + W::TT);
  look_up(first + 2 * W::TT);
  __syncthreads();

  // m: of the weights so far, a whole number, so that scaling by another is exact
  float m = -INFINITY, l = 0.0f;
  floatx16 acc[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[t][j] = 0.0f;
  float x[16];            // scores of the tile less m, in base 2
  bf16x8 part[2][3] = {};  // weights of the tile before it: steps of 16 tokens, parts

  // A tile's scores less m, and the largest
  auto scores = [&](const floatx16& sc, const float* ks, float* top) {
    const float mu = m == -INFINITY ? 0.0f : m;
    float t = -INFINITY;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const floatx4 f = *reinterpret_cast<const floatx4*>(ks + 8 * b + 4 * hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * b + j] = fmaf(sc[4 * b + j], f[j], -mu);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) t = fmaxf(t, x[j]);
    *top = t;
  };
  // What is seldom: tokens that are not there, and a larger maximum.  m is set kAhead
  // beyond it, so that it stays while the maximum grows less than that: no weight
  // passes 1, so none times a value passes what the narrow workgroups can hold, and
  // the largest is 2^-kAhead at least, far from where numbers end below (64 sequences
  // behind 16384 tokens: 77 us, with 4 for kAhead 79, with 2 84, with 0 92).
  constexpr float kAhead = 8.0f;
  auto settle = [&](int ok, const float* bias, float top) {
    if (!__builtin_amdgcn_readfirstlane(ok)) {
      top = -INFINITY;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const floatx4 f = *reinterpret_cast<const floatx4*>(bias + 8 * b + 4 * hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (f[j] != 0.0f) x[4 * b + j] = f[j];
          top = fmaxf(top, x[4 * b + j]);
        }
      }
    }
    if (!__ballot(top > 0.0f || m == -INFINITY)) return;
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const bool up = top > 0.0f || (m == -INFINITY && top > -INFINITY);
    if (!__ballot(up)) return;
    const float by = up ? ceilf(top) + kAhead : 0.0f;  // m moves by it
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(-by);
    if (up) m = (m == -INFINITY ? 0.0f : m) + by;
    l *= f;
#pragma unroll
    for (int t = 0; t < DP / 32; ++t)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[t][j] *= f;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] -= by;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[h][k][j] = (__bf16)((float)part[h][k][j] * f);
  };
  // V^T of 16 tokens: reduction slot e of a lane is token 8 (e / 4) + 4 hi + e %
  // 4, as the scores have them
  auto read_v = [&](const __bf16* v, int h, int t) {
    const int g = lane >> 4, y = lane & 15;
    const __bf16* src = v + (16 * h + 4 * hi + (y >> 2)) * W::VP + 16 * (g & 1) + 4 * (y & 3) + 32 * t;
    const short8_t f = __builtin_shufflevector(ds_read_tr16(src), ds_read_tr16(src + 8 * W::VP), 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, f);
  };
  auto weighted = [&](const __bf16* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < DP / 32; ++t) {
        const bf16x8 f = read_v(v, h, t);
#pragma unroll
        for (int k = 0; k < 3; ++k) acc[t] = mfma32(f, part[h][k], acc[t]);
      }
  };
  auto products = [&](const __bf16* k) {
    floatx16 sc;
#pragma unroll
    for (int j = 0; j < 16; ++j) sc[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) sc = mfma32(frag_kc(k, W::KP, 0, 16 * i, lane), q[i], sc);
    return sc;
  };
  auto whole = [&](int nk, int tok) { return lds.ok[nk][tok / 16] & lds.ok[nk][tok / 16 + 1]; };

  {
    float top;
    scores(products(lds.k[0] + mine * W::KP), lds.ks[0] + mine, &top);
    settle(whole(0, mine), lds.bias[0] + mine, top);
  }
  // nv: buffers of the values of the step before this one, this one and the next
  int nk = 0, nv[3] = {W::NV - 1, 0, 1};
  for (int t0 = first; t0 < last; t0 += W::TT) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s == NS - 1) {
        // the keys of the next step are needed from here on
        store(nk ^ 1, nv[2]);
        load(t0 + 2 * W::TT);
        look_up(t0 + 3 * W::TT);
        __syncthreads();
      }
      const int kb = s == NS - 1 ? nk ^ 1 : nk, next = mine + (s == NS - 1 ? 0 : 32 * (s + 1));
      const floatx16 sc = products(lds.k[kb] + next * W::KP);
      weighted(lds.v[s == 0 ? nv[0] : nv[1]] + (mine + (s == 0 ? 32 * (NS - 1) : 32 * (s - 1))) * W::VP);
      // weights of this tile
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = __builtin_amdgcn_exp2f(x[j]);
        l += x[j];
      }
      if constexpr (CODED) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const floatx4 f = *reinterpret_cast<const floatx4*>(lds.vs[nv[1]] + mine + 32 * s + 8 * b + 4 * hi);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[4 * b + j] *= f[j];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = x[8 * h + j];
        split<!CODED>(w, part[h]);
      }
      float top;
      scores(sc, lds.ks[kb] + next, &top);
      // the weights are formed here, beside the products, not where they are used
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 3; ++k) asm volatile("" : "+v"(part[h][k]));
      settle(whole(kb, next), lds.bias[kb] + next, top);
    }
    nk ^= 1;
    nv[0] = nv[1], nv[1] = nv[2], nv[2] = nv[2] + 1 == W::NV ? 0 : nv[2] + 1;
  }
  weighted(lds.v[nv[0]] + (mine + 32 * (NS - 1)) * W::VP);

  l += __shfl_xor(l, 32, 64);
  if constexpr (WT > 1) {  // the waves of the same rows join, in order
    __syncthreads();
    float* const all = reinterpret_cast<float*>(bytes) + (wq * 32 + (lane & 31)) * W::OP;
    if (wt > 0) {
      float* o = all + (wt - 1) * WQ * 32 * W::OP;
#pragma unroll
      for (int t = 0; t < DP / 32; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[32 * t + acc_row32(j, lane)] = acc[t][j];
      if (hi == 0) o[DP] = m, o[DP + 1] = l;
    }
    __syncthreads();
    if (wt > 0) return;
#pragma unroll
    for (int w = 1; w < WT; ++w) {
      const float* o = all + (w - 1) * WQ * 32 * W::OP;
      const float om = o[DP], mx = fmaxf(m, om), mu = mx == -INFINITY ? 0.0f : mx;
      const float f0 = __builtin_amdgcn_exp2f(m - mu), f1 = __builtin_amdgcn_exp2f(om - mu);
      m = mx, l = l * f0 + o[DP + 1] * f1;
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

template <int DP, int CT, int WQ, int WT, int NS>
hipError_t prefix_as(const KvAttnArgs& a, hipStream_t stream) {
  using W = Wide<DP, CT, WQ, WT, NS>;
  static_assert(W::BYTES <= 160 * 1024, "LDS of a CU");
  const int64_t rows = a.S * (a.q_heads / a.c.kv_heads), tiles = (rows + 32 * WQ - 1) / (32 * WQ);
  hipLaunchKernelGGL((kv_prefix_kernel<DP, CT, WQ, WT, NS>), dim3((unsigned)(tiles * a.c.kv_heads * a.psplits)),
                     dim3(W::THREADS), 0, stream, a);
  return hipGetLastError();
}

template <int DP, int CT>
hipError_t prefix_rows(const KvAttnArgs& a, hipStream_t stream) {
  if constexpr (DP > 128) return prefix_as<DP, CT, 4, 1, 1>(a, stream);
  else if (a.wide > 128) return prefix_as<DP, CT, 8, 1, 2>(a, stream);
  else return prefix_as<DP, CT, 4, 2, 1>(a, stream);
}

template <int CT>
hipError_t prefix_type(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.head_dim <= 64) return prefix_rows<64, CT>(a, stream);
  if (a.c.head_dim <= 96) return prefix_rows<96, CT>(a, stream);
  if (a.c.head_dim <= 128) return prefix_rows<128, CT>(a, stream);
  return prefix_rows<256, CT>(a, stream);
}

}  // namespace

hipError_t launch_kv_prefix(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.type == kCacheInt8) return prefix_type<kCacheInt8>(a, stream);
  if (a.c.type == kCacheE4m3) return prefix_type<kCacheE4m3>(a, stream);
  return prefix_type<kCacheBf16>(a, stream);
}

}  // namespace qlora
