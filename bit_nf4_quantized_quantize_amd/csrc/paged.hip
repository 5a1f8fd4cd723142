// The paged key-value cache, gfx950: the plan of a batch (pages, slots and
// positions from the requests' lengths) and the attention of one new token
// per sequence over the cache (definitions in include/qlora_decoder.h).
#include "decoder.h"
#include "device.h"
#include "paged_device.h"

namespace qlora {

namespace {

// ------------------------------------------------------------------- plan
//
// One launch: every workgroup forms the prefix sums of the new tokens and of
// the pages taken over all S sequences in LDS (a scan over at most 4096
// sequences, a few microseconds, against the second launch and the round trip
// through memory it saves), then takes its share of the token rows (the
// sequence of a row by binary search in the prefix sums) and of the
// sequences' new table entries.  Slots of fresh pages come from the free list
// itself, so no workgroup waits for another's table entries.

constexpr int kPlanThreads = 512;

__device__ __forceinline__ int pages_of(int32_t tokens, const Div& page) {
  return tokens > 0 ? (tokens - 1) / page + 1 : 0;
}
// A sequence's length from one of the caller's: not negative.
__device__ __forceinline__ int32_t length_of(const int32_t* v, int64_t s) { return v[s] < 0 ? 0 : v[s]; }
// a + b of numbers that are not negative, at most 2^31 - 1: sums of lengths that
// make no sense stay in order, so nothing is searched or addressed out of
// bounds by them.
__device__ __forceinline__ int32_t add_sat(int32_t a, int32_t b) {
  const uint32_t v = (uint32_t)a + (uint32_t)b;
  return v > INT32_MAX ? INT32_MAX : (int32_t)v;
}
// Pages of a sequence of `tokens` that the table has room for.
__device__ __forceinline__ int32_t held(int32_t tokens, const Div& page, int64_t cols) {
  const int32_t p = pages_of(tokens, page);
  return p < cols ? p : (int32_t)cols;
}

// The largest s < n with v[s] <= i (v[0] <= i).
__device__ __forceinline__ int last_at_most(const int32_t* v, int n, int64_t i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanArgs a, int per, Div page) {
  extern __shared__ int32_t lds[];  // starts [S + 1], first page taken [S + 1]
  __shared__ int32_t wave[2][kPlanThreads / 64];
  int32_t* starts = lds;
  int32_t* first = lds + a.S + 1;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  // thread t sums sequences t * per .., then the threads' sums are scanned
  const int s0 = threadIdx.x * per, s1 = s0 + per < a.S ? s0 + per : a.S;
  int32_t nt = 0, np = 0;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const int32_t c = length_of(a.cached, s), n = length_of(a.fresh, s);
    const int32_t p = held(add_sat(c, n), page, a.table_cols) - held(c, page, a.table_cols);
    starts[s] = n, first[s] = p;
    nt = add_sat(nt, n), np = add_sat(np, p);
  }
  int32_t vt = nt, vp = np;  // inclusive sums over the wave
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t ut = __shfl_up(vt, o, 64), up = __shfl_up(vp, o, 64);
    if (lane >= o) vt = add_sat(vt, ut), vp = add_sat(vp, up);
  }
  if (lane == 63) wave[0][wv] = vt, wave[1][wv] = vp;
  vt = __shfl_up(vt, 1, 64), vp = __shfl_up(vp, 1, 64);  // the sums before this thread's
  if (lane == 0) vt = vp = 0;
  __syncthreads();
  int32_t run_t = 0, run_p = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w == wv) vt = add_sat(vt, run_t), vp = add_sat(vp, run_p);
    run_t = add_sat(run_t, wave[0][w]), run_p = add_sat(run_p, wave[1][w]);
  }
  for (int s = s0; s < s1; ++s) {
    const int32_t n = starts[s], p = first[s];
    starts[s] = vt, first[s] = vp;
    vt = add_sat(vt, n), vp = add_sat(vp, p);
  }
  if (threadIdx.x == 0) starts[a.S] = run_t, first[a.S] = run_p;
  __syncthreads();

  const int64_t gid = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  const int64_t gsz = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t s = gid; s <= a.S; s += gsz) {
    a.starts[s] = starts[s];
    if (s < a.S) a.total[s] = add_sat(length_of(a.cached, s), length_of(a.fresh, s));
  }
  if (gid == 0) *a.pages_needed = run_p;
  // new table entries, in the order of the free list
  for (int64_t i = gid; i < run_p; i += gsz) {
    const int q = last_at_most(first, a.S, i);
    const int64_t col = held(length_of(a.cached, q), page, a.table_cols) + (i - first[q]);
    if (col < a.table_cols) a.table[q * a.table_cols + col] = i < a.n_free ? a.free_pages[i] : -1;
  }
  for (int64_t t = gid; t < a.T; t += gsz) {  // token rows
    int32_t slot = -1;
    int64_t pos = 0;
    if (t < run_t) {
      const int q = last_at_most(starts, a.S, t);
      const int32_t c = length_of(a.cached, q);
      pos = c + (t - starts[q]);
      if (pos <= INT32_MAX) {
        const int32_t col = (int32_t)pos / page, have = pages_of(c, page);
        int32_t pg = -1;
        if (col < a.table_cols) {
          if (col < have) {
            pg = a.table[q * a.table_cols + col];
          } else {
            const int64_t i = (int64_t)first[q] + col - have;
            if (i < a.n_free) pg = a.free_pages[i];
          }
        }
        if (pg >= 0) {
          const int64_t v = (int64_t)pg * a.page_size + ((int32_t)pos - col * a.page_size);
          if (v <= INT32_MAX) slot = (int32_t)v;
        }
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos <= INT32_MAX ? (int32_t)pos : INT32_MAX;
  }
}

}  // namespace

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream) {
  // a row per thread (263000 rows of 1024 sequences: 7.0 us, four in a row per
  // thread 9.0; 16 rows: 3.8 us)
  int64_t wgs = (a.T + kPlanThreads - 1) / kPlanThreads;
  wgs = wgs < 1 ? 1 : wgs > 1024 ? 1024 : wgs;
  hipLaunchKernelGGL(paged_plan_kernel, dim3((unsigned)wgs), dim3(kPlanThreads),
                     2 * (size_t)(a.S + 1) * sizeof(int32_t), stream, a, (a.S + kPlanThreads - 1) / kPlanThreads,
                     div_by((uint32_t)a.page_size));
  return hipGetLastError();
}

// -------------------------------------------------------------- attention
//
// Bound by HBM: every key and value of a sequence is read once, by the
// workgroup that takes its kv head (and its share of the length).  The work
// per byte is small but grows with the query heads that share a kv head, so
// the products run on MFMA with those heads as the 16 columns; a wave works
// alone on tiles of 32 tokens, with the running maximum and sum of its own:
//   scores^T [32 tokens x 16 heads] = K Q^T, K straight from memory as the
//     row operand (a lane holds 8 elements of a token's row), Q kept in
//     registers;
//   out^T [d x 16 heads] += V^T P, where the reduction index runs over the
//     tokens in the order in which the scores' lanes hold them, so P goes from
//     the exponentials into the operand without leaving its lane; V^T comes
//     from a [token][d] tile in LDS by transposed reads.
// A weight enters the product as three bfloat16 parts whose sum it is, with all
// of its 24 bits, and which are all positive, so an infinity of V stays one: of
// 65536 outputs 26 are not the rounding of the exact value (8 sequences of 32768
// to 65536, 64 heads on 8), where fp32 products in a serial sum leave 133.  The
// products of the remainders hide under the loads: with 16 bits of a weight and
// with all 290.3 and 290.6 us there, 49.8 and 49.9 for 10 of 5165, 9.7 and 10.2
// for one of 512.  The sums of the weights are fp32.  The rows of V behind the
// length are put as zeros into LDS (0 times what lies there would not be 0 for an
// infinity), the scores there are replaced, not added to.
// Measured: 8 sequences of 32768 to 65536 tokens, 64 query heads on 8 kv heads of
// 128, 279-290 us (5.6-5.8 TB/s; a streaming read reaches 5.6); 16 of 1 to 4096, 32
// heads, 106 us (5.1 TB/s); 8 of 16384 to 32768, 32 heads on 8 kv heads of 256, 274
// us (5.7 TB/s); one of 512, 32 heads, in a table of 512 9.6-10.2 us, at what 32 CUs
// read: eight waves take as long, two workgroups per head with half of V's columns
// each 0.5 us less, but 1 us more at 128 heads.

namespace {

__device__ __forceinline__ int64_t tokens_of(const AttnArgs& a, int64_t s) {
  const int64_t n = a.lengths[s], cap = a.table_cols << a.page_shift;
  return n < 0 ? 0 : n > cap ? cap : n;
}

// The pages of the two halves of a tile (-1: none, or behind the length).
struct Pages {
  int32_t of[2];
};
__device__ __forceinline__ Pages pages_at(const AttnArgs& a, const int32_t* table, int64_t tok, int64_t n) {
  Pages p;
#pragma unroll
  for (int h = 0; h < 2; ++h) p.of[h] = tok + 16 * h < n ? table[(tok + 16 * h) >> a.page_shift] : -1;
  return p;
}

// What the lanes of a wave hold of one tile.
template <int DP>
struct Tile {
  uint4 k[2][DP / 32];  // tokens 16 half + lane % 16, elements 32 i + 8 (lane / 16) ..
  uint4 v[DP / 16];     // pieces i * 64 + lane of the 32 rows
  bool ok[2];           // the halves lie in pages of the cache
};

template <int DP>
__device__ __forceinline__ void load_tile(Tile<DP>& t, const AttnArgs& a, const Pages& p, int64_t tok, int kv,
                                          int lane) {
  constexpr int CH = DP / 8;  // 16-byte pieces of a padded row
  const int d = a.head_dim;
  int64_t base[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t page = __builtin_amdgcn_readfirstlane(p.of[h]);
    t.ok[h] = page >= 0 && page < a.num_pages;
    // without a page the loads go to the cache's first rows and count nothing
    const int64_t first = (tok + 16 * h) & ((1 << a.page_shift) - 1);
    base[h] = t.ok[h] ? ((((int64_t)page * a.kv_heads + kv) << a.page_shift) + first) * d : 0;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint16_t* row = a.k_cache + base[h] + (lane & 15) * d;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) {
      const int c = 32 * i + 8 * (lane >> 4);
      t.k[h][i] = *reinterpret_cast<const uint4*>(row + (c < d ? c : 0));
    }
  }
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) {
    const int idx = i * 64 + lane, r = idx / CH, c = idx % CH * 8;
    t.v[i] = *reinterpret_cast<const uint4*>(a.v_cache + (r < 16 ? base[0] : base[1]) + (r & 15) * d + (c < d ? c : 0));
  }
}

template <int DP, int W>
__global__ __launch_bounds__(64 * W) void paged_attention_kernel(AttnArgs a, int qtiles) {
  constexpr int CH = DP / 8;
  constexpr int PITCH = DP + 16;  // of the V tile: 16 rows of one column go to different banks
  constexpr int OP = DP + 4;      // of the partial outputs
  constexpr int WAVE_BYTES = kTile * PITCH * 2;
  static_assert(16 * OP * 4 <= WAVE_BYTES, "a wave's outputs take the place of its V tile");
  __shared__ __attribute__((aligned(16))) char lds[W * WAVE_BYTES];
  __shared__ float s_m[W][16], s_l[W][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15, d = a.head_dim;
  const int64_t s = blockIdx.y;
  int id = blockIdx.x;
  const int z = id % a.splits;
  id /= a.splits;
  const int qt = id % qtiles, kv = id / qtiles;
  const int group = a.q_heads / a.kv_heads;
  const int h0 = kv * group + qt * 16, heads = group - qt * 16 < 16 ? group - qt * 16 : 16;
  const int64_t n = tokens_of(a, s);
  const Cut cut = cut_of(n, a.splits, W);
  if (a.splits > 1 && z >= cut.parts) return;
  const int64_t first = z * cut.per;
  const int64_t last = first + cut.per < cut.tiles ? first + cut.per : cut.tiles;

  // Q^T: column col (a query head), reduction elements 32 i + 8 g ..
  bf16x8 q[DP / 32];
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) {
    const int c = 32 * i + 8 * g;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (col < heads && c < d)
      v = *reinterpret_cast<const uint4*>(a.q + s * a.q_stride + (int64_t)(h0 + col) * d + c);
    q[i] = __builtin_bit_cast(bf16x8, v);
  }
  const int32_t* table = a.table + s * a.table_cols;
  const float scale2 = a.scale * 1.44269504088896340736f;  // scores in base 2
  float m = -INFINITY, l = 0.0f;
  floatx4 acc[DP / 16];
#pragma unroll
  for (int t = 0; t < DP / 16; ++t) acc[t] = (floatx4){0, 0, 0, 0};
  __bf16* vt = reinterpret_cast<__bf16*>(lds + wave * WAVE_BYTES);

  // the loads of the next tile run under the products of this one, and the
  // look-up of the pages after that, so neither waits for the other
  Tile<DP> t;
  int64_t ti = first + wave;
  Pages pages = pages_at(a, table, ti * kTile, n);
  if (ti < last) load_tile<DP>(t, a, pages, ti * kTile, kv, lane);
  pages = pages_at(a, table, (ti + W) * kTile, n);
  for (; ti < last; ti += W) {
    const int64_t tok = ti * kTile;
    const bool full = tok + kTile <= n && t.ok[0] && t.ok[1];
    // V to LDS
    lds_in_order();
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int idx = i * 64 + lane, r = idx / CH, c = idx % CH * 8;
      uint4 v = t.v[i];
      if (!full && !(tok + r < n && (r < 16 ? t.ok[0] : t.ok[1]))) v = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(vt + r * PITCH + c) = v;
    }
    // scores
    floatx4 sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h] = (floatx4){0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        uint4 k = t.k[h][i];
        if (d < DP && 32 * i + 8 * g >= d) k = make_uint4(0, 0, 0, 0);
        sc[h] = mfma16(__builtin_bit_cast(bf16x8, k), q[i], sc[h]);
      }
    }
    const bool ok0 = t.ok[0], ok1 = t.ok[1];
    if (ti + W < last) load_tile<DP>(t, a, pages, tok + W * kTile, kv, lane);
    pages = pages_at(a, table, tok + 2 * W * kTile, n);
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = sc[j >> 2][j & 3] * scale2;
    if (!full) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(tok + 16 * (j >> 2) + 4 * g + (j & 3) < n && (j < 4 ? ok0 : ok1))) p[j] = -INFINITY;
    }
    float mt = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) mt = fmaxf(mt, p[j]);
    mt = fmaxf(mt, __shfl_xor(mt, 16, 64));
    mt = fmaxf(mt, __shfl_xor(mt, 32, 64));
    const float mu = mt == -INFINITY ? 0.0f : mt;
    if (__ballot(mt > m)) {
      const float old = __builtin_amdgcn_exp2f(m - mu);
      l *= old;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) acc[i] *= old;
    }
    m = mt;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = __builtin_amdgcn_exp2f(p[j] - mu);
      l += p[j];
    }
    bf16x8 part[3];
    split<true>(p, part);
    lds_in_order();
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const __bf16* src = vt + (4 * g + (col >> 2)) * PITCH + 16 * i + 4 * (col & 3);
      const short4_t v0 = ds_read_tr16(src), v1 = ds_read_tr16(src + 16 * PITCH);
      const short8_t v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int k = 0; k < 3; ++k) acc[i] = mfma16(__builtin_bit_cast(bf16x8, v), part[k], acc[i]);
    }
  }

  // join the waves: each lane group holds the sum of its own tokens
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
  lds_in_order();
  float* ow = reinterpret_cast<float*>(lds + wave * WAVE_BYTES);
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) *reinterpret_cast<floatx4*>(ow + col * OP + 16 * i + 4 * g) = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < heads * (d / 4); e += 64 * W) {
    const int h = e / (d / 4), c = e % (d / 4) * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w][h]);
    const float mu = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
    floatx4 o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][h] - mu);
      sum += s_l[w][h] * f;
      o += *reinterpret_cast<const floatx4*>(reinterpret_cast<const float*>(lds + w * WAVE_BYTES) + h * OP + c) * f;
    }
    const int64_t row = s * a.q_heads + h0 + h;
    if (a.splits > 1) {
      *reinterpret_cast<floatx4*>(a.part_o + (row * a.splits + z) * d + c) = o;
      if (c == 0) a.part_ml[(row * a.splits + z) * 2] = mx, a.part_ml[(row * a.splits + z) * 2 + 1] = sum;
    } else {
      o *= sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<uint2*>(a.out + row * d + c) = make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
      if (a.lse && c == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

// Joins the parts of a sequence, one workgroup per sequence and head: its
// threads hold four elements of the head each and take the parts in turns of
// 1024 / head_dim, then the turns' sums are added in order.
constexpr int kMaxSplits = 256;

__global__ __launch_bounds__(256) void paged_join_kernel(AttnArgs a) {
  __shared__ float s_f[kMaxSplits], s_m[4], s_l[4];
  __shared__ floatx4 s_o[256];
  const int64_t s = blockIdx.y, row = s * a.q_heads + blockIdx.x;
  const int d = a.head_dim, dq = d / 4, t = threadIdx.x;
  const int parts = (int)cut_of(tokens_of(a, s), a.splits, a.waves).parts;
  float m = -INFINITY, l = 0.0f;
  if (t < parts) {
    const float2 v = *reinterpret_cast<const float2*>(a.part_ml + (row * a.splits + t) * 2);
    m = v.x, l = v.y;
  }
  const float wm = wave_max(m);
  if ((t & 63) == 0) s_m[t >> 6] = wm;
  __syncthreads();
  const float mx = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), mu = mx == -INFINITY ? 0.0f : mx;
  const float f = __builtin_amdgcn_exp2f(m - mu);
  l *= f;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) l += __shfl_xor(l, o, 64);
  s_f[t] = f;
  if ((t & 63) == 0) s_l[t >> 6] = l;
  __syncthreads();
  const float sum = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]), inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.lse && t == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994530942f;
  const int turns = 256 / dq, turn = t / dq, c = t - turn * dq;
  floatx4 o = {0, 0, 0, 0};
  if (turn < turns) {
    const float* src = a.part_o + row * a.splits * d + 4 * c;
#pragma unroll 4
    for (int z = turn; z < parts; z += turns) o += *reinterpret_cast<const floatx4*>(src + (int64_t)z * d) * s_f[z];
  }
  s_o[t] = o;
  __syncthreads();
  if (t < dq) {
    for (int k = 1; k < turns; ++k) o += s_o[k * dq + t];
    o *= inv;
    *reinterpret_cast<uint2*>(a.out + row * d + 4 * t) = make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
  }
}

template <int DP, int W>
void attention_as(const AttnArgs& a, hipStream_t stream) {
  const int qtiles = (a.q_heads / a.kv_heads + 15) / 16;
  hipLaunchKernelGGL((paged_attention_kernel<DP, W>), dim3((unsigned)(a.kv_heads * qtiles * a.splits), (unsigned)a.S),
                     dim3(64 * W), 0, stream, a, qtiles);
}

template <int DP>
void attention_waves(const AttnArgs& a, hipStream_t stream) {
  if (a.waves == 8) attention_as<DP, 8>(a, stream);
  else attention_as<DP, 4>(a, stream);
}

}  // namespace

// Eight waves per workgroup for large calls (by what the table can hold: 128
// tiles per CU), else four: with fewer, longer streams large calls read a little
// faster (64 sequences of 1 to 2048, 32 heads: 197 us with four, 188 with eight;
// 8 of 32768 to 65536, 8 kv heads: 284 and 280), in smaller ones the waves run
// out of tiles (10 of 5165, 8 kv heads: 47 us and 53; 4 of 2048, 32 heads: 31
// and 38).  Heads of more than 128 keep four: eight waves' registers and V tiles
// would leave a CU nothing else.
static int waves_for(int64_t groups, int head_dim, int64_t max_len) {
  return groups * ((max_len + kTile - 1) / kTile) >= 128 * 256 && head_dim <= 128 ? 8 : 4;
}
static int64_t groups_of(int64_t S, int q_heads, int kv_heads) {
  return S * kv_heads * ((q_heads / kv_heads + 15) / 16);
}

// No split for tables of up to 512 tokens, where one launch takes less than two
// (1 sequence of 512, 32 heads: 9.5 us against 10.9; 16 of 384: 18.5 and 25); else
// enough workgroups for four per CU, which evens out sequences of different
// lengths as far as it cuts them, or two for less than four sequences (1 of 131072,
// 32 on 8 heads: 105 us with four, 100 with two), as far as the table gives each
// wave its tiles.  The rule knows the table, not the lengths: one of 512 tokens
// takes 13.8 us in a table of 4096; and 1024 groups or more are not cut at all, so
// one long sequence among them sets the time (one of 65536 and 31 of 256, 32 kv
// heads: 714 us, where the bytes take 215).
int paged_splits(int64_t S, int q_heads, int kv_heads, int head_dim, int64_t max_len) {
  if (S == 0 || max_len <= 512) return 1;
  const int64_t groups = groups_of(S, q_heads, kv_heads), waves = waves_for(groups, head_dim, max_len);
  int64_t n = ((S < 4 ? 2 : 4) * 256 + groups - 1) / groups;
  const int64_t least = waves * kMinTiles * kTile, most = (max_len + least - 1) / least;
  if (n > most) n = most;
  if (n > kMaxSplits) n = kMaxSplits;
  return n < 1 ? 1 : (int)n;
}

hipError_t launch_paged_attention(const AttnArgs& args, hipStream_t stream) {
  AttnArgs a = args;
  a.waves = waves_for(groups_of(a.S, a.q_heads, a.kv_heads), a.head_dim, a.table_cols << a.page_shift);
  if (a.head_dim <= 64) attention_waves<64>(a, stream);
  else if (a.head_dim <= 96) attention_waves<96>(a, stream);
  else if (a.head_dim <= 128) attention_waves<128>(a, stream);
  else attention_as<256, 4>(a, stream);
  if (a.splits > 1)
    hipLaunchKernelGGL(paged_join_kernel, dim3(a.q_heads, (unsigned)a.S), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlora
