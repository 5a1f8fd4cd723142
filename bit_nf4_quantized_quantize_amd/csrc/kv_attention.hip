// Attention of one new token per sequence over a paged cache of any type, and
// over a prefix that the sequences share, gfx950 (definitions in
// include/qlora_kvcache.h).
//
// The narrow workgroups below are those of the bfloat16 cache's attention: the
// query heads of a kv head are the 16 columns of the products, a wave works alone
// on tiles of 32 tokens with a running maximum and sum, weights enter the product
// with V as three bfloat16 parts with all of their 24 bits, long lengths are cut
// and joined.  Over a prefix the columns are heads of any sequences, so its keys
// are read once for 16 rows.  Codes are read 16 bytes per lane and made bfloat16
// numbers, exactly, where they enter the products (E4M3: one instruction for two;
// whole numbers: three); a key's scale is put on its score and a value's on its
// weight in fp32, four of each per lane and tile.
// Bound by HBM, at half the bytes per token of bfloat16, so at twice the work per
// byte: 8 sequences of 32768 to 65536 tokens, 64 on 8 heads of 128, in int8 155-159
// us (830 MB, 5.3 TB/s; a streaming read reaches 5.6); 16 of 1 to 4096, 32 heads, in
// E4M3 57-60 us and 4 to 5 for the join (277 MB); one of 512, 32 heads, in int8 8.6
// us; 16 sequences behind 8191 shared tokens, 32 heads, bf16, 41 us (201 MB) and 5.
// Short own lengths behind a prefix are further off: 256 of 0 to 700, 32 on 8
// heads, E4M3, 50 us (189 MB take 34; 45 with even lengths), the first loads of a
// workgroup and its end being half of its life.  Behind a prefix of many rows these
// workgroups, the last to touch a row, also join its parts: 55 us, where a kernel
// for that took 11.  Not kept: Q in LDS (164 registers as before), registers for
// four waves per SIMD (spills, 57 -> 87 us).
#include <type_traits>

#include "device.h"
#include "kv_codes.h"
#include "kvcache.h"
#include "paged_device.h"

namespace qlora {

// ------------------------------------------- few rows or tokens: narrow workgroups

namespace {

template <int CT>
constexpr bool kCoded = CT != kCacheBf16;

__device__ __forceinline__ int64_t cut_length(int64_t n, int64_t cols, int shift) {
  const int64_t cap = cols << shift;
  return n < 0 ? 0 : n > cap ? cap : n;
}

// The table's entries for the two halves of a tile.  Any tile may be asked for:
// behind the table's end the last entry is read, and whether tokens are there is
// asked when the pages are used.
struct Halves {
  int32_t of[2];
};
__device__ __forceinline__ Halves halves_at(const int32_t* table, int64_t cols, int64_t tok, int shift) {
  Halves p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = (tok + 16 * h) >> shift;
    p.of[h] = table[at < cols ? at : cols - 1];
  }
  return p;
}

// What the lanes of a wave hold of one tile of 32 tokens.
//   bf16:  k token 16 half + lane % 16, elements 32 i + 8 (lane / 16) ..
//   codes: the same token, elements 64 i + 16 (lane / 16) .., two steps of the
//          product in one load; the order of the elements in the reduction is
//          free as long as Q has the same
//   v: pieces i * 64 + lane of the 32 rows
template <int DP, int CT>
struct KvTile {
  static constexpr int EV = kCoded<CT> ? 16 : 8;                    // elements in 16 bytes
  static constexpr int KI = kCoded<CT> ? (DP + 63) / 64 : DP / 32;  // loads of a key per lane
  static constexpr int STEPS = kCoded<CT> ? 2 * KI : KI;            // of 32 elements
  static constexpr int VI = kTile * DP / EV / 64;
  uint4 k[2][KI];
  uint4 v[VI];
  float4 ks[2], vs[2];  // scales of the tokens 16 half + 4 (lane / 16) ..
  bool ok[2];           // the halves lie in pages of the cache
};

// Where the halves' rows are; sets t.ok.
struct Rows {
  int64_t of[2];
};
template <int DP, int CT>
__device__ __forceinline__ Rows rows_at(KvTile<DP, CT>& t, const KvCache& c, const Halves& p, int64_t tok, int64_t n,
                                        int kv) {
  Rows r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int32_t page = __builtin_amdgcn_readfirstlane(p.of[h]);
    t.ok[h] = tok + 16 * h < n && page >= 0 && page < c.num_pages;
    // without a page the loads go to the cache's first rows and count nothing
    const int64_t first = (tok + 16 * h) & ((1 << c.page_shift) - 1);
    r.of[h] = t.ok[h] ? (((int64_t)page * c.kv_heads + kv) << c.page_shift) + first : 0;
  }
  return r;
}
template <int DP, int CT>
__device__ __forceinline__ void load_v(KvTile<DP, CT>& t, const KvCache& c, const Rows& row, int lane) {
  using Tile = KvTile<DP, CT>;
  typedef typename std::conditional<kCoded<CT>, uint8_t, uint16_t>::type Elem;
  constexpr int CH = DP / Tile::EV;
  const int d = c.head_dim;
#pragma unroll
  for (int i = 0; i < Tile::VI; ++i) {
    const int idx = i * 64 + lane, r = idx / CH, e = idx % CH * Tile::EV;
    t.v[i] = *reinterpret_cast<const uint4*>((const Elem*)c.v + ((r < 16 ? row.of[0] : row.of[1]) + (r & 15)) * d +
                                             (e < d ? e : 0));
  }
}
template <int DP, int CT>
__device__ __forceinline__ void load_k(KvTile<DP, CT>& t, const KvCache& c, const Rows& row, int lane) {
  using Tile = KvTile<DP, CT>;
  typedef typename std::conditional<kCoded<CT>, uint8_t, uint16_t>::type Elem;
  const int d = c.head_dim;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const Elem* key = (const Elem*)c.k + (row.of[h] + (lane & 15)) * d;
#pragma unroll
    for (int i = 0; i < Tile::KI; ++i) {
      const int e = (4 * i + (lane >> 4)) * Tile::EV;
      t.k[h][i] = *reinterpret_cast<const uint4*>(key + (e < d ? e : 0));
    }
    if constexpr (kCoded<CT>) {
      t.ks[h] = *reinterpret_cast<const float4*>(c.k_scale + row.of[h] + 4 * (lane >> 4));
      t.vs[h] = *reinterpret_cast<const float4*>(c.v_scale + row.of[h] + 4 * (lane >> 4));
    }
  }
}

__device__ __forceinline__ float part_of(const float4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// The query rows of a workgroup are the 16 columns of its products: heads that
// share a kv head, of one sequence or, over the prefix, of any.
struct Columns {
  int64_t s;    // sequence, or -1: rows of all of them from r0
  int64_t r0;   // first row (sequence * group + head of the group), or head
  int n, group, kv;
};
__device__ __forceinline__ void place_of(const Columns& c, int col, int64_t* s, int* head) {
  const int64_t r = c.r0 + col;
  if (c.s >= 0) {
    *s = c.s, *head = c.kv * c.group + (int)r;
  } else {
    *s = (uint32_t)r / (uint32_t)c.group, *head = c.kv * c.group + (int)((uint32_t)r % (uint32_t)c.group);
  }
}

// Grid: with ptiles tiles of 16 rows of a prefix first their kv heads and parts, then
// the sequences' kv heads, tiles of heads and parts, all in x; else those in x and
// the sequences in y.
template <int DP, int W, int CT>
__global__ __launch_bounds__(64 * W, DP > 128 ? 1 : 2) void kv_attention_kernel(KvAttnArgs a, int qtiles, int ptiles) {
  using Tile = KvTile<DP, CT>;
  constexpr int CH = DP / Tile::EV;
  constexpr int PITCH = DP + 16;  // of the V tile: 16 rows of one column go to different banks
  constexpr int OP = DP + 4;      // of the partial outputs
  constexpr int WAVE_BYTES = kTile * PITCH * 2;
  static_assert(16 * OP * 4 <= WAVE_BYTES, "a wave's outputs take the place of its V tile");
  __shared__ __attribute__((aligned(16))) char lds[W * WAVE_BYTES];
  __shared__ float s_m[W][16], s_l[W][16];

  const KvCache& kc = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15, d = kc.head_dim;
  const int group = a.q_heads / kc.kv_heads, parts = a.psplits + a.splits;
  uint32_t id = blockIdx.x;
  const uint32_t jobs = (uint32_t)kc.kv_heads * a.psplits, own = (uint32_t)(kc.kv_heads * qtiles) * a.splits;
  const bool shared = id < ptiles * jobs;
  Columns cols;
  cols.group = group;
  int z;
  int64_t n, table_cols;
  const int32_t* table;
  Cut32 cut;
  Halves pages = {{-1, -1}};  // of the first tile, asked for beside the length where it does not depend on it
  if (shared) {
    const uint32_t tile = id / jobs;
    id -= tile * jobs;
    z = id % (uint32_t)a.psplits;
    cols.kv = id / (uint32_t)a.psplits;
    cols.s = -1, cols.r0 = (int64_t)tile * 16;
    const int64_t left = a.S * group - cols.r0;
    cols.n = left < 16 ? (int)left : 16;
    table = a.prefix_table, table_cols = a.prefix_cols;
    if (z == 0) pages = halves_at(table, table_cols, wave * kTile, kc.page_shift);
    n = cut_length(*a.prefix_len, a.prefix_cols, kc.page_shift);
    cut = cut32_of((uint32_t)n, a.psplits, W);
  } else {
    uint32_t s = blockIdx.y;
    if (ptiles) id -= ptiles * jobs, s = id / own, id -= s * own;
    z = id % (uint32_t)a.splits;
    id /= (uint32_t)a.splits;
    const int qt = id % (uint32_t)qtiles;
    cols.kv = id / (uint32_t)qtiles;
    cols.s = s, cols.r0 = qt * 16;
    cols.n = group - qt * 16 < 16 ? group - qt * 16 : 16;
    table = a.table + cols.s * a.table_cols, table_cols = a.table_cols;
    if (z == 0 && table_cols) pages = halves_at(table, table_cols, wave * kTile, kc.page_shift);
    n = cut_length(a.lengths[cols.s], a.table_cols, kc.page_shift);
    cut = cut32_of((uint32_t)n, a.splits, W);
  }
  if (parts > 1 && !a.joined && (uint32_t)z >= cut.parts) return;
  const int64_t first = (int64_t)z * cut.per;
  const int64_t last = first + cut.per < cut.tiles ? first + cut.per : cut.tiles;

  // Q^T: column col (a query row), reduction elements as the keys' lanes hold them
  bf16x8 q[Tile::STEPS];
  {
    int64_t s = 0;
    int head = 0;
    if (col < cols.n) place_of(cols, col, &s, &head);
    const uint16_t* src = a.q + s * a.q_stride + (int64_t)head * d;
#pragma unroll
    for (int i = 0; i < Tile::STEPS; ++i) {
      const int e = kCoded<CT> ? 64 * (i / 2) + 16 * g + 8 * (i % 2) : 32 * i + 8 * g;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (col < cols.n && e < d) v = *reinterpret_cast<const uint4*>(src + e);
      q[i] = __builtin_bit_cast(bf16x8, v);
    }
  }
  const float scale2 = a.scale * 1.44269504088896340736f;  // scores in base 2
  float m = -INFINITY, l = 0.0f;
  floatx4 acc[DP / 16];
#pragma unroll
  for (int t = 0; t < DP / 16; ++t) acc[t] = (floatx4){0, 0, 0, 0};
  __bf16* vt = reinterpret_cast<__bf16*>(lds + wave * WAVE_BYTES);

  // The loads of the next tile run under the products of this one, its values'
  // from the moment that this one's are in LDS, and the look-up of the pages after
  // that, so neither waits for the other.
  Tile t;
  int64_t ti = first + wave;
  if (ti < last) {
    if (z) pages = halves_at(table, table_cols, ti * kTile, kc.page_shift);
    const Rows r = rows_at(t, kc, pages, ti * kTile, n, cols.kv);
    load_k(t, kc, r, lane);
    load_v(t, kc, r, lane);
    pages = halves_at(table, table_cols, (ti + W) * kTile, kc.page_shift);
  }
  for (; ti < last; ti += W) {
    const int64_t tok = ti * kTile;
    const bool full = tok + kTile <= n && t.ok[0] && t.ok[1], more = ti + W < last;
    // V to LDS
    lds_in_order();
#pragma unroll
    for (int i = 0; i < Tile::VI; ++i) {
      const int idx = i * 64 + lane, r = idx / CH, e = idx % CH * Tile::EV;
      uint4 v = t.v[i];
      if (!full && !(tok + r < n && (r < 16 ? t.ok[0] : t.ok[1]))) v = make_uint4(0, 0, 0, 0);
      uint4* dst = reinterpret_cast<uint4*>(vt + r * PITCH + e);
      if constexpr (kCoded<CT>) {
        dst[0] = numbers<CT>(v.x, v.y);
        dst[1] = numbers<CT>(v.z, v.w);
      } else {
        dst[0] = v;
      }
    }
    const bool ok0 = t.ok[0], ok1 = t.ok[1];
    Rows next;
    if (more) {
      next = rows_at(t, kc, pages, tok + W * kTile, n, cols.kv);
      load_v(t, kc, next, lane);
    }
    // scores
    floatx4 sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h] = (floatx4){0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < Tile::KI; ++i) {
        uint4 k = t.k[h][i];
        if (d < 4 * Tile::KI * Tile::EV && (4 * i + g) * Tile::EV >= d) k = make_uint4(0, 0, 0, 0);
        if constexpr (kCoded<CT>) {
          sc[h] = mfma16(__builtin_bit_cast(bf16x8, numbers<CT>(k.x, k.y)), q[2 * i], sc[h]);
          sc[h] = mfma16(__builtin_bit_cast(bf16x8, numbers<CT>(k.z, k.w)), q[2 * i + 1], sc[h]);
        } else {
          sc[h] = mfma16(__builtin_bit_cast(bf16x8, k), q[i], sc[h]);
        }
      }
    }
    float p[8], vs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = sc[j >> 2][j & 3] * (kCoded<CT> ? part_of(t.ks[j >> 2], j & 3) * scale2 : scale2);
      vs[j] = kCoded<CT> ? part_of(t.vs[j >> 2], j & 3) : 1.0f;
    }
    if (more) {
      load_k(t, kc, next, lane);
      pages = halves_at(table, table_cols, tok + 2 * W * kTile, kc.page_shift);
    }
    if (!full) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(tok + 16 * (j >> 2) + 4 * g + (j & 3) < n && (j < 4 ? ok0 : ok1))) p[j] = -INFINITY, vs[j] = 0.0f;
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
      if constexpr (kCoded<CT>) p[j] *= vs[j];
    }
    bf16x8 part[3];
    split<!kCoded<CT>>(p, part);
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
  uint32_t pre = 0;
  if (a.joined)
    pre = cut32_of((uint32_t)cut_length(*a.prefix_len, a.prefix_cols, kc.page_shift), a.psplits, a.pwaves).parts;
  for (int e = threadIdx.x; e < cols.n * (d / 4); e += 64 * W) {
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
    int64_t s;
    int head;
    place_of(cols, h, &s, &head);
    const int64_t row = s * a.q_heads + head;
    if (a.joined) {  // the prefix's parts are there: this is the row's last one
      const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * parts;
      const float* src = a.part_o + row * parts * d + c;
      float all = mx;
      for (uint32_t i = 0; i < pre; ++i) all = fmaxf(all, ml[i].x);
      const float au = all == -INFINITY ? 0.0f : all, f = __builtin_amdgcn_exp2f(mx - au);
      sum *= f, o *= f;
#pragma unroll 8
      for (uint32_t i = 0; i < pre; ++i) {
        const float2 v = ml[i];
        const float g2 = __builtin_amdgcn_exp2f(v.x - au);
        sum += v.y * g2;
        o += *reinterpret_cast<const floatx4*>(src + (int64_t)i * d) * g2;
      }
      mx = all;
    }
    if (parts > 1 && !a.joined) {
      const int64_t at = row * parts + (shared ? z : a.psplits + z);
      *reinterpret_cast<floatx4*>(a.part_o + at * d + c) = o;
      if (c == 0) a.part_ml[at * 2] = mx, a.part_ml[at * 2 + 1] = sum;
    } else {
      o *= sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<uint2*>(a.out + row * d + c) = make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
      if (a.lse && c == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994530942f;
    }
  }
}

// Joins the parts of a row: TEAM waves each take the parts in turns, a turn being
// as many parts as fit into the wave with four elements of the head per lane (256 /
// head_dim); the turns' sums are added in order.  Four waves per workgroup.
constexpr int kMaxParts = 256;

template <int TEAM>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttnArgs a, Div heads) {
  __shared__ floatx4 s_o[TEAM > 1 ? TEAM : 1][64];
  __shared__ float s_sum[TEAM > 1 ? TEAM : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, member = wave % TEAM;
  const int d = a.c.head_dim, dq = d / 4, all = a.psplits + a.splits;
  const int64_t row = ((int64_t)blockIdx.x * 4 + wave) / TEAM;
  if (row >= a.S * a.q_heads) return;  // never part of a team
  const int s = (int)row / heads;
  const int own = cut32_of((uint32_t)cut_length(a.lengths[s], a.table_cols, a.c.page_shift), a.splits, a.waves).parts;
  int pre = 0;
  if (a.psplits)
    pre = cut32_of((uint32_t)cut_length(*a.prefix_len, a.prefix_cols, a.c.page_shift), a.psplits, a.pwaves).parts;
  // part i of those there are lies at i, behind the prefix's at psplits ..
  const int parts = pre + own, gap = a.psplits - pre;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + row * all;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 64) m = fmaxf(m, ml[i < pre ? i : i + gap].x);
  const float mx = wave_max(m), mu = mx == -INFINITY ? 0.0f : mx;
  const int turns = 64 / dq, turn = lane / dq, c = lane - turn * dq;
  float sum = 0.0f;
  floatx4 o = {0, 0, 0, 0};
  if (turn < turns) {
    const float* src = a.part_o + row * all * d + 4 * c;
#pragma unroll 8
    for (int i = member * turns + turn; i < parts; i += TEAM * turns) {
      const int at = i < pre ? i : i + gap;
      const float2 v = ml[at];
      const float f = __builtin_amdgcn_exp2f(v.x - mu);
      sum += v.y * f;
      o += *reinterpret_cast<const floatx4*>(src + (int64_t)at * d) * f;
    }
  }
  // the other turns' lanes hold the same elements
  float all_sum = sum;
  floatx4 all_o = o;
  for (int k = 1; k < turns; ++k) {
    const int from = k * dq + c;
    all_sum += __shfl(sum, from, 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) all_o[j] += __shfl(o[j], from, 64);
  }
  if constexpr (TEAM > 1) {
    s_o[member][lane] = all_o;
    if (lane == 0) s_sum[member] = all_sum;
    __syncthreads();
    if (member > 0) return;
#pragma unroll
    for (int k = 1; k < TEAM; ++k) all_o += s_o[k][lane], all_sum += s_sum[k];
  }
  if (lane >= dq) return;
  all_o *= all_sum == 0.0f ? 0.0f : 1.0f / all_sum;
  *reinterpret_cast<uint2*>(a.out + row * d + 4 * lane) = make_uint2(pack_bf2(all_o[0], all_o[1]), pack_bf2(all_o[2], all_o[3]));
  if (a.lse && lane == 0) a.lse[row] = all_sum == 0.0f ? -INFINITY : (mx + log2f(all_sum)) * 0.69314718055994530942f;
}

template <int DP, int W, int CT>
void attention_as(const KvAttnArgs& a, hipStream_t stream) {
  const int group = a.q_heads / a.c.kv_heads, qtiles = (group + 15) / 16;
  const int64_t ptiles = a.psplits && !a.wide ? (a.S * group + 15) / 16 : 0;
  const int64_t own = (int64_t)a.c.kv_heads * qtiles * a.splits, jobs = ptiles * a.c.kv_heads * a.psplits;
  const dim3 grid = ptiles ? dim3((unsigned)(jobs + a.S * own)) : dim3((unsigned)own, (unsigned)a.S);
  hipLaunchKernelGGL((kv_attention_kernel<DP, W, CT>), grid, dim3(64 * W), 0, stream, a, qtiles, (int)ptiles);
}

template <int DP, int CT>
void attention_waves(const KvAttnArgs& a, hipStream_t stream) {
  if (a.waves == 8) attention_as<DP, 8, CT>(a, stream);
  else attention_as<DP, 4, CT>(a, stream);
}

template <int CT>
void attention_of(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.head_dim <= 64) attention_waves<64, CT>(a, stream);
  else if (a.c.head_dim <= 96) attention_waves<96, CT>(a, stream);
  else if (a.c.head_dim <= 128) attention_waves<128, CT>(a, stream);
  else attention_as<256, 4, CT>(a, stream);
}

// Eight waves per workgroup for large calls, by what the table can hold (128 tiles
// per CU), where fewer, longer streams read a little faster (8 sequences of 32768 to
// 65536 in int8, 64 on 8 heads: 162 us with four, 155 with eight; 16 of 1 to 4096,
// 32 heads in E4M3: 58 and 57), and for codes where one launch has fewer workgroups
// than the card CUs (one of 512, 32 heads: 10.3 and 8.6); else four: in between the
// waves run out of tiles (256 of 0 to 700 behind a prefix, 32 on 8 heads: 49 and
// 62, two waves 51).  Heads of more than 128 keep four: eight waves' registers and V
// tiles would leave a CU nothing else.
int waves_for(const KvAttnArgs& a) {
  if (a.psplits || a.c.head_dim > 128) return 4;
  const int64_t group = a.q_heads / a.c.kv_heads, groups = a.S * a.c.kv_heads * ((group + 15) / 16);
  const int64_t tiles = ((a.table_cols << a.c.page_shift) + kTile - 1) / kTile;
  if (a.splits == 1 && a.c.type != kCacheBf16 && groups <= 256) return 8;
  return groups * tiles >= 128 * 256 ? 8 : 4;
}

}  // namespace

// Rows of a prefix's workgroup: narrow ones (0) up to 32, and as long as they read
// little in all, in the launch of the own tokens instead of one before it (128 rows,
// 8 kv heads, int8, 1000 tokens 20 us, wide 27; 4000, at the limit, 31 and 33; 8000
// 46 and 38; with 32 kv heads even at twice the limit or four times, 128 rows of 2000
// 56 and 63, of 4000 76 and 73).  1024 rows at most, so that a grid holds them.  Wide
// ones of 128 up to 256 rows (256 of 8 kv heads, 4000 tokens 37 us, with 256 42; 8000
// 45 and 50; 512 of 16000 101 and 93).
static int wide_rows(int64_t rows, const KvCache& c, int64_t prefix_cols) {
  const int64_t reads = ((rows + 15) / 16) * c.kv_heads * (prefix_cols << c.page_shift);
  if (rows <= 32 || (rows <= 1024 && reads <= 1 << 18)) return 0;
  return rows <= 256 || c.head_dim > 128 ? 128 : 256;
}
constexpr int kWideWaves = 2;  // a part of the prefix has the tiles of that many narrow waves at least

// Own tokens stay whole up to that many of them, so that their workgroups can join
// the prefix's parts.
constexpr int64_t kWholeOwn = 1024;

// The own tokens' parts as without a prefix; but whole where their workgroups then
// join the prefix's parts (launch_kv_attention), if these are enough and lengths
// end at kWholeOwn (64 sequences of 100 to 800, 64 on 8 heads: 26 us, against 23 and
// 11 for the join; finer parts, for the join, do not pay: 256 of 0 to 700 in parts
// of 256 tokens 52 us, whole 50).  Behind 8000 tokens, 64 sequences of 1 to 1024, 32
// on 8 heads, int8: whole 57 us, cut 63; of 1 to 2048 75 and 74; 32 of 1 to 16384
// 270 and 164, one of 16384 among 31 of 256 262 and 95.
// The prefix's: a workgroup per CU, as far as its length gives each some tiles (16 rows
// of 8191 tokens, 32 heads: 41 us so, 45 with two, 49 with four).
KvParts kv_parts(const KvCache& c, int64_t S, int q_heads, int64_t table_cols, int64_t prefix_cols) {
  KvParts p;
  const int64_t max_len = table_cols << c.page_shift;
  p.own = paged_splits(S, q_heads, c.kv_heads, c.head_dim, max_len);
  p.prefix = 0;
  if (!prefix_cols || !S) return p;
  const int64_t rows = S * (q_heads / c.kv_heads), cap = prefix_cols << c.page_shift;
  const int wide = wide_rows(rows, c, prefix_cols);
  const int64_t groups = c.kv_heads * (wide ? (rows + wide - 1) / wide : (rows + 15) / 16);
  if (wide && q_heads > c.kv_heads && max_len <= kWholeOwn &&
      S * c.kv_heads * ((q_heads / c.kv_heads + 15) / 16) >= 256)
    p.own = 1;
  int64_t n = (256 + groups - 1) / groups;
  const int64_t least = (wide ? kWideWaves : 4) * kMinTiles * kTile, most = (cap + least - 1) / least;
  if (n > most) n = most;
  if (n > kMaxParts / 2) n = kMaxParts / 2;
  p.prefix = n < 1 ? 1 : (int)n;
  if (p.own > kMaxParts / 2) p.own = kMaxParts / 2;
  return p;
}

hipError_t launch_kv_attention(const KvAttnArgs& args, hipStream_t stream) {
  KvAttnArgs a = args;
  const int64_t group = a.q_heads / a.c.kv_heads;
  a.waves = waves_for(a);
  a.wide = a.psplits ? wide_rows(a.S * group, a.c, a.prefix_cols) : 0;
  a.pwaves = a.wide ? kWideWaves : a.waves;
  // A workgroup of one row would join it with a few of its threads only (behind 2000
  // tokens, bf16, 256 sequences on 32 of 32 heads: joined 148 us, by the kernel below
  // 122; 128 on 8 of 32: 45 and 49).
  a.joined = a.wide && a.splits == 1 && group > 1;
  if (a.wide) {
    const hipError_t e = launch_kv_prefix(a, stream);
    if (e != hipSuccess) return e;
  }
  if (a.c.type == kCacheInt8) attention_of<kCacheInt8>(a, stream);
  else if (a.c.type == kCacheE4m3) attention_of<kCacheE4m3>(a, stream);
  else attention_of<kCacheBf16>(a, stream);
  if (a.psplits + a.splits > 1 && !a.joined) {
    // a wave per row once the rows fill the card (4096 rows of 9 parts: 7.0 us, with
    // four waves 12.6; 512 rows of 16: 9.5 and 4.2)
    const int64_t rows = a.S * a.q_heads;
    if (rows >= 2048)
      hipLaunchKernelGGL(kv_join_kernel<1>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, div_by(a.q_heads));
    else
      hipLaunchKernelGGL(kv_join_kernel<4>, dim3((unsigned)rows), dim3(256), 0, stream, a, div_by(a.q_heads));
  }
  return hipGetLastError();
}

}  // namespace qlora
