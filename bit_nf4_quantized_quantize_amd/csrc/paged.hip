// The paged key-value cache, gfx950: the plan of a batch (pages, slots and
// positions from the requests' lengths) and the attention of one new token
// per sequence over the cache (definitions in include/qlora_decoder.h).
#include "decoder.h"
#include "device.h"

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

__device__ __forceinline__ int pages_of(int64_t tokens, int page) { return (int)((tokens + page - 1) / page); }

__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanArgs a) {
  extern __shared__ int32_t lds[];  // starts [S + 1], first page taken [S + 1]
  __shared__ int32_t wave[2][kPlanThreads / 64];
  int32_t* starts = lds;
  int32_t* first = lds + a.S + 1;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int32_t run_t = 0, run_p = 0;
  for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    int32_t c = 0, n = 0;
    if (s < a.S) {
      c = a.cached[s] < 0 ? 0 : a.cached[s];
      n = a.fresh[s] < 0 ? 0 : a.fresh[s];
    }
    const int32_t p = pages_of((int64_t)c + n, a.page_size) - pages_of(c, a.page_size);
    int32_t vt = n, vp = p;  // inclusive sums over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t ut = __shfl_up(vt, o, 64), up = __shfl_up(vp, o, 64);
      if (lane >= o) vt += ut, vp += up;
    }
    if (lane == 63) wave[0][wv] = vt, wave[1][wv] = vp;
    __syncthreads();
    int32_t bt = run_t, bp = run_p;
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      if (w < wv) bt += wave[0][w], bp += wave[1][w];
      run_t += wave[0][w], run_p += wave[1][w];
    }
    if (s < a.S) {
      starts[s] = bt + vt - n;
      first[s] = bp + vp - p;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) starts[a.S] = run_t, first[a.S] = run_p;
  __syncthreads();

  const int64_t gid = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  const int64_t gsz = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t s = gid; s <= a.S; s += gsz) {
    a.starts[s] = starts[s];
    if (s < a.S) a.total[s] = (a.cached[s] < 0 ? 0 : a.cached[s]) + starts[s + 1] - starts[s];
  }
  if (gid == 0) *a.pages_needed = run_p;
  // new table entries, in the order of the free list
  for (int64_t i = gid; i < run_p; i += gsz) {
    int lo = 0, hi = a.S;  // the last sequence whose first page is at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid;
    }
    const int64_t col = pages_of(a.cached[lo] < 0 ? 0 : a.cached[lo], a.page_size) + (i - first[lo]);
    if (col < a.table_cols) a.table[lo * a.table_cols + col] = i < a.n_free ? a.free_pages[i] : -1;
  }
  for (int64_t t = gid; t < a.T; t += gsz) {
    int32_t slot = -1;
    int64_t pos = 0;
    if (t < run_t) {
      int lo = 0, hi = a.S;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid;
      }
      const int32_t c = a.cached[lo] < 0 ? 0 : a.cached[lo];
      pos = c + (t - starts[lo]);
      const int64_t col = pos / a.page_size, have = pages_of(c, a.page_size);
      int32_t page = -1;
      if (col < a.table_cols) {
        if (col < have) {
          page = a.table[lo * a.table_cols + col];
        } else {
          const int64_t i = first[lo] + col - have;
          if (i < a.n_free) page = a.free_pages[i];
        }
      }
      if (page >= 0) {
        const int64_t v = (int64_t)page * a.page_size + pos % a.page_size;
        slot = v < ((int64_t)1 << 31) ? (int32_t)v : -1;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = (int32_t)pos;
  }
}

}  // namespace

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream) {
  int64_t wgs = (a.T + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  wgs = wgs < 1 ? 1 : wgs > 256 ? 256 : wgs;
  hipLaunchKernelGGL(paged_plan_kernel, dim3((unsigned)wgs), dim3(kPlanThreads),
                     2 * (size_t)(a.S + 1) * sizeof(int32_t), stream, a);
  return hipGetLastError();
}

// -------------------------------------------------------------- attention
//
// One wave per sequence and query head: scores of 64 tokens at a time, a
// token per lane; then the weighted sum of their values, four elements of the
// head per lane.

namespace {

__global__ __launch_bounds__(64) void paged_attention_kernel(AttnArgs a) {
  __shared__ float p_s[64];
  __shared__ int64_t row_s[64];
  const int64_t s = blockIdx.y;
  const int h = blockIdx.x, lane = threadIdx.x, d = a.head_dim;
  const int j = h / (a.q_heads / a.kv_heads);
  const int page = 1 << a.page_shift;
  int64_t n = a.lengths[s];
  const int64_t cap = a.table_cols << a.page_shift;
  n = n < 0 ? 0 : n > cap ? cap : n;
  const uint16_t* q = a.q + s * a.q_stride + (int64_t)h * d;
  float m = -INFINITY, l = 0.0f, acc[4] = {0, 0, 0, 0};
  for (int64_t t0 = 0; t0 < n; t0 += 64) {
    const int64_t t = t0 + lane;
    int64_t row = -1;
    float sc = -INFINITY;
    if (t < n) {
      const int32_t pg = a.table[s * a.table_cols + (t >> a.page_shift)];
      if (pg >= 0 && pg < a.num_pages) {
        row = ((((int64_t)pg * a.kv_heads + j) << a.page_shift) + (t & (page - 1))) * d;
        float dot = 0.0f;
        for (int e = 0; e < d; ++e) dot = __builtin_fmaf(bf2f(q[e]), bf2f(a.k_cache[row + e]), dot);
        sc = dot * a.scale;
      }
    }
    const float mt = fmaxf(m, wave_max(sc));
    const float mu = mt == -INFINITY ? 0.0f : mt;
    const float p = row < 0 ? 0.0f : expf(sc - mu), old = expf(m - mu);
    m = mt;
    float ps = p;
    for (int o = 1; o < 64; o <<= 1) ps += __shfl_xor(ps, o, 64);
    l = l * old + ps;
    p_s[lane] = p;
    row_s[lane] = row;
    __syncthreads();
    for (int i = 0; i < 4; ++i) acc[i] *= old;
    for (int i = 0; i < 64; ++i) {
      if (row_s[i] < 0) continue;
      for (int e = 0; e < 4; ++e)
        if (lane * 4 + e < d) acc[e] = __builtin_fmaf(p_s[i], bf2f(a.v_cache[row_s[i] + lane * 4 + e]), acc[e]);
    }
    __syncthreads();
  }
  for (int e = 0; e < 4; ++e)
    if (lane * 4 + e < d) a.out[(s * a.q_heads + h) * d + lane * 4 + e] = f2bf(l > 0.0f ? acc[e] / l : 0.0f);
  if (a.lse && lane == 0) a.lse[s * a.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

int paged_splits(int64_t, int, int, int64_t) { return 1; }

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(paged_attention_kernel, dim3(a.q_heads, (unsigned)a.S), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlora
