// The residual update of a decoder block with its norms, gfx950: forward and
// backward (formulas in include/qlora_decoder.h).
//
// Both directions are streams over rows of D elements with one or two row
// means in between, bound by HBM: the forward reads x and h and writes xo and
// n once, the backward reads dxo, xo, dn and h and writes dx and dh once.  A
// row is held in the registers of its threads (TPR threads, NV chunks of 8
// elements each), so nothing is read twice; rows of up to 512 x 2 elements
// take one wave, wider ones a workgroup.
#include "decoder.h"
#include "device.h"

namespace qlora {

namespace {

// Eight elements of a row as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
};

__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// How a thread's chunk c maps to elements of its row.  VEC (D % 8 == 0, so
// every row starts 16-byte aligned): 8 consecutive elements; otherwise
// element by element, consecutive threads on consecutive elements.
template <int TPR, bool VEC>
struct Map {
  static __device__ __forceinline__ int at(int c, int i, int t) {
    return VEC ? (c * TPR + t) * 8 + i : (c * 8 + i) * TPR + t;
  }
  static __device__ __forceinline__ Raw8<uint16_t> load(const uint16_t* row, int c, int t, int D) {
    Raw8<uint16_t> r = {{0, 0, 0, 0}};
    if (VEC) {
      const int j = at(c, 0, t);
      if (j < D) {
        const uint4 q = *reinterpret_cast<const uint4*>(row + j);
        r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = at(c, i, t);
        const uint32_t e = j < D ? row[j] : 0;
        r.w[i >> 1] |= e << (16 * (i & 1));
      }
    }
    return r;
  }
  static __device__ __forceinline__ Raw8<float> load(const float* row, int c, int t, int D) {
    Raw8<float> r;
    if (VEC) {
      const int j = at(c, 0, t);
      float4 a = make_float4(0, 0, 0, 0), b = a;
      if (j < D) {
        a = *reinterpret_cast<const float4*>(row + j);
        b = *reinterpret_cast<const float4*>(row + j + 4);
      }
      r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
      r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = at(c, i, t);
        r.v[i] = j < D ? row[j] : 0.0f;
      }
    }
    return r;
  }
  static __device__ __forceinline__ void store(uint16_t* row, const float (&v)[8], int c, int t, int D) {
    if (VEC) {
      const int j = at(c, 0, t);
      if (j < D)
        *reinterpret_cast<uint4*>(row + j) =
            make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at(c, i, t) < D) put(row + at(c, i, t), v[i]);
    }
  }
  static __device__ __forceinline__ void store(float* row, const float (&v)[8], int c, int t, int D) {
    if (VEC) {
      const int j = at(c, 0, t);
      if (j < D) {
        *reinterpret_cast<float4*>(row + j) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(row + j + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at(c, i, t) < D) put(row + at(c, i, t), v[i]);
    }
  }
};

template <int S>
__device__ __forceinline__ float dpp_ror(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + S, 0xF, 0xF, false));
}

// Sums of N values over the 64 lanes (every lane gets them).
template <int N>
__device__ __forceinline__ void wave_sum(float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] += dpp_ror<1>(v[k]);
    v[k] += dpp_ror<2>(v[k]);
    v[k] += dpp_ror<4>(v[k]);
    v[k] += dpp_ror<8>(v[k]);
  }
#pragma unroll
  for (int o = 16; o <= 32; o <<= 1) {
    float w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __shfl_xor(v[k], o, 64);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += w[k];
  }
}

// Sums over the TPR threads of a row.  `buf` holds two sets of wave sums used
// in turn, so one barrier per sum suffices: a set is written again only after
// the barrier of the sum in between, which every thread passes after it has
// read the set.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[3][16], int& turn) {
  wave_sum<N>(v);
  if (TPR == 64) return;
  float(*s)[16] = buf[turn];
  turn ^= 1;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k][threadIdx.x >> 6] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) t += s[k][w];
    v[k] = t;
  }
}

constexpr int wg_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <typename XT, typename HT, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(wg_threads(TPR)) void norm_fwd_kernel(NormArgs a) {
  using M = Map<TPR, VEC>;
  __shared__ float buf[2][3][16];
  constexpr int ROWS = wg_threads(TPR) / TPR;
  const int t = threadIdx.x % TPR, D = a.D;
  const float inv = 1.0f / (float)D;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR; r < a.T; r += (int64_t)gridDim.x * ROWS) {
    float x[NV][8];
    const XT* xr = (const XT*)a.x + r * D;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const auto v = M::load(xr, c, t, D);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[c][i] = v.get(i);
    }
    if (a.h) {
      Raw8<HT> h[NV];
      const HT* hr = (const HT*)a.h + r * D;
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NV; ++c) h[c] = M::load(hr, c, t, D);
      float k = a.alpha;
      if (a.w_post) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] += h[c].get(i) * h[c].get(i);
        row_sum<TPR, 1>(s, buf, turn);
        k *= 1.0f / sqrtf(s[0] * inv + a.eps);
      }
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        Raw8<float> w, g;
        if (a.w_post) w = M::load(a.w_post, c, t, D);
        if (a.gate) g = M::load(a.gate, c, t, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float u = h[c].get(i) * k;
          if (a.w_post) u *= w.get(i);
          if (a.gate) u *= g.get(i);
          x[c][i] += u;
        }
      }
    }
    if (a.xo) {
      XT* o = (XT*)a.xo + r * D;
#pragma unroll
      for (int c = 0; c < NV; ++c) M::store(o, x[c], c, t, D);
    }
    if (a.n) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += x[c][i] * x[c][i];
      row_sum<TPR, 1>(s, buf, turn);
      const float rs = 1.0f / sqrtf(s[0] * inv + a.eps);
      HT* o = (HT*)a.n + r * D;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const Raw8<float> w = M::load(a.w_pre, c, t, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * rs * w.get(i);
        M::store(o, x[c], c, t, D);
      }
    }
  }
}

// The backward of one row needs two rounds of row sums: first sum xo^2, sum a
// xo (for dx) and sum h^2, then sum b w_post h (for dh).  SUMS: the sums over
// tokens are kept in the thread's registers, one per element it owns, and
// written once per workgroup row group; norm_sums_kernel adds those.
template <typename XT, typename HT, int TPR, int NV, bool VEC, bool SUMS>
__global__ __launch_bounds__(wg_threads(TPR)) void norm_bwd_kernel(NormArgs a, int64_t parts) {
  using M = Map<TPR, VEC>;
  __shared__ float buf[2][3][16];
  constexpr int ROWS = wg_threads(TPR) / TPR;
  const int t = threadIdx.x % TPR, D = a.D;
  const float inv = 1.0f / (float)D;
  int turn = 0;
  float sp[NV][8], sg[NV][8], sw[NV][8];
  if (SUMS) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sp[c][i] = sg[c][i] = sw[c][i] = 0.0f;
  }
  const int64_t first = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  for (int64_t r = first; r < a.T; r += (int64_t)gridDim.x * ROWS) {
    Raw8<XT> xo[NV], dxo[NV];
    Raw8<HT> dn[NV], h[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      xo[c] = M::load((const XT*)a.x + r * D, c, t, D);
      if (a.dxo) dxo[c] = M::load((const XT*)a.dxo + r * D, c, t, D);
      if (a.dn) dn[c] = M::load((const HT*)a.dn + r * D, c, t, D);
      if (a.h) h[c] = M::load((const HT*)a.h + r * D, c, t, D);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};  // xo^2, a xo, h^2
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (a.dn) {
        const Raw8<float> w = M::load(a.w_pre, c, t, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = xo[c].get(i);
          s[0] += x * x;
          s[1] += dn[c].get(i) * w.get(i) * x;
        }
      }
      if (a.w_post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += h[c].get(i) * h[c].get(i);
      }
    }
    row_sum<TPR, 3>(s, buf, turn);
    const float rs = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float back = rs * rs * (s[1] * inv);
    const float rh = a.w_post ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    float g[NV][8];  // dx, then alpha * dx
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[c][i] = a.dxo ? dxo[c].get(i) : 0.0f;
      if (a.dn) {
        const Raw8<float> w = M::load(a.w_pre, c, t, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = xo[c].get(i), d = dn[c].get(i);
          g[c][i] += rs * (d * w.get(i) - x * back);
          if (SUMS) sw[c][i] += d * (x * rs);
        }
      }
      M::store((XT*)a.xo + r * D, g[c], c, t, D);
      Raw8<float> wp, gt;
      if (a.w_post) wp = M::load(a.w_post, c, t, D);
      if (a.gate) gt = M::load(a.gate, c, t, D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = a.h ? h[c].get(i) * rh : 0.0f;
        float b = g[c][i] * a.alpha;
        if (SUMS) sg[c][i] += b * (a.w_post ? y * wp.get(i) : y);
        if (a.gate) b *= gt.get(i);
        if (SUMS) sp[c][i] += b * y;
        if (a.w_post) b *= wp.get(i);
        q[0] += b * y;
        g[c][i] = b;
      }
    }
    if (a.n) {
      if (a.w_post) {
        row_sum<TPR, 1>(q, buf, turn);
        const float m = q[0] * inv;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] = rh * (g[c][i] - h[c].get(i) * rh * m);
      }
#pragma unroll
      for (int c = 0; c < NV; ++c) M::store((HT*)a.n + r * D, g[c], c, t, D);
    }
  }
  if (SUMS) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (a.dw_post) M::store(a.part + (0 * parts + first) * D, sp[c], c, t, D);
      if (a.dgate) M::store(a.part + (1 * parts + first) * D, sg[c], c, t, D);
      if (a.dw_pre) M::store(a.part + (2 * parts + first) * D, sw[c], c, t, D);
    }
  }
}

// The three sums over tokens from the partial sums, in a fixed order: a
// workgroup takes 64 columns, its wave w the partials w, w + 16, ...
__global__ __launch_bounds__(1024) void norm_sums_kernel(NormArgs a, int64_t parts) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? a.dw_post : blockIdx.y == 1 ? a.dgate : a.dw_pre;
  if (!out) return;
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int64_t col = (int64_t)blockIdx.x * 64 + l;
  float acc = 0.0f;
  if (col < a.D) {
    const float* p = a.part + (int64_t)blockIdx.y * parts * a.D + col;
#pragma unroll 8
    for (int64_t i = w; i < parts; i += 16) acc += p[i * a.D];
  }
  s[w][l] = acc;
  __syncthreads();
  if (w == 0 && col < a.D) {
#pragma unroll
    for (int k = 1; k < 16; ++k) acc += s[k][l];
    out[col] = acc;
  }
}

__global__ __launch_bounds__(256) void norm_zero_sums_kernel(NormArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.D) return;
  if (a.dw_post) a.dw_post[i] = 0.0f;
  if (a.dgate) a.dgate[i] = 0.0f;
  if (a.dw_pre) a.dw_pre[i] = 0.0f;
}

constexpr int kBwdGroups = 512;  // workgroups of the backward when it keeps sums

// Threads per row of the backward for width D (the forward takes the same).
int row_threads(int64_t D) { return D <= 1024 ? 64 : D <= 2048 ? 256 : D <= 4096 ? 512 : 1024; }

template <typename XT, typename HT, int TPR, int NV>
hipError_t fwd_as(const NormArgs& a, hipStream_t stream) {
  constexpr int ROWS = wg_threads(TPR) / TPR;
  const int64_t need = (a.T + ROWS - 1) / ROWS;
  const unsigned grid = (unsigned)(need < 65536 ? need : 65536);
  if (a.D % 8 == 0)
    hipLaunchKernelGGL((norm_fwd_kernel<XT, HT, TPR, NV, true>), dim3(grid), dim3(wg_threads(TPR)), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<XT, HT, TPR, NV, false>), dim3(grid), dim3(wg_threads(TPR)), 0, stream, a);
  return hipGetLastError();
}

template <typename XT, typename HT, int TPR, int NV>
hipError_t bwd_as(const NormArgs& a, hipStream_t stream) {
  constexpr int ROWS = wg_threads(TPR) / TPR;
  const int64_t parts = norm_bwd_parts(a.T, a.D);
  const unsigned grid = (unsigned)(parts / ROWS);
  const dim3 wg(wg_threads(TPR));
  const bool vec = a.D % 8 == 0, sums = a.dw_post || a.dgate || a.dw_pre;
  if (vec && sums)
    hipLaunchKernelGGL((norm_bwd_kernel<XT, HT, TPR, NV, true, true>), dim3(grid), wg, 0, stream, a, parts);
  else if (vec)
    hipLaunchKernelGGL((norm_bwd_kernel<XT, HT, TPR, NV, true, false>), dim3(grid), wg, 0, stream, a, parts);
  else if (sums)
    hipLaunchKernelGGL((norm_bwd_kernel<XT, HT, TPR, NV, false, true>), dim3(grid), wg, 0, stream, a, parts);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<XT, HT, TPR, NV, false, false>), dim3(grid), wg, 0, stream, a, parts);
  if (sums)
    hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((a.D + 63) / 64), 3), dim3(1024), 0, stream, a, parts);
  return hipGetLastError();
}

template <typename XT, typename HT>
hipError_t fwd_types(const NormArgs& a, hipStream_t stream) {
  if (a.D <= 512) return fwd_as<XT, HT, 64, 1>(a, stream);
  if (a.D <= 1024) return fwd_as<XT, HT, 64, 2>(a, stream);
  if (a.D <= 2048) return fwd_as<XT, HT, 256, 1>(a, stream);
  if (a.D <= 4096) return fwd_as<XT, HT, 512, 1>(a, stream);
  if (a.D <= 8192) return fwd_as<XT, HT, 1024, 1>(a, stream);
  return fwd_as<XT, HT, 1024, 2>(a, stream);
}

template <typename XT, typename HT>
hipError_t bwd_types(const NormArgs& a, hipStream_t stream) {
  if (a.D <= 512) return bwd_as<XT, HT, 64, 1>(a, stream);
  if (a.D <= 1024) return bwd_as<XT, HT, 64, 2>(a, stream);
  if (a.D <= 2048) return bwd_as<XT, HT, 256, 1>(a, stream);
  if (a.D <= 4096) return bwd_as<XT, HT, 512, 1>(a, stream);
  if (a.D <= 8192) return bwd_as<XT, HT, 1024, 1>(a, stream);
  return bwd_as<XT, HT, 1024, 2>(a, stream);
}

}  // namespace

// One partial row per row group of a workgroup; a multiple of the row groups
// per workgroup, every one of which writes its partials (zeros past the end).
int64_t norm_bwd_parts(int64_t T, int64_t D) {
  const int tpr = row_threads(D), rows = wg_threads(tpr) / tpr;
  int64_t groups = (T + rows - 1) / rows;
  if (groups > kBwdGroups) groups = kBwdGroups;
  return groups * rows;
}

hipError_t launch_norm_fwd(const NormArgs& a, bool x_f32, bool h_f32, hipStream_t stream) {
  if (!x_f32) return fwd_types<uint16_t, uint16_t>(a, stream);
  return h_f32 ? fwd_types<float, float>(a, stream) : fwd_types<float, uint16_t>(a, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, bool x_f32, bool h_f32, hipStream_t stream) {
  if (a.T == 0) {
    hipLaunchKernelGGL(norm_zero_sums_kernel, dim3((unsigned)((a.D + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (!x_f32) return bwd_types<uint16_t, uint16_t>(a, stream);
  return h_f32 ? bwd_types<float, float>(a, stream) : bwd_types<float, uint16_t>(a, stream);
}

}  // namespace qlora
