// The residual update of a decoder block with its norms, gfx950: forward and
// backward (formulas in include/qlora_decoder.h).
//
// Both directions are streams over rows of D elements with one or two row
// means in between, bound by HBM: the forward reads x and h and writes xo and
// n once, the backward reads dxo, xo, dn and h and writes dx and dh once.  A
// row is held in the registers of its threads (NV chunks of 8 elements each), so
// nothing is read twice, but for the backward of rows beyond 8192, which takes
// them from the caches again; 512 elements to a wave (1024 beyond 8192).
// Measured: 8192 x 8192 in bfloat16 with every part, forward 108-113 us (4.8-4.95
// TB/s, a device copy's rate is 4.9), backward 178 us with the sums (4.5 TB/s) and
// 163 without; 8191 x 4096 with an fp32 stream, backward 127 us (4.75 TB/s) and
// 120; 4096 x 16384 in bfloat16, backward 233 us (3.5 TB/s).  With few rows the sums
// set the pace, two rows of partials per workgroup and a second kernel: 256 x 8192
// in bfloat16 26.5 us with them, 13.8 without.
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
  __device__ __forceinline__ void set(int i, uint16_t e) { w[i >> 1] |= (uint32_t)e << (16 * (i & 1)); }
  static __device__ __forceinline__ Raw8 of(const float (&v)[8]) {
    return {{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])}};
  }
  __device__ __forceinline__ uint16_t elem(int i) const { return (uint16_t)(w[i >> 1] >> (16 * (i & 1))); }
};
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(int i, float e) { v[i] = e; }
  static __device__ __forceinline__ Raw8 of(const float (&v)[8]) {
    return {{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}};
  }
  __device__ __forceinline__ float elem(int i) const { return v[i]; }
};

// Elements j .. j + 7 of a row of D (those that exist; the rest reads as zero
// and is not written).  ALIGNED: D % 8 == 0, so the pieces of every row lie on
// 16-byte boundaries and are there whole or not at all; otherwise they are
// moved with the same 16-byte accesses at element alignment, which global
// memory allows, and the row's last piece element by element (8000 rows of
// 4097 forward: 211 us with element accesses throughout).
template <bool ALIGNED, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* row, int j, int D) {
  Raw8<T> r = {};
  if (ALIGNED) {
    if (j < D) r = *reinterpret_cast<const Raw8<T>*>(__builtin_assume_aligned(row + j, 16));
  } else if (j + 8 <= D) {
    __builtin_memcpy(&r, row + j, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (j + i < D) r.set(i, row[j + i]);
  }
  return r;
}
template <bool ALIGNED, typename T>
__device__ __forceinline__ void store8(T* row, const float (&v)[8], int j, int D) {
  const Raw8<T> r = Raw8<T>::of(v);
  if (ALIGNED) {
    if (j < D) *reinterpret_cast<Raw8<T>*>(__builtin_assume_aligned(row + j, 16)) = r;
  } else if (j + 8 <= D) {
    __builtin_memcpy(row + j, &r, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (j + i < D) row[j + i] = r.elem(i);
  }
}

// A value that is the same in all lanes of a wave, as the compiler is to see
// it: row addresses made from it stay in scalar registers.
__device__ __forceinline__ int wave_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

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

// Sums over the `tpr` threads of a row (a multiple of 64, at most 1024; the
// rows of a workgroup take theirs together).  `buf` holds two sets of wave sums
// used in turn, so one barrier per sum suffices: a set is written again only
// after the barrier of the sum in between, which every thread passes after it
// has read the set.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[3][16], int& turn, int tpr) {
  wave_sum<N>(v);
  if (tpr == 64) return;
  float(*s)[16] = buf[turn];
  turn ^= 1;
  const int wave = threadIdx.x >> 6, waves = tpr >> 6, first = wave / waves * waves;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k][wave] = v[k];
  }
  __syncthreads();
  // lane i of 16 takes the sum of the row's wave i; rotations add them
  const int i = threadIdx.x & 15;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float t = i < waves ? s[k][first + i] : 0.0f;
    t += dpp_ror<1>(t);
    t += dpp_ror<2>(t);
    t += dpp_ror<4>(t);
    t += dpp_ror<8>(t);
    v[k] = t;
  }
}

// A row per workgroup of tpr threads, or four rows of one wave each (rows of
// one workgroup end at different times, which only waves may).
template <typename XT, typename HT, int NV, bool AL>
__global__ __launch_bounds__(1024, NV == 1 ? 8 : 4) void norm_fwd_kernel(NormArgs a, int tpr) {
  __shared__ float buf[2][3][16];
  const int rows = tpr == 64 ? 4 : 1, sub = tpr == 64 ? wave_uniform(threadIdx.x >> 6) : 0;
  const int t = threadIdx.x - sub * tpr, D = a.D;
  const float inv = 1.0f / (float)D;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * rows + sub; r < a.T; r += (int64_t)gridDim.x * rows) {
    float x[NV][8];
    Raw8<XT> rx[NV];
    Raw8<HT> h[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      rx[c] = load8<AL>((const XT*)a.x + r * D, (c * tpr + t) * 8, D);
      if (a.h) h[c] = load8<AL>((const HT*)a.h + r * D, (c * tpr + t) * 8, D);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[c][i] = rx[c].get(i);
    if (a.h) {
      float s[1] = {0.0f};
      float k = a.alpha;
      if (a.w_post) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(h[c].get(i), h[c].get(i), s[0]);
        row_sum<1>(s, buf, turn, tpr);
        k *= 1.0f / sqrtf(s[0] * inv + a.eps);
      }
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        Raw8<float> w, g;
        if (a.w_post) w = load8<AL>(a.w_post, (c * tpr + t) * 8, D);
        if (a.gate) g = load8<AL>(a.gate, (c * tpr + t) * 8, D);
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
#pragma unroll
      for (int c = 0; c < NV; ++c) store8<AL>((XT*)a.xo + r * D, x[c], (c * tpr + t) * 8, D);
    }
    if (a.n) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(x[c][i], x[c][i], s[0]);
      row_sum<1>(s, buf, turn, tpr);
      const float rs = 1.0f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const Raw8<float> w = load8<AL>(a.w_pre, (c * tpr + t) * 8, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * rs * w.get(i);
        store8<AL>((HT*)a.n + r * D, x[c], (c * tpr + t) * 8, D);
      }
    }
  }
}

// What a thread reads of one row in the backward.
template <typename XT, typename HT, int NV>
struct BwdRow {
  Raw8<XT> xo[NV], dxo[NV];
  Raw8<HT> dn[NV], h[NV];
};

// The backward of one row needs two rounds of row sums: first sum xo^2, sum a
// xo (for dx) and sum h^2, then sum b w_post h (for dh).  One workgroup of up
// to 1024 threads per CU walks over the rows, as many at a time as it holds, with the next rows'
// loads in flight under the present ones' sums and barriers.  SUMS: the sums
// over tokens are kept in the threads' registers, one per element a thread
// owns, added over the workgroup's row groups in LDS at the end and written
// once per workgroup; norm_sums_kernel adds those.  The gains lie in LDS for the
// whole walk: registers have no room for them beside the sums, the row and the
// next row, and from the L2 they would double its reads.  Rows beyond 8192
// (NV = 2) keep the sums in the LDS and read the row and the gains where they are
// used, from the caches after the first time (all in registers spilled: 4096 x
// 16384 in bfloat16 839 us).
constexpr int kBwdThreads = 1024;

template <typename XT, typename HT, int NV, bool AL, bool SUMS>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormArgs a, int tpr, int rows) {
  __shared__ float buf[2][3][16];
  extern __shared__ __attribute__((aligned(16))) float lds[];  // the gains, at the end the row groups' sums
  constexpr bool LDS_GAINS = NV == 1, AHEAD = NV == 1;
  // an fp32 row of dxo has no room in flight beside the rest (spills: 65536 x
  // 256 in fp32 111 us against 82); it is loaded with its own row, whose first
  // sums do not need it
  constexpr bool DXO_AHEAD = sizeof(XT) == 2;
  using Row = BwdRow<XT, HT, NV>;
  const int sub = wave_uniform(threadIdx.x / tpr), t = threadIdx.x - sub * tpr, D = a.D;
  const float inv = 1.0f / (float)D;
  int turn = 0;
  // sums of dx y and of dn xo r: in registers, or in the thread's own places of
  // the LDS
  constexpr bool LDS_SUMS = SUMS && NV == 2;
  float sums[2][NV][8];
  auto place = [&](int which, int c, int i) { return ((which * NV + c) * 8 + i) * tpr + t; };
  if (SUMS) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[k][c][i] = 0.0f;
          if (LDS_SUMS) lds[place(k, c, i)] = 0.0f;
        }
  }
  auto add = [&](int which, int c, int i, float u, float v) {
    if (LDS_SUMS) lds[place(which, c, i)] = __builtin_fmaf(u, v, lds[place(which, c, i)]);
    else sums[which][c][i] = __builtin_fmaf(u, v, sums[which][c][i]);
  };
  auto load = [&](Row& w, int64_t r) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int j = (c * tpr + t) * 8;
      w.xo[c] = load8<AL>((const XT*)a.x + r * D, j, D);
      if (a.dxo && DXO_AHEAD) w.dxo[c] = load8<AL>((const XT*)a.dxo + r * D, j, D);
      if (a.dn) w.dn[c] = load8<AL>((const HT*)a.dn + r * D, j, D);
      if (a.h) w.h[c] = load8<AL>((const HT*)a.h + r * D, j, D);
    }
  };
  const float* const gains[3] = {a.w_pre, a.w_post, a.gate};
  if (LDS_GAINS) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (!gains[k]) continue;
      for (int i = threadIdx.x; i < tpr * 8; i += blockDim.x) lds[k * tpr * 8 + i] = i < D ? gains[k][i] : 0.0f;
    }
    __syncthreads();
  }
  auto gain = [&](int k, int c) {
    Raw8<float> w;
    if (LDS_GAINS) {
      w = *reinterpret_cast<const Raw8<float>*>(lds + (k * tpr + t) * 8);
    } else {
      int j = (c * tpr + t) * 8;
      asm volatile("" : "+v"(j));  // loaded again for every row, not kept in registers
      w = load8<AL>(gains[k], j, D);
    }
    return w;
  };
  // every row group makes the same number of turns (barriers); a group whose
  // rows have run out repeats the last row and keeps nothing of it
  const int64_t step = (int64_t)gridDim.x * rows;
  Row nx;
  int64_t r0 = (int64_t)blockIdx.x * rows;
  if (AHEAD) load(nx, r0 + sub < a.T ? r0 + sub : a.T - 1);
  for (; r0 < a.T; r0 += step) {
    const int64_t r = r0 + sub, rr = r < a.T ? r : a.T - 1;
    const bool mine = r < a.T;
    Row w;
    if (AHEAD) {
      w = nx;
      if (a.dxo && !DXO_AHEAD) {
#pragma unroll
        for (int c = 0; c < NV; ++c) w.dxo[c] = load8<AL>((const XT*)a.dxo + rr * D, (c * tpr + t) * 8, D);
      }
      if (r0 + step < a.T) load(nx, r + step < a.T ? r + step : a.T - 1);
    }
    // chunk c of the row: held, or (NV = 2) loaded where it is used
    auto xo_of = [&](int c) -> decltype(auto) {
      if constexpr (AHEAD) return (w.xo[c]);
      else return load8<AL>((const XT*)a.x + rr * D, (c * tpr + t) * 8, D);
    };
    auto dxo_of = [&](int c) -> decltype(auto) {
      if constexpr (AHEAD) return (w.dxo[c]);
      else return a.dxo ? load8<AL>((const XT*)a.dxo + rr * D, (c * tpr + t) * 8, D) : Raw8<XT>{};
    };
    auto dn_of = [&](int c) -> decltype(auto) {
      if constexpr (AHEAD) return (w.dn[c]);
      else return load8<AL>((const HT*)a.dn + rr * D, (c * tpr + t) * 8, D);
    };
    auto h_of = [&](int c) -> decltype(auto) {
      if constexpr (AHEAD) return (w.h[c]);
      else return a.h ? load8<AL>((const HT*)a.h + rr * D, (c * tpr + t) * 8, D) : Raw8<HT>{};
    };
    float s[3] = {0.0f, 0.0f, 0.0f};  // xo^2, a xo, h^2
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (a.dn) {
        const Raw8<float> wp = gain(0, c);
        const Raw8<XT>& xo = xo_of(c);
        const Raw8<HT>& dn = dn_of(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = xo.get(i);
          s[0] = __builtin_fmaf(x, x, s[0]);
          s[1] = __builtin_fmaf(dn.get(i) * wp.get(i), x, s[1]);
        }
      }
      if (a.w_post) {
        const Raw8<HT>& h = h_of(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] = __builtin_fmaf(h.get(i), h.get(i), s[2]);
      }
    }
    row_sum<3>(s, buf, turn, tpr);
    const float rs = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float back = rs * rs * (s[1] * inv);
    const float rh = a.w_post ? 1.0f / sqrtf(s[2] * inv + a.eps) : 1.0f;
    float g[NV][8];  // dx, then the gradient of y
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int j = (c * tpr + t) * 8;
      const Raw8<XT>& dxo = dxo_of(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[c][i] = a.dxo ? dxo.get(i) : 0.0f;
      if (a.dn) {
        const Raw8<float> wp = gain(0, c);
        const Raw8<XT>& xo = xo_of(c);
        const Raw8<HT>& dn = dn_of(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = xo.get(i), d = dn.get(i);
          g[c][i] = __builtin_fmaf(rs, __builtin_fmaf(d, wp.get(i), -(x * back)), g[c][i]);
          if (SUMS && mine) add(1, c, i, d, x * rs);
        }
      }
      if (mine) store8<AL>((XT*)a.xo + r * D, g[c], j, D);
      Raw8<float> wp, gt;
      if (a.w_post) wp = gain(1, c);
      if (a.gate) gt = gain(2, c);
      const Raw8<HT>& h = h_of(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = a.h ? h.get(i) * rh : 0.0f;
        float b = g[c][i] * a.alpha;
        if (SUMS && mine) add(0, c, i, g[c][i], y);
        if (a.gate) b *= gt.get(i);
        if (a.w_post) b *= wp.get(i);
        q[0] = __builtin_fmaf(b, y, q[0]);
        g[c][i] = b;
      }
    }
    if (a.n) {
      if (a.w_post) {
        row_sum<1>(q, buf, turn, tpr);
        const float m = q[0] * inv;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const Raw8<HT>& h = h_of(c);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] = rh * (g[c][i] - h.get(i) * rh * m);
        }
      }
      if (mine) {
#pragma unroll
        for (int c = 0; c < NV; ++c) store8<AL>((HT*)a.n + r * D, g[c], (c * tpr + t) * 8, D);
      }
    }
  }
  if (SUMS) {
    auto flush = [&](int which) {
      float(&v)[NV][8] = sums[which];
      if (LDS_SUMS) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = lds[place(which, c, i)];
      } else if (rows > 1) {  // add the row groups' sums, in order
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) lds[((sub * NV + c) * 8 + i) * tpr + t] = v[c][i];
        __syncthreads();
        if (sub == 0) {
          for (int k = 1; k < rows; ++k)
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[c][i] += lds[((k * NV + c) * 8 + i) * tpr + t];
        }
      }
      if (sub == 0) {
        float* row = a.part + ((int64_t)which * gridDim.x + blockIdx.x) * D;
#pragma unroll
        for (int c = 0; c < NV; ++c) store8<AL>(row, v[c], (c * tpr + t) * 8, D);
      }
    };
    if (a.dw_post || a.dgate) flush(0);
    if (a.dw_pre) flush(1);
  }
}

// The gradients of the gains and the gate from the partial sums, added in a
// fixed order: a workgroup takes 64 columns, its wave w the partials w, w + 16,
// ...  One sum, of dx y, serves two of them: dw_post = alpha gate sum and dgate =
// alpha w_post sum.
__global__ __launch_bounds__(1024) void norm_sums_kernel(NormArgs a, int64_t parts) {
  __shared__ float s[16][64];
  const bool pre = blockIdx.y != 0;
  if (pre ? !a.dw_pre : !a.dw_post && !a.dgate) return;
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
    if (pre) {
      a.dw_pre[col] = acc;
    } else {
      acc *= a.alpha;
      if (a.dw_post) a.dw_post[col] = a.gate ? acc * a.gate[col] : acc;
      if (a.dgate) a.dgate[col] = a.w_post ? acc * a.w_post[col] : acc;
    }
  }
}

__global__ __launch_bounds__(256) void norm_zero_sums_kernel(NormArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.D) return;
  if (a.dw_post) a.dw_post[i] = 0.0f;
  if (a.dgate) a.dgate[i] = 0.0f;
  if (a.dw_pre) a.dw_pre[i] = 0.0f;
}

// Threads per row: 8 elements each up to 8192, then 16.
int row_threads(int64_t D) {
  const int64_t each = D <= 8192 ? 512 : 1024;  // elements per wave
  return (int)((D + each - 1) / each) * 64;
}

// The backward: one workgroup per CU at most, with as many rows at a time as
// 1024 threads hold.
constexpr int kBwdGroups = 256;
int bwd_rows(int64_t D) { return kBwdThreads / row_threads(D); }

template <typename XT, typename HT>
hipError_t fwd_types(const NormArgs& a, hipStream_t stream) {
  const int tpr = row_threads(a.D), rows = tpr == 64 ? 4 : 1;
  const int64_t need = (a.T + rows - 1) / rows;
  const unsigned grid = (unsigned)(need < 65536 ? need : 65536);
  const bool al = a.D % 8 == 0;
  const auto kernel = a.D <= 8192 ? (al ? norm_fwd_kernel<XT, HT, 1, true> : norm_fwd_kernel<XT, HT, 1, false>)
                                  : (al ? norm_fwd_kernel<XT, HT, 2, true> : norm_fwd_kernel<XT, HT, 2, false>);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(tpr * rows), 0, stream, a, tpr);
  return hipGetLastError();
}

template <typename XT, typename HT, int NV, bool AL>
hipError_t bwd_as(const NormArgs& a, hipStream_t stream) {
  const int tpr = row_threads(a.D), rows = bwd_rows(a.D);
  const int64_t parts = norm_bwd_parts(a.T, a.D);
  const bool sums = a.dw_post || a.dgate || a.dw_pre;
  // NV = 1: the gains, then the row groups' sums; NV = 2 (one row): the sums
  const size_t gains = NV == 1 ? 3 * (size_t)tpr * 32 : 0;
  const size_t add = !sums ? 0 : NV == 2 ? 2 * (size_t)tpr * NV * 32 : rows > 1 ? (size_t)rows * tpr * 32 : 0;
  const auto kernel = sums ? norm_bwd_kernel<XT, HT, NV, AL, true> : norm_bwd_kernel<XT, HT, NV, AL, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)parts), dim3(tpr * rows), gains > add ? gains : add, stream, a, tpr, rows);
  if (sums)
    hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((a.D + 63) / 64), 2), dim3(1024), 0, stream, a, parts);
  return hipGetLastError();
}

template <typename XT, typename HT>
hipError_t bwd_types(const NormArgs& a, hipStream_t stream) {
  const bool al = a.D % 8 == 0;
  if (a.D <= 8192) return al ? bwd_as<XT, HT, 1, true>(a, stream) : bwd_as<XT, HT, 1, false>(a, stream);
  return al ? bwd_as<XT, HT, 2, true>(a, stream) : bwd_as<XT, HT, 2, false>(a, stream);
}

}  // namespace

int64_t norm_bwd_parts(int64_t T, int64_t D) {
  const int64_t rows = bwd_rows(D), groups = (T + rows - 1) / rows;
  return groups < kBwdGroups ? groups : kBwdGroups;
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
