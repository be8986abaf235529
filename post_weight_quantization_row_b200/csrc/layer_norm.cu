// layer_norm: y = (x - mean) rstd w + b per row, and its backward pass with
// the reduction of the parameters' gradients.
//
// Both are bound by HBM, and next by the issue of instructions: a bf16 element
// of 2 bytes leaves about 18 issue slots of a lane at the copy rate, so the
// arithmetic runs on packed pairs (f32x2) and decodes each element once.  A
// row is held in the registers of a group of G threads, NV vectors of 8
// elements each, so it is read once: the mean, then the variance around it,
// then the output.  The backward pass adds dw and db on the way: every block
// walks rows with a fixed stride and each of its threads keeps the same
// columns, so the sums stay in registers and leave the block once, as one
// partial row per block; a second kernel adds the partial rows in a fixed
// order.
//
// Measured at 16384 x 4096 bf16 with fp32 parameters: forward 55 us (4.8 TB/s),
// backward 81 us (5.0 TB/s; 63% of the issue slots at four warps a scheduler).
// Rows that start at odd addresses pay for shifting their vectors: 2000 x 5001
// bf16 takes 21 us and 60 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "layer_ops.cuh"

namespace mpq {
namespace {

constexpr int64_t LN_BACK_BLOCKS = 1184;       // partial rows of dw and db at most
constexpr int64_t LN_REG_MAX = 32768;      // widest row held in registers (forward)
constexpr int LN_PART = 8192;              // columns per CTA of the backward kernel
constexpr int64_t LN_BACK_MAX = 4 * LN_PART;  // widest row of a cluster of them
constexpr int LN_COL_ROWS = 64;            // rows per partial of the wide rows' column sums

// Sums over a group of G threads (a power of two): shuffles within a warp,
// shared memory across warps (then the block is one group).  `buf` alternates
// between two halves of the scratch, so one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G, float* scratch, int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o < G) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
  if (G > 32) {
    float* s = scratch + buf * (32 * N);
    buf ^= 1;
    const int nw = G >> 5;  // 2, 4, .. 32 warps
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i * 32 + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (nw == 2) {
        v[i] = s[i * 32] + s[i * 32 + 1];
      } else {
        float t = 0.0f;
        for (int w = 0; w < nw; w += 4) {
          const float4 q = *reinterpret_cast<const float4*>(s + i * 32 + w);
          t += (q.x + q.y) + (q.z + q.w);
        }
        v[i] = t;
      }
    }
  }
}

struct LnArgs {
  const void* x;
  int64_t ldx, rows, n;
  const void* w;
  const void* b;
  bool p_f32, x_vec, p_vec, o_vec;
  int G, C;
  int sms;  // of the device
};

// How rows and parameters come.  Parameters: none, all in T, all in fp32, on
// 16-byte boundaries.  Rows: on 16-byte boundaries and of whole vectors of 8,
// or PM_SHIFT: at any address and of any length (from 129 on, so that a warp
// holds one row).  PM_ANY: everything else, element by element.
enum { PM_NONE = 0, PM_T = 1, PM_F32 = 2, PM_ANY = 3, PM_SHIFT = 4 };

// The column of element i of vector j of a thread t of G: 8 neighbours, or for
// PM_ANY single elements G apart, so that a warp's accesses still cover
// neighbouring ones.
template <int PM>
__device__ __forceinline__ int ln_col(int t, int G, int j, int i) {
  return PM != PM_ANY ? (t + j * G) * 8 + i : (j * 8 + i) * G + t;
}
template <int PM, typename T>
__device__ __forceinline__ Raw8<T> ln_load(const T* row, int n, int t, int G, int j) {
  Raw8<T> r;
  if (PM != PM_ANY) {
    const int c = (t + j * G) * 8;
    if (PM & PM_SHIFT) {
      if (c < n) return load_row8<T>(row, c, n);
#pragma unroll
      for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.q[i] = make_uint4(0, 0, 0, 0);
      return r;
    }
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
      r.q[i] = c < n ? reinterpret_cast<const uint4*>(row + c)[i] : make_uint4(0, 0, 0, 0);
    return r;
  }
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = ln_col<PM>(t, G, j, i) < n ? row[ln_col<PM>(t, G, j, i)] : from_f<T>(0.0f);
  memcpy(&r, e, sizeof(r));
  return r;
}
// A vector on its way: as it will be used, or (PM_SHIFT) before its shift.
template <int PM, typename T>
using Fetched = typename std::conditional<PM != PM_ANY && (PM & PM_SHIFT), RawWindow<T>, Raw8<T>>::type;
template <int PM, typename T>
__device__ __forceinline__ Fetched<PM, T> ln_fetch(const T* row, int n, int t, int G, int j) {
  if constexpr (PM != PM_ANY && (PM & PM_SHIFT)) {
    const int c = (t + j * G) * 8;
    if (c < n) return load_window<T>(row, c, n);
    RawWindow<T> w;
#pragma unroll
    for (int i = 0; i <= (int)(sizeof(T) / 2); ++i) w.q[i] = make_uint4(0, 0, 0, 0);
    w.halfwords = 0;
    return w;
  } else {
    return ln_load<PM, T>(row, n, t, G, j);
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> ln_take(const RawWindow<T>& w) { return shift_window<T>(w); }
template <typename T>
__device__ __forceinline__ const Raw8<T>& ln_take(const Raw8<T>& r) { return r; }

// A warp's staging for rows at any address
template <int PM, typename T>
struct Stage {
  uint4 v[PM != PM_ANY && (PM & PM_SHIFT) ? 32 * (16 * sizeof(T) + 1) : 1];
  __device__ __forceinline__ T* warp() { return reinterpret_cast<T*>(v + (threadIdx.x >> 5) * (16 * sizeof(T) + 1)); }
};
template <int PM, typename T>
__device__ __forceinline__ void ln_store(T* row, const float (&v)[8], int n, int t, int G, int j, Stage<PM, T>& stage) {
  if (PM != PM_ANY) {
    const int c = (t + j * G) * 8;
    if (PM & PM_SHIFT) {
      const int cw = c - (int)(threadIdx.x & 31) * 8;  // the warp's first column
      if (cw < n) warp_store<T>(row + cw, v, min(256, n - cw), stage.warp());
    } else if (c < n) {
      store_vec<8>(row + c, v, true);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (ln_col<PM>(t, G, j, i) < n) row[ln_col<PM>(t, G, j, i)] = from_f<T>(v[i]);
  }
}
template <int PM, typename T>
__device__ __forceinline__ void ln_param(const LnArgs& a, const void* p, float dflt, int t, int j, float (&w)[8]) {
  const int n = (int)a.n;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = dflt;
  if ((PM & 3) == PM_NONE) return;
  if (PM != PM_ANY) {
    const int c = (t + j * a.G) * 8;
    if (c >= n) return;
    const int have = (PM & PM_SHIFT) ? n - c : 8;
    if ((PM & 3) == PM_T) load_edge<8>(static_cast<const T*>(p) + c, w, have, true);
    else load_edge<8>(static_cast<const float*>(p) + c, w, have, true);
    return;
  }
  if (!p) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = ln_col<PM>(t, a.G, j, i);
    if (c < n) w[i] = a.p_f32 ? static_cast<const float*>(p)[c] : to_f(static_cast<const T*>(p)[c]);
  }
}

__device__ __forceinline__ float f2_sum(uint64_t a) {
  float x, y;
  f2_unpack(a, x, y);
  return x + y;
}
// NR rows at a time per group (narrow rows): more loads in flight, and the
// parameters are read once for NR rows.
template <typename T, int NV, int NR, int PM>
__global__ void __launch_bounds__(NV * NR >= 8 ? 256 : 1024)
    k_ln_fwd(const __grid_constant__ LnArgs a, float eps, T* __restrict__ y, float* __restrict__ mean_out,
             float* __restrict__ rstd_out) {
  __shared__ __align__(16) float scratch[2 * 32 * NR];
  __shared__ Stage<PM, T> stage;
  int buf = 0;
  const int t = threadIdx.x & (a.G - 1);
  const int64_t row0 = ((int64_t)blockIdx.x * (blockDim.x / a.G) + threadIdx.x / a.G) * NR;
  const int n = (int)a.n;
  const float inv_n = 1.0f / (float)n;
  F8 v[NR][NV];
  {
    Raw8<T> x[NR][NV];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const T* xr = static_cast<const T*>(a.x) + (row0 + r < a.rows ? row0 + r : 0) * a.ldx;
#pragma unroll
      for (int j = 0; j < NV; ++j) x[r][j] = ln_load<PM, T>(xr, n, t, a.G, j);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < NV; ++j) v[r][j] = pairs<T>(x[r][j]);
  }
  float mean[NR], rstd[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s0 = f2_add(s0, f2_add(v[r][j].p[0], v[r][j].p[1]));
      s1 = f2_add(s1, f2_add(v[r][j].p[2], v[r][j].p[3]));
    }
    mean[r] = f2_sum(f2_add(s0, s1));
  }
  group_sum<NR>(mean, a.G, scratch, buf);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    mean[r] *= inv_n;
    const uint64_t m2 = f2_pack(-mean[r], -mean[r]);
    uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][j].p[i] = f2_add(v[r][j].p[i], m2);
      // columns that do not exist hold -mean: out
      if (PM == PM_ANY || ((PM & PM_SHIFT) && (t + j * a.G) * 8 + 8 > n)) {
        float e[8];
        unpairs(v[r][j], e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (ln_col<PM>(t, a.G, j, i) >= n) e[i] = 0.0f;
        v[r][j] = pairs(e);
      }
      if (PM == PM_ANY || (t + j * a.G) * 8 < n) {
        s0 = f2_fma(v[r][j].p[0], v[r][j].p[0], s0);
        s1 = f2_fma(v[r][j].p[1], v[r][j].p[1], s1);
        s0 = f2_fma(v[r][j].p[2], v[r][j].p[2], s0);
        s1 = f2_fma(v[r][j].p[3], v[r][j].p[3], s1);
      }
    }
    rstd[r] = f2_sum(f2_add(s0, s1));
  }
  group_sum<NR>(rstd, a.G, scratch, buf);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    rstd[r] = 1.0f / sqrtf(fmaf(rstd[r], inv_n, eps));
    if (t == 0 && row0 + r < a.rows) {
      if (mean_out) mean_out[row0 + r] = mean[r];
      if (rstd_out) rstd_out[row0 + r] = rstd[r];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float w[8], b[8];
    ln_param<PM, T>(a, a.w, 1.0f, t, j, w);
    ln_param<PM, T>(a, a.b, 0.0f, t, j, b);
    const F8 w2 = pairs(w), b2 = pairs(b);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (row0 + r >= a.rows) break;
      const uint64_t r2 = f2_pack(rstd[r], rstd[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][j].p[i] = f2_fma(f2_mul(v[r][j].p[i], r2), w2.p[i], b2.p[i]);
      float o[8];
      unpairs(v[r][j], o);
      ln_store<PM, T>(y + (row0 + r) * a.n, o, n, t, a.G, j, stage);
    }
  }
}

// Rows too wide for registers: three passes over the row, which L2 serves
// after the first.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_ln_fwd_wide(const __grid_constant__ LnArgs a, float eps, T* __restrict__ y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out) {
  __shared__ __align__(16) float scratch[2 * 32];
  int buf = 0;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
  const int n = (int)a.n;
  float s[1] = {0.0f};
  for (int c = threadIdx.x * 8; c < n; c += 8192) {
    float v[8];
    load_edge<8>(xr + c, v, n - c, a.x_vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += v[i];
  }
  group_sum<1>(s, 1024, scratch, buf);
  const float mean = s[0] / (float)n;
  float q[1] = {0.0f};
  for (int c = threadIdx.x * 8; c < n; c += 8192) {
    float v[8];
    load_edge<8>(xr + c, v, n - c, a.x_vec);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) q[0] = fmaf(v[i] - mean, v[i] - mean, q[0]);
  }
  group_sum<1>(q, 1024, scratch, buf);
  const float rstd = 1.0f / sqrtf(q[0] / (float)n + eps);
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
  for (int c = threadIdx.x * 8; c < n; c += 8192) {
    float v[8], w[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { w[i] = 1.0f; b[i] = 0.0f; }
    load_edge<8>(xr + c, v, n - c, a.x_vec);
    if (a.w) load_param<8, T>(a.w, a.p_f32, c, w, n - c, a.p_vec);
    if (a.b) load_param<8, T>(a.b, a.p_f32, c, b, n - c, a.p_vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fmaf((v[i] - mean) * rstd, w[i], b[i]);
    store_edge<8>(y + row * a.n + c, w, n - c, a.o_vec);
  }
}

// --------------------------------------------------------------- backward --
// dx of a row at a time per group, walking the rows with a fixed stride, and
// (SUMS) per block the column sums of dy xh and dy over its rows.  The next
// row's loads are issued before this row's sums are joined.  CL: a cluster of
// CTAs shares the rows, LN_PART columns each; their sums meet over distributed
// shared memory.
template <typename T, int NV, int PM, bool SUMS, bool CL>
__global__ void __launch_bounds__(NV == 1 && !(PM & PM_SHIFT) ? 128 : 512)
    k_ln_bwd(const __grid_constant__ LnArgs a, const T* __restrict__ dy, int64_t ldy,
             const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
             float* __restrict__ part) {
  __shared__ __align__(16) float scratch[2 * 64];
  __shared__ Stage<PM, T> stage;
  __shared__ float meet[2][2];     // CL: this CTA's sums, alternating between rows
  extern __shared__ float join[];  // several groups: dw[n], db[n]
  int buf = 0;
  const int t = threadIdx.x & (a.G - 1), groups = blockDim.x / a.G;
  const int C = CL ? a.C : 1, rank = CL ? (int)tcx::cluster_ctarank() : 0;
  const int c0 = CL ? rank * LN_PART : 0;
  const int n = CL ? min(LN_PART, (int)a.n - c0) : (int)a.n;  // this CTA's columns
  const int64_t block = blockIdx.x / C, nblocks = gridDim.x / C;
  const float inv_n = 1.0f / (float)a.n;
  LnArgs pa = a;  // the parameters of these columns
  pa.n = n;
  if (CL && a.w) pa.w = static_cast<const char*>(a.w) + (int64_t)c0 * (a.p_f32 ? 4 : (int)sizeof(T));
  F8 dw2[NV], db2[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw2[j].p[i] = db2[j].p[i] = 0ull;
  const int64_t step = nblocks * groups;
  int64_t row = block * groups + threadIdx.x / a.G;
  Fetched<PM, T> xs[NV], ds[NV];
  float m = 0.0f, r = 0.0f;
  const auto fetch = [&](int64_t at) {  // (rows that do not exist: zeros)
    const bool live = at < a.rows;
    const T* xr = static_cast<const T*>(a.x) + (live ? at : 0) * a.ldx + c0;
    const T* yr = dy + (live ? at : 0) * ldy + c0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xs[j] = ln_fetch<PM, T>(xr, live ? n : 0, t, a.G, j);
      ds[j] = ln_fetch<PM, T>(yr, live ? n : 0, t, a.G, j);
    }
    m = live ? mean[at] : 0.0f;
    r = live ? rstd[at] : 0.0f;
  };
  fetch(row);
  // every thread of the block takes the same number of turns (group_sum)
  for (int64_t base = block * groups; base < a.rows; base += step, row += step) {
    F8 xh[NV], g[NV];
    const uint64_t m2 = f2_pack(-m, -m), r2 = f2_pack(r, r);
    const float rr = r;
    uint64_t t0 = 0ull, t1 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8];
      ln_param<PM, T>(pa, pa.w, 1.0f, t, j, w);
      const F8 w2 = pairs(w);
      xh[j] = pairs<T>(ln_take<T>(xs[j]));
      g[j] = pairs<T>(ln_take<T>(ds[j]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (columns that do not exist: dy = 0 there, and xh is finite)
        xh[j].p[i] = f2_mul(f2_add(xh[j].p[i], m2), r2);
        if (SUMS) {
          dw2[j].p[i] = f2_fma(g[j].p[i], xh[j].p[i], dw2[j].p[i]);
          db2[j].p[i] = f2_add(g[j].p[i], db2[j].p[i]);
        }
        g[j].p[i] = f2_mul(g[j].p[i], w2.p[i]);
        t0 = f2_add(t0, g[j].p[i]);
        t1 = f2_fma(g[j].p[i], xh[j].p[i], t1);
      }
    }
    fetch(row + step);
    if (dx) {
      float s[2] = {f2_sum(t0), f2_sum(t1)};
      group_sum<2>(s, a.G, scratch, buf);
      if (CL) {
        if (threadIdx.x == 0) {
          meet[buf][0] = s[0];
          meet[buf][1] = s[1];
        }
        __syncwarp();
        tcx::cluster_sync();
        s[0] = s[1] = 0.0f;
        for (int q = 0; q < C; ++q) {
          s[0] += ld_cluster(&meet[buf][0], q);
          s[1] += ld_cluster(&meet[buf][1], q);
        }
      }
      if (row < a.rows) {
        const uint64_t s0 = f2_pack(-s[0] * inv_n, -s[0] * inv_n), s1 = f2_pack(-s[1] * inv_n, -s[1] * inv_n);
        const uint64_t q2 = f2_pack(rr, rr);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            g[j].p[i] = f2_mul(q2, f2_fma(xh[j].p[i], s1, f2_add(g[j].p[i], s0)));
          unpairs(g[j], o);
          ln_store<PM, T>(dx + row * a.n + c0, o, n, t, a.G, j, stage);
        }
      }
    }
  }
  if (CL) {
    __syncwarp();
    tcx::cluster_sync();  // no peer still reads this CTA's sums
  }
  if (!SUMS) return;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    unpairs(dw2[j], dw[j]);
    unpairs(db2[j], db[j]);
  }
  float* pw = part + block * 2 * a.n + c0;
  float* pb = pw + a.n;
  if (groups == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (PM != PM_ANY && !(PM & PM_SHIFT)) {
        const int c = (t + j * a.G) * 8;
        if (c < n) {
          store_vec<8>(pw + c, dw[j], true);
          store_vec<8>(pb + c, db[j], true);
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = ln_col<PM>(t, a.G, j, i);
        if (c < n) { pw[c] = dw[j][i]; pb[c] = db[j][i]; }
      }
    }
    return;
  }
  // several rows at a time: the groups add up in order
  for (int q = 0; q < groups; ++q) {
    if (threadIdx.x / a.G == q) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = ln_col<PM>(t, a.G, j, i);
          if (c < n) {
            join[c] = (q ? join[c] : 0.0f) + dw[j][i];
            join[n + c] = (q ? join[n + c] : 0.0f) + db[j][i];
          }
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < n; c += blockDim.x) { pw[c] = join[c]; pb[c] = join[n + c]; }
}

// Rows too wide for the kernel above: dx in two passes over the row, and the
// column sums by blocks of 256 columns x LN_COL_ROWS rows.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_ln_dx_wide(const __grid_constant__ LnArgs a, const T* __restrict__ dy, int64_t ldy, bool y_vec,
                 const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx) {
  __shared__ __align__(16) float scratch[2 * 64];
  int buf = 0;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
  const T* yr = dy + row * ldy;
  const int n = (int)a.n;
  const float m = mean[row], r = rstd[row];
  float s[2] = {0.0f, 0.0f};
  for (int pass = 0; pass < 2; ++pass) {
    for (int c = threadIdx.x * 8; c < n; c += 8192) {
      float x[8], g[8], w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      load_edge<8>(xr + c, x, n - c, a.x_vec);
      load_edge<8>(yr + c, g, n - c, y_vec);
      if (a.w) load_param<8, T>(a.w, a.p_f32, c, w, n - c, a.p_vec);
      if (pass == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < n) {
            s[0] = fmaf(g[i], w[i], s[0]);
            s[1] = fmaf(g[i] * w[i], (x[i] - m) * r, s[1]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = r * (g[i] * w[i] - fmaf((x[i] - m) * r, s[1], s[0]));
        store_edge<8>(dx + row * a.n + c, g, n - c, a.o_vec);
      }
    }
    if (pass == 0) {
      group_sum<2>(s, 1024, scratch, buf);
      s[0] /= (float)n;
      s[1] /= (float)n;
    }
  }
}
template <typename T>
__global__ void __launch_bounds__(256)
    k_ln_cols_wide(const __grid_constant__ LnArgs a, const T* __restrict__ dy, int64_t ldy, bool y_vec,
                   const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part) {
  __shared__ float red[2][8][256 + 8];
  const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.y * 256 + cg * 8;
  const int64_t lo = (int64_t)blockIdx.x * LN_COL_ROWS, hi = min(a.rows, lo + LN_COL_ROWS);
  float dw[8] = {}, db[8] = {};
  if (c < a.n) {
    const int left = (int)min((int64_t)8, a.n - c);
    for (int64_t row = lo + rl; row < hi; row += 8) {
      float x[8], g[8];
      load_edge<8>(static_cast<const T*>(a.x) + row * a.ldx + c, x, left, a.x_vec);
      load_edge<8>(dy + row * ldy + c, g, left, y_vec);
      const float m = mean[row], r = rstd[row];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[i] = fmaf(g[i], (x[i] - m) * r, dw[i]);
        db[i] += g[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) { red[0][rl][cg * 8 + i] = dw[i]; red[1][rl][cg * 8 + i] = db[i]; }
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (col < a.n) {
    float s = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) { s += red[0][i][threadIdx.x]; b += red[1][i][threadIdx.x]; }
    part[((int64_t)blockIdx.x * 2) * a.n + col] = s;
    part[((int64_t)blockIdx.x * 2 + 1) * a.n + col] = b;
  }
}

// dw and db from the blocks' partial rows, in a fixed order.
template <typename O>
__global__ void __launch_bounds__(1024)
    k_ln_dparam(const float* __restrict__ part, int blocks, int64_t n, O* __restrict__ dw, O* __restrict__ db) {
  __shared__ float red[2][32][33];
  const int cl = threadIdx.x & 31, bl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.0f, t = 0.0f;
  if (c < n) {
#pragma unroll 8
    for (int b = bl; b < blocks; b += 32) {
      s += part[(2 * (int64_t)b) * n + c];
      t += part[(2 * (int64_t)b + 1) * n + c];
    }
  }
  red[0][bl][cl] = s;
  red[1][bl][cl] = t;
  __syncthreads();
  if (bl < 2 && c < n) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) u += red[bl][i][cl];
    O* out = bl ? db : dw;
    if (out) out[c] = from_f<O>(u);
  }
}

// The smallest group (a power of two) that holds n columns in nv vectors a
// thread, between lo and 1024 threads.
int group_threads(int64_t n, int nv, int lo) {
  int g = lo;
  while ((int64_t)g * nv * 8 < n) g *= 2;
  return g;
}

mpq_status ln_check(const char* who, int64_t rows, int64_t n, int32_t dtype, const void* w, const void* b,
                    int32_t pd) {
  if (rows < 0 || rows > MAX_ROWS || n < 1 || n > (1 << 20))
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": need 0 <= rows < 2^31 and 1 <= n <= 2^20");
  if (!any_dtype(dtype)) return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": unknown element type");
  if ((w || b) && pd != dtype && pd != MPQ_F32)
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": weight and bias must have x's type or fp32");
  return MPQ_OK;
}

template <typename T, int PM>
void ln_fwd_rows(LnArgs a, float e, T* y, float* mean, float* rstd, cudaStream_t st) {
  const auto go = [&](auto kernel, int nv, int nr) {
    a.G = group_threads(a.n, nv, 4);
    const int block = a.G > 32 ? a.G : 128;  // a group of several warps is the whole block
    kernel<<<(unsigned)cdiv(a.rows, (int64_t)(block / a.G) * nr), block, 0, st>>>(a, e, y, mean, rstd);
  };
  // One vector a thread where there are too few rows to fill the device with
  // small groups; 4 otherwise: a row of 4096 then has one barrier between 4
  // warps per sum, and 8 rows are at work on an SM.
  const bool few = a.rows * cdiv(a.n, 1024) < 8 * a.sms;
  if (few && a.n <= 8192) go(k_ln_fwd<T, 1, 1, PM>, 1, 1);
  else if (a.n <= 256) go(k_ln_fwd<T, 1, 4, PM>, 1, 4);
  else if (a.n <= 512) go(k_ln_fwd<T, 2, 2, PM>, 2, 2);
  // (fp32 parameters weigh as much as four rows of 16-bit elements: 16384 x
  // 4096 takes 55 us with two rows a group, 61 with one; with 16-bit
  // parameters 8000 x 8192 takes 64 and 56)
  else if (PM == PM_F32 && sizeof(T) == 2 && a.n <= 8192) go(k_ln_fwd<T, 4, 2, PM>, 4, 2);
  else go(k_ln_fwd<T, 4, 1, PM>, 4, 1);
}
template <typename T>
mpq_status ln_fwd(const LnArgs& a, double eps, void* y, float* mean, float* rstd, cudaStream_t st) {
  T* yo = static_cast<T*>(y);
  const float e = (float)eps;
  ProfScope ps_("k_layer_norm", st);
  if (a.n > LN_REG_MAX) k_ln_fwd_wide<T><<<(unsigned)a.rows, 1024, 0, st>>>(a, e, yo, mean, rstd);
  else if (!a.p_vec || !a.w != !a.b) ln_fwd_rows<T, PM_ANY>(a, e, yo, mean, rstd, st);
  else if (!a.x_vec || !a.o_vec || a.n % 8) {
    if (a.n <= 128) ln_fwd_rows<T, PM_ANY>(a, e, yo, mean, rstd, st);
    else if (!a.w) ln_fwd_rows<T, PM_NONE | PM_SHIFT>(a, e, yo, mean, rstd, st);
    else if (a.p_f32) ln_fwd_rows<T, PM_F32 | PM_SHIFT>(a, e, yo, mean, rstd, st);
    else ln_fwd_rows<T, PM_T | PM_SHIFT>(a, e, yo, mean, rstd, st);
  }
  else if (!a.w) ln_fwd_rows<T, PM_NONE>(a, e, yo, mean, rstd, st);
  else if (a.p_f32) ln_fwd_rows<T, PM_F32>(a, e, yo, mean, rstd, st);
  else ln_fwd_rows<T, PM_T>(a, e, yo, mean, rstd, st);
  count_launch();
  return check_launch("k_layer_norm");
}

template <typename T, int PM, bool SUMS>
mpq_status ln_bwd_rows(LnArgs a, const T* dy, int64_t ldy, const float* mean, const float* rstd, T* dx, float* part,
                       int64_t* blocks, cudaStream_t st) {
  const auto go = [&](auto kernel, int nv) -> mpq_status {
    a.C = (int)cdiv(a.n, LN_PART);
    a.G = a.C > 1 ? LN_PART / 16 : group_threads(a.n, nv, 4);
    const int block = a.G > 32 ? a.G : 128;
    const int64_t groups = block / a.G;
    *blocks = std::min<int64_t>({cdiv(a.rows, groups), (int64_t)a.sms * std::max(1, std::min(8, 512 / block)) / a.C,
                                 LN_BACK_BLOCKS});  // (the workspace has no more partial rows)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(*blocks * a.C));
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = SUMS && groups > 1 ? (size_t)(2 * a.n * 4) : 0;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.C > 1 ? 1 : 0;
    MPQ_CUDA(cudaLaunchKernelEx(&cfg, kernel, (const LnArgs)a, dy, ldy, mean, rstd, dx, part));
    return MPQ_OK;
  };
  // (rows at any address hold one vector more on its way)
  if (a.n <= (PM != PM_ANY && (PM & PM_SHIFT) ? 4096 : 256)) return go(k_ln_bwd<T, 1, PM, SUMS, false>, 1);
  if (a.n <= LN_PART) return go(k_ln_bwd<T, 2, PM, SUMS, false>, 2);
  return go(k_ln_bwd<T, 2, PM, SUMS, true>, 2);
}
template <typename T>
mpq_status ln_bwd(LnArgs a, const void* dy, int64_t ldy, bool y_vec, const float* mean, const float* rstd,
                  void* dx, void* dw, void* db, float* part, cudaStream_t st) {
  const T* dyp = static_cast<const T*>(dy);
  T* dxp = static_cast<T*>(dx);
  const bool sums = dw || db;
  int64_t blocks = 0;
  if (a.n > LN_BACK_MAX) {
    if (dx) {
      ProfScope ps_("k_ln_dx_wide", st);
      k_ln_dx_wide<T><<<(unsigned)a.rows, 1024, 0, st>>>(a, dyp, ldy, y_vec, mean, rstd, dxp);
      count_launch();
      MPQ_TRY(check_launch("k_ln_dx_wide"));
    }
    blocks = cdiv(a.rows, LN_COL_ROWS);
    if (sums) {
      ProfScope ps_("k_ln_cols_wide", st);
      k_ln_cols_wide<T><<<dim3((unsigned)blocks, (unsigned)cdiv(a.n, 256)), 256, 0, st>>>(
          a, dyp, ldy, y_vec, mean, rstd, part);
      count_launch();
      MPQ_TRY(check_launch("k_ln_cols_wide"));
    }
  } else {
    ProfScope ps_("k_ln_bwd", st);
    const auto go = [&](auto pm) {
      constexpr int PM = decltype(pm)::value;
      return sums ? ln_bwd_rows<T, PM, true>(a, dyp, ldy, mean, rstd, dxp, part, &blocks, st)
                  : ln_bwd_rows<T, PM, false>(a, dyp, ldy, mean, rstd, dxp, part, &blocks, st);
    };
    const bool rows_vec = a.x_vec && y_vec && a.o_vec && a.n % 8 == 0;
    if (!a.p_vec || (!rows_vec && a.n <= 128)) MPQ_TRY(go(std::integral_constant<int, PM_ANY>{}));
    else if (!rows_vec && !a.w) MPQ_TRY(go(std::integral_constant<int, PM_NONE | PM_SHIFT>{}));
    else if (!rows_vec && a.p_f32) MPQ_TRY(go(std::integral_constant<int, PM_F32 | PM_SHIFT>{}));
    else if (!rows_vec) MPQ_TRY(go(std::integral_constant<int, PM_T | PM_SHIFT>{}));
    else if (!a.w) MPQ_TRY(go(std::integral_constant<int, PM_NONE>{}));
    else if (a.p_f32) MPQ_TRY(go(std::integral_constant<int, PM_F32>{}));
    else MPQ_TRY(go(std::integral_constant<int, PM_T>{}));
    count_launch();
    MPQ_TRY(check_launch("k_ln_bwd"));
  }
  if (sums) {
    ProfScope ps_("k_ln_dparam", st);
    const unsigned grid = (unsigned)cdiv(a.n, 32);
    if (a.p_f32) k_ln_dparam<float><<<grid, 1024, 0, st>>>(part, (int)blocks, a.n, static_cast<float*>(dw), static_cast<float*>(db));
    else k_ln_dparam<T><<<grid, 1024, 0, st>>>(part, (int)blocks, a.n, static_cast<T*>(dw), static_cast<T*>(db));
    count_launch();
    return check_launch("k_ln_dparam");
  }
  return MPQ_OK;
}

}  // namespace

mpq_status current_device(int* dev, int* sms) {
  static std::atomic<int> cached[64] = {};  // (host threads may call at once)
  MPQ_CUDA(cudaGetDevice(dev));
  if (*dev < 0 || *dev >= 64) return fail(MPQ_ERR_CUDA, "device index out of range");
  int n = cached[*dev].load(std::memory_order_relaxed);
  if (!n) {
    MPQ_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev));
    cached[*dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return MPQ_OK;
}

}  // namespace mpq

using namespace mpq;

extern "C" mpq_status mpq_layer_norm(const void* x, int64_t ldx, int64_t rows, int64_t n, int32_t dtype,
                                     const void* weight, const void* bias, int32_t param_dtype, double eps,
                                     void* y, float* mean, float* rstd, mpq_stream_t stream) {
  MPQ_TRY(ln_check("layer_norm", rows, n, dtype, weight, bias, param_dtype));
  if (!(eps > 0.0) || !((float)eps > 0.0f) || eps > 1e30)
    return fail(MPQ_ERR_INVALID_ARG, "layer_norm: eps must be > 0");
  if (rows == 0) return MPQ_OK;
  if (!x || !y) return fail(MPQ_ERR_INVALID_ARG, "layer_norm: missing buffer");
  const int64_t es = dtype_size(dtype), ps = dtype_size(param_dtype);
  MPQ_TRY(check_elements("layer_norm", {{x, es}, {y, es}, {weight, ps}, {bias, ps}, {mean, 4}, {rstd, 4}}));
  LnArgs a{};
  int dev = 0;
  MPQ_TRY(current_device(&dev, &a.sms));
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.n = n;
  a.w = weight;
  a.b = bias;
  a.p_f32 = param_dtype == MPQ_F32;
  a.x_vec = aligned_rows(x, ldx, es, 16);
  a.p_vec = ((uintptr_t)weight & 15) == 0 && ((uintptr_t)bias & 15) == 0;
  a.o_vec = aligned_rows(y, n, es, 16);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MPQ_BF16) return ln_fwd<__nv_bfloat16>(a, eps, y, mean, rstd, st);
  if (dtype == MPQ_F16) return ln_fwd<__half>(a, eps, y, mean, rstd, st);
  return ln_fwd<float>(a, eps, y, mean, rstd, st);
}

extern "C" int64_t mpq_layer_norm_backward_workspace_bytes(int64_t rows, int64_t n, int32_t need_dparam) {
  if (rows < 1 || n < 1 || !need_dparam) return 0;
  const int64_t blocks = n > LN_BACK_MAX ? cdiv(rows, LN_COL_ROWS) : std::min<int64_t>(rows, LN_BACK_BLOCKS);
  return round_up(blocks * 2 * n * 4, 256);
}

extern "C" mpq_status mpq_layer_norm_backward(const void* dy, int64_t ldy, const void* x, int64_t ldx,
                                              const float* mean, const float* rstd, int64_t rows, int64_t n,
                                              int32_t dtype, const void* weight, int32_t param_dtype, void* dx,
                                              void* dweight, void* dbias, void* workspace,
                                              int64_t workspace_bytes, mpq_stream_t stream) {
  const bool sums = dweight || dbias;
  MPQ_TRY(ln_check("layer_norm_backward", rows, n, dtype, weight ? weight : dweight, dbias, param_dtype));
  const int64_t es = dtype_size(dtype), ps = dtype_size(param_dtype);
  MPQ_TRY(check_elements("layer_norm_backward", {{dy, es}, {x, es}, {mean, 4}, {rstd, 4}, {weight, ps}, {dx, es},
                                                 {dweight, ps}, {dbias, ps}}));
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {
    const size_t bytes = (size_t)(n * dtype_size(param_dtype));
    if (dweight) MPQ_CUDA(cudaMemsetAsync(dweight, 0, bytes, st));
    if (dbias) MPQ_CUDA(cudaMemsetAsync(dbias, 0, bytes, st));
    return MPQ_OK;
  }
  if (!dy || !x || !mean || !rstd) return fail(MPQ_ERR_INVALID_ARG, "layer_norm_backward: missing buffer");
  if (!dx && !sums) return MPQ_OK;
  const int64_t need = mpq_layer_norm_backward_workspace_bytes(rows, n, sums ? 1 : 0);
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
    return fail(MPQ_ERR_INVALID_ARG, "layer_norm_backward: needs " + std::to_string(need) +
                                         " bytes of workspace on a 256-byte boundary");
  LnArgs a{};
  int dev = 0;
  MPQ_TRY(current_device(&dev, &a.sms));
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.n = n;
  a.w = weight;
  a.p_f32 = param_dtype == MPQ_F32;
  a.x_vec = aligned_rows(x, ldx, es, 16);
  a.p_vec = ((uintptr_t)weight & 15) == 0;
  a.o_vec = aligned_rows(dx, n, es, 16);
  const bool y_vec = aligned_rows(dy, ldy, es, 16);
  float* part = static_cast<float*>(workspace);
  if (dtype == MPQ_BF16)
    return ln_bwd<__nv_bfloat16>(a, dy, ldy, y_vec, mean, rstd, dx, dweight, dbias, part, st);
  if (dtype == MPQ_F16) return ln_bwd<__half>(a, dy, ldy, y_vec, mean, rstd, dx, dweight, dbias, part, st);
  return ln_bwd<float>(a, dy, ldy, y_vec, mean, rstd, dx, dweight, dbias, part, st);
}
