// layer_norm: y = (x - mean) rstd w + b per row, and its backward pass with
// the reduction of the parameters' gradients.
//
// Both are bound by HBM: the forward pass reads x and writes y, the backward
// pass reads x and dy and writes dx.  A row is held in the registers of a
// group of G threads (G = 4 .. 1024 by its width, 8 consecutive elements per
// thread and vector), so it is read once: the mean, then the variance around
// it, then the output.  The backward pass adds dw and db on the way: every
// block walks rows with a fixed stride and each of its threads keeps the same
// columns, so the sums stay in registers (in shared memory for wide rows) and
// leave the block once, as one partial row per block; a second kernel adds
// the partial rows in a fixed order.
#include <algorithm>

#include "layer_ops.cuh"

namespace mpq {
namespace {

constexpr int LN_BACK_BLOCKS = 296;        // partial rows of dw and db at most
constexpr int64_t LN_REG_MAX = 32768;      // widest row held in registers (forward)
constexpr int64_t LN_BACK_MAX = 16384;     // and in the one-pass backward kernel
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = G >> 5;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[warp * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < nw ? s[lane * N + i] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
}

struct LnArgs {
  const void* x;
  int64_t ldx, rows, n;
  const void* w;
  const void* b;
  bool p_f32, x_vec, p_vec, o_vec;
  int G;
};

template <typename T, int NV>
__global__ void __launch_bounds__(1024)
    k_ln_fwd(const __grid_constant__ LnArgs a, float eps, T* __restrict__ y, float* __restrict__ mean_out,
             float* __restrict__ rstd_out) {
  __shared__ float scratch[2 * 32];
  int buf = 0;
  const int t = threadIdx.x & (a.G - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / a.G) + threadIdx.x / a.G;
  const bool live = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
  const int n = (int)a.n;
  float v[NV][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * a.G) * 8;
    if (live && c < n) load_edge<8>(xr + c, v[j], n - c, a.x_vec);
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += v[j][i];
  }
  group_sum<1>(s, a.G, scratch, buf);
  const float mean = s[0] / (float)n;
  float q[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * a.G) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[j][i] -= mean;
      if (c + i < n) q[0] = fmaf(v[j][i], v[j][i], q[0]);
    }
  }
  group_sum<1>(q, a.G, scratch, buf);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(q[0] / (float)n + eps);
  if (t == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * a.G) * 8;
    if (c >= n) break;
    float w[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { w[i] = 1.0f; b[i] = 0.0f; }
    if (a.w) load_param<8, T>(a.w, a.p_f32, c, w, n - c, a.p_vec);
    if (a.b) load_param<8, T>(a.b, a.p_f32, c, b, n - c, a.p_vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fmaf(v[j][i] * rstd, w[i], b[i]);
    store_edge<8>(y + row * a.n + c, w, n - c, a.o_vec);
  }
}

// Rows too wide for registers: three passes over the row, which L2 serves
// after the first.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_ln_fwd_wide(const __grid_constant__ LnArgs a, float eps, T* __restrict__ y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out) {
  __shared__ float scratch[2 * 32];
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
enum { ACC_NONE = 0, ACC_REG = 1, ACC_SMEM = 2 };

// dx of rows row0, row0 + step, ... and, per block, the column sums of dy xh
// and dy over those rows.  The next row's loads are issued before this row's
// sums are joined.
template <typename T, int NV, int ACC>
__global__ void __launch_bounds__(1024)
    k_ln_bwd(const __grid_constant__ LnArgs a, const T* __restrict__ dy, int64_t ldy, bool y_vec,
             const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
             float* __restrict__ part) {
  __shared__ float scratch[2 * 64];
  extern __shared__ float accs[];  // ACC_SMEM: dw[n8], db[n8]; ACC_REG with several groups: the join
  int buf = 0;
  const int t = threadIdx.x & (a.G - 1), groups = blockDim.x / a.G;
  const int n = (int)a.n;
  const float inv_n = 1.0f / (float)n;
  constexpr int NA = ACC == ACC_REG ? NV : 1;
  float dw[NA][8], db[NA][8];
#pragma unroll
  for (int j = 0; j < NA; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) { dw[j][i] = 0.0f; db[j][i] = 0.0f; }
  const int n8 = (n + 7) / 8 * 8;
  if (ACC == ACC_SMEM) {  // each thread clears and later adds to its own columns only
    for (int c = t * 8; c < n8; c += a.G * 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) { accs[c + i] = 0.0f; accs[n8 + c + i] = 0.0f; }
  }
  const int64_t step = (int64_t)gridDim.x * groups;
  // every thread of the block takes the same number of turns (group_sum)
  for (int64_t base = (int64_t)blockIdx.x * groups; base < a.rows; base += step) {
    const int64_t row = base + threadIdx.x / a.G;
    const bool live = row < a.rows;
    const T* xr = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
    const T* yr = dy + (live ? row : 0) * ldy;
    float xh[NV][8], g[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * a.G) * 8;
      if (live && c < n) {
        load_edge<8>(xr + c, xh[j], n - c, a.x_vec);
        load_edge<8>(yr + c, g[j], n - c, y_vec);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) { xh[j][i] = 0.0f; g[j][i] = 0.0f; }
      }
    }
    const float m = live ? mean[row] : 0.0f, r = live ? rstd[row] : 0.0f;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * a.G) * 8;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      if (a.w && c < n) load_param<8, T>(a.w, a.p_f32, c, w, n - c, a.p_vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] = (live && c + i < n) ? (xh[j][i] - m) * r : 0.0f;
        const float d = g[j][i];
        if (ACC == ACC_REG) {
          dw[ACC == ACC_REG ? j : 0][i] = fmaf(d, xh[j][i], dw[ACC == ACC_REG ? j : 0][i]);
          db[ACC == ACC_REG ? j : 0][i] += d;
        }
        if (ACC == ACC_SMEM && c < n) {
          accs[c + i] = fmaf(d, xh[j][i], accs[c + i]);
          accs[n8 + c + i] += d;
        }
        g[j][i] = d * w[i];
        s[0] += g[j][i];
        s[1] = fmaf(g[j][i], xh[j][i], s[1]);
      }
    }
    if (dx) {
      group_sum<2>(s, a.G, scratch, buf);
      const float s0 = s[0] * inv_n, s1 = s[1] * inv_n;
      if (live) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (t + j * a.G) * 8;
          if (c >= n) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) g[j][i] = r * (g[j][i] - fmaf(xh[j][i], s1, s0));
          store_edge<8>(dx + row * a.n + c, g[j], n - c, a.o_vec);
        }
      }
    }
  }
  if (ACC == ACC_NONE) return;
  float* pw = part + (int64_t)blockIdx.x * 2 * n;
  float* pb = pw + n;
  if (ACC == ACC_SMEM) {
    for (int c = t * 8; c < n; c += a.G * 8)
      for (int i = 0; i < 8 && c + i < n; ++i) { pw[c + i] = accs[c + i]; pb[c + i] = accs[n8 + c + i]; }
    return;
  }
  if (groups == 1) {
#pragma unroll
    for (int j = 0; j < NA; ++j) {
      const int c = (t + j * a.G) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) { pw[c + i] = dw[j][i]; pb[c + i] = db[j][i]; }
    }
    return;
  }
  // several rows at a time: the groups add up in order
  for (int q = 0; q < groups; ++q) {
    if (threadIdx.x / a.G == q) {
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        const int c = (t + j * a.G) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < n) {
            accs[c + i] = (q ? accs[c + i] : 0.0f) + dw[j][i];
            accs[n8 + c + i] = (q ? accs[n8 + c + i] : 0.0f) + db[j][i];
          }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < n; c += blockDim.x) { pw[c] = accs[c]; pb[c] = accs[n8 + c]; }
}

// Rows too wide for the kernel above: dx in two passes over the row, and the
// column sums by blocks of 256 columns x LN_COL_ROWS rows.
template <typename T>
__global__ void __launch_bounds__(1024)
    k_ln_dx_wide(const __grid_constant__ LnArgs a, const T* __restrict__ dy, int64_t ldy, bool y_vec,
                 const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx) {
  __shared__ float scratch[2 * 64];
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
__global__ void __launch_bounds__(512)
    k_ln_dparam(const float* __restrict__ part, int64_t blocks, int64_t n, O* __restrict__ dw, O* __restrict__ db) {
  __shared__ float red[2][16][32];
  const int cl = threadIdx.x & 31, bl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.0f, t = 0.0f;
  if (c < n)
    for (int64_t b = bl; b < blocks; b += 16) {
      s += part[(2 * b) * n + c];
      t += part[(2 * b + 1) * n + c];
    }
  red[0][bl][cl] = s;
  red[1][bl][cl] = t;
  __syncthreads();
  if (bl < 2 && c < n) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) u += red[bl][i][cl];
    O* out = bl ? db : dw;
    if (out) out[c] = from_f<O>(u);
  }
}

// Threads per row for nv vectors of 8 per thread
int group_threads(int64_t n, int nv) {
  int g = 4;
  while ((int64_t)g * nv * 8 < n) g *= 2;
  return g;
}
int fwd_vectors(int64_t n) { return n <= 8192 ? 1 : n <= 16384 ? 2 : 4; }
int bwd_vectors(int64_t n) { return n <= 8192 ? 1 : 2; }
mpq_status ln_check(const char* who, int64_t rows, int64_t n, int32_t dtype, const void* w, const void* b,
                    int32_t pd) {
  if (rows < 0 || rows > MAX_ROWS || n < 1 || n > (1 << 20))
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": need 0 <= rows < 2^31 and 1 <= n <= 2^20");
  if (!any_dtype(dtype)) return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": unknown element type");
  if ((w || b) && pd != dtype && pd != MPQ_F32)
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": weight and bias must have x's type or fp32");
  return MPQ_OK;
}

template <typename T>
mpq_status ln_fwd(LnArgs a, double eps, void* y, float* mean, float* rstd, cudaStream_t st) {
  T* yo = static_cast<T*>(y);
  const float e = (float)eps;
  ProfScope ps_("k_layer_norm", st);
  if (a.n > LN_REG_MAX) {
    k_ln_fwd_wide<T><<<(unsigned)a.rows, 1024, 0, st>>>(a, e, yo, mean, rstd);
  } else {
    const int nv = fwd_vectors(a.n);
    a.G = group_threads(a.n, nv);
    const int block = std::max(a.G, 128);
    const unsigned grid = (unsigned)cdiv(a.rows, block / a.G);
    if (a.G > 32 && block != a.G) {  // a group of several warps is the whole block
      const unsigned rows = (unsigned)a.rows;
      k_ln_fwd<T, 1><<<rows, a.G, 0, st>>>(a, e, yo, mean, rstd);
    } else if (nv == 1) {
      k_ln_fwd<T, 1><<<grid, block, 0, st>>>(a, e, yo, mean, rstd);
    } else if (nv == 2) {
      k_ln_fwd<T, 2><<<grid, block, 0, st>>>(a, e, yo, mean, rstd);
    } else {
      k_ln_fwd<T, 4><<<grid, block, 0, st>>>(a, e, yo, mean, rstd);
    }
  }
  count_launch();
  return check_launch("k_layer_norm");
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
    const int nv = bwd_vectors(a.n);
    a.G = group_threads(a.n, nv);
    const int block = a.G < 256 ? (a.G > 32 ? a.G : 256) : a.G;
    const int groups = block / a.G;
    blocks = std::min<int64_t>(cdiv(a.rows, groups), LN_BACK_BLOCKS);
    const int n8 = (int)round_up(a.n, 8);
    ProfScope ps_("k_ln_bwd", st);
    if (!sums) {
      const unsigned grid = (unsigned)std::min<int64_t>(cdiv(a.rows, groups), 148 * 8);
      if (nv == 1) k_ln_bwd<T, 1, ACC_NONE><<<grid, block, 0, st>>>(a, dyp, ldy, y_vec, mean, rstd, dxp, nullptr);
      else k_ln_bwd<T, 2, ACC_NONE><<<grid, block, 0, st>>>(a, dyp, ldy, y_vec, mean, rstd, dxp, nullptr);
    } else if (nv == 1) {
      const int smem = groups > 1 ? 2 * n8 * 4 : 0;
      k_ln_bwd<T, 1, ACC_REG><<<(unsigned)blocks, block, smem, st>>>(a, dyp, ldy, y_vec, mean, rstd, dxp, part);
    } else {
      MPQ_CUDA(cudaFuncSetAttribute(k_ln_bwd<T, 2, ACC_SMEM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(2 * LN_BACK_MAX * 4)));
      k_ln_bwd<T, 2, ACC_SMEM><<<(unsigned)blocks, block, 2 * n8 * 4, st>>>(a, dyp, ldy, y_vec, mean, rstd, dxp, part);
    }
    count_launch();
    MPQ_TRY(check_launch("k_ln_bwd"));
  }
  if (sums) {
    ProfScope ps_("k_ln_dparam", st);
    const unsigned grid = (unsigned)cdiv(a.n, 32);
    if (a.p_f32) k_ln_dparam<float><<<grid, 512, 0, st>>>(part, blocks, a.n, static_cast<float*>(dw), static_cast<float*>(db));
    else k_ln_dparam<T><<<grid, 512, 0, st>>>(part, blocks, a.n, static_cast<T*>(dw), static_cast<T*>(db));
    count_launch();
    return check_launch("k_ln_dparam");
  }
  return MPQ_OK;
}

}  // namespace

mpq_status current_device(int* dev, int* sms) {
  static int cached[64] = {};
  MPQ_CUDA(cudaGetDevice(dev));
  if (*dev < 0 || *dev >= 64) return fail(MPQ_ERR_CUDA, "device index out of range");
  if (!cached[*dev]) {
    int n = 0;
    MPQ_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev));
    cached[*dev] = n;
  }
  *sms = cached[*dev];
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
  const int64_t es = dtype_size(dtype);
  LnArgs a{};
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
  const int64_t es = dtype_size(dtype);
  LnArgs a{};
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
