// Operators over rows of logits: token_logprobs (log probability of given
// tokens, entropy, top alternatives) and topk_distill (KL divergence from a
// teacher's top logits and the student's gradient).
//
// One pass over a row of v logits with the running maximum and sums of a
// softmax, in powers of two: with k = log2(e) / T, M the row's largest logit and
// y = (l - M) k, S = sum 2^y and U = sum y 2^y, so that
//   log p_t = (l_t - M) / T - ln S,   H = ln S - ln2 U / S.
// The maximum is subtracted before the scaling, so that its own y is 0 whatever
// its size: in l k - M k a rounded M k leaves half a step of M k, which for a
// finite mask of -1e10 is hundreds.  A cluster of C CTAs shares a row when there are few rows
// (each takes a stretch of the columns; sums and top lists meet over
// distributed shared memory in rank order).
//
// Top alternatives without a second pass: every thread keeps the largest
// logit it met.  The top-th largest of the maxima of 128 disjoint sets of
// columns is a lower bound of the row's top-th largest logit, and only
// threads whose maximum reaches it can hold a candidate (about `top` of 256),
// so only their columns are read again, from L2.  The candidates are ranked
// by counting.  The order is (logit descending, id ascending) throughout: a
// total order, so the result does not depend on the order of any atomics.
//
// What bounds them: HBM by the bytes, and before it the issue of an exponential
// and its arithmetic per element.  At 1024 rows of 131072 bf16 logits (268 MB):
// token_logprobs without alternatives 60 us (4.5 TB/s), with 20 alternatives 78
// (3.4 TB/s; 61% of the issue slots); topk_distill, which reads the row twice
// and writes the gradient, 125 us against 82 for the bytes read once.
#include <algorithm>
#include <type_traits>

#include "layer_ops.cuh"

namespace mpq {
namespace {

constexpr int TOP_SETS = 128;      // sets of columns whose maxima bound the top list
constexpr int CAND = 4096;         // candidates ranked at once
constexpr int64_t L2_ROWS = 96ll << 20;  // logits at work that L2 (126 MB) is trusted with
constexpr float M_FLOOR = -3.4028234663852886e38f;  // start of the running maximum: fp32's lowest value
constexpr float Y_FLOOR = -150.0f;  // an exponent whose power is 0, and stays finite times a sum
constexpr float LN2 = 0.69314718055994531f, LOG2E = 1.4426950408889634f;
static_assert(TOP_SETS >= MPQ_TOP_MAX, "a bound needs `top` sets");

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A row cut into vectors of 8 columns that start on 16-byte boundaries:
// vector g covers columns first + 8 g .. first + 8 g + 7, of which those
// outside [0, v) do not exist (first is -7 .. 0).
template <typename T>
struct Row {
  const T* p;
  int v, first, nvec;
  __device__ __forceinline__ Row(const T* row, int v_) : p(row), v(v_) {
    const int off = (int)(((uintptr_t)row & 15) / sizeof(T));  // elements past a boundary
    first = -off;
    nvec = (v + off + 7) / 8;
  }
  __device__ __forceinline__ int col(int g) const { return first + 8 * g; }
  __device__ __forceinline__ Raw8<T> load(int g) const {  // columns that do not exist: -inf
    Raw8<T> r;
    const int c = col(g);
    if (c >= 0 && c + 8 <= v) {
      const uint4* s = reinterpret_cast<const uint4*>(p + c);
#pragma unroll
      for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.q[i] = __ldg(s + i);
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = (c + i >= 0 && c + i < v) ? p[c + i] : from_f<T>(-INFINITY);
      memcpy(&r, e, sizeof(r));
    }
    return r;
  }
};

template <typename T>
__device__ __forceinline__ Raw8<T> encode(const float (&x)[8]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    memcpy(&r, x, sizeof(r));
  } else {
    const T* t = nullptr;
    r.q[0] = make_uint4(pack2(x[0], x[1], t), pack2(x[2], x[3], t), pack2(x[4], x[5], t), pack2(x[6], x[7], t));
  }
  return r;
}

struct Soft {  // the running softmax: maximum, sums
  float m, s, u;
};
template <bool ENT>
__device__ __forceinline__ Soft merge(const Soft& a, const Soft& b, float k) {
  const float m = fmaxf(a.m, b.m);
  // (a maximum of +inf has a NaN for its sum already)
  const float da = fmaxf((a.m - m) * k, Y_FLOOR), db = fmaxf((b.m - m) * k, Y_FLOOR);
  const float ca = ex2(da), cb = ex2(db);
  Soft r;
  r.m = m;
  r.s = fmaf(ca, a.s, cb * b.s);
  r.u = ENT ? fmaf(ca, fmaf(da, a.s, a.u), cb * fmaf(db, b.s, b.u)) : 0.0f;
  return r;
}
template <bool ENT>
__device__ __forceinline__ Soft warp_merge(Soft a, float k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Soft b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.u = ENT ? __shfl_xor_sync(0xffffffffu, a.u, o) : 0.0f;
    a = merge<ENT>(a, b, k);
  }
  return a;
}

__device__ __forceinline__ uint32_t order_key(float x) {  // order-preserving
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);  // -0 ties with 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint64_t full_key(float x, uint32_t id) {
  return ((uint64_t)order_key(x) << 32) | (0xffffffffu - id);
}

// One pass over vectors [lo, hi) of the row: the running softmax, and (TOP)
// the thread's largest logit with its vector.  `best_g` stays -1 where no
// logit above -inf was met.
template <int AT, typename T, bool ENT, bool TOP>
__device__ __forceinline__ Soft scan_row(const Row<T>& row, int lo, int hi, float k, float& best, int& best_g) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;  // 64 bytes in flight per thread
  float m = M_FLOOR;
  uint64_t s2 = 0ull, u2 = 0ull;
  const uint64_t k2 = f2_pack(k, k);
  best = -INFINITY;
  best_g = -1;
  for (int g0 = lo + (int)threadIdx.x; g0 < hi; g0 += AT * U) {
    Raw8<T> r[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (g0 + j * AT < hi) r[j] = row.load(g0 + j * AT);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g0 + j * AT >= hi) break;
      float x[8];
      decode<T>(r[j], x);
      const float top = fmax3(fmax3(fmax3(x[0], x[1], x[2]), x[3], x[4]), fmaxf(x[5], x[6]), x[7]);
      if (TOP && top > best) {
        best = top;
        best_g = g0 + j * AT;
      }
      const float old = m;
      m = fmaxf(m, top);
      const float d = fmaxf((old - m) * k, Y_FLOOR), c = ex2(d);
      const uint64_t c2 = f2_pack(c, c);
      if (ENT) u2 = f2_mul(c2, f2_fma(f2_pack(d, d), s2, u2));
      s2 = f2_mul(s2, c2);
      const uint64_t m2 = f2_pack(-m, -m);
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f2_unpack(f2_mul(f2_add(f2_pack(x[2 * i], x[2 * i + 1]), m2), k2), y[2 * i], y[2 * i + 1]);
      if (ENT) {
        // masked logits: keeps 0 * (-inf) out of the entropy's sum
        const float low = fmin3(fmin3(fmin3(y[0], y[1], y[2]), y[3], y[4]), fminf(y[5], y[6]), y[7]);
        if (low < Y_FLOOR) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = max_nan(y[i], Y_FLOOR);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t e2 = f2_pack(ex2(y[2 * i]), ex2(y[2 * i + 1]));
        s2 = f2_add(s2, e2);
        if (ENT) u2 = f2_fma(f2_pack(y[2 * i], y[2 * i + 1]), e2, u2);
      }
    }
  }
  Soft a{m, 0.0f, 0.0f};
  float e0, e1;
  f2_unpack(s2, e0, e1);
  a.s = e0 + e1;
  f2_unpack(u2, e0, e1);
  a.u = e0 + e1;
  return a;
}

struct RowStat {
  Soft a;
  float logs;   // ln S
  bool empty;   // all logits are -inf: S = 0 (else the largest adds 1)
};

template <int AT>
struct AnsShared {
  Soft warp[AT / 32];
  Soft cta;               // this CTA's part of the row (read by the cluster)
};

template <bool CL>
__device__ __forceinline__ void sync_row() {
  if (CL) {
    __syncwarp();
    tcx::cluster_sync();
  } else {
    __syncthreads();
  }
}
__device__ __forceinline__ uint64_t ld_cluster64(const uint64_t* p, int rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(tcx::map_to_rank(tcx::smem_u32(p), (uint32_t)rank)) : "memory");
  return v;
}

// Joins the threads' softmaxes over the CTA and the cluster of C CTAs; every
// thread gets the row's.
template <int AT, bool ENT, bool CL>
__device__ __forceinline__ RowStat join_row(Soft a, float k, int C, AnsShared<AT>& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  a = warp_merge<ENT>(a, k);
  if (lane == 0) sh.warp[warp] = a;
  __syncthreads();
  if (warp == 0) {
    Soft b{M_FLOOR, 0.0f, 0.0f};
    if (lane < AT / 32) b = sh.warp[lane];
    b = warp_merge<ENT>(b, k);
    if (lane == 0) sh.cta = b;
  }
  sync_row<CL>();
  RowStat st;
  if (CL) {
    Soft b{M_FLOOR, 0.0f, 0.0f};
    if (lane < C) {  // a lane per CTA, so that the remote loads overlap
      b.m = ld_cluster(&sh.cta.m, lane);
      b.s = ld_cluster(&sh.cta.s, lane);
      b.u = ENT ? ld_cluster(&sh.cta.u, lane) : 0.0f;
    }
    st.a = warp_merge<ENT>(b, k);
  } else {
    st.a = sh.cta;
  }
  st.empty = st.a.s == 0.0f;
  st.logs = st.empty ? 0.0f : logf(st.a.s);
  return st;
}

// log p of a logit x of the row
__device__ __forceinline__ float log_prob(const RowStat& st, float x, float inv_t) {
  if (st.empty) return -INFINITY;
  const float d = x - st.a.m;
  if (d == -INFINITY && x > -INFINITY)  // their distance overflows, which a temperature may bring back
    return fmaf(x, inv_t, -fmaf(st.a.m, inv_t, st.logs));
  return fmaf(d, inv_t, -st.logs);
}

// ---------------------------------------------------------- token_logprobs --
template <int AT>
struct TopShared {
  uint64_t sets[TOP_SETS];
  uint64_t cand[CAND];
  uint64_t list[MPQ_TOP_MAX];  // this CTA's top list, descending (read by the cluster)
  uint64_t bound;
  int flagged[AT];
  int n_flagged, n_cand;
  uint64_t warp_best[AT / 32];
};

// Hands the `top` largest of n <= CAND keys to put(position, key), zeros
// behind the last.  Few keys are ranked by counting; many are sorted
// (bitonic; the buffer is padded to a power of two).
template <int AT, typename F>
__device__ __forceinline__ void rank_keys(uint64_t* keys, int n, int top, F put) {
  const int tid = threadIdx.x;
  if (n <= 2 * TOP_SETS) {
    for (int i = tid; i < n; i += AT) {
      const uint64_t key = keys[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += (keys[j] > key || (keys[j] == key && j < i)) ? 1 : 0;
      if (rank < top) put(rank, key);
    }
    for (int i = n + tid; i < top; i += AT) put(i, 0ull);
    return;
  }
  int p = 4 * TOP_SETS;
  while (p < n) p *= 2;
  for (int i = n + tid; i < p; i += AT) keys[i] = 0;
  __syncthreads();
  for (int size = 2; size <= p; size *= 2)
    for (int half = size / 2; half > 0; half /= 2) {
      for (int i = tid; i < p / 2; i += AT) {
        const int a = 2 * half * (i / half) + i % half, b = a + half;
        const uint64_t x = keys[a], y = keys[b];
        const bool down = (a & size) == 0;  // this run descends
        if (down ? x < y : x > y) {
          keys[a] = y;
          keys[b] = x;
        }
      }
      __syncthreads();
    }
  for (int i = tid; i < top; i += AT) put(i, keys[i]);  // p > top
}

// The CTA's `top` largest (logit, id) of vectors [lo, hi) into sh.list, zeros
// behind the last.  best, best_g: as scan_row left them; nan: the thread met a
// NaN.
template <int AT, typename T>
__device__ __forceinline__ void cta_top(const Row<T>& row, int lo, int hi, int top, float best, int best_g,
                                        bool nan, TopShared<AT>& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a thread that met nothing above -inf stands for its first vector, if it
  // has one; where that may hold NaN only, with the lowest key there is
  const int own_g = best_g >= 0 ? best_g : lo + tid;
  const uint64_t mine = own_g >= hi ? 0ull : (best_g < 0 && nan) ? 1ull : full_key(best, (uint32_t)own_g);
  uint64_t q = mine;
#pragma unroll
  for (int o = 1; o < AT / TOP_SETS; o *= 2) q = max(q, __shfl_xor_sync(0xffffffffu, q, o));
  if (tid % (AT / TOP_SETS) == 0) sh.sets[tid / (AT / TOP_SETS)] = q;
  if (tid == 0) {
    sh.n_flagged = 0;
    sh.n_cand = 0;
    sh.bound = 0;
  }
  if (tid < MPQ_TOP_MAX) sh.list[tid] = 0;
  __syncthreads();
  if (tid < TOP_SETS) {
    const uint64_t key = sh.sets[tid];
    int rank = 0;
#pragma unroll 16
    for (int i = 0; i < TOP_SETS; ++i) {
      const uint64_t o = sh.sets[i];
      rank += (o > key || (o == key && i < tid)) ? 1 : 0;
    }
    if (rank == top - 1) sh.bound = key;
  }
  __syncthreads();
  // keys of vectors: (largest logit, vector); every one of the top logits has
  // (logit, its vector) >= bound
  const uint64_t bound = sh.bound;
  // (a thread with the lowest key may hold logits of -inf next to its NaN: read
  // where the bound is one)
  const bool hidden = mine == 1 && bound <= full_key(-INFINITY, 0);
  if (hidden || (mine != 0 && mine >= bound)) sh.flagged[atomicAdd(&sh.n_flagged, 1)] = tid;
  __syncthreads();
  const int per = (hi - lo + AT - 1) / AT, items = sh.n_flagged * per;
  const float floor_x = bound > 1 ? key_value((uint32_t)(bound >> 32)) : -INFINITY;
  constexpr int RU = 4;  // loads in flight
  for (int i0 = tid; i0 < items; i0 += AT * RU) {
    Raw8<T> raw[RU];
    int gs[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int i = i0 + u * AT;
      gs[u] = i < items ? lo + sh.flagged[i / per] + (i % per) * AT : hi;
      if (gs[u] < hi) raw[u] = row.load(gs[u]);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      if (gs[u] >= hi) continue;
      float x[8];
      decode<T>(raw[u], x);
      const float mx = fmax3(fmax3(fmax3(x[0], x[1], x[2]), x[3], x[4]), fmaxf(x[5], x[6]), x[7]);
      if (!(mx >= floor_x)) continue;  // few vectors hold a candidate
      const int c = row.col(gs[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (x[j] >= floor_x && c + j >= 0 && c + j < row.v && full_key(x[j], (uint32_t)gs[u]) >= bound) {
          const int at = atomicAdd(&sh.n_cand, 1);
          if (at < CAND) sh.cand[at] = full_key(x[j], (uint32_t)(c + j));
        }
      }
    }
  }
  __syncthreads();
  const int n = sh.n_cand;
  if (n <= CAND) {
    rank_keys<AT>(sh.cand, n, top, [&](int at, uint64_t key) { sh.list[at] = key; });
    __syncthreads();
    return;
  }
  // a few threads hold most of the row's largest logits: take the list one
  // by one, the largest key below the last one taken
  uint64_t last = ~0ull;
  for (int t = 0; t < top; ++t) {
    uint64_t b = 0;
    for (int i = tid; i < items; i += AT) {
      const int g = lo + sh.flagged[i / per] + (i % per) * AT;
      if (g >= hi) continue;
      float x[8];
      decode<T>(row.load(g), x);
      const int c = row.col(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (c + j < 0 || c + j >= row.v || x[j] != x[j]) continue;
        const uint64_t key = full_key(x[j], (uint32_t)(c + j));
        if (key < last && key > b) b = key;
      }
    }
    for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
    if (lane == 0) sh.warp_best[warp] = b;
    __syncthreads();
    b = sh.warp_best[0];
    for (int w = 1; w < AT / 32; ++w) b = max(b, sh.warp_best[w]);
    if (tid == 0) sh.list[t] = b;
    last = b;
    __syncthreads();
    if (b == 0) break;
  }
}

struct LogprobArgs {
  const void* logits;
  int64_t ldl, rows;
  int v, top, C;
  const int64_t* tokens;
  int64_t ignore;
  float* logprob;
  float* entropy;
  float* top_logprob;
  int64_t* top_id;
};

template <int AT, typename T, bool TOP, bool CL>
__global__ void __launch_bounds__(AT, 1024 / AT) k_token_logprobs(const __grid_constant__ LogprobArgs a) {
  __shared__ AnsShared<AT> sh;
  __shared__ typename std::conditional<TOP, TopShared<AT>, int>::type top_sh;
  const int rank = CL ? (int)tcx::cluster_ctarank() : 0;
  const int64_t r = CL ? blockIdx.x / (unsigned)a.C : blockIdx.x;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ldl, a.v);
  const int lo = CL ? (int)((int64_t)row.nvec * rank / a.C) : 0;
  const int hi = CL ? (int)((int64_t)row.nvec * (rank + 1) / a.C) : row.nvec;
  float best;
  int best_g;
  const Soft part = scan_row<AT, T, true, TOP>(row, lo, hi, LOG2E, best, best_g);
  if constexpr (TOP) cta_top<AT, T>(row, lo, hi, a.top, best, best_g, part.s != part.s, top_sh);
  const RowStat st = join_row<AT, true, CL>(part, LOG2E, a.C, sh);  // (its barriers publish the top lists)
  if (rank == 0 && threadIdx.x == 0) {
    if (a.logprob) {
      const int64_t t = a.tokens[r];
      float lp = 0.0f;
      if (t != a.ignore) lp = (t < 0 || t >= a.v) ? NAN : log_prob(st, to_f(row.p[t]), 1.0f);
      a.logprob[r] = lp;
    }
    if (a.entropy) a.entropy[r] = st.empty ? 0.0f : max_nan(0.0f, fmaf(-LN2, st.a.u / st.a.s, st.logs));
  }
  if constexpr (TOP) {
    auto put = [&](int at, uint64_t key) {
      const int64_t o = r * a.top + at;
      a.top_id[o] = key ? (int64_t)(0xffffffffu - (uint32_t)key) : -1;
      a.top_logprob[o] = (key || st.a.s != st.a.s) ? log_prob(st, key_value((uint32_t)(key >> 32)), 1.0f) : -INFINITY;
    };
    if (!CL) {
      if ((int)threadIdx.x < a.top) put((int)threadIdx.x, top_sh.list[threadIdx.x]);
    } else {
      if (rank == 0) {  // the CTAs' lists become one
        const int n = a.C * a.top;  // <= 8 * MPQ_TOP_MAX
        for (int i = threadIdx.x; i < n; i += AT)
          top_sh.cand[i] = ld_cluster64(&top_sh.list[i % a.top], i / a.top);
        __syncthreads();
        rank_keys<AT>(top_sh.cand, n, a.top, put);
      }
    }
  }
  if (CL) sync_row<true>();  // no peer still reads this CTA's memory
}

// ------------------------------------------------------------ topk_distill --
struct DistillArgs {
  const void* logits;
  int64_t ldl, rows;
  int v, top, C;
  const float* top_logits;
  const int64_t* top_ids;
  const float* weight;
  float k, inv_t;
  float* loss;
  void* dlogits;
};

struct TeacherShared {
  float q[MPQ_TOP_MAX], logq[MPQ_TOP_MAX];
  int id[MPQ_TOP_MAX];  // -1: padding
  int bad, live;
};

// The teacher's q and log q over its entries, in one warp.
__device__ __forceinline__ void teacher_row(const DistillArgs& a, int64_t r, TeacherShared& sh) {
  const int lane = threadIdx.x;
  float t[MPQ_TOP_MAX / 32], mx = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < MPQ_TOP_MAX / 32; ++j) {
    const int e = lane + 32 * j;
    t[j] = -INFINITY;
    if (e < a.top) {
      const int64_t id = a.top_ids[r * a.top + e];
      if (id >= a.v) bad = true;
      const bool use = id >= 0 && id < a.v;
      if (use) t[j] = a.top_logits[r * a.top + e];
      sh.id[e] = use ? (int)id : -1;
    }
    mx = max_nan(mx, t[j]);
  }
  for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const bool live = mx != -INFINITY;  // an entry is left (a NaN one makes the row NaN)
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < MPQ_TOP_MAX / 32; ++j)
    if (lane + 32 * j < a.top && live) sum += expf((t[j] - mx) * a.inv_t);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float ls = live ? logf(sum) : 0.0f;
#pragma unroll
  for (int j = 0; j < MPQ_TOP_MAX / 32; ++j) {
    const int e = lane + 32 * j;
    if (e < a.top) {
      const float d = (t[j] - mx) * a.inv_t;
      sh.q[e] = live ? expf(d) / sum : 0.0f;
      sh.logq[e] = live ? d - ls : 0.0f;
    }
  }
  const unsigned any_bad = __ballot_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.bad = any_bad != 0;
    sh.live = live;
  }
}

template <int AT, typename T, bool CL>
__global__ void __launch_bounds__(AT, 1024 / AT) k_topk_distill(const __grid_constant__ DistillArgs a) {
  __shared__ AnsShared<AT> sh;
  __shared__ TeacherShared te;
  const int rank = CL ? (int)tcx::cluster_ctarank() : 0;
  const int64_t r = CL ? blockIdx.x / (unsigned)a.C : blockIdx.x;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ldl, a.v);
  const int lo = CL ? (int)((int64_t)row.nvec * rank / a.C) : 0;
  const int hi = CL ? (int)((int64_t)row.nvec * (rank + 1) / a.C) : row.nvec;
  if (threadIdx.x < 32) teacher_row(a, r, te);
  float best;
  int best_g;
  const Soft part = scan_row<AT, T, false, false>(row, lo, hi, a.k, best, best_g);
  const RowStat st = join_row<AT, false, CL>(part, a.k, a.C, sh);
  if (rank == 0 && threadIdx.x < 32) {
    float l = 0.0f;
    for (int e = threadIdx.x; e < a.top; e += 32) {
      const float q = te.q[e];
      if (te.id[e] >= 0 && q != 0.0f)  // (a NaN entry counts)
        l = fmaf(q, te.logq[e] - log_prob(st, to_f(row.p[te.id[e]]), a.inv_t), l);
    }
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (threadIdx.x == 0) a.loss[r] = te.bad ? NAN : te.live ? l : 0.0f;
  }
  if (a.dlogits) {
    T* out = static_cast<T*>(a.dlogits) + r * a.v;
    const float w = a.weight ? a.weight[r] : 1.0f;
    const bool zero = w == 0.0f || (!te.live && !te.bad);
    const float c = te.bad ? NAN : w * a.inv_t, cs = st.empty ? c : c / st.a.s;
    // vectors by the output's alignment now: wide stores, and loads that are
    // shifted where the two rows are aligned differently
    const Row<T> dst(out, a.v);
    const bool same = dst.first == row.first;
    const int lo2 = CL ? (int)((int64_t)dst.nvec * rank / a.C) : 0;
    const int hi2 = CL ? (int)((int64_t)dst.nvec * (rank + 1) / a.C) : dst.nvec;
    const auto fetch = [&](int g) {
      if (same) return row.load(g);
      const int col = dst.col(g);
      if constexpr (sizeof(T) == 2) {
        if (col >= 0) return load_row8<T>(row.p, col, a.v);
      }
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = col + i >= 0 && col + i < a.v ? row.p[col + i] : from_f<T>(0.0f);
      Raw8<T> r;
      memcpy(&r, e, sizeof(r));
      return r;
    };
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    const uint64_t k2 = f2_pack(a.k, a.k), m2 = f2_pack(-st.a.m, -st.a.m), c2 = f2_pack(cs, cs);
    // from the end of the row, which L2 got last (132 us become 128 at 1024 rows
    // of 131072 bf16; stores that leave L2 to the logits: 125)
    for (int tile = (hi2 - lo2 + AT * U - 1) / (AT * U) - 1; tile >= 0; --tile) {
      const int g0 = lo2 + tile * (AT * U) + (int)threadIdx.x;
      Raw8<T> raw[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (g0 + j * AT < hi2) raw[j] = fetch(g0 + j * AT);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int g = g0 + j * AT;
        if (g >= hi2) break;
        float x[8];
        decode<T>(raw[j], x);
        if (zero) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // cs 2^y
            float y0, y1;
            f2_unpack(f2_mul(f2_add(f2_pack(x[2 * i], x[2 * i + 1]), m2), k2), y0, y1);
            f2_unpack(f2_mul(f2_pack(ex2(y0), ex2(y1)), c2), x[2 * i], x[2 * i + 1]);
          }
        }
        const int col = dst.col(g);
        if (col >= 0 && col + 8 <= a.v) {
          Raw8<T> y = encode<T>(x);
          uint4* d = reinterpret_cast<uint4*>(out + col);
#pragma unroll
          for (int i = 0; i < (int)(sizeof(T) / 2); ++i) __stcs(d + i, y.q[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i >= 0 && col + i < a.v) out[col + i] = from_f<T>(x[i]);
        }
      }
    }
    // the teacher's entries in this CTA's columns, each from p and q at once
    // (one rounding); the first of equal ids takes them all
    __syncthreads();
    const int c_lo = dst.col(lo2), c_hi = dst.col(hi2);
    for (int e = threadIdx.x; e < a.top && !zero; e += AT) {
      const int id = te.id[e];
      if (id < c_lo || id >= c_hi || id < 0) continue;
      float q = 0.0f;
      bool first = true;
      for (int j = 0; j < a.top; ++j)
        if (te.id[j] == id) {
          if (j < e) first = false;
          q += te.q[j];
        }
      if (!first) continue;
      const float p = st.empty ? 0.0f : ex2((to_f(row.p[id]) - st.a.m) * a.k) / st.a.s;
      out[id] = from_f<T>(c * (p - q));
    }
  }
  if (CL) sync_row<true>();  // no peer still reads this CTA's memory
}

// CTAs per row: one where the rows fill the device; more, down to 4096
// columns each, where they do not.
int row_ctas(int64_t rows, int64_t v, int sms) {
  int c = 1;
  while (c < 8 && rows * c * 2 <= 2 * sms && v / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename A>
mpq_status launch_rows(void (*kernel)(A), const A& a, int threads, cudaStream_t st, const char* name) {
  const int C = a.C;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * C));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  ProfScope ps_(name, st);
  MPQ_CUDA(cudaLaunchKernelEx(&cfg, kernel, a));
  count_launch();
  return check_launch(name);
}

// Whether four CTAs an SM, a row each, would hold more than L2 does: then two of
// twice the threads.
template <typename T>
bool large_rows(int C, int64_t v, int sms) {
  return C == 1 && 4ll * sms * v * (int64_t)sizeof(T) > L2_ROWS;
}

template <typename T>
mpq_status run_logprobs(const LogprobArgs& a, int sms, cudaStream_t st) {
  // (the columns that are read again should still be in L2: 1024 rows of
  // 131072 bf16 with 64 alternatives take 92 us with 512 threads, 104 with 256;
  // 4096 rows of 32000 with 20 take 125 and 101)
  if (a.top && large_rows<T>(a.C, a.v, sms))
    return launch_rows(k_token_logprobs<512, T, true, false>, a, 512, st, "k_token_logprobs");
  const bool cl = a.C > 1;
  if (a.top) return launch_rows(cl ? k_token_logprobs<256, T, true, true> : k_token_logprobs<256, T, true, false>, a, 256, st, "k_token_logprobs");
  return launch_rows(cl ? k_token_logprobs<256, T, false, true> : k_token_logprobs<256, T, false, false>, a, 256, st, "k_token_logprobs");
}
template <typename T>
mpq_status run_distill(const DistillArgs& a, int sms, cudaStream_t st) {
  // the second reading of a row should find it in L2 (1024 rows of 131072
  // bf16, 20 entries, in row order: 132 us with 512 threads, 144 with 256; from
  // the row's end with streaming stores 125; 4096 rows of 32000: 139 with 512,
  // 121 with 256.  Clusters of 2 and 4 CTAs a row: 137 to 181, 169 to 450)
  if (a.dlogits && large_rows<T>(a.C, a.v, sms)) return launch_rows(k_topk_distill<512, T, false>, a, 512, st, "k_topk_distill");
  return launch_rows(a.C > 1 ? k_topk_distill<256, T, true> : k_topk_distill<256, T, false>, a, 256, st, "k_topk_distill");
}

mpq_status rows_check(const char* who, int64_t rows, int64_t v, int32_t dtype) {
  if (rows < 0 || rows > (1 << 24) || v < 1 || v > (1 << 24))
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": need 0 <= rows <= 2^24 and 1 <= v <= 2^24");
  if (!any_dtype(dtype)) return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": unknown element type");
  return MPQ_OK;
}

}  // namespace
}  // namespace mpq

using namespace mpq;

extern "C" mpq_status mpq_token_logprobs(const void* logits, int64_t ldl, int64_t rows, int64_t v, int32_t dtype,
                                         const int64_t* tokens, int64_t ignore_index, int32_t top, float* logprob,
                                         float* entropy, float* top_logprob, int64_t* top_id,
                                         mpq_stream_t stream) {
  MPQ_TRY(rows_check("token_logprobs", rows, v, dtype));
  if (top < 0 || top > MPQ_TOP_MAX || top > v)
    return fail(MPQ_ERR_INVALID_ARG, "token_logprobs: need 0 <= top <= min(v, " + std::to_string(MPQ_TOP_MAX) + ")");
  if ((logprob == nullptr) != (tokens == nullptr))
    return fail(MPQ_ERR_INVALID_ARG, "token_logprobs: tokens and logprob go together");
  if (rows == 0) return MPQ_OK;
  if (!logits || (top > 0 && (!top_logprob || !top_id)))
    return fail(MPQ_ERR_INVALID_ARG, "token_logprobs: missing buffer");
  MPQ_TRY(check_elements("token_logprobs", {{logits, dtype_size(dtype)}, {tokens, 8}, {logprob, 4}, {entropy, 4},
                                            {top_logprob, 4}, {top_id, 8}}));
  int dev = 0, sms = 0;
  MPQ_TRY(current_device(&dev, &sms));
  LogprobArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.rows = rows;
  a.v = (int)v;
  a.top = top;
  a.C = row_ctas(rows, v, sms);
  a.tokens = tokens;
  a.ignore = ignore_index;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_logprob = top_logprob;
  a.top_id = top_id;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MPQ_BF16) return run_logprobs<__nv_bfloat16>(a, sms, st);
  if (dtype == MPQ_F16) return run_logprobs<__half>(a, sms, st);
  return run_logprobs<float>(a, sms, st);
}

extern "C" mpq_status mpq_topk_distill(const void* logits, int64_t ldl, int64_t rows, int64_t v, int32_t dtype,
                                       const float* top_logits, const int64_t* top_ids, int32_t top,
                                       const float* weight, double temperature, float* loss, void* dlogits,
                                       mpq_stream_t stream) {
  MPQ_TRY(rows_check("topk_distill", rows, v, dtype));
  if (top < 1 || top > MPQ_TOP_MAX)
    return fail(MPQ_ERR_INVALID_ARG, "topk_distill: need 1 <= top <= " + std::to_string(MPQ_TOP_MAX));
  if (!(temperature >= 1e-3 && temperature <= 1e3))
    return fail(MPQ_ERR_INVALID_ARG, "topk_distill: temperature must be in [1e-3, 1e3]");
  if (rows == 0) return MPQ_OK;
  if (!logits || !top_logits || !top_ids || !loss) return fail(MPQ_ERR_INVALID_ARG, "topk_distill: missing buffer");
  MPQ_TRY(check_elements("topk_distill", {{logits, dtype_size(dtype)}, {top_logits, 4}, {top_ids, 8}, {weight, 4},
                                          {loss, 4}, {dlogits, dtype_size(dtype)}}));
  int dev = 0, sms = 0;
  MPQ_TRY(current_device(&dev, &sms));
  DistillArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.rows = rows;
  a.v = (int)v;
  a.top = top;
  a.C = row_ctas(rows, v, sms);
  a.top_logits = top_logits;
  a.top_ids = top_ids;
  a.weight = weight;
  a.k = (float)(1.4426950408889634 / temperature);
  a.inv_t = (float)(1.0 / temperature);
  a.loss = loss;
  a.dlogits = dlogits;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MPQ_BF16) return run_distill<__nv_bfloat16>(a, sms, st);
  if (dtype == MPQ_F16) return run_distill<__half>(a, sms, st);
  return run_distill<float>(a, sms, st);
}
