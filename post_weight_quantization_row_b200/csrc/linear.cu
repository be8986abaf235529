// linear: y = act(x W^T + b) + residual with bf16 or fp16 operands, and its
// backward pass dz = dy * act'(z), dx = dz W, dW = dz^T x, db = sum dz.
//
// All three products run on tcgen05 (kind::f16, fp32 accumulators in TMEM)
// with operands staged by TMA in the layout they have in memory: x W^T has
// both operands contiguous along the contraction (K-major); dz W reads W with
// its output index contiguous (MN-major), and dz^T x reads both so.  The
// instruction and shared-memory descriptors take either order, so no operand
// is transposed or copied.  Two kernels share the tile format (128-byte
// swizzled boxes of 64 contiguous elements):
//  - k_lin_pair: CTA pairs (cta_group::2), 256 x 256 tiles, persistent, two
//    accumulators in TMEM so that a tile's epilogue overlaps the next tile's
//    MMAs.  For products with tiles enough to fill the SMs.
//  - k_lin_split: one 128 x (16..128) tile per cluster of S CTAs, each taking
//    1/S of the contraction; the partial tiles are joined over distributed
//    shared memory in a fixed order.  For few rows and for small outputs.
// One row of x W^T, and two of small or unaligned W, need no tensor cores:
// k_lin_gemv reads W once with a warp per row of it (and any alignment).
// The epilogue adds the bias, applies the activation, adds the residual and
// rounds once, in fp32 before that.
//
// Measured: 4096 x 14336 -> 4096 bf16 with a residual takes 300 to 337 us in a
// replayed graph (1.43 to 1.60 PFLOP/s; the tensor pipe active in 91% of the
// cycles) and 395 in a long loop of calls, where the power cap lowers the clock;
// with an fp32 result 338 to 363; its backward products run at the same rate.  One
// row of 4096 -> 4096: 9.0 us for the 33.6 MB of W (3.7 TB/s; at the
// copy rate 5.1).  In between the fixed part of a launch counts:
// 256 x 2048 -> 512 takes 10.9.
//
// The tensor cores' accumulator drops what falls below its last bit instead of
// rounding it, so a long chain of products drifts towards zero: 2.4e-6 of the
// result over a contraction of 2000, 8.7e-6 over 14336, and for terms of one
// sign 7.8e-4 over 2^20, more than half a step of fp16.  So a chain ends after
// chain_steps<O>() steps and the chains are added, rounded, in the epilogue's
// registers: after 512 products for fp32 results, which keeps their error below
// 1e-6 at any length, and after 4096 for 16-bit ones: 256 last bits at most,
// 3e-5 (measured: 7e-6 over 14336, 2e-5 for terms of one sign), where their half
// step is 5e-4 or 4e-3.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "layer_ops.cuh"

namespace mpq {
namespace {
using namespace tcx;

// Counts the waits that ran out.  It only grows, and mpq_ops_status compares it
// with what its thread saw last: nothing is cleared, so that no call takes a
// timeout from another stream's or thread's.
__device__ uint32_t g_timeouts;
__device__ __forceinline__ void report_timeout() { atomicAdd(&g_timeouts, 1u); }

// ------------------------------------------------------------ activations --
// All from one 2^x and one reciprocal each (special function unit), in forms
// that keep the relative accuracy of small results at large negative z.
__device__ __forceinline__ float rcp_approx(float x) {  // 1 ulp; 0 for inf
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;
// The normal distribution's upper tail Phi(-a) for a >= 0, and e = e^(-a^2/2):
// Phi(-a) e^(a^2/2) as a polynomial in t = 1/(1 + 0.3 a) without constant
// term, fitted to erfcx(a / sqrt 2) / 2 on [0, 13.3] by reweighted least
// squares for the least relative error (1.2e-7; in fp32 2.2e-7 absolute, and
// 1.4e-6 relative up to a = 5, from the rounding of the exponent).
// Half the instructions of erfcf and expf.
__device__ constexpr float TAIL[8] = {0.11962516605854034f, 0.12081687152385712f,  0.09952317178249359f,
                                      0.1298430860042572f,  -0.05609530583024025f, 0.2089640498161316f,
                                      -0.15871335566043854f, 0.03603625297546387f};
__device__ __forceinline__ float normal_tail(float a, float& e) {
  e = ex2(-0.5f * LOG2E * a * a);
  const float t = rcp_approx(fmaf(0.3f, a, 1.0f));
  float q = TAIL[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) q = fmaf(q, t, TAIL[i]);
  return q * t * e;
}
// Bounds that keep a NaN.  Where a factor of the result underflows, the other
// is held finite, so that -inf gives the limit 0 and not inf * 0.
__device__ __forceinline__ float at_most(float x, float hi) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(hi));
  return y;
}
__device__ __forceinline__ float at_least(float x, float lo) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MPQ_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case MPQ_ACT_GELU: {
      float e;
      const float a = at_most(fabsf(z), 30.0f), u = a * normal_tail(a, e);  // |z| Phi(-|z|)
      return z >= 0.0f ? z - u : -u;
    }
    case MPQ_ACT_GELU_TANH: {
      z = at_least(z, -30.0f);
      const float u2 = 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);  // 2 sqrt(2/pi) (...)
      return z * rcp_approx(1.0f + ex2(-LOG2E * u2));
    }
    case MPQ_ACT_SILU:
      z = at_least(z, -128.0f);
      return z * rcp_approx(1.0f + ex2(-LOG2E * z));
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == MPQ_ACT_NONE) return 1.0f;
  if (act == MPQ_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  // beyond |z| = 30 the other three slopes are 0 or 1 to fp32; the clip keeps
  // z^3 and e^-z finite (a NaN stays one)
  const float c = at_most(at_least(z, -30.0f), 30.0f);
  if (act == MPQ_ACT_GELU) {
    float e;
    const float u = normal_tail(fabsf(c), e);
    return fmaf(0.3989422804014327f * c, e, c >= 0.0f ? 1.0f - u : u);
  }
  float u = c, du = 1.0f;
  if (act == MPQ_ACT_GELU_TANH) {
    const float c2 = c * c;
    u = 1.5957691216057308f * fmaf(0.044715f * c2, c, c);
    du = fmaf(0.2140644488f, c2, 1.5957691216057308f);  // u' = 2 sqrt(2/pi) (1 + 0.134145 c^2)
  }
  const float e = ex2(-LOG2E * fabsf(u)), d = rcp_approx(1.0f + e);
  const float s = u >= 0.0f ? d : e * d;  // 1/(1 + e^-u)
  return fmaf(c * (e * d * d), du, s);    // s + c s (1 - s) u'
}

// normal_tail of two values: Q = Phi(-a) / e, e = e^(-a^2/2)
__device__ __forceinline__ uint64_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ void normal_tail2(uint64_t a, uint64_t& q, uint64_t& e) {
  float x0, x1;
  f2_unpack(f2_mul(f2_mul(a, f2_both(-0.5f * LOG2E)), a), x0, x1);
  e = f2_pack(ex2(x0), ex2(x1));
  f2_unpack(f2_fma(a, f2_both(0.3f), f2_both(1.0f)), x0, x1);
  const uint64_t t = f2_pack(rcp_approx(x0), rcp_approx(x1));
  q = f2_both(TAIL[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) q = f2_fma(q, t, f2_both(TAIL[i]));
  q = f2_mul(q, t);
}
// The activation of N values: one choice for all, so that its code is there
// once.
template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int act) {
  switch (act) {
    case MPQ_ACT_GELU:
      if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {  // z Phi(z) with u = |z| Phi(-|z|): z - u for z >= 0, -u below
          const uint64_t a = f2_pack(at_most(fabsf(v[i]), 30.0f), at_most(fabsf(v[i + 1]), 30.0f));
          uint64_t q, e;
          normal_tail2(a, q, e);
          float u0, u1;
          f2_unpack(f2_mul(f2_mul(q, e), a), u0, u1);
          v[i] = (v[i] >= 0.0f ? v[i] : 0.0f) - u0;
          v[i + 1] = (v[i + 1] >= 0.0f ? v[i + 1] : 0.0f) - u1;
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MPQ_ACT_GELU);
      }
      return;
    case MPQ_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MPQ_ACT_RELU);
      return;
    case MPQ_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MPQ_ACT_GELU_TANH);
      return;
    case MPQ_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_value(v[i], MPQ_ACT_SILU);
      return;
    default: return;
  }
}
// dy * act'(z) of 8 elements.  gelu on packed pairs: with a = |z| and w =
// Phi(-a) - a phi(a), act'(z) is 1 - w for z >= 0 and w below.
__device__ __forceinline__ void act_grad8(F8& g, const F8& z, int act) {
  if (act == MPQ_ACT_NONE) return;
  if (act != MPQ_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float z0, z1;
      f2_unpack(z.p[i], z0, z1);
      g.p[i] = f2_mul(g.p[i], f2_pack(act_slope(z0, act), act_slope(z1, act)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float z0, z1;
    f2_unpack(z.p[i], z0, z1);
    const uint64_t a = f2_pack(at_most(fabsf(z0), 30.0f), at_most(fabsf(z1), 30.0f));  // w is 0 from there on
    uint64_t q, e;
    normal_tail2(a, q, e);
    const uint64_t w = f2_mul(f2_fma(a, f2_both(-0.3989422804014327f), q), e);
    float w0, w1, v0, v1;
    f2_unpack(w, w0, w1);
    f2_unpack(f2_sub(f2_both(1.0f), w), v0, v1);
    g.p[i] = f2_mul(g.p[i], f2_pack(z0 >= 0.0f ? v0 : w0, z1 >= 0.0f ? v1 : w1));
  }
}

// ------------------------------------------------------------- the operand --
constexpr int BK = 64;              // contraction per stage
constexpr int BOX = 64 * 64 * 2;    // bytes of a 64 x 64 box (8 KiB)
// Steps accumulated at a stretch: 512 products for fp32 results, 4096 for 16-bit
// ones.  A second chain costs 16-bit results 3 us of code that runs for the
// first time (1024 x 4096 -> 4096, GELU: 37.4 us with chains of 2048, 34.5 with
// 4096); 4096 x 14336 -> 4096 takes 302 us against 300 in one chain, 307 with
// chains of 2048 and 326 with 512.
template <typename O>
__host__ __device__ constexpr int chain_steps() { return sizeof(O) == 4 ? 8 : 64; }

// Operand tiles of 64 (contraction) x 64 .. 128, with 128-byte swizzle.
// K-major (rows of 64 contraction elements): 8 rows are 1024 B apart; 16
// elements further along the contraction starts 32 B on.  MN-major (rows of
// 64 output elements, one per contraction element): 8 rows are 1024 B apart
// (stride offset), the next 64 output elements one box further (leading
// offset); 16 contraction elements further starts 2048 B on.
template <bool MN>
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr) {
  uint64_t d = sw128_desc(saddr);
  if (MN) d += (uint64_t)((BOX >> 4) - 1) << 16;
  return d;
}
template <bool MN>
constexpr uint32_t KSTEP = (MN ? 2048u : 32u) >> 4;  // descriptor step of 16 along the contraction

// The copies of n rows (output elements) from r0 at contraction k0: K-major
// one box of n x 64 (the map's), MN-major boxes of 64 x 64.
template <bool MN, bool PAIR>
__device__ __forceinline__ void load_tile(const CUtensorMap* tm, uint32_t bar, uint8_t* dst, int r0, int k0, int n) {
  for (int h = 0; h < (MN ? n : 1); h += 64) {
    const int c0 = MN ? r0 + h : k0, c1 = MN ? k0 : r0;
    if (PAIR)
      asm volatile(
          "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst) + (uint32_t)h * 128u),
          "l"((uint64_t)tm), "r"(bar), "r"(c0), "r"(c1)
          : "memory");
    else
      asm volatile(
          "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst) + (uint32_t)h * 128u),
          "l"((uint64_t)tm), "r"(bar), "r"(c0), "r"(c1)
          : "memory");
  }
}
// One lane of a converged warp.  The MMA loops run in the whole warp, with the
// issuing instructions alone in one lane, so that descriptors and counters stay
// in uniform registers (moving them there cost 65 cycles per MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Whether a phase is complete (asked one stage ahead, while MMAs are issued)
__device__ __forceinline__ bool mbar_done_cl(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// completion of the pair's MMAs issued so far, on the barrier at the same
// place in both CTAs
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// instruction descriptor: fp32 accumulator, A and B fp16 or bf16 (bits 7-9
// and 10-12), MN-major flags (bits 15 and 16), N / 8 and M / 16
template <typename T, bool A_MN, bool B_MN>
__host__ __device__ constexpr uint32_t lin_idesc(int M, int N) {
  const uint32_t f = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The contraction of a product: `steps` of BK in all.  An operand in two parts
// (dz of a smooth activation: what 16 bits hold, and what they leave) takes
// two steps per BK, first part first, so that the other operand's second copy
// comes from L2.
struct Contraction {
  int steps, two;
  __device__ __forceinline__ int at(int i) const { return (i >> two) * BK; }
  __device__ __forceinline__ bool second(int i) const { return (i & two) != 0; }
};

struct LinOut {
  const void* bias;      // n values in T or fp32, or NULL
  const void* residual;  // rows x n in the output's type, or NULL
  void* preact;          // rows x n in T, or NULL
  void* out;             // rows x n
  int64_t ldr, ldo;
  int rows, cols, act;
  bool bias_f32, bias_vec, res_vec, out_vec;
};

// The residual of W consecutive columns of a row (zeros without one).  Read
// for several runs before the first is stored: the compiler may not move loads
// over stores, and one at a time they cost a memory latency each.
template <int W, typename O>
__device__ __forceinline__ void lin_residual(const LinOut& o, int row, int col, float (&r)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = 0.0f;
  if (o.residual)
    load_edge<W>(static_cast<const O*>(o.residual) + (int64_t)row * o.ldr + col, r, o.cols - col, o.res_vec);
}
// One run of W consecutive columns of a row: bias, activation, residual, store.
template <int W, typename T, typename O>
__device__ __forceinline__ void lin_finish(const LinOut& o, int row, int col, float (&v)[W],
                                           const float (&bias)[W], const float (&r)[W]) {
  const int n = o.cols - col;  // >= 1
  const int64_t at = (int64_t)row * o.ldo + col;
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] += bias[i];
  if (o.preact) store_edge<W>(static_cast<T*>(o.preact) + at, v, n, o.out_vec);
  if (o.act != MPQ_ACT_NONE) act_apply<W>(v, o.act);
  if (o.residual) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += r[i];
  }
  store_edge<W>(static_cast<O*>(o.out) + at, v, n, o.out_vec);
}

// ----------------------------------------------------------- CTA-pair GEMM --
constexpr int PT = 256;                    // tile: 256 rows x 256 columns
constexpr int P_RING = 6 * 2 * 128 * BK * 2;  // 6 stages of 128 rows of A and 128 of B per CTA,
constexpr int P_STAGES = 8;                   // or 8 of 128 and 64 (128-column tiles only)
constexpr int P_EPI = 8;                   // epilogue warps
// Three warpgroups: copies and MMAs (a warp is idle), and two of epilogue warps,
// which take over registers for their part of a tile's sums, 128 a thread.
constexpr int P_THREADS = 32 * (4 + P_EPI);
// (Each role sets its own share in its own branch: where branches of different
// shares meet, the compiler keeps to the smaller one.)
constexpr int P_REGS = 168, P_REGS_ISSUE = 72, P_REGS_EPI = 216;
static_assert(P_THREADS * P_REGS <= 65536 && 128 * P_REGS_ISSUE + 256 * P_REGS_EPI <= P_THREADS * P_REGS,
              "a block moves the registers that it was launched with");
constexpr int P_SMEM = P_RING + P_EPI * 4096 + 1024 + 256;
static_assert(P_SMEM <= 232448, "pair kernel's shared memory");

// The walk over tiles: whole waves of 256 x 256 tiles; what is left for a last
// wave runs as two 128-column halves each where that fills no more workers
// than there are.
struct Walk {
  int mt, nt, whole, total;
};
__host__ __device__ inline Walk make_walk(int rows, int cols, int workers) {
  Walk w;
  w.mt = (rows + PT - 1) / PT;
  w.nt = (cols + PT - 1) / PT;
  const int t = w.mt * w.nt, left = t % workers;
  w.whole = 2 * left <= workers ? t - left : t;
  w.total = w.whole + 2 * (t - w.whole);
  return w;
}
// Tiles run in groups of 8 row tiles (rows fastest), so that the panels of
// both operands in flight stay in L2.
__device__ __forceinline__ void walk_tile(const Walk& w, int t, int& m0, int& n0, int& wn) {
  int s = t, half = 0;
  wn = PT;
  if (t >= w.whole) {
    s = w.whole + (t - w.whole) / 2;
    half = (t - w.whole) & 1;
    wn = PT / 2;
  }
  const int per = 8 * w.nt, g = s / per, q = s % per;
  const int gm = min(8, w.mt - g * 8);
  m0 = (g * 8 + q % gm) * PT;
  n0 = (q / gm) * PT + half * (PT / 2);
}

// The issuing threads set the pace next to the MMAs (512 cycles per stage of a
// 256-column tile): with one thread for both operands' copies, two commits a
// stage and descriptors built per MMA they took 450 and 540 cycles a stage, and
// 600 with the waits.  So A and B have a copying warp each, a copy is as large
// as a box may be, a commit reaches both CTAs, and descriptors are added up.
template <typename T, typename O, bool A_MN, bool B_MN, bool FEAT>
__global__ void __launch_bounds__(P_THREADS, 1)
    k_lin_pair(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap ta_second,
               const __grid_constant__ CUtensorMap tb, const __grid_constant__ CUtensorMap tb_half,
               const __grid_constant__ Contraction kc, const __grid_constant__ LinOut o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* stg_all = smem + P_RING;
  uint64_t* full = (uint64_t*)(stg_all + P_EPI * 4096);
  uint64_t* empty = full + P_STAGES;
  uint64_t* tm_full = empty + P_STAGES;
  uint64_t* tm_empty = tm_full + 2;
  uint32_t* tmem_slot = (uint32_t*)(tm_empty + 2);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // rank 0 issues the pair's MMAs
  const int worker = (int)cluster_id_x(), nworkers = (int)(gridDim.x / 2);
  constexpr int CHAIN = chain_steps<O>();
  const Walk walk = make_walk(o.rows, o.cols, nworkers);
  const int KT = kc.steps;
  const int stages = walk.whole ? 6 : 8, stage = walk.whole ? P_RING / 6 : P_RING / 8;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tm_full[b], 1);
      mbar_init(&tm_empty[b], 2 * P_EPI);  // the epilogue warps of both CTAs
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ta) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tb) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tb_half) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(2 * PT));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full_r0 = map_to_rank(smem_u32(full), 0);
  const uint32_t tm_empty_r0 = map_to_rank(smem_u32(tm_empty), 0);

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P_REGS_ISSUE));
  if ((warp == 0 || warp == 2) && lane == 0) {
    // ------------------------------------------------- producers: A and B
    const bool is_a = warp == 0;
    uint8_t* dst0 = smem + (is_a ? 0 : 128 * BK * 2);
    uint32_t it = 0;
    int s = 0;
    uint32_t phase = 1;  // of `empty`: the first turn over the ring passes at once
    bool ok = true;
    for (int t = worker; t < walk.total && ok; t += nworkers) {
      int m0, n0, wn;
      walk_tile(walk, t, m0, n0, wn);
      const int r0 = is_a ? m0 + (int)rank * 128 : n0 + (int)rank * (wn / 2);
      const uint32_t bytes = (uint32_t)((128 + wn / 2) * BK * 2);
      const CUtensorMap* tm = wn == PT ? &tb : &tb_half;
      for (int i = 0; i < KT; ++i, ++it) {
        const int k0 = kc.at(i);
        if (!mbar_wait(&empty[s], phase)) {
          report_timeout();
          ok = false;
          break;
        }
        const uint32_t fb = full_r0 + 8u * (uint32_t)s;  // rank 0's barrier counts both CTAs' bytes
        uint8_t* dst = dst0 + s * stage;
        if (is_a) {
          if (rank == 0) mbar_expect_tx(&full[s], 2 * bytes);
          load_tile<A_MN, true>(kc.second(i) ? &ta_second : &ta, fb, dst, r0, k0, 128);
        } else {
          load_tile<B_MN, true>(tm, fb, dst, r0, k0, wn / 2);
        }
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // every copy lands before the CTA leaves (rank 0's barriers count both
    // CTAs' copies; rank 1 waits for rank 0 at the closing cluster barrier)
    if (rank == 0)
      for (uint32_t q = (it > (uint32_t)stages ? it - stages : 0); q < it; ++q)
        for (uint32_t i = 0; i < (1u << 25) && !mbar_try_wait(&full[q % stages], (q / stages) & 1); ++i)
          if (i > 256) __nanosleep(64);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t ID_W = lin_idesc<T, A_MN, B_MN>(256, PT), ID_N = lin_idesc<T, A_MN, B_MN>(256, PT / 2);
    const uint64_t da0 = op_desc<A_MN>(smem_u32(smem)), db0 = op_desc<B_MN>(smem_u32(smem) + 128 * BK * 2);
    uint32_t tl = 0;  // accumulators filled
    int s = 0;
    uint32_t phase = 0;
    bool ok = true, ready = false;
    for (int t = worker; t < walk.total; t += nworkers) {
      const uint32_t idesc = t < walk.whole ? ID_W : ID_N;
      for (int k0 = 0; k0 < KT; k0 += CHAIN, ++tl) {  // a chain into an accumulator
        const int buf = tl & 1, n = min(CHAIN, KT - k0);
        // elect.sync needs every lane, so a wait that runs out ends no loop: its
        // lane waits no more, and the result is reported as undefined
        if (ok && tl >= 2) ok = mbar_wait_cl(&tm_empty[buf], (tl / 2 - 1) & 1);
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * PT;
        for (int kt = 0; kt < n; ++kt) {
          if (ok && !ready) ok = mbar_wait_cl(&full[s], phase);
          tc_fence_after();
          const uint64_t da = da0 + (uint32_t)s * (uint32_t)(stage >> 4), db = db0 + (uint32_t)s * (uint32_t)(stage >> 4);
          uint64_t* freed = &empty[s];
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
          ready = mbar_done_cl(&full[s], phase);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_f16_cg2(d, da + kk * KSTEP<A_MN>, db + kk * KSTEP<B_MN>, idesc, (kt | kk) != 0 ? 1u : 0u);
            commit_both(freed);
            if (kt == n - 1) commit_both(&tm_full[buf]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) report_timeout();
    for (uint32_t q = (tl > 2 ? tl - 2 : 0); q < tl; ++q)  // MMAs finish before TMEM is freed
      for (uint32_t i = 0; i < (1u << 25) && !mbar_try_wait(&tm_full[q & 1], (q / 2) & 1); ++i)
        if (i > 256) __nanosleep(64);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P_REGS_EPI));
    // -------------------------------------------------------------- epilogue
    // two warps per TMEM lane quadrant, alternating over 32-column chunks: up to
    // four each, whose chains are added up here.  Then a chunk goes through a
    // swizzled 32 x 32 fp32 staging tile, which turns the lane-per-row layout
    // into 8 consecutive columns per lane.
    const int q = warp & 3, side = (warp - 4) >> 2;
    float4* stg = reinterpret_cast<float4*>(stg_all + (warp - 4) * 4096);
    const int c8 = (lane & 3) * 8, r8 = lane >> 2;
    const bool wide = o.out_vec && (!o.residual || o.res_vec);
    uint32_t tl = 0;
    for (int t = worker; t < walk.total; t += nworkers) {
      int m0, n0, wn;
      walk_tile(walk, t, m0, n0, wn);
      const int row0 = m0 + (int)rank * 128 + q * 32;
      if (FEAT && o.residual && row0 + lane < o.rows) {  // this warp's residual comes to L2 during the MMAs
        const O* rl = static_cast<const O*>(o.residual) + (int64_t)(row0 + lane) * o.ldr;
        for (int c = n0 + side * 32; c < min(n0 + wn, o.cols); c += 64) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rl + c));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rl + min(c + 31, o.cols - 1)));
        }
      }
      // Chains of this warp's two or four chunks: all of them for fp32 results,
      // those before the last for 16-bit ones, which are often a single one.
      constexpr bool ALL = sizeof(O) == 4;
      float sum[4][32];
      const auto add = [&](int c, uint32_t at) {
        uint32_t a[32];
        tmem_ld32(at + 64u * (uint32_t)c, a);
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[c][i] += __uint_as_float(a[i]);
      };
      const bool chains = ALL || KT > CHAIN;
      bool ok = true;
      if (chains) {
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[0][i] = sum[1][i] = 0.0f;
        if (wn == PT) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[2][i] = sum[3][i] = 0.0f;
        }
        for (int k = ALL ? 0 : CHAIN; k < KT && ok; k += CHAIN, ++tl) {
          const int buf = tl & 1;
          ok = __all_sync(0xffffffffu, mbar_wait_cl(&tm_full[buf], (tl / 2) & 1));
          tc_fence_after();
          const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * PT + side * 32);
          add(0, tb);
          add(1, tb);
          if (wn == PT) {
            add(2, tb);
            add(3, tb);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cl(tm_empty_r0 + 8u * (uint32_t)buf);  // read: hand the accumulator back
        }
      }
      const int buf = tl & 1;  // (not ALL: the last chain's)
      if constexpr (!ALL) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_cl(&tm_full[buf], (tl / 2) & 1));
        tc_fence_after();
        ++tl;
      }
      if (!ok) {
        if (lane == 0) report_timeout();
        break;
      }
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)buf * PT;
#pragma unroll 1
      for (int c0 = side * 32; c0 < wn; c0 += 64) {
        const int left = o.cols - (n0 + c0), top = o.rows - row0;  // columns and rows from this chunk on
        const bool inside = wide && left >= 32 && top >= 32;
        // bias and residual in the layout of the stores, in flight while the
        // accumulator is read
        float bias[8] = {};
        Raw8<O> res[4] = {};
        const bool has_res = FEAT && o.residual;
        const O* rp = static_cast<const O*>(o.residual) + (int64_t)row0 * o.ldr + n0 + c0;
        if (inside) {
          if (o.bias) load_param<8, T>(o.bias, o.bias_f32, n0 + c0 + c8, bias, 8, o.bias_vec);
          if (has_res) {
#pragma unroll
            for (int i = 0; i < 4; ++i) res[i] = load_raw<O>(rp + (int64_t)(i * 8 + r8) * o.ldr + c8, 8, true);
          }
        }
        uint32_t v[32];
        if constexpr (!ALL) {
          tmem_ld32(tbase + (uint32_t)c0, v);
          if (c0 + 64 >= wn) {  // this warp's part is read: hand the accumulator back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cl(tm_empty_r0 + 8u * (uint32_t)buf);
          }
        }
        // (the loop is not unrolled: selects)
        const auto take = [&](const float (&even)[32], const float (&odd)[32]) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float w = c0 & 64 ? odd[i] : even[i];
            v[i] = __float_as_uint(ALL ? w : __uint_as_float(v[i]) + w);
          }
        };
        if (chains && c0 < 128) take(sum[0], sum[1]);
        else if (chains) take(sum[2], sum[3]);
        if (left <= 0 || top <= 0) continue;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          stg[lane * 8 + (k ^ (lane & 7))] =
              make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                          __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
        __syncwarp();
        // rolled loops: a tile's epilogue runs its code once or a few times,
        // and its length is paid in instruction fetches
        if (inside) {
          const int64_t at0 = (int64_t)(row0 + r8) * o.ldo + n0 + c0 + c8;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int rr = i * 8 + r8;
            const float4 x0 = stg[rr * 8 + ((c8 / 4) ^ (rr & 7))];
            const float4 x1 = stg[rr * 8 + ((c8 / 4 + 1) ^ (rr & 7))];
            float w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] += bias[j];
            const int64_t at = at0 + (int64_t)(i * 8) * o.ldo;
            if (FEAT) {
              if (o.preact) store_vec<8>(static_cast<T*>(o.preact) + at, w, true);
              if (o.act != MPQ_ACT_NONE) act_apply<8>(w, o.act);
              if (has_res) {
                float r[8];
                decode<O>(i == 0 ? res[0] : i == 1 ? res[1] : i == 2 ? res[2] : res[3], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] += r[j];
              }
            }
            store_vec<8>(static_cast<O*>(o.out) + at, w, true);
          }
        } else if (lane < left) {
          // edges and unaligned rows: a column a lane, 8 rows at a time, the
          // residual of the next 8 in flight
          const int64_t at0 = (int64_t)row0 * o.ldo + n0 + c0 + lane;
          float b1[1] = {}, r0[8] = {}, r1[8] = {};
          if (o.bias) load_param<1, T>(o.bias, o.bias_f32, n0 + c0 + lane, b1, 1, false);
          if (has_res) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < top) r0[i] = to_f(rp[(int64_t)i * o.ldr + lane]);
          }
#pragma unroll 1
          for (int q = 0; q < min(32, top); q += 8) {
            if (has_res) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (q < 24 && q + 8 + i < top) r1[i] = to_f(rp[(int64_t)(q + 8 + i) * o.ldr + lane]);
            }
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              w[i] = reinterpret_cast<const float*>(stg + (q + i) * 8 + ((lane >> 2) ^ i))[lane & 3] + b1[0];
              if (FEAT && o.preact && q + i < top) static_cast<T*>(o.preact)[at0 + (int64_t)(q + i) * o.ldo] = from_f<T>(w[i]);
            }
            if (FEAT && o.act != MPQ_ACT_NONE) act_apply<8>(w, o.act);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (q + i < top) static_cast<O*>(o.out)[at0 + (int64_t)(q + i) * o.ldo] = from_f<O>(w[i] + r0[i]);
              r0[i] = r1[i];
            }
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no peer still reads this CTA's memory or barriers
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * PT));
  }
}

// -------------------------------------------------------------- split GEMM --
// Roles are swapped: the operand with the output's columns (W, or x for dW)
// fills the 128 TMEM lanes, the one with its rows (the tokens) the NT columns
// of the accumulator, so few rows waste no tensor work.
constexpr int S_THREADS = 320;  // copies, MMAs, 8 epilogue warps
constexpr int S_NARROW = 32;    // rows of a tile of which two CTAs fit on an SM

struct SplitGeom {
  int NT;      // rows of the output per tile (accumulator columns)
  int stages;
  int S;       // CTAs per cluster, each with its share of the contraction
  int KT;      // contraction steps in all
  uint32_t tmem_cols;
  bool chains;
};
__host__ __device__ inline int split_stage_bytes(int NT) { return 128 * BK * 2 + NT * BK * 2; }
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Elements of a partial tile (row-major, 128 columns) that each of S CTAs
// joins: whole runs of 32.
__host__ __device__ inline int split_share(int rows, int S) { return ((rows * 128 + S - 1) / S + 31) / 32 * 32; }
// Shared memory behind the ring for the partial tiles of S > 1 CTAs
__host__ __device__ inline int split_recv_bytes(int NT, int S) { return S > 1 ? S * split_share(NT, S) * 4 : 0; }

// CHAINS: the chains of a CTA's contraction are added up in registers, NC blocks
// of 16 rows a warp (one for tiles of up to S_NARROW rows); else it is one chain.
template <typename T, typename O, bool A_MN, bool B_MN, bool CHAINS, int NC>
__global__ void __launch_bounds__(S_THREADS, NC == 1 || !CHAINS ? 2 : 1)
    k_lin_split(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const __grid_constant__ CUtensorMap tb_second, const __grid_constant__ Contraction kc,
                const __grid_constant__ SplitGeom g, const __grid_constant__ LinOut o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int stage = split_stage_bytes(g.NT);
  float* recv = (float*)(smem + g.stages * stage);
  uint64_t* full = (uint64_t*)(smem + g.stages * stage + split_recv_bytes(g.NT, g.S));
  uint64_t* empty = full + g.stages;
  uint64_t* done = empty + g.stages;
  uint64_t* arrived = done + 1;  // S > 1: every CTA's part of this CTA's share is in recv
  uint64_t* ch_full = arrived + 1;  // chains (fp32 results): two accumulators in turn
  uint64_t* ch_empty = ch_full + 2;
  uint32_t* tmem_slot = (uint32_t*)(ch_empty + 2);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = g.S > 1 ? (int)cluster_ctarank() : 0;
  const int a0 = blockIdx.y * 128, b0 = blockIdx.z * g.NT;
  const int k_lo = (int)((int64_t)g.KT * rank / g.S), k_hi = (int)((int64_t)g.KT * (rank + 1) / g.S);
  const int nk = k_hi - k_lo;  // >= 1
  const int nrow = min(g.NT, o.rows - b0), share = split_share(nrow, g.S);
  const int e_lo = rank * share, e_hi = min(nrow * 128, e_lo + share);  // what this CTA joins

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(arrived, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ch_full[b], 1);
      mbar_init(&ch_empty[b], 8);  // the epilogue warps
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (g.S > 1) mbar_expect_tx(arrived, (uint32_t)(g.S * max(e_hi - e_lo, 0) * 4));
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ta) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tb) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(g.tmem_cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (g.S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  if (warp == 0 && lane == 0) {
    int i = 0, s = 0;
    uint32_t phase = 1;
    for (; i < nk; ++i) {
      if (!mbar_wait(&empty[s], phase)) {
        report_timeout();
        break;
      }
      uint8_t* a = smem + s * stage;
      const int k0 = kc.at(k_lo + i);
      const uint32_t fb = smem_u32(&full[s]);
      mbar_expect_tx(&full[s], (uint32_t)stage);
      load_tile<A_MN, false>(&ta, fb, a, a0, k0, 128);
      load_tile<B_MN, false>(kc.second(k_lo + i) ? &tb_second : &tb, fb, a + 128 * BK * 2, b0, k0, g.NT);
      if (++s == g.stages) {
        s = 0;
        phase ^= 1;
      }
    }
    for (int q = (i > g.stages ? i - g.stages : 0); q < i; ++q)  // every copy lands
      for (uint32_t w = 0; w < (1u << 25) && !mbar_try_wait(&full[q % g.stages], (q / g.stages) & 1); ++w)
        if (w > 256) __nanosleep(64);
  } else if (warp == 1) {
    const uint32_t idesc = lin_idesc<T, A_MN, B_MN>(128, g.NT);
    const uint64_t da0 = op_desc<A_MN>(smem_u32(smem)), db0 = op_desc<B_MN>(smem_u32(smem) + 128 * BK * 2);
    const int CH = CHAINS ? chain_steps<O>() : nk;
    int s = 0;
    uint32_t phase = 0, tl = 0;
    bool ok = true, ready = false;
    for (int i0 = 0; i0 < nk; i0 += CH, ++tl) {
      const int buf = CHAINS ? (int)(tl & 1) : 0, n = min(CH, nk - i0);
      // (as in the pair kernel, a wait that runs out ends no loop)
      if (CHAINS) {
        if (ok && tl >= 2) ok = mbar_wait(&ch_empty[buf], (tl / 2 - 1) & 1);
        tc_fence_after();
      }
      const uint32_t d = tmem + (uint32_t)buf * (g.tmem_cols / 2);
      for (int i = 0; i < n; ++i) {
        if (ok && !ready) ok = mbar_wait(&full[s], phase);
        tc_fence_after();
        const uint64_t da = da0 + (uint32_t)s * (uint32_t)(stage >> 4), db = db0 + (uint32_t)s * (uint32_t)(stage >> 4);
        uint64_t* freed = &empty[s];
        if (++s == g.stages) {
          s = 0;
          phase ^= 1;
        }
        ready = mbar_test_wait(&full[s], phase);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma_f16(d, da + kk * KSTEP<A_MN>, db + kk * KSTEP<B_MN>, idesc, (i | kk) != 0 ? 1u : 0u);
          umma_commit(freed);
          if (CHAINS && i == n - 1) umma_commit(&ch_full[buf]);
        }
        __syncwarp();
      }
    }
    if (!ok) report_timeout();
    __syncwarp();
    if (elect_one()) umma_commit(done);
    __syncwarp();
    for (uint32_t w = 0; w < (1u << 25) && !mbar_try_wait(done, 0); ++w)
      if (w > 256) __nanosleep(64);
  }
  // chains: this warp's rows of the tile, 16 at a time from (warp - 2) / 4 * 16
  float sums[CHAINS ? NC : 1][16];
  if (warp >= 2) {
    if constexpr (CHAINS) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[c][j] = 0.0f;
      uint32_t tl = 0;
      bool ok = true;
      for (int i = 0; i < nk && ok; i += chain_steps<O>(), ++tl) {
        const int buf = tl & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&ch_full[buf], (tl / 2) & 1));
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int c0 = ((warp - 2) >> 2) * 16 + c * 32;
          if (c0 >= nrow) break;
          uint32_t v[16];
          tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)buf * (g.tmem_cols / 2) + (uint32_t)c0, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sums[c][j] += __uint_as_float(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ch_empty[buf]);
      }
      if (!ok && lane == 0) report_timeout();
    }
    if (!__all_sync(0xffffffffu, mbar_wait(done, 0)) && lane == 0) report_timeout();
  }
  // All copies have landed and all MMAs have read them: the ring becomes the
  // partial tile part[row][128 columns].  Lane l of quadrant q holds column
  // 32 q + l of the output, one row per accumulator column.
  __syncthreads();
  tc_fence_after();
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int q = warp & 3;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int c0 = ((warp - 2) >> 2) * 16 + c * 32;
      if (c0 >= nrow) break;
      uint32_t v[16];
      if constexpr (CHAINS) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(sums[c][j]);
      } else {
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
      }
      float* p = part + c0 * 128 + q * 32 + lane;  // (rows up to NT fit)
#pragma unroll
      for (int j = 0; j < 16; ++j) p[j * 128] = __uint_as_float(v[j]);
    }
  }
  const float* from = part;
  if (g.S > 1) {
    // every CTA sends every other (and itself) its share of the partial tile,
    // by bulk copies between the CTAs' shared memories
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all CTAs have begun
    if (threadIdx.x == 0) {
      for (int p = 0; p < g.S; ++p) {
        const int lo = p * share, n = min(nrow * 128, lo + share) - lo;
        if (n <= 0) break;
        asm volatile(
            "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                map_to_rank(smem_u32(recv + rank * share), (uint32_t)p)),
            "r"(smem_u32(part + lo)), "r"((uint32_t)(n * 4)), "r"(map_to_rank(smem_u32(arrived), (uint32_t)p))
            : "memory");
      }
    }
    __syncwarp();
    if (!mbar_wait_cl(arrived, 0) && threadIdx.x == 0) report_timeout();
    __syncwarp();
    // (what this CTA receives has arrived; when all say so, all copies are done)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    from = recv;
  } else {
    __syncthreads();
  }
  {
    // each CTA joins its share of the tile, in rank order, two runs a turn
    // (their loads are in flight together)
    const auto join = [&](auto width) {
      constexpr int W = decltype(width)::value, R = W == 1 ? 8 : 2;
      for (int e0 = e_lo + (int)threadIdx.x * W; e0 < e_hi; e0 += R * S_THREADS * W) {
        float res[R][W], bias[R][W], v[R][W];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int e = e0 + i * S_THREADS * W, r = e >> 7, c = a0 + (e & 127);
          if (e >= e_hi || c >= o.cols) continue;
          lin_residual<W, O>(o, b0 + r, c, res[i]);
#pragma unroll
          for (int j = 0; j < W; ++j) bias[i][j] = v[i][j] = 0.0f;
          if (o.bias) load_param<W, T>(o.bias, o.bias_f32, c, bias[i], o.cols - c, o.bias_vec);
          for (int p = 0; p < g.S; ++p) {
            const float* x = from + p * share + (e - e_lo);
            if constexpr (W == 8) {
              const float4 q = reinterpret_cast<const float4*>(x)[0], u = reinterpret_cast<const float4*>(x)[1];
              v[i][0] += q.x; v[i][1] += q.y; v[i][2] += q.z; v[i][3] += q.w;
              v[i][4] += u.x; v[i][5] += u.y; v[i][6] += u.z; v[i][7] += u.w;
            } else {
              v[i][0] += *x;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int e = e0 + i * S_THREADS * W, r = e >> 7, c = a0 + (e & 127);
          if (e >= e_hi || c >= o.cols) continue;
          lin_finish<W, T, O>(o, b0 + r, c, v[i], bias[i], res[i]);
        }
      }
    };
    if (o.out_vec && (!o.residual || o.res_vec)) join(std::integral_constant<int, 8>{});
    else join(std::integral_constant<int, 1>{});  // unaligned rows: neighbouring threads, neighbouring columns
  }
  __syncwarp();
  if (g.S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no copy still reads this CTA's tile
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_cols));
  }
}

// ------------------------------------------------------------- few rows --
// y = x W^T for one or two rows of x, bound by the read of W: WPR warps share a
// row of W, 16 bytes a lane and load, four loads in flight; the sums meet by
// shuffles and, for WPR > 1, in shared memory.  x comes from L1.
constexpr int GEMV_ROWS = 2, GEMV_WARPS = 8;
template <typename T, typename O, int MR, bool VEC>
__global__ void __launch_bounds__(GEMV_WARPS * 32, 4)
    k_lin_gemv(const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, int64_t ldw, int K, int wpr,
               const __grid_constant__ LinOut o) {
  __shared__ float sums[GEMV_WARPS][MR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = GEMV_WARPS / wpr;  // outputs per block
  const int n0 = blockIdx.x * per, col = n0 + warp / wpr;
  uint64_t acc[MR][2];
#pragma unroll
  for (int m = 0; m < MR; ++m) acc[m][0] = acc[m][1] = 0ull;
  const auto add = [&](const Raw8<T>& wv, int k) {
    float a[8];
    decode<T>(wv, a);
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      float b[8];
      if (VEC) decode<T>(load_raw<T>(x + m * ldx + k, K - k, true), b);
      else decode<T>(load_row8<T>(x + m * ldx, k, K), b);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[m][i & 1] = f2_fma(f2_pack(a[2 * i], a[2 * i + 1]), f2_pack(b[2 * i], b[2 * i + 1]), acc[m][i & 1]);
    }
  };
  if (col < o.cols) {
    const T* wr = w + (int64_t)col * ldw;
    constexpr int U = 4;
    const int step = wpr * 256;
    int k = (warp % wpr) * 256 + lane * 8;
    if (VEC) {
      for (; k + (U - 1) * step + 8 <= K; k += U * step) {
        Raw8<T> wv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) wv[u].q[0] = __ldcs(reinterpret_cast<const uint4*>(wr + k + u * step));
#pragma unroll
        for (int u = 0; u < U; ++u) add(wv[u], k + u * step);
      }
    }
    for (; k < K; k += step) add(load_row8<T>(wr, k, K), k);
  }
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float a, b;
    f2_unpack(f2_add(acc[m][0], acc[m][1]), a, b);
    float s = a + b;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    if (lane == 0) sums[warp][m] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < per * MR; i += GEMV_WARPS * 32) {
    const int m = i / per, c = i % per;
    if (n0 + c >= o.cols) continue;
    float v[1] = {0.0f}, bias[1] = {};
    for (int q = 0; q < wpr; ++q) v[0] += sums[c * wpr + q][m];
    if (o.bias) bias[0] = o.bias_f32 ? static_cast<const float*>(o.bias)[n0 + c] : to_f(static_cast<const T*>(o.bias)[n0 + c]);
    float res[1];
    lin_residual<1, O>(o, m, n0 + c, res);
    lin_finish<1, T, O>(o, m, n0 + c, v, bias, res);
  }
}

// -------------------------------------------------- rows and pre-activation --
// Copies rows x cols 16-bit elements of up to two operands to leading
// dimensions that TMA can take (multiples of 8).  Only for operands whose base
// or row stride is not a multiple of 16 bytes.
struct PackJob {
  const __half* src;  // 16-bit elements, copied as they are
  __half* dst;
  int64_t ld, rows, cols, ldd;
};
__global__ void __launch_bounds__(256)
    k_lin_pack(const __grid_constant__ PackJob a, const __grid_constant__ PackJob b) {
  const int64_t na = a.rows * (a.ldd / 8), nb = b.rows * (b.ldd / 8);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < na + nb; i += (int64_t)gridDim.x * 256) {
    const PackJob& j = i < na ? a : b;
    const int64_t at = i < na ? i : i - na, groups = j.ldd / 8;
    const int64_t r = at / groups;
    const int c = (int)(at % groups) * 8;
    const Raw8<__half> v = load_row8<__half>(j.src + r * j.ld, c, (int)j.cols);
    *reinterpret_cast<uint4*>(j.dst + r * j.ldd + c) = v.q[0];
  }
}

// x as two values of 16 bits, for the tensor cores: x rounded, and what that
// leaves, rounded.  Together within 2^-16 of x in bf16 and 2^-22 in fp16 (and
// 2^-25 absolute).  What a first part of 16 bits cannot hold, the second does
// (fp16: up to 131008).
template <typename T>
__device__ __forceinline__ void two_parts(float x, float& first, float& second) {
  constexpr float top = std::is_same<T, __half>::value ? 65504.0f : 3.3895313892515355e38f;
  first = to_f(from_f<T>(x));
  if (isinf(first) && !isinf(x)) first = copysignf(top, x);
  second = isfinite(first) ? x - first : 0.0f;
}
// dz = dy * act'(z) as the tensor cores take it, and per block of 64 rows the
// column sums of its fp32 values.  The slopes of relu are 0 and 1, so its dz has
// dy's type as it is; that of the smooth activations comes in two parts
// (dz_second), or rounded to one (half a step of the type per element) where the
// caller asked for that.
constexpr int DZ_ROWS = 64;
template <typename T>
__global__ void __launch_bounds__(256, 3)
    k_lin_dz(const T* __restrict__ dy, int64_t ldy, const T* __restrict__ z, int64_t ldz, int act,
             int64_t rows, int64_t n, T* __restrict__ dz, T* __restrict__ dz_second, int64_t ldd,
             float* __restrict__ part, bool vec_y, bool vec_z) {
  __shared__ float red[8][256 + 8];
  const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.y * 256 + cg * 8;
  const int64_t r_lo = (int64_t)blockIdx.x * DZ_ROWS, r_hi = min(rows, r_lo + DZ_ROWS);
  F8 sum = {};
  if (c < n) {
    const int left = (int)min((int64_t)8, n - c);
    constexpr int NR = 2;  // rows in flight
    for (int64_t r0 = r_lo + rl; r0 < r_hi; r0 += 8 * NR) {
      Raw8<T> gy[NR], zz[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int64_t r = r0 + 8 * q;
        const int have = r < r_hi ? left : 0;
        gy[q] = load_raw<T>(dy + (r < r_hi ? r : r0) * ldy + c, have, vec_y);
        if (act != MPQ_ACT_NONE) zz[q] = load_raw<T>(z + (r < r_hi ? r : r0) * ldz + c, have, vec_z);
      }
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int64_t r = r0 + 8 * q;
        if (r >= r_hi) break;
        F8 g = pairs<T>(gy[q]);
        if (act != MPQ_ACT_NONE) act_grad8(g, pairs<T>(zz[q]), act);
        if (dz) {  // ldd is a multiple of 8: the pad is zero
          float v[8];
          unpairs(g, v);
          if (dz_second) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) two_parts<T>(v[j], v[j], w[j]);
            store_vec<8>(dz_second + r * ldd + c, w, true);
          }
          store_vec<8>(dz + r * ldd + c, v, true);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum.p[j] = f2_add(sum.p[j], g.p[j]);
      }
    }
  }
  if (!part) return;
  float total[8];
  unpairs(sum, total);
#pragma unroll
  for (int j = 0; j < 8; ++j) red[rl][cg * 8 + j] = total[j];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (col < n) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    part[(int64_t)blockIdx.x * n + col] = s;
  }
}

// Column sums of `blocks` partial rows, in a fixed order.
template <typename O>
__global__ void __launch_bounds__(256)
    k_lin_colsum(const float* __restrict__ part, int64_t blocks, int64_t n, O* __restrict__ out) {
  __shared__ float red[8][32];
  const int cl = threadIdx.x & 31, bl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.0f;
  if (c < n)
    for (int64_t b = bl; b < blocks; b += 8) s += part[b * n + c];
  red[bl][cl] = s;
  __syncthreads();
  if (bl == 0 && c < n) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][cl];
    out[c] = from_f<O>(t);
  }
}

// A wait that nothing ends, over at once: 64 tests of a barrier with no arrivals.
__global__ void k_expire() {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) mbar_init(&bar, 1);
  __syncthreads();
  bool done = false;
  for (uint32_t i = 0; i < WAIT_SPIN && !done; ++i) done = mbar_test_wait(&bar, 0);
  if (!done && threadIdx.x == 0) report_timeout();
}

// -------------------------------------------------------------------- host --
PFN_cuTensorMapEncodeTiled_v12000 g_lin_encode = nullptr;
std::mutex g_lin_mu;
struct LinDevice {
  bool ready = false;
  int pairs = 0;
};
LinDevice g_lin_dev[64];

mpq_status encode_box(CUtensorMap* tm, const void* base, int64_t inner, int64_t rows, int64_t ld,
                      bool bf16, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = g_lin_encode(
      tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
      const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MPQ_ERR_CUDA, "linear: cuTensorMapEncodeTiled failed with code " + std::to_string((int)r));
  return MPQ_OK;
}

// An operand in memory: `rows` rows of `inner` contiguous elements; `second`:
// its second part, laid out alike, or NULL.
struct Operand {
  const void* p;
  int64_t inner, rows, ld;
  const void* second = nullptr;
};
bool tma_ok(const void* p, int64_t inner, int64_t rows, int64_t ld) {
  return ((uintptr_t)p & 15) == 0 && (rows <= 1 || (ld % 8 == 0 && ld >= inner));
}
int64_t packed_bytes(int64_t inner, int64_t rows) {
  return round_up(rows * round_up(inner, 8) * 2, 256);
}
// A row stride for TMA where there is one row (its stride is not read).
int64_t tma_ld(const Operand& a) { return a.rows <= 1 ? round_up(a.inner, 8) : a.ld; }

// Packs those of two operands that have somewhere to go.
mpq_status pack(Operand* a, void* dst_a, Operand* b, void* dst_b, cudaStream_t st) {
  int dev = 0, sms = 0;
  const auto job = [](Operand* q, void* dst) {
    PackJob j{};
    if (!dst) return j;
    j = PackJob{static_cast<const __half*>(q->p), static_cast<__half*>(dst), q->ld, q->rows, q->inner, round_up(q->inner, 8)};
    q->p = dst;
    q->ld = j.ldd;
    return j;
  };
  const PackJob ja = job(a, dst_a), jb = job(b, dst_b);
  const int64_t work = (ja.rows * ja.ldd + jb.rows * jb.ldd) / 8;
  if (work == 0) return MPQ_OK;
  MPQ_TRY(current_device(&dev, &sms));
  {
    ProfScope ps_("k_lin_pack", st);
    k_lin_pack<<<(unsigned)std::min<int64_t>(cdiv(work, 256), sms * 16), 256, 0, st>>>(ja, jb);
  }
  count_launch();
  return check_launch("k_lin_pack");
}

// The split kernel of a product: chains where a CTA's part of the contraction is
// longer than one (always for fp32 results, whose chains are short).
template <typename T, typename O, bool RN, bool CN>
auto split_kernel(bool chains, int NT) {
  auto k = k_lin_split<T, O, CN, RN, true, 4>;
  if constexpr (!RN)
    if (chains && NT <= S_NARROW) return k_lin_split<T, O, CN, RN, true, 1>;
  if constexpr (sizeof(O) == 2)
    if (!chains) return k_lin_split<T, O, CN, RN, false, 4>;
  return k;
}

// Its epilogue warps wait for the registers that the issuing warps give up: a
// build that launched the block with fewer than it moves would wait for good.
template <typename K>
mpq_status pair_attrs(K kernel) {
  cudaFuncAttributes a{};
  MPQ_CUDA(cudaFuncGetAttributes(&a, kernel));
  if (a.numRegs != P_REGS)
    return fail(MPQ_ERR_CUDA, "linear: the pair kernel was built with " + std::to_string(a.numRegs) + " registers");
  MPQ_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM));
  return MPQ_OK;
}
template <typename T, typename O, bool RN, bool CN>
mpq_status set_attrs() {
  MPQ_TRY(pair_attrs(k_lin_pair<T, O, RN, CN, false>));
  if constexpr (!RN && !CN) MPQ_TRY(pair_attrs(k_lin_pair<T, O, RN, CN, true>));
  for (const bool chains : {false, true})
    for (const int NT : {S_NARROW, 128})
      MPQ_CUDA(cudaFuncSetAttribute(split_kernel<T, O, RN, CN>(chains, NT), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    220 * 1024));
  return MPQ_OK;
}

mpq_status lin_device(int* dev_out, int* sms_out) {
  int dev = 0;
  MPQ_TRY(current_device(&dev, sms_out));
  std::lock_guard<std::mutex> lk(g_lin_mu);
  if (!g_lin_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
      return fail(MPQ_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    g_lin_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  if (!g_lin_dev[dev].ready) {
    using B = __nv_bfloat16;
    using H = __half;
    MPQ_TRY((set_attrs<B, B, false, false>()));
    MPQ_TRY((set_attrs<B, float, false, false>()));
    MPQ_TRY((set_attrs<B, B, false, true>()));
    MPQ_TRY((set_attrs<B, B, true, true>()));
    MPQ_TRY((set_attrs<H, H, false, false>()));
    MPQ_TRY((set_attrs<H, float, false, false>()));
    MPQ_TRY((set_attrs<H, H, false, true>()));
    MPQ_TRY((set_attrs<H, H, true, true>()));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)*sms_out);
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = P_SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int nc = 0;
    if (cudaOccupancyMaxActiveClusters(&nc, k_lin_pair<B, B, false, false, true>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      nc = 0;
    }
    g_lin_dev[dev].pairs = nc;
    g_lin_dev[dev].ready = true;
  }
  *dev_out = dev;
  return MPQ_OK;
}

// Geometry of the split kernel.  Tiles of up to 32 rows leave room for two
// CTAs on an SM; the contraction is split while that finds free SMs and each
// CTA keeps 2 steps.  Clusters of 8 only where they leave half of the SMs
// free: 16 of them (256 x 1024 over 2048) find no place at once and take 18.7
// us, clusters of 4 11.0.
SplitGeom split_geom(const LinOut& o, bool rows_mn, int64_t KT, int sms, int chain) {
  SplitGeom g{};
  g.NT = rows_mn ? (o.rows <= 64 ? 64 : 128) : (int)std::min<int64_t>(128, round_up(o.rows, 16));
  const int64_t tiles = cdiv(o.cols, 128) * cdiv(o.rows, g.NT);
  const int per_sm = g.NT <= S_NARROW ? 2 : 1;
  g.S = 1;
  while (g.S < 4 && tiles * g.S * 2 <= per_sm * sms && KT >= 4 * g.S) g.S *= 2;
  if (g.S == 4 && tiles * 8 <= sms / 2 && KT >= 16) g.S = 8;
  g.KT = (int)KT;
  const int budget = 216 * 1024 / per_sm - split_recv_bytes(g.NT, g.S);
  g.stages = (int)std::min<int64_t>(std::min(budget / split_stage_bytes(g.NT), 12), std::max<int64_t>(cdiv(KT, g.S), 1));
  // the ring must also hold the partial tile
  g.stages = std::max(g.stages, (int)cdiv(round_up(g.NT, 32) * 128 * 4, split_stage_bytes(g.NT)));
  g.chains = chain <= chain_steps<float>() || cdiv(KT, g.S) > chain;
  g.tmem_cols = 32;
  while ((int)g.tmem_cols < g.NT * (g.chains ? 2 : 1)) g.tmem_cols *= 2;
  return g;
}
// What the two kernels take, in microseconds, fitted to 90 shapes of 130 to
// 2560 rows, 128 to 4096 columns and contractions of 512 to 8192 (within 15%
// where the two are near each other): a fixed part (launch, first copies, last
// epilogue) and a part per step of 64.  256 x 512 over 2048: pair 11.7, split
// 10.9; over 8192: 27.9 and 15.6; 1280 x 1024 over 8192: 29.9 and 35.3.
double pair_us(const LinOut& o, int64_t KT, int pairs) {
  const Walk w = make_walk(o.rows, o.cols, (int)std::min<int64_t>(2 * cdiv(o.rows, PT) * cdiv(o.cols, PT), pairs));
  return 6.2 + (double)KT * (0.33 * (double)cdiv(w.whole, pairs) + 0.17 * (double)cdiv(w.total - w.whole, pairs));
}
double split_us(int64_t tiles, const SplitGeom& g, int sms) {
  return 8.8 + 0.21 * (double)(cdiv(tiles * g.S, sms) * cdiv(g.KT, g.S));
}

// out[rows x cols] = R C^T over KC, the epilogue as `o` says.  RN / CN: the
// operand that gives the output's rows / columns is stored with that index
// contiguous (else with the contraction contiguous).
template <typename T, typename O, bool RN, bool CN>
mpq_status lin_product(const Operand& R, const Operand& Cc, int64_t KC, const LinOut& o, cudaStream_t st,
                       const char* tag) {
  int dev = 0, sms = 0;
  MPQ_TRY(lin_device(&dev, &sms));
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  const Contraction kc{(int)cdiv(KC, BK) * (R.second ? 2 : 1), R.second ? 1 : 0};
  const int64_t KT = kc.steps;
  const int64_t big = cdiv(o.rows, PT) * cdiv(o.cols, PT);
  const int pairs = g_lin_dev[dev].pairs;
  const SplitGeom g = split_geom(o, RN, KT, sms, chain_steps<O>());
  const int64_t at_ = cdiv(o.cols, 128), bt = cdiv(o.rows, g.NT);
  ProfScope ps_(tag, st);
  if (pairs > 0 && o.rows > 128 && (bt > 65535 || pair_us(o, KT, pairs) <= split_us(at_ * bt, g, sms))) {
    CUtensorMap ta, ta_second, tb, tb_half;
    MPQ_TRY(encode_box(&ta, R.p, R.inner, R.rows, tma_ld(R), bf, RN ? 64 : 128));
    MPQ_TRY(encode_box(&ta_second, R.second ? R.second : R.p, R.inner, R.rows, tma_ld(R), bf, RN ? 64 : 128));
    MPQ_TRY(encode_box(&tb, Cc.p, Cc.inner, Cc.rows, tma_ld(Cc), bf, CN ? 64 : 128));
    MPQ_TRY(encode_box(&tb_half, Cc.p, Cc.inner, Cc.rows, tma_ld(Cc), bf, 64));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(2 * big, pairs));
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = P_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto kern = k_lin_pair<T, O, RN, CN, false>;
    if constexpr (!RN && !CN)
      if (o.act != MPQ_ACT_NONE || o.residual || o.preact) kern = k_lin_pair<T, O, RN, CN, true>;
    MPQ_CUDA(cudaLaunchKernelEx(&cfg, kern, ta, ta_second, tb, tb_half, kc, o));
  } else {
    if (bt > 65535 || at_ > 65535) return fail(MPQ_ERR_INVALID_ARG, "linear: too many tiles");
    const int smem = g.stages * split_stage_bytes(g.NT) + split_recv_bytes(g.NT, g.S) + (2 * g.stages + 6) * 8 + 16 + 1024;
    CUtensorMap ta, tb, tb_second;
    MPQ_TRY(encode_box(&ta, Cc.p, Cc.inner, Cc.rows, tma_ld(Cc), bf, CN ? 64 : 128));
    MPQ_TRY(encode_box(&tb, R.p, R.inner, R.rows, tma_ld(R), bf, RN ? 64 : g.NT));
    MPQ_TRY(encode_box(&tb_second, R.second ? R.second : R.p, R.inner, R.rows, tma_ld(R), bf, RN ? 64 : g.NT));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.S, (unsigned)at_, (unsigned)bt);
    cfg.blockDim = dim3(S_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)g.S;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    MPQ_CUDA(cudaLaunchKernelEx(&cfg, split_kernel<T, O, RN, CN>(g.chains, g.NT), ta, tb, tb_second, kc, g, o));
  }
  count_launch();
  return check_launch(tag);
}

mpq_status check_dims(const char* who, int64_t rows, int64_t n, int64_t k, int32_t dtype, int32_t act) {
  if (rows < 0 || rows > (1 << 23) || n < 1 || n > (1 << 22) || k < 1 || k > (1 << 22))
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": need 0 <= rows <= 2^23, 1 <= n, k <= 2^22");
  if (!half_dtype(dtype)) return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": operands must be bf16 or fp16");
  if (act < MPQ_ACT_NONE || act > MPQ_ACT_SILU)
    return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": unknown activation");
  return MPQ_OK;
}

// Two rows double the arithmetic per byte of W, which then sets the pace where W
// is large: 4096 -> 4096 takes 12.1 us (the split kernel 10.1), 4096 -> 14336
// 30.6 (24.3), but 8192 -> 512 4.9 (9.5) and 1024 -> 1024 3.5 (6.2).  One row: 8.9
// (10.4), 23.9 (24.3), and 1024 -> 8192 6.9 (8.1).  Without packing W first only
// this kernel reads rows at any address.
bool use_gemv(const Operand& x, const Operand& w) {
  if (x.rows <= 1) return true;
  return x.rows <= GEMV_ROWS && (w.rows * w.inner <= (1 << 23) || !tma_ok(x.p, x.inner, x.rows, x.ld) ||
                                 !tma_ok(w.p, w.inner, w.rows, w.ld));
}

template <typename T, typename O>
mpq_status linear_fwd(Operand x, Operand w, const LinOut& o, char* ws, cudaStream_t st) {
  if (use_gemv(x, w)) {
    // a warp per row of W fills the device from 24 warps an SM on; below that
    // more warps share a row, as long as each has 512 elements
    int wpr = 1, dev = 0, sms = 0;
    MPQ_TRY(current_device(&dev, &sms));
    while (wpr < GEMV_WARPS && w.rows * wpr < sms * 24 && x.inner >= 1024 * wpr) wpr *= 2;
    const unsigned grid = (unsigned)cdiv(w.rows, GEMV_WARPS / wpr);
    const bool vec = aligned_rows(x.p, x.ld, 2, 16) && aligned_rows(w.p, w.ld, 2, 16);
    const auto go = [&](auto kernel) {
      kernel<<<grid, GEMV_WARPS * 32, 0, st>>>(static_cast<const T*>(x.p), x.ld, static_cast<const T*>(w.p), w.ld,
                                               (int)x.inner, wpr, o);
    };
    ProfScope ps_("k_linear", st);
    if (x.rows == 1) vec ? go(k_lin_gemv<T, O, 1, true>) : go(k_lin_gemv<T, O, 1, false>);
    else vec ? go(k_lin_gemv<T, O, 2, true>) : go(k_lin_gemv<T, O, 2, false>);
    count_launch();
    return check_launch("k_linear");
  }
  char* to_x = tma_ok(x.p, x.inner, x.rows, x.ld) ? nullptr : ws;
  char* to_w = tma_ok(w.p, w.inner, w.rows, w.ld) ? nullptr : ws + (to_x ? packed_bytes(x.inner, x.rows) : 0);
  MPQ_TRY(pack(&x, to_x, &w, to_w, st));
  return lin_product<T, O, false, false>(x, w, x.inner, o, st, "k_linear");
}

struct BackPlan {  // workspace of a backward pass, in order
  bool make_dz, two_parts, pack_x, pack_w, sums;
  int64_t dz, dz_second, x, w, part, total;
};
BackPlan back_plan(const void* dy, int64_t ldy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                   int64_t rows, int64_t n, int64_t k, int32_t act_flags, bool need_dx, bool need_dw, bool need_db) {
  BackPlan p{};
  const int32_t act = act_flags & ~MPQ_DZ_ROUNDED;
  const bool prod = need_dx || need_dw;
  p.make_dz = prod && (act != MPQ_ACT_NONE || !tma_ok(dy, n, rows, ldy));
  p.two_parts = prod && act > MPQ_ACT_RELU && !(act_flags & MPQ_DZ_ROUNDED);
  p.pack_x = need_dw && !tma_ok(x, k, rows, ldx);
  p.pack_w = need_dx && !tma_ok(w, k, n, ldw);
  p.sums = need_db;
  p.dz = 0;
  p.dz_second = p.dz + rows * round_up(n, 8) * 2;
  p.x = p.dz + (p.make_dz ? packed_bytes(n, rows * (p.two_parts ? 2 : 1)) : 0);
  p.w = p.x + (p.pack_x ? packed_bytes(k, rows) : 0);
  p.part = p.w + (p.pack_w ? packed_bytes(k, n) : 0);
  p.total = p.part + (p.sums ? round_up(cdiv(rows, DZ_ROWS) * n * 4, 256) : 0);
  return p;
}

template <typename T>
mpq_status linear_bwd(const void* dy, int64_t ldy, Operand x, Operand w, const void* z, int64_t ldz,
                      int64_t rows, int64_t n, int64_t k, int32_t act, void* dx, void* dw, void* db,
                      bool db_f32, const BackPlan& p, char* ws, cudaStream_t st) {
  Operand dz{dy, n, rows, ldy};
  if (p.make_dz || p.sums) {
    T* dzp = p.make_dz ? reinterpret_cast<T*>(ws + p.dz) : nullptr;
    T* dz2 = p.two_parts ? reinterpret_cast<T*>(ws + p.dz_second) : nullptr;
    float* part = p.sums ? reinterpret_cast<float*>(ws + p.part) : nullptr;
    const int64_t ldd = round_up(n, 8), blocks = cdiv(rows, DZ_ROWS);
    {
      ProfScope ps_("k_lin_dz", st);
      k_lin_dz<T><<<dim3((unsigned)blocks, (unsigned)cdiv(n, 256)), 256, 0, st>>>(
          static_cast<const T*>(dy), ldy, static_cast<const T*>(z), ldz, act, rows, n, dzp, dz2, ldd, part,
          aligned_rows(dy, ldy, 2, 16), aligned_rows(z, ldz, 2, 16));
    }
    count_launch();
    MPQ_TRY(check_launch("k_lin_dz"));
    if (p.sums) {
      ProfScope ps_("k_lin_colsum", st);
      if (db_f32)
        k_lin_colsum<float><<<(unsigned)cdiv(n, 32), 256, 0, st>>>(part, blocks, n, static_cast<float*>(db));
      else
        k_lin_colsum<T><<<(unsigned)cdiv(n, 32), 256, 0, st>>>(part, blocks, n, static_cast<T*>(db));
      count_launch();
      MPQ_TRY(check_launch("k_lin_colsum"));
    }
    if (p.make_dz) dz = Operand{dzp, n, rows, ldd, dz2};
  }
  MPQ_TRY(pack(&x, p.pack_x ? ws + p.x : nullptr, &w, p.pack_w ? ws + p.w : nullptr, st));
  LinOut o{};
  if (dx) {  // dx[rows x k] = dz[rows x n] W[n x k]: W has the output's columns contiguous
    o.out = dx;
    o.ldo = k;
    o.rows = (int)rows;
    o.cols = (int)k;
    o.out_vec = aligned_rows(dx, k, 2, 16);
    MPQ_TRY((lin_product<T, T, false, true>(dz, w, n, o, st, "k_linear_dx")));
  }
  if (dw) {  // dW[n x k] = dz^T x: both have their output index contiguous
    o.out = dw;
    o.ldo = k;
    o.rows = (int)n;
    o.cols = (int)k;
    o.out_vec = aligned_rows(dw, k, 2, 16);
    MPQ_TRY((lin_product<T, T, true, true>(dz, x, rows, o, st, "k_linear_dw")));
  }
  return MPQ_OK;
}

}  // namespace
}  // namespace mpq

using namespace mpq;

extern "C" int64_t mpq_linear_workspace_bytes(const void* x, int64_t ldx, const void* weight, int64_t ldw,
                                              int64_t rows, int64_t n, int64_t k) {
  if (rows < 1 || n < 1 || k < 1 || use_gemv({x, k, rows, ldx}, {weight, k, n, ldw})) return 0;
  return (tma_ok(x, k, rows, ldx) ? 0 : packed_bytes(k, rows)) + (tma_ok(weight, k, n, ldw) ? 0 : packed_bytes(k, n));
}

extern "C" mpq_status mpq_linear(const void* x, int64_t ldx, const void* weight, int64_t ldw, int64_t rows,
                                 int64_t n, int64_t k, int32_t dtype, const void* bias, int32_t bias_dtype,
                                 int32_t act, const void* residual, int64_t ldr, void* preact, void* y,
                                 int32_t y_dtype, void* workspace, int64_t workspace_bytes, mpq_stream_t stream) {
  MPQ_TRY(check_dims("linear", rows, n, k, dtype, act));
  if (y_dtype != dtype && y_dtype != MPQ_F32)
    return fail(MPQ_ERR_INVALID_ARG, "linear: the output must have the operands' type or fp32");
  if (bias && bias_dtype != dtype && bias_dtype != MPQ_F32)
    return fail(MPQ_ERR_INVALID_ARG, "linear: the bias must have the operands' type or fp32");
  if (rows == 0) return MPQ_OK;
  if (!x || !weight || !y) return fail(MPQ_ERR_INVALID_ARG, "linear: missing buffer");
  MPQ_TRY(check_elements("linear", {{x, 2}, {weight, 2}, {bias, bias ? dtype_size(bias_dtype) : 1},
                                    {residual, dtype_size(y_dtype)}, {preact, 2}, {y, dtype_size(y_dtype)}}));
  const int64_t need = mpq_linear_workspace_bytes(x, ldx, weight, ldw, rows, n, k);
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
    return fail(MPQ_ERR_INVALID_ARG, "linear: needs " + std::to_string(need) +
                                         " bytes of workspace on a 256-byte boundary");
  LinOut o{};
  const int64_t os = dtype_size(y_dtype);
  o.bias = bias;
  o.residual = residual;
  o.preact = preact;
  o.out = y;
  o.ldr = ldr;
  o.ldo = n;
  o.rows = (int)rows;
  o.cols = (int)n;
  o.act = act;
  o.bias_f32 = bias_dtype == MPQ_F32;
  o.bias_vec = ((uintptr_t)bias & 15) == 0;
  o.res_vec = aligned_rows(residual, ldr, os, 16);
  o.out_vec = aligned_rows(y, n, os, 16) && aligned_rows(preact, n, 2, 16);
  const Operand xo{x, k, rows, ldx}, wo{weight, k, n, ldw};
  char* ws = static_cast<char*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MPQ_BF16)
    return y_dtype == MPQ_F32 ? linear_fwd<__nv_bfloat16, float>(xo, wo, o, ws, st)
                              : linear_fwd<__nv_bfloat16, __nv_bfloat16>(xo, wo, o, ws, st);
  return y_dtype == MPQ_F32 ? linear_fwd<__half, float>(xo, wo, o, ws, st)
                            : linear_fwd<__half, __half>(xo, wo, o, ws, st);
}

extern "C" int64_t mpq_linear_backward_workspace_bytes(const void* dy, int64_t ldy, const void* x, int64_t ldx,
                                                       const void* weight, int64_t ldw, int64_t rows, int64_t n,
                                                       int64_t k, int32_t act, int32_t need_dx,
                                                       int32_t need_dweight, int32_t need_dbias) {
  if (rows < 1 || n < 1 || k < 1) return 0;
  return back_plan(dy, ldy, x, ldx, weight, ldw, rows, n, k, act, need_dx != 0, need_dweight != 0,
                   need_dbias != 0).total;
}

extern "C" mpq_status mpq_linear_backward(const void* dy, int64_t ldy, const void* x, int64_t ldx,
                                          const void* weight, int64_t ldw, const void* preact, int64_t ldz,
                                          int64_t rows, int64_t n, int64_t k, int32_t dtype, int32_t act,
                                          void* dx, void* dweight, void* dbias, int32_t dbias_dtype,
                                          void* workspace, int64_t workspace_bytes, mpq_stream_t stream) {
  const int32_t act_flags = act;
  act &= ~MPQ_DZ_ROUNDED;
  MPQ_TRY(check_dims("linear_backward", rows, n, k, dtype, act));
  if (dbias && dbias_dtype != dtype && dbias_dtype != MPQ_F32)
    return fail(MPQ_ERR_INVALID_ARG, "linear_backward: dbias must have the operands' type or fp32");
  MPQ_TRY(check_elements("linear_backward", {{dy, 2}, {x, 2}, {weight, 2}, {preact, 2}, {dx, 2}, {dweight, 2},
                                             {dbias, dbias ? dtype_size(dbias_dtype) : 1}}));
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // nothing to sum: the parameters' gradients are zero
    if (dweight) MPQ_CUDA(cudaMemsetAsync(dweight, 0, (size_t)(n * k * 2), st));
    if (dbias) MPQ_CUDA(cudaMemsetAsync(dbias, 0, (size_t)(n * dtype_size(dbias_dtype)), st));
    return MPQ_OK;
  }
  if (!dy || (dweight && !x) || (dx && !weight) || (act != MPQ_ACT_NONE && !preact))
    return fail(MPQ_ERR_INVALID_ARG, "linear_backward: missing buffer");
  const BackPlan p = back_plan(dy, ldy, x, ldx, weight, ldw, rows, n, k, act_flags, dx != nullptr, dweight != nullptr,
                               dbias != nullptr);
  if (p.total > 0 && (!workspace || workspace_bytes < p.total || ((uintptr_t)workspace & 255)))
    return fail(MPQ_ERR_INVALID_ARG, "linear_backward: needs " + std::to_string(p.total) +
                                         " bytes of workspace on a 256-byte boundary");
  const Operand xo{x, k, rows, ldx}, wo{weight, k, n, ldw};
  char* ws = static_cast<char*>(workspace);
  const bool f32 = dbias_dtype == MPQ_F32;
  if (dtype == MPQ_BF16)
    return linear_bwd<__nv_bfloat16>(dy, ldy, xo, wo, preact, ldz, rows, n, k, act, dx, dweight, dbias, f32, p, ws, st);
  return linear_bwd<__half>(dy, ldy, xo, wo, preact, ldz, rows, n, k, act, dx, dweight, dbias, f32, p, ws, st);
}

extern "C" mpq_status mpq_ops_status(mpq_stream_t stream) {
  static thread_local uint32_t seen[64] = {};
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0, sms = 0;
  MPQ_TRY(current_device(&dev, &sms));
  uint32_t now = 0;
  MPQ_CUDA(cudaMemcpyFromSymbolAsync(&now, g_timeouts, sizeof(now), 0, cudaMemcpyDeviceToHost, st));
  MPQ_CUDA(cudaStreamSynchronize(st));
  if (now == seen[dev]) return MPQ_OK;
  seen[dev] = now;
  return fail(MPQ_ERR_TIMEOUT, "a bounded wait of a linear kernel ran out");
}

extern "C" mpq_status mpq_ops_expire(mpq_stream_t stream) {
  k_expire<<<1, 32, 0, (cudaStream_t)stream>>>();
  count_launch();
  return check_launch("k_expire");
}
