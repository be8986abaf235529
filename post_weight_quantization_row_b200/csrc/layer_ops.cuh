// Shared parts of the layer and answer operators (linear, layer norm, token
// log probabilities, top-logits distillation): element types and vector access.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <initializer_list>

#include "f32x2.cuh"
#include "mpq_internal.cuh"
#include "tc_ptx.cuh"

namespace mpq {

inline int64_t dtype_size(int32_t dt) { return dt == MPQ_F32 ? 4 : 2; }
inline bool half_dtype(int32_t dt) { return dt == MPQ_BF16 || dt == MPQ_F16; }
inline bool any_dtype(int32_t dt) { return dt == MPQ_F32 || half_dtype(dt); }

// Index and SM count of the current device.
mpq_status current_device(int* dev, int* sms);

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

__device__ __forceinline__ float2 unpack2(uint32_t w, const __nv_bfloat16*) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, const __half*) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// W consecutive elements (W = 1, 4 or 8) as floats.  vec: the address is aligned
// to W elements (at most 16 bytes are read at once); otherwise one by one.
template <int W, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[W], bool vec) {
  if (!vec || W == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = to_f(p[i]);
    return;
  }
  if constexpr (W == 1) return;
  else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else if constexpr (W == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(w[i], p);
      v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2(q.x, p), b = unpack2(q.y, p);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
}
template <int W, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[W], bool vec) {
  if (!vec || W == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) p[i] = from_f<T>(v[i]);
    return;
  }
  if constexpr (W == 1) return;
  else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (W == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1], p), pack2(v[2], v[3], p),
                                              pack2(v[4], v[5], p), pack2(v[6], v[7], p));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1], p), pack2(v[2], v[3], p));
  }
}
// The same with the first n elements only (n < W at an edge); missing ones
// read as zero.
template <int W, typename T>
__device__ __forceinline__ void load_edge(const T* p, float (&v)[W], int n, bool vec) {
  if (n >= W) {
    load_vec<W>(p, v, vec);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = i < n ? to_f(p[i]) : 0.0f;
  }
}
template <int W, typename T>
__device__ __forceinline__ void store_edge(T* p, const float (&v)[W], int n, bool vec) {
  if (n >= W) {
    store_vec<W>(p, v, vec);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) p[i] = from_f<T>(v[i]);
  }
}
// A parameter vector (bias, norm weight) held in T or in fp32.
template <int W, typename T>
__device__ __forceinline__ void load_param(const void* p, bool f32, int64_t at, float (&v)[W],
                                           int n, bool vec) {
  if (f32) load_edge<W>(static_cast<const float*>(p) + at, v, n, vec);
  else load_edge<W>(static_cast<const T*>(p) + at, v, n, vec);
}

// 8 consecutive elements as they lie in memory: half the registers of floats
// for 16-bit types.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void decode(const Raw8<T>& r, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(w[i], static_cast<const T*>(nullptr));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
// 8 elements as 4 packed pairs
struct F8 {
  uint64_t p[4];
};
template <typename T>
__device__ __forceinline__ F8 pairs(const Raw8<T>& r) {
  float v[8];
  decode<T>(r, v);
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f2_pack(v[2 * i], v[2 * i + 1]);
  return f;
}
__device__ __forceinline__ F8 pairs(const float (&v)[8]) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f2_pack(v[2 * i], v[2 * i + 1]);
  return f;
}
__device__ __forceinline__ void unpairs(const F8& f, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f.p[i], v[2 * i], v[2 * i + 1]);
}
// The first n of 8 elements (all for n >= 8, none for n <= 0), the others 0;
// vec: the address is on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p, int n, bool vec) {
  Raw8<T> r;
  if (n >= 8 && vec) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : from_f<T>(0.0f);
    memcpy(&r, e, sizeof(r));
  }
  return r;
}

// Words s .. s + 3 of 8, counted in bytes 2 s2 .. (0 .. 14): a 16-byte window at
// any even byte of two vectors.
__device__ __forceinline__ uint4 window16(const uint4& u, const uint4& v, int halfwords) {
  uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  if (halfwords & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (halfwords & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t s = (halfwords & 1) * 16;
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                    __funnelshift_r(w[3], w[4], s));
}
// Elements at .. at + 7 of a row of n elements at any address, those past the
// end 0.  Aligned 16-byte loads and shifts where all of them lie within the
// row, single elements at its ends.  In two parts, so that the loads can be in
// flight before the shift needs them.
template <typename T>
struct RawWindow {
  uint4 q[sizeof(T) / 2 + 1];
  int halfwords;  // how far into q the elements begin
};
template <typename T>
__device__ __forceinline__ RawWindow<T> load_window(const T* row, int at, int n) {
  const T* p = row + at;
  const uintptr_t a = (uintptr_t)p;
  constexpr int V = 16 / (int)sizeof(T);           // elements of a 16-byte vector
  const int off = (int)(a & 15) / (int)sizeof(T);  // elements past the boundary
  RawWindow<T> w;
  if (off && at >= off && at - off + 8 + V <= n) {
    const uint4* q = reinterpret_cast<const uint4*>(a & ~(uintptr_t)15);
#pragma unroll
    for (int i = 0; i <= (int)(sizeof(T) / 2); ++i) w.q[i] = q[i];
    w.halfwords = (int)(a & 15) >> 1;
  } else {
    const Raw8<T> r = load_raw<T>(p, n - at, off == 0);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w.q[i] = r.q[i];
    w.q[sizeof(T) / 2] = make_uint4(0, 0, 0, 0);
    w.halfwords = 0;
  }
  return w;
}
template <typename T>
__device__ __forceinline__ Raw8<T> shift_window(const RawWindow<T>& w) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.q[i] = window16(w.q[i], w.q[i + 1], w.halfwords);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw8<T> load_row8(const T* row, int at, int n) {
  return shift_window<T>(load_window<T>(row, at, n));
}
// Stores a warp's 8 elements a lane, 256 neighbours of a row of which `total`
// exist, at any address: through `stage` (shared memory of the warp, 256
// elements and 16 bytes, on a 16-byte boundary) to whole aligned vectors, and
// single elements at the ends.  All lanes take part.
template <typename T>
__device__ __forceinline__ void warp_store(T* row, const float (&v)[8], int total, T* stage) {
  const int lane = threadIdx.x & 31;
  constexpr int V = 16 / (int)sizeof(T);
  __syncwarp();
  store_vec<8>(stage + lane * 8, v, true);
  __syncwarp();
  const int past = (int)((uintptr_t)row & 15) / (int)sizeof(T), lead = min(total, past ? V - past : 0);
  const int nv = (total - lead) / V;
  const uint4* q = reinterpret_cast<const uint4*>(stage);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
    const int k = lane + 32 * i;
    if (k < nv)
      reinterpret_cast<uint4*>(row + lead)[k] = lead ? window16(q[k], q[k + 1], lead * (int)sizeof(T) / 2) : q[k];
  }
  const int e = lane < lead ? lane : lead + nv * V + (lane - lead);
  if (e < total) row[e] = stage[e];
}

__device__ __forceinline__ float ex2(float x) {  // 2^x, 2 ulp; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a float at the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];"
               : "=f"(v)
               : "r"(tcx::map_to_rank(tcx::smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}

// Buffers that do not start on a multiple of their elements' size are refused:
// a load or store of such an element is a fault on the device.
struct Buffer {
  const void* p;
  int64_t elem;
};
inline mpq_status check_elements(const char* who, std::initializer_list<Buffer> buffers) {
  for (const Buffer& b : buffers)
    if ((uintptr_t)b.p % (uintptr_t)b.elem)
      return fail(MPQ_ERR_INVALID_ARG, std::string(who) + ": a buffer is not aligned to its elements");
  return MPQ_OK;
}

inline bool aligned_rows(const void* p, int64_t ld, int64_t elem, int64_t bytes) {
  return ((uintptr_t)p % bytes) == 0 && (ld * elem) % bytes == 0;
}

}  // namespace mpq
