// Rows of the root-mean-square norm's kernels: how a team of threads holds one
// row, in groups of eight values or value by value, and sums over the team.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace flce {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Eight values at a 16-byte boundary (32 bytes of fp32 in two loads).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values as they lie in memory.
template <class T>
struct Raw {
  uint4 q[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const T* p) {
    q[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (sizeof(T) == 4) q[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() {
    q[0] = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 4) q[1] = q[0];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same_v<T, __half>) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        } else {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
};

// A team's columns value by value, for rows that start anywhere: value j of a
// thread's i-th group of eight lies TEAM columns after the one before, so that a
// warp's loads are neighbours.
template <int TEAM>
struct Columns {
  static __device__ __forceinline__ int64_t first(int64_t e0, int i, int t) {
    return e0 + i * 8 * TEAM + t;
  }
  // Zeros past the row's end.
  template <class T>
  static __device__ __forceinline__ void load(const T* row, int64_t e, int64_t h, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e + j * TEAM < h ? to_f32(row[e + j * TEAM]) : 0.0f;
  }
  template <class T>
  static __device__ __forceinline__ void store(T* row, int64_t e, int64_t h,
                                               const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j * TEAM < h) row[e + j * TEAM] = from_f32<T>(v[j]);
  }
  // A tensor that is fp32 where `wide` and T otherwise.
  template <class T>
  static __device__ __forceinline__ void load_either(const void* p, int64_t row_at, int wide,
                                                     int64_t e, int64_t h, float (&v)[8]) {
    if (sizeof(T) == 4 || wide)
      load(static_cast<const float*>(p) + row_at, e, h, v);
    else
      load(static_cast<const T*>(p) + row_at, e, h, v);
  }
  template <class T>
  static __device__ __forceinline__ void store_either(void* p, int64_t row_at, int wide,
                                                      int64_t e, int64_t h,
                                                      const float (&v)[8]) {
    if (sizeof(T) == 4 || wide)
      store(static_cast<float*>(p) + row_at, e, h, v);
    else
      store(static_cast<T*>(p) + row_at, e, h, v);
  }
};

// Eight fp32 weights from column e on; zeros past the row's end.
__device__ __forceinline__ void load_weights(const void* weight, int e, int64_t h, float (&v)[8]) {
  if (e < h) {
    load8(static_cast<const float*>(weight) + e, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
}

// Whether every row of a tensor starts at a 16-byte boundary.
inline bool rows_of_16(const void* p, int64_t pitch, int size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch * size % 16 == 0);
}

// The sum (or, for MaxOp, the maximum) of `v` over the team: a warp, or all
// TEAM threads of the CTA, in a fixed order. `buf` holds a value a warp; calls
// one after the other use different buffers or have a barrier between them.
struct SumOp {
  template <class V>
  __device__ __forceinline__ V operator()(V a, V b) const {
    return a + b;
  }
};
struct MaxOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return a > b ? a : b;
  }
};
template <int TEAM, class V, class Op>
__device__ __forceinline__ V team_all(V v, V* buf, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (TEAM > 32) {
    constexpr int kWarps = TEAM / 32;
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

}  // namespace flce
