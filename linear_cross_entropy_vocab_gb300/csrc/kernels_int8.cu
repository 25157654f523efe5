// 8-bit integer rows with a scale each:
//
//   scale_i = max_h |x_ih| / 127,  q_ih = round(x_ih / scale_i)
//
// as bytes for the caller, or as halves in the operand order of the linear
// kernel (kernels_qlinear.cu). Bound by memory: a CTA takes one row, keeps up
// to 4096 values of it in registers between the maximum and the rounding, and
// reads longer rows a second time, from L2.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int8_internal.h"

namespace flce {
namespace {

constexpr int kThreads = 128;
constexpr int kVecs = 4;  // groups of 8 values per thread and sweep
constexpr int kSweep = kThreads * kVecs * 8;

template <class T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(int8_t x) { return static_cast<float>(x); }

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const int8_t* p, float (&x)[8]) {
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = static_cast<float>(static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3))));
}

// 8 values from element e of a row of h; zeros past its end.
template <class T>
__device__ __forceinline__ void load_group(const T* row, int64_t e, int64_t h, bool vec,
                                           float (&x)[8]) {
  if (vec && e + 8 <= h) {
    load8(row + e, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = e + j < h ? to_float(row[e + j]) : 0.0f;
  }
}

// round(x / scale), halves to even. The product with the reciprocal is within
// 2^-16 of the quotient (at most 127, two roundings): only near a half does
// the division decide.
__device__ __forceinline__ void round8(float (&x)[8], float scale, float inv) {
  if (!(scale > 0.0f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    return;
  }
  bool close = scale < 1.0e-37f;  // its reciprocal may overflow
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = x[j] * inv;
    r[j] = rintf(y);
    close |= fabsf(y - r[j]) > 0.4999f;
  }
  if (close) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = rintf(__fdiv_rn(x[j], scale));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = fminf(127.0f, fmaxf(-127.0f, r[j]));
}

__device__ __forceinline__ void put_bytes(int8_t* q, int64_t e, int64_t h, bool vec,
                                          const float (&x)[8]) {
  if (vec && e + 8 <= h) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t b0 = static_cast<uint32_t>(__float2int_rn(x[4 * i])) & 0xffu;
      const uint32_t b1 = static_cast<uint32_t>(__float2int_rn(x[4 * i + 1])) & 0xffu;
      const uint32_t b2 = static_cast<uint32_t>(__float2int_rn(x[4 * i + 2])) & 0xffu;
      const uint32_t b3 = static_cast<uint32_t>(__float2int_rn(x[4 * i + 3]));
      w[i] = b0 | (b1 << 8) | (b2 << 16) | (b3 << 24);
    }
    *reinterpret_cast<uint2*>(q + e) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < h) q[e + j] = static_cast<int8_t>(__float2int_rn(x[j]));
  }
}

__device__ __forceinline__ void put_halves(__half* wide, int64_t e, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 a = __floats2half2_rn(x[4 * i], x[4 * i + 2]);
    const __half2 b = __floats2half2_rn(x[4 * i + 1], x[4 * i + 3]);
    w[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
    w[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(wide + e) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per row; WIDE: halves in operand order instead of bytes.
template <class T, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
  __shared__ uint32_t buf[kThreads / 32];
  if (WIDE) grid_launch_dependents();
  constexpr bool kInt = sizeof(T) == 1;
  const int64_t row = blockIdx.x;
  const T* const x0 = static_cast<const T*>(p.x) + row * p.x_pitch;
  const bool vec = (reinterpret_cast<uintptr_t>(x0) & (kInt ? 7u : 15u)) == 0;
  int8_t* const q0 = WIDE ? nullptr : p.q + row * p.q_pitch;
  const bool qvec = (reinterpret_cast<uintptr_t>(q0) & 7u) == 0;
  __half* const w0 = WIDE ? static_cast<__half*>(p.wide) + row * p.wide_pitch : nullptr;
  const int64_t end = WIDE ? p.wide_pitch : p.h;
  float x[kVecs][8];
  float scale = 1.0f, inv = 1.0f;
  if constexpr (!kInt) {
    // largest magnitude by the order of the bits: NaN is above infinity
    uint32_t m = 0;
    for (int64_t e0 = 0; e0 < p.h; e0 += kSweep) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int64_t e = e0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
        load_group(x0, e, p.h, vec, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[i][j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, buf[w]);
    const float peak = __uint_as_float(m);
    // NaN and infinity: the scale is NaN, and so is every product with it
    scale = peak < INFINITY ? __fdiv_rn(peak, 127.0f) : NAN;
    inv = __fdiv_rn(1.0f, scale);
    if (threadIdx.x == 0) p.scale[row] = scale;
  }
  for (int64_t e0 = 0; e0 < end; e0 += kSweep) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int64_t e = e0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
      if (e >= end) break;
      if (kInt || p.h > kSweep) load_group(x0, e, p.h, vec, x[i]);
      if constexpr (!kInt) round8(x[i], scale, inv);
      if constexpr (WIDE)
        put_halves(w0, e, x[i]);
      else
        put_bytes(q0, e, p.h, qvec, x[i]);
    }
  }
}

// Four bytes at a time into aligned rows; the source may start anywhere.
__global__ void __launch_bounds__(256)
    align_rows_kernel(const int8_t* src, int64_t rows, int64_t h, int64_t src_pitch, int8_t* dst,
                      int64_t dst_pitch) {
  const int64_t words = dst_pitch / 4;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int8_t* const s = src + row * src_pitch;
    for (int64_t w = threadIdx.x; w < words; w += 256) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * w + j < h)
          v |= static_cast<uint32_t>(static_cast<uint8_t>(s[4 * w + j])) << (8 * j);
      reinterpret_cast<uint32_t*>(dst + row * dst_pitch)[w] = v;
    }
  }
}

template <bool WIDE>
cudaError_t launch_rows(const QuantParams& p, int dtype, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.n);
  if (dtype == FLCE_F32)
    quantize_rows_kernel<float, WIDE><<<grid, kThreads, 0, s>>>(p);
  else if (dtype == FLCE_BF16)
    quantize_rows_kernel<__nv_bfloat16, WIDE><<<grid, kThreads, 0, s>>>(p);
  else if (dtype == FLCE_F16)
    quantize_rows_kernel<__half, WIDE><<<grid, kThreads, 0, s>>>(p);
  else if constexpr (WIDE)
    quantize_rows_kernel<int8_t, WIDE><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantParams& p, int dtype, cudaStream_t s) {
  return launch_rows<false>(p, dtype, s);
}

cudaError_t launch_widen_rows(const QuantParams& p, int dtype, cudaStream_t s) {
  return launch_rows<true>(p, dtype, s);
}

cudaError_t launch_align_rows(const int8_t* src, int64_t rows, int64_t h, int64_t src_pitch,
                              int8_t* dst, int64_t dst_pitch, cudaStream_t s) {
  const unsigned grid = rows < 65536 ? static_cast<unsigned>(rows) : 65536u;
  align_rows_kernel<<<grid, 256, 0, s>>>(src, rows, h, src_pitch, dst, dst_pitch);
  return cudaGetLastError();
}

}  // namespace flce
