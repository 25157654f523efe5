// 8-bit integer rows with a scale each, and the linear layer on them:
//
//   scale_i = max_h |x_ih| / 127,  q_ih = round(x_ih / scale_i)
//   out_ij  = f(scale_i * weight_scale_j * sum_h q_ih w_jh + bias_j)
//
// with f the logit transform of the losses (scale and softcap).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int8_internal.h"

namespace flce {
namespace {

__device__ __forceinline__ float load_as_float(const void* p, int dtype, int64_t i) {
  if (dtype == FLCE_F32) return static_cast<const float*>(p)[i];
  if (dtype == FLCE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_float(void* p, int dtype, int64_t i, float x) {
  if (dtype == FLCE_F32)
    static_cast<float*>(p)[i] = x;
  else if (dtype == FLCE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16(x);
  else
    static_cast<__half*>(p)[i] = __float2half(x);
}

// ------------------------------------------------------------ quantisation
constexpr int kQuantThreads = 128;

// Largest magnitude of a row by the order of the bits: NaN is above infinity.
__device__ __forceinline__ uint32_t row_peak(uint32_t m, uint32_t* buf) {
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
  __syncthreads();
  m = buf[0];
#pragma unroll
  for (int w = 1; w < kQuantThreads / 32; ++w) m = max(m, buf[w]);
  return m;
}

// One CTA per row.
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const QuantParams p, int dtype) {
  __shared__ uint32_t buf[kQuantThreads / 32];
  const int64_t row = blockIdx.x;
  const int64_t x0 = row * p.x_pitch;
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < p.h; i += kQuantThreads)
    m = max(m, __float_as_uint(load_as_float(p.x, dtype, x0 + i)) & 0x7fffffffu);
  const float peak = __uint_as_float(row_peak(m, buf));
  // NaN and infinity: the scale is NaN, and so is every product with it
  const float scale = peak < INFINITY ? __fdiv_rn(peak, 127.0f) : NAN;
  if (threadIdx.x == 0) p.scale[row] = scale;
  for (int64_t i = threadIdx.x; i < p.h; i += kQuantThreads) {
    const float x = load_as_float(p.x, dtype, x0 + i);
    int q = 0;
    if (scale > 0.0f) q = min(127, max(-127, __float2int_rn(__fdiv_rn(x, scale))));
    p.q[row * p.q_pitch + i] = static_cast<int8_t>(q);
  }
}

// ------------------------------------------------------------------ linear
// 64 x 64 outputs per CTA, 4 x 4 per thread, dot products of four bytes at a
// time; rows of any pitch and address.
constexpr int kTile = 64;
constexpr int kTileK = 64;
constexpr int kPad = kTileK / 4 + 1;  // words of a staged row

__device__ __forceinline__ void stage_tile(int (*dst)[kPad], const int8_t* src, int64_t row0,
                                           int64_t rows, int64_t pitch, int64_t k0, int64_t h) {
  for (int i = threadIdx.x; i < kTile * kTileK / 4; i += 256) {
    const int r = i / (kTileK / 4), w = i % (kTileK / 4);
    uint32_t v = 0;
    if (row0 + r < rows) {
      const int8_t* const p = src + (row0 + r) * pitch + k0 + 4 * w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + 4 * w + j < h) v |= static_cast<uint32_t>(static_cast<uint8_t>(p[j])) << (8 * j);
    }
    dst[r][w] = static_cast<int>(v);
  }
}

__global__ void __launch_bounds__(256) qlinear_simple_kernel(const QLinearParams p) {
  __shared__ int xs[kTile][kPad];
  __shared__ int ws[kTile][kPad];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.h; k0 += kTileK) {
    __syncthreads();
    stage_tile(xs, p.x, n0, p.n, p.x_pitch, k0, p.h);
    stage_tile(ws, p.weight, v0, p.v, p.weight_pitch, k0, p.h);
    __syncthreads();
#pragma unroll 4
    for (int w = 0; w < kTileK / 4; ++w) {
      int a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = xs[ty + 16 * i][w];
        b[i] = ws[tx + 16 * i][w];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[i], b[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + ty + 16 * i;
    if (n >= p.n) continue;
    const float xsc = p.x_scale[n];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t v = v0 + tx + 16 * j;
      if (v >= p.v) continue;
      const float b = p.bias != nullptr ? load_as_float(p.bias, p.bias_dtype, v) : 0.0f;
      const float lin = static_cast<float>(acc[i][j]) * p.weight_scale[v] * xsc;
      store_float(p.out, p.out_dtype, n * p.out_pitch + v, p.xf(lin, b));
    }
  }
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantParams& p, int dtype, cudaStream_t s) {
  quantize_rows_kernel<<<static_cast<unsigned>(p.n), kQuantThreads, 0, s>>>(p, dtype);
  return cudaGetLastError();
}

cudaError_t launch_qlinear_simple(const QLinearParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.v + kTile - 1) / kTile),
                  static_cast<unsigned>((p.n + kTile - 1) / kTile));
  qlinear_simple_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flce
