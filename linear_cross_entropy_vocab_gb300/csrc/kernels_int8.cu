// 8-bit integer rows with a scale each:
//
//   scale_i = max_h |x_ih| * (1/127),  q_ih = round(x_ih / scale_i)
//
// as bytes for the caller, or as halves in the operand order of the linear
// kernel (kernels_qlinear.cu).
//
// Bound by memory: a team of threads takes one row, keeps it in registers, as
// it came, between the maximum and the rounding, and reads rows of more than
// 4096 values a second time, from L2. The team is 8 threads for rows of up to
// 256 values, a warp up to 2048, a CTA beyond: 128256 bf16 rows of 128 take
// 32 us with 8 threads each and 54 with 32; rows of 2048 144 with a warp and
// 192 with a CTA; rows of 4096 266 with a CTA and 314 with a warp (calls with
// their host side). What keeps it near that bound is the
// number of instructions for a value: the maximum is taken on the raw bits, two
// 16-bit values at a time; the quotient is a product with the reciprocal and one
// correction; and adding 1.5 * 2^23 rounds it and leaves the integer in the low
// byte.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int8_internal.h"

namespace flce {
namespace {

constexpr int kThreads = 128;

// A group of 8 values: how it is loaded, its largest magnitude by the order of
// the bits (NaN is above infinity), and its values.
template <class T>
struct Group;
template <>
struct Group<float> {
  static constexpr int kAlign = 16;
  uint4 q[2];
  __device__ __forceinline__ void load(const float* p) {
    q[0] = __ldg(reinterpret_cast<const uint4*>(p));
    q[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void load_some(const float* p, int64_t n) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __float_as_uint(p[j]) : 0u;
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ uint32_t peak(uint32_t m) const {
    const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7fffffffu);
    return m;
  }
  static __device__ __forceinline__ float peak_value(uint32_t m) { return __uint_as_float(m); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
  }
};

// The same for 16-bit types, two values in a word.
struct Group16 {
  static constexpr int kAlign = 16;
  uint4 q;
  __device__ __forceinline__ void load(const void* p) {
    q = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_some(const void* p, int64_t n) {
    const uint16_t* const u = static_cast<const uint16_t*>(p);
    uint32_t w[4];
    if (n >= 8 && (reinterpret_cast<uintptr_t>(p) & 3u) == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __ldg(static_cast<const uint32_t*>(p) + j);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (2 * j < n ? u[2 * j] : 0u) | ((2 * j + 1 < n ? u[2 * j + 1] : 0u) << 16);
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint32_t peak(uint32_t m) const {
    m = __vmaxu2(m, q.x & 0x7fff7fffu);
    m = __vmaxu2(m, q.y & 0x7fff7fffu);
    m = __vmaxu2(m, q.z & 0x7fff7fffu);
    return __vmaxu2(m, q.w & 0x7fff7fffu);
  }
};
template <>
struct Group<__nv_bfloat16> : Group16 {
  static __device__ __forceinline__ float peak_value(uint32_t m) {
    return __uint_as_float(max(m >> 16, m & 0xffffu) << 16);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Group<__half> : Group16 {
  static __device__ __forceinline__ float peak_value(uint32_t m) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(max(m >> 16, m & 0xffffu))));
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
// Integers already: nothing to scale.
template <>
struct Group<int8_t> {
  static constexpr int kAlign = 8;
  uint2 q;
  __device__ __forceinline__ void load(const int8_t* p) {
    q = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void load_some(const int8_t* p, int64_t n) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[j])) << (8 * (j & 3));
    q = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ uint32_t peak(uint32_t m) const { return m; }
  static __device__ __forceinline__ float peak_value(uint32_t) { return 0.0f; }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3))));
  }
};

constexpr float kToInt = 12582912.0f;  // 1.5 * 2^23: adding it rounds to whole numbers

// x / scale rounded to whole numbers, halves to even, plus kToInt (the integer
// is in the low byte). Values of a short type are multiples of few scales, and
// halves are common: the quotient has to be the correctly rounded one. It is,
// from a product with the correctly rounded reciprocal and one correction by
// the exact remainder (Markstein 1990, theorem on division), where nothing
// leaves the normal range: quotients below a half need no more than to stay
// there.
__device__ __forceinline__ void round8(float (&x)[8], float scale, float inv) {
  if (scale >= 1.0e-28f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = x[j] * inv;
      x[j] = fmaf(fmaf(-q, scale, x[j]), inv, q) + kToInt;
    }
    return;
  }
  // a tiny scale, 0 or NaN
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = scale > 0.0f ? rintf(__fdiv_rn(x[j], scale)) : 0.0f;
    x[j] = fminf(127.0f, fmaxf(-127.0f, q)) + kToInt;
  }
}

__device__ __forceinline__ void put_bytes(int8_t* q, int64_t e, int64_t h, bool vec,
                                          const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __byte_perm(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), 0x40);
    const uint32_t hi =
        __byte_perm(__float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]), 0x40);
    w[i] = __byte_perm(lo, hi, 0x5410);
  }
  if (vec && e + 8 <= h) {
    *reinterpret_cast<uint2*>(q + e) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < h) q[e + j] = static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
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

// One row per team of TEAM threads; WIDE: halves in operand order instead of
// bytes.
template <class T, bool WIDE, int TEAM, int VECS>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
  __shared__ uint32_t buf[kThreads / 32];
  if (WIDE) grid_launch_dependents();
  constexpr bool kInt = sizeof(T) == 1;
  constexpr int kSweep = TEAM * VECS * 8;
  const int in_team = static_cast<int>(threadIdx.x) % TEAM;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TEAM) +
                      static_cast<int>(threadIdx.x) / TEAM;
  if (TEAM < kThreads && row >= p.n) return;
  const T* const x0 = static_cast<const T*>(p.x) + row * p.x_pitch;
  const bool vec = (reinterpret_cast<uintptr_t>(x0) & (Group<T>::kAlign - 1)) == 0;
  int8_t* const q0 = WIDE ? nullptr : p.q + row * p.q_pitch;
  const bool qvec = (reinterpret_cast<uintptr_t>(q0) & 7u) == 0;
  __half* const w0 = WIDE ? static_cast<__half*>(p.wide) + row * p.wide_pitch : nullptr;
  const int64_t end = WIDE ? p.wide_pitch : p.h;
  Group<T> g[VECS];
  // the thread's groups of the sweep from e0 on; zeros past the row's end
  auto load = [&](int64_t e0) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int64_t e = e0 + (i * TEAM + in_team) * 8;
      if (vec && e + 8 <= p.h)
        g[i].load(x0 + e);
      else if (e < p.h)
        g[i].load_some(x0 + e, p.h - e);
      else
        g[i] = Group<T>{};
    }
  };
  float scale = 1.0f, inv = 1.0f;
  if constexpr (!kInt) {
    uint32_t m = 0;
    for (int64_t e0 = 0; e0 < p.h; e0 += kSweep) {
      load(e0);
#pragma unroll
      for (int i = 0; i < VECS; ++i) m = g[i].peak(m);
    }
    m = __float_as_uint(Group<T>::peak_value(m));
    if constexpr (TEAM < 32) {
#pragma unroll
      for (int o = TEAM / 2; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffu << (threadIdx.x & 24u), m, o, TEAM));
    } else {
      m = __reduce_max_sync(0xffffffffu, m);
    }
    if constexpr (TEAM == kThreads) {
      if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = max(m, buf[w]);
    }
    const float peak = __uint_as_float(m);
    // NaN and infinity: the scale is NaN, and so is every product with it
    scale = peak < INFINITY ? peak * (1.0f / 127.0f) : NAN;
    inv = __fdiv_rn(1.0f, scale);
    if (in_team == 0) p.scale[row] = scale;
  }
  for (int64_t e0 = 0; e0 < end; e0 += kSweep) {
    if (kInt || p.h > kSweep) load(e0);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int64_t e = e0 + (i * TEAM + in_team) * 8;
      if (e >= end) break;
      float x[8];
      g[i].values(x);
      if constexpr (!kInt) {
        round8(x, scale, inv);
        if constexpr (WIDE) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] -= kToInt;
        }
      }
      if constexpr (WIDE)
        put_halves(w0, e, x);
      else
        put_bytes(q0, e, p.h, qvec, x);
    }
  }
}

// Rows that start anywhere into rows that start at multiples of 16 bytes: a
// thread makes 16 bytes from the five aligned words that hold them. At the
// buffer's two ends, where such a word would reach past it, and in a row's
// last bytes it takes them one by one.
__global__ void __launch_bounds__(256)
    align_rows_kernel(const int8_t* src, int64_t rows, int64_t h, int64_t src_pitch, int8_t* dst,
                      int64_t dst_pitch) {
  const int64_t per_row = dst_pitch / 16;
  const int64_t total = rows * per_row;
  const uintptr_t begin = reinterpret_cast<uintptr_t>(src);
  const uintptr_t end = begin + static_cast<uintptr_t>((rows - 1) * src_pitch + h);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = total <= 0xffffffffll
                            ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row)
                            : i / per_row;
    const int64_t c = (i - row * per_row) * 16;
    const int8_t* const s = src + row * src_pitch + c;
    const uintptr_t word = reinterpret_cast<uintptr_t>(s) & ~uintptr_t(3);
    uint32_t v[4] = {0, 0, 0, 0};
    if (c + 16 <= h && word >= begin && word + 20 <= end) {
      const uint32_t* const w = reinterpret_cast<const uint32_t*>(word);
      const uint32_t shift = 8u * static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s) & 3u);
      uint32_t lo = __ldg(w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t hi = __ldg(w + j + 1);
        v[j] = __funnelshift_r(lo, hi, shift);
        lo = hi;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < h)
          v[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(s[j])) << (8 * (j & 3));
    }
    *reinterpret_cast<uint4*>(dst + row * dst_pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

template <class T, bool WIDE, int TEAM, int VECS>
cudaError_t launch_team(const QuantParams& p, cudaStream_t s) {
  const int64_t rows = kThreads / TEAM;  // of a CTA
  const unsigned grid = static_cast<unsigned>((p.n + rows - 1) / rows);
  quantize_rows_kernel<T, WIDE, TEAM, VECS><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T, bool WIDE>
cudaError_t launch_typed(const QuantParams& p, cudaStream_t s) {
  const int64_t len = WIDE ? p.wide_pitch : p.h;
  if (len <= 256) return launch_team<T, WIDE, 8, 4>(p, s);
  if (len <= 1024) return launch_team<T, WIDE, 32, 4>(p, s);
  if (len <= 2048) return launch_team<T, WIDE, 32, 8>(p, s);
  return launch_team<T, WIDE, kThreads, 4>(p, s);
}

template <bool WIDE>
cudaError_t launch_rows(const QuantParams& p, int dtype, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_typed<float, WIDE>(p, s);
  if (dtype == FLCE_BF16) return launch_typed<__nv_bfloat16, WIDE>(p, s);
  if (dtype == FLCE_F16) return launch_typed<__half, WIDE>(p, s);
  if constexpr (WIDE) return launch_typed<int8_t, WIDE>(p, s);
  return cudaErrorInvalidValue;
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
  const int64_t blocks = (rows * (dst_pitch / 16) + 255) / 256;
  const unsigned grid = blocks < (1 << 20) ? static_cast<unsigned>(blocks) : 1u << 20;
  align_rows_kernel<<<grid, 256, 0, s>>>(src, rows, h, src_pitch, dst, dst_pitch);
  return cudaGetLastError();
}

}  // namespace flce
