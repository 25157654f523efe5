// The norm of a set of gradients taken together, and the clipping by it:
//
//   norm = (sum_i |g_i|^p)^(1/p)  for p = 1, 2;  max_i |g_i|  for p = inf
//   coef = min(1, max_norm / (norm + eps)),  out_i = g_i * coef
//
// over every element of every tensor. Two launches: each CTA of the first
// leaves one 64-bit partial; each CTA of the second adds all partials in the
// same order (so all get the same norm, and the same in every run), and the
// clip scales with it, rounding products to fp32 and then to the type. Nothing
// is read back to the host. A clip of little data is one launch of a cluster of
// eight CTAs, which exchange their partials through each other's shared memory.
//
// Both are bound by memory: the norm reads each gradient once, the clip reads
// and writes it once more. The tensors are cut into chunks of 32 KB of source
// (256 threads x 8 loads of 16 bytes, all in flight before the first is
// used); a table of the tensors and of their first chunks travels in the
// kernel's parameters, so that a call copies nothing to the device and can be
// captured into a graph. The clip takes the chunks from the last to the first:
// what the norm read last is still in L2.
//
// Sums: a thread adds the at most 64 terms of a chunk in 32 bits and those
// sums in 64 bits. Where a 32-bit sum overflows or is so small that squares
// below the normal range could matter, the thread reads the same values again
// (the caches hold them) and adds them in 64 bits: the norm of gradients around
// 1e25 or 1e-25 is right as well.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grads_internal.h"
#include "tc_ptx.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kGradChunkBytes / (kThreads * 16);  // 16-byte loads per thread

template <int DT>
struct Elem;
template <>
struct Elem<FLCE_F32> {
  using T = float;
  static constexpr int kPer16 = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float to_f(T x) { return x; }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Elem<FLCE_BF16> {
  using T = __nv_bfloat16;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float to_f(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Elem<FLCE_F16> {
  using T = __half;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float to_f(T x) { return __half2float(x); }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 b = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ void store_one(void* dst, int dtype, int64_t i, float x) {
  if (dtype == FLCE_F32)
    static_cast<float*>(dst)[i] = x;
  else if (dtype == FLCE_BF16)
    static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16(x);
  else
    static_cast<__half*>(dst)[i] = __float2half(x);
}

// One term of the sum (P = 1, 2), or of the maximum (P = 0: |x| with NaN
// above infinity, which the order of the bits gives).
template <int P>
struct Acc {
  float s = 0.0f;
  uint32_t m = 0;
  __device__ __forceinline__ void add(float x) {
    if constexpr (P == 0)
      m = max(m, __float_as_uint(x) & 0x7fffffffu);
    else if constexpr (P == 1)
      s += fabsf(x);
    else
      s = fmaf(x, x, s);
  }
};

// A 32-bit sum that has to be taken again in 64 bits. For p = 2 a term below
// the normal range is off by up to 2^-126: 64 of them are within 2^-27 of a
// sum of at least 2^-93.
template <int P>
__device__ __forceinline__ bool recount(float s) {
  if constexpr (P == 1) return !(s < 3.0e38f);
  if constexpr (P == 2) return !(s < 3.0e38f) || s < 1.0e-28f;
  return false;
}

template <int P>
__device__ __forceinline__ double term64(float x) {
  const double d = static_cast<double>(x);
  return P == 1 ? fabs(d) : d * d;
}

// Elements from p to the next 128-byte line, at most n: the 16-byte accesses of
// a warp then cover whole lines.
template <class T>
__device__ __forceinline__ int to_line(const T* p, int n) {
  const int head =
      static_cast<int>(((128u - (reinterpret_cast<uintptr_t>(p) & 127u)) & 127u) / sizeof(T));
  return head < n ? head : n;
}

// The partial of one chunk: elements [e0, e1) of tensor t. Ordinary loads: the
// cluster's kernel writes the same memory afterwards.
template <int P, int DT>
__device__ __forceinline__ void chunk_norm(const GradEntry& t, int64_t e0, int64_t e1,
                                           double& sum, uint32_t& peak) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16;
  const T* const src = static_cast<const T*>(t.src);
  if (t.cols < t.n) {  // rows with a pitch: one element at a time
    Acc<P> a;
    double extra = 0.0;
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
      const int64_t r = e / t.cols;
      const float x = E::to_f(src[r * t.src_pitch + (e - r * t.cols)]);
      if constexpr (P == 0)
        a.add(x);
      else
        extra += term64<P>(x);
    }
    sum += extra;
    peak = max(peak, a.m);
    return;
  }
  // elements before the first line, whole groups of 16 bytes, and the rest
  const T* const p = src + e0;
  const int n = static_cast<int>(e1 - e0);
  const int head = to_line(p, n);
  const int groups = (n - head) / N;
  const uint4* const v = reinterpret_cast<const uint4*>(p + head);
  uint4 q[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int g = static_cast<int>(threadIdx.x) + i * kThreads;
    q[i] = g < groups ? v[g] : make_uint4(0, 0, 0, 0);
  }
  const int rest = n - groups * N;  // head and tail elements: at most 70
  float edge = 0.0f;
  if (static_cast<int>(threadIdx.x) < rest) {
    const int i = static_cast<int>(threadIdx.x);
    edge = E::to_f(p[i < head ? i : groups * N + i]);
  }
  Acc<P> a[4];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float x[N];
    E::unpack(q[i], x);
#pragma unroll
    for (int j = 0; j < N; ++j) a[j & 3].add(x[j]);
  }
  if constexpr (P == 0) {
    a[0].add(edge);
    peak = max(peak, max(max(a[0].m, a[1].m), max(a[2].m, a[3].m)));
  } else {
    const float s = (a[0].s + a[1].s) + (a[2].s + a[3].s);
    bool again = recount<P>(s);
    if (P == 2 && s == 0.0f) {  // all zero is common (unused embedding rows) and needs no recount
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) any |= q[i].x | q[i].y | q[i].z | q[i].w;
      again = (any & (DT == FLCE_F32 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
    }
    if (again) {
      double d = 0.0;
#pragma unroll 1
      for (int i = 0; i < kVecs; ++i) {
        const int g = static_cast<int>(threadIdx.x) + i * kThreads;
        if (g >= groups) break;
        float x[N];
        E::unpack(v[g], x);
#pragma unroll
        for (int j = 0; j < N; ++j) d += term64<P>(x[j]);
      }
      sum += d;
    } else {
      sum += static_cast<double>(s);
    }
    if (edge != 0.0f) sum += term64<P>(edge);
  }
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the CTA, on every thread.
__device__ __forceinline__ double block_sum(double x, double* buf) {
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += buf[w];
  return t;
}
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* buf) {
  x = __reduce_max_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t = max(t, buf[w]);
  return t;
}

// The tensor that chunk c belongs to.
template <int CAP>
__device__ __forceinline__ int find_tensor(const GradTable<CAP>& tab, uint32_t c) {
  int lo = 0, hi = tab.count;  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void chunk_range(const GradEntry& t, uint32_t c, uint32_t first,
                                            int64_t& e0, int64_t& e1) {
  const int64_t len = kGradChunkBytes / (t.src_dtype == FLCE_F32 ? 4 : 2);
  e0 = static_cast<int64_t>(c - first) * len;
  e1 = e0 + len < t.n ? e0 + len : t.n;
}

template <int P>
__device__ __forceinline__ void any_chunk_norm(const GradEntry& t, int64_t e0, int64_t e1,
                                               double& sum, uint32_t& peak) {
  if (t.src_dtype == FLCE_F32)
    chunk_norm<P, FLCE_F32>(t, e0, e1, sum, peak);
  else if (t.src_dtype == FLCE_BF16)
    chunk_norm<P, FLCE_BF16>(t, e0, e1, sum, peak);
  else
    chunk_norm<P, FLCE_F16>(t, e0, e1, sum, peak);
}

// partials[blockIdx.x]: the sum of powers of this CTA's chunks, or for
// P = 0 the bits of their largest magnitude.
template <int P, int CAP>
__global__ void __launch_bounds__(kThreads, kGradNormCtasPerSm)
    grad_partials_kernel(const __grid_constant__ GradTable<CAP> tab, double* partials) {
  __shared__ double buf[kThreads / 32];
  grid_launch_dependents();
  double sum = 0.0;
  uint32_t peak = 0;
  for (uint32_t c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
    const int i = find_tensor(tab, c);
    const GradEntry& t = tab.t[i];
    int64_t e0, e1;
    chunk_range(t, c, tab.first[i], e0, e1);
    any_chunk_norm<P>(t, e0, e1, sum, peak);
  }
  if constexpr (P == 0) {
    peak = block_max(peak, reinterpret_cast<uint32_t*>(buf));
    if (threadIdx.x == 0) partials[blockIdx.x] = static_cast<double>(__uint_as_float(peak));
  } else {
    sum = block_sum(sum, buf);
    if (threadIdx.x == 0) partials[blockIdx.x] = sum;
  }
}

// The norm from all partials: the same additions in the same order in every
// CTA that calls it.
__device__ __forceinline__ float norm_of(const double* partials, int n, int p, double* buf) {
  if (p == 0) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i < n; i += kThreads)
      m = max(m, __float_as_uint(static_cast<float>(partials[i])));
    return __uint_as_float(block_max(m, reinterpret_cast<uint32_t*>(buf)));
  }
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partials[i];
  s = block_sum(s, buf);
  return static_cast<float>(p == 2 ? sqrt(s) : s);
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const double* partials, int n, int p, float* norm_out) {
  __shared__ double buf[kThreads / 32];
  grid_dependency_wait();
  const float norm = norm_of(partials, n, p, buf);
  if (threadIdx.x == 0) *norm_out = norm;
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const GradEntry& t, int64_t e0, int64_t e1,
                                            float coef) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int N = E::kPer16;
  const T* const src = static_cast<const T*>(t.src);
  if (t.cols < t.n) {
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
      const int64_t r = e / t.cols, c = e - r * t.cols;
      store_one(t.dst, t.dst_dtype, r * t.dst_pitch + c, E::to_f(src[r * t.src_pitch + c]) * coef);
    }
    return;
  }
  const T* const p = src + e0;
  const int n = static_cast<int>(e1 - e0);
  const int head = to_line(p, n);
  const int groups = (n - head) / N;
  const uint4* const v = reinterpret_cast<const uint4*>(p + head);
  uint4 q[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int g = static_cast<int>(threadIdx.x) + i * kThreads;
    if (g < groups) q[i] = v[g];
  }
  const int rest = n - groups * N;
  const int ei = static_cast<int>(threadIdx.x) < head ? static_cast<int>(threadIdx.x)
                                                      : groups * N + static_cast<int>(threadIdx.x);
  float edge = 0.0f;
  if (static_cast<int>(threadIdx.x) < rest) edge = E::to_f(p[ei]);
  const bool same = t.dst_dtype == DT;
  const int64_t d0 = e0 + head;  // first element of the groups
  const bool vec = same && ((reinterpret_cast<uintptr_t>(t.dst) + d0 * sizeof(T)) & 15u) == 0;
  const bool wide = !same && t.dst_dtype == FLCE_F32 &&
                    ((reinterpret_cast<uintptr_t>(t.dst) + d0 * 4) & 15u) == 0;
  // each kind of store in a loop of its own: merged, they become single ones
  auto each = [&](auto put) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int g = static_cast<int>(threadIdx.x) + i * kThreads;
      if (g >= groups) break;
      float x[N];
      E::unpack(q[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] *= coef;
      put(g, x);
    }
  };
  if (vec) {
    uint4* const o = reinterpret_cast<uint4*>(static_cast<T*>(t.dst) + d0);
    each([&](int g, const float(&x)[N]) { o[g] = E::pack(x); });
  } else if (wide) {
    float4* const o = reinterpret_cast<float4*>(static_cast<float*>(t.dst) + d0);
    each([&](int g, const float(&x)[N]) {
#pragma unroll
      for (int j = 0; j < N; j += 4)
        o[g * (N / 4) + j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    });
  } else {
    each([&](int g, const float(&x)[N]) {
#pragma unroll
      for (int j = 0; j < N; ++j) store_one(t.dst, t.dst_dtype, d0 + g * N + j, x[j]);
    });
  }
  if (static_cast<int>(threadIdx.x) < rest) store_one(t.dst, t.dst_dtype, e0 + ei, edge * coef);
}

__device__ __forceinline__ void any_chunk_scale(const GradEntry& t, int64_t e0, int64_t e1,
                                                float coef) {
  if (t.src_dtype == FLCE_F32)
    chunk_scale<FLCE_F32>(t, e0, e1, coef);
  else if (t.src_dtype == FLCE_BF16)
    chunk_scale<FLCE_BF16>(t, e0, e1, coef);
  else
    chunk_scale<FLCE_F16>(t, e0, e1, coef);
}

// min(1, max_norm / (norm + eps)); NaN stays NaN. All gradients 0 and eps 0
// leave nothing to scale, whatever max_norm is.
__device__ __forceinline__ float clip_factor(float norm, float max_norm, float eps) {
  if (norm + eps == 0.0f) return 1.0f;
  const float coef = max_norm / (norm + eps);
  return coef > 1.0f ? 1.0f : coef;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kGradClipCtasPerSm)
    grad_clip_kernel(const __grid_constant__ GradTable<CAP> tab, const double* partials, int n,
                     int p, float max_norm, float eps, float* norm_out, int write_norm) {
  __shared__ double buf[kThreads / 32];
  grid_dependency_wait();
  const float norm = norm_of(partials, n, p, buf);
  if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float coef = clip_factor(norm, max_norm, eps);
  if (tab.in_place && coef == 1.0f) return;
  const uint32_t total = tab.first[tab.count];
  for (uint32_t k = blockIdx.x; k < total; k += gridDim.x) {
    const uint32_t c = total - 1 - k;
    const int i = find_tensor(tab, c);
    const GradEntry& t = tab.t[i];
    int64_t e0, e1;
    chunk_range(t, c, tab.first[i], e0, e1);
    any_chunk_scale(t, e0, e1, coef);
  }
}

// Norm and clip in one launch of one cluster: rank r takes chunks r, r + 8, ...
template <int P, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    grad_clip_cluster_kernel(const __grid_constant__ GradTable<CAP> tab, float max_norm, float eps,
                             float* norm_out) {
  __shared__ double buf[kThreads / 32];
  __shared__ double all[kGradCluster];  // every rank's partial
  // every CTA of the cluster has started before any writes to another's memory
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const uint32_t rank = cluster_ctarank();
  const uint32_t total = tab.first[tab.count];
  double sum = 0.0;
  uint32_t peak = 0;
  for (uint32_t c = rank; c < total; c += kGradCluster) {
    const int i = find_tensor(tab, c);
    int64_t e0, e1;
    chunk_range(tab.t[i], c, tab.first[i], e0, e1);
    any_chunk_norm<P>(tab.t[i], e0, e1, sum, peak);
  }
  if constexpr (P == 0)
    sum = static_cast<double>(__uint_as_float(block_max(peak, reinterpret_cast<uint32_t*>(buf))));
  else
    sum = block_sum(sum, buf);
  asm volatile("barrier.cluster.wait;" ::: "memory");
  if (threadIdx.x < kGradCluster) {
    const uint32_t to = map_to_rank(smem_addr(&all[rank]), threadIdx.x);
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(sum) : "memory");
  }
  cluster_sync();
  double t = all[0];
#pragma unroll
  for (int r = 1; r < kGradCluster; ++r) {
    if constexpr (P == 0)  // magnitudes, NaN above infinity
      t = __double_as_longlong(all[r]) > __double_as_longlong(t) ? all[r] : t;
    else
      t += all[r];
  }
  const float norm = static_cast<float>(P == 2 ? sqrt(t) : t);
  if (rank == 0 && threadIdx.x == 0) *norm_out = norm;
  const float coef = clip_factor(norm, max_norm, eps);
  if (tab.in_place && coef == 1.0f) return;
  for (uint32_t c = rank; c < total; c += kGradCluster) {
    const int i = find_tensor(tab, c);
    int64_t e0, e1;
    chunk_range(tab.t[i], c, tab.first[i], e0, e1);
    any_chunk_scale(tab.t[i], e0, e1, coef);
  }
}

// A launch that may be placed while the kernel before it drains; it waits for
// that kernel's end before it reads anything.
template <class... P, class... A>
cudaError_t launch_after(void (*kern)(P...), unsigned grid, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int CAP>
unsigned grid_of(const GradTable<CAP>& tab, int max_ctas) {
  const uint32_t chunks = tab.first[tab.count];
  return chunks < static_cast<uint32_t>(max_ctas) ? chunks : static_cast<unsigned>(max_ctas);
}

}  // namespace

template <int CAP>
cudaError_t launch_grad_partials(const GradTable<CAP>& tab, int p, int max_ctas, double* partials,
                                 int* n_partials, cudaStream_t s) {
  const unsigned grid = grid_of(tab, max_ctas);
  *n_partials = static_cast<int>(grid);
  if (p == 0)
    grad_partials_kernel<0, CAP><<<grid, kThreads, 0, s>>>(tab, partials);
  else if (p == 1)
    grad_partials_kernel<1, CAP><<<grid, kThreads, 0, s>>>(tab, partials);
  else
    grad_partials_kernel<2, CAP><<<grid, kThreads, 0, s>>>(tab, partials);
  return cudaGetLastError();
}

cudaError_t launch_grad_norm(const double* partials, int n, int p, float* norm_out,
                             cudaStream_t s) {
  return launch_after(grad_norm_kernel, 1, s, partials, n, p, norm_out);
}

template <int CAP>
cudaError_t launch_grad_clip(const GradTable<CAP>& tab, const double* partials, int n, int p,
                             float max_norm, float eps, float* norm_out, bool write_norm,
                             int max_ctas, cudaStream_t s) {
  return launch_after(grad_clip_kernel<CAP>, grid_of(tab, max_ctas), s, tab, partials, n, p,
                      max_norm, eps, norm_out, write_norm ? 1 : 0);
}

cudaError_t launch_grad_clip_cluster(const GradTable<kGradTableSmall>& tab, int p, float max_norm,
                                     float eps, float* norm_out, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(kGradCluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kGradCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = p == 0   ? grad_clip_cluster_kernel<0, kGradTableSmall>
              : p == 1 ? grad_clip_cluster_kernel<1, kGradTableSmall>
                       : grad_clip_cluster_kernel<2, kGradTableSmall>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tab, max_norm, eps, norm_out);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template cudaError_t launch_grad_partials(const GradTable<kGradTableSmall>&, int, int, double*,
                                          int*, cudaStream_t);
template cudaError_t launch_grad_partials(const GradTable<kGradTableMedium>&, int, int, double*,
                                          int*, cudaStream_t);
template cudaError_t launch_grad_partials(const GradTable<kGradTableLarge>&, int, int, double*,
                                          int*, cudaStream_t);
template cudaError_t launch_grad_clip(const GradTable<kGradTableSmall>&, const double*, int, int,
                                      float, float, float*, bool, int, cudaStream_t);
template cudaError_t launch_grad_clip(const GradTable<kGradTableMedium>&, const double*, int, int,
                                      float, float, float*, bool, int, cudaStream_t);
template cudaError_t launch_grad_clip(const GradTable<kGradTableLarge>&, const double*, int, int,
                                      float, float, float*, bool, int, cudaStream_t);

}  // namespace flce
