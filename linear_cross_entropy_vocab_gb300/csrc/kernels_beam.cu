// One step of a beam search over the vocabulary, and the reordering of the
// states that its choice asks for.
//
// Selection. For each prompt b, over its K beams and V tokens:
//
//   s_kv = score_bk + (z_kv - lse_k),   lse_k = log sum_v e^{z_kv}
//
// and the M largest s_kv, equal ones in the order of k V + v. Within a beam
// the order of s is the order of the logits, so the first kernel never needs
// lse: it reads each logit once, keeps the M best of a slice of the row with
// their indices, and the slice's maximum and sum of exponentials. The second
// takes one prompt: lse of each beam from its slices, the scores of the
// K x slices x M survivors in 64 bits (what is chosen hangs on comparisons
// that 32 bits would decide by rounding), and the M best of them.
//
// Finding the M best without sorting: the threads are put into G >= M groups;
// the smallest of the groups' maxima has at least M values at or above it, and
// about G ln G of them for values in no particular order. Those few go into a
// buffer, and a key's place is the number of larger keys in it. Keys hold the
// value's order and the complement of the index, so they are all different
// and ties go to the lowest index. Where the buffer would overflow (thousands
// of equal logits at the top), the M best are taken one after the other.
//
// Bound: the logits are read once. A thread holds its part of the slice in
// registers, so that nothing is read a second time.
//
// Reordering. state[b K + j] = state[b K + parent_bj], in place: a thread owns
// the same 16 bytes (or less, by alignment) of all K beams of a prompt, reads
// what moves, and only then writes. Beams that continue themselves are neither
// read nor written.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam_internal.h"
#include "flce_math.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBuffer = 2048;  // keys that may pass a slice's threshold

// Order-preserving bits of a float that is not NaN (-0 counts as +0).
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
  return (static_cast<uint64_t>(order_bits(x)) << 32) | (0xffffffffu - index);
}

template <class T>
struct Load8;
template <>
struct Load8<float> {
  static __device__ __forceinline__ void vec(const float* p, float (&x)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldcs(p); }
};
template <>
struct Load8<__nv_bfloat16> {
  static __device__ __forceinline__ void vec(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
};
template <>
struct Load8<__half> {
  static __device__ __forceinline__ void vec(const __half* p, float (&x)[8]) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float one(const __half* p) { return __half2float(*p); }
};

// A value with its place in the order of all candidates: larger scores first,
// then lower indices.
struct Scored {
  double s;
  uint64_t at;
};
__device__ __forceinline__ bool better(const Scored& a, const Scored& b) {
  return a.s > b.s || (a.s == b.s && a.at < b.at);
}
__device__ __forceinline__ bool better(uint64_t a, uint64_t b) { return a > b; }

__device__ __forceinline__ Scored shfl_xor(const Scored& a, int o) {
  return Scored{__shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.at, o)};
}
__device__ __forceinline__ uint64_t shfl_xor(uint64_t a, int o) {
  return __shfl_xor_sync(0xffffffffu, a, o);
}

template <class K>
__device__ __forceinline__ K block_best(K x, K* warp_buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const K y = shfl_xor(x, o);
    if (better(y, x)) x = y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_buf[threadIdx.x >> 5] = x;
  __syncthreads();
  x = warp_buf[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w)
    if (better(warp_buf[w], x)) x = warp_buf[w];
  return x;
}

// Places of the n <= kBuffer different keys in buf: out(rank, key) for the
// ranks below m.
template <class K, class Out>
__device__ __forceinline__ void rank_keys(const K* buf, int n, int m, Out out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const K mine = buf[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += better(buf[j], mine) ? 1 : 0;
    if (rank < m) out(rank, mine);
  }
}

// The warps of a group of 256 / g threads (g a power of two, at most 256) and
// the smallest of the groups' maxima, for a 32-bit order: on every thread.
__device__ __forceinline__ uint32_t group_floor(uint32_t x, int g, uint32_t* warp_buf) {
  const int width = kThreads / g;  // threads per group
  for (int o = 1; o < 32 && o < width; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (width <= 32) {
    x = __reduce_min_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_buf[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t t = warp_buf[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) t = min(t, warp_buf[w]);
    return t;
  }
  // fewer groups than warps: the maximum of each run of width / 32 warps
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_buf[threadIdx.x >> 5] = x;
  __syncthreads();
  uint32_t t = 0xffffffffu;
  const int per = width / 32;
  for (int a = 0; a < kWarps; a += per) {
    uint32_t m = 0;
    for (int w = a; w < a + per; ++w) m = max(m, warp_buf[w]);
    t = min(t, m);
  }
  return t;
}

__device__ __forceinline__ int groups_for(int m) {
  int g = 1;
  while (g < m) g <<= 1;
  return g;
}

// One slice of one row: its M best logits, maximum and sum of exponentials.
// VECS groups of 8 logits per thread.
template <class T, int VECS>
__global__ void __launch_bounds__(kThreads, VECS == 1 ? 6 : 3)
    beam_slices_kernel(const BeamSelectParams p) {
  __shared__ uint64_t buf[kBuffer];
  __shared__ uint64_t warp_key[kWarps];
  __shared__ uint32_t warp_u32[kWarps];
  __shared__ float warp_f32[kWarps];
  __shared__ int count;
  const int64_t row = blockIdx.x / p.splits;
  const int slice = static_cast<int>(blockIdx.x - row * p.splits);
  const int b = static_cast<int>(row / p.beams), k = static_cast<int>(row - b * static_cast<int64_t>(p.beams));
  const float score = p.beam_scores[row];
  // a finished beam and one that cannot be continued need none of their logits
  if (p.finished != nullptr && p.finished[row] != 0) return;
  if (score == -INFINITY) return;
  const T* const z = static_cast<const T*>(p.logits) + b * p.stride_b + k * p.stride_k;
  const uint8_t* const ok =
      p.allowed != nullptr ? p.allowed + b * p.allowed_b + k * p.allowed_k : nullptr;
  const int64_t v0 = static_cast<int64_t>(slice) * (kThreads * 8 * VECS);
  const bool z16 = (reinterpret_cast<uintptr_t>(z) & 15u) == 0;
  const bool ok8 = ok != nullptr && (reinterpret_cast<uintptr_t>(ok) & 7u) == 0;
  float x[VECS][8];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int64_t v = v0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
    if (z16 && v + 8 <= p.v) {
      Load8<T>::vec(z + v, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = v + j < p.v ? Load8<T>::one(z + v + j) : -INFINITY;
    }
  }
  if (ok != nullptr) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int64_t v = v0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
      if (ok8 && v + 8 <= p.v) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(ok + v));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((((j < 4 ? a.x : a.y) >> (8 * (j & 3))) & 0xffu) == 0) x[i][j] = -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v + j < p.v && ok[v + j] == 0) x[i][j] = -INFINITY;
      }
    }
  }
  if (threadIdx.x == 0) count = 0;

  // maximum (NaN and +infinity make the row invalid: the stats say so)
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top = fmaxf(top, x[i][j]);
      bad |= !(x[i][j] < INFINITY);
    }
  bad = __syncthreads_or(bad ? 1 : 0) != 0;
  const int64_t out = row * p.splits + slice;
  uint64_t* const keys = p.keys + out * p.m;
  if (bad) {
    if (threadIdx.x == 0) p.stats[out] = make_float2(NAN, 0.0f);
    for (int i = threadIdx.x; i < p.m; i += kThreads) keys[i] = 0;
    return;
  }
  const uint32_t floor_bits = group_floor(order_bits(top), groups_for(p.m), warp_u32);
  float row_top = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    row_top = fmaxf(row_top, __shfl_xor_sync(0xffffffffu, row_top, o));
  if ((threadIdx.x & 31) == 0) warp_f32[threadIdx.x >> 5] = row_top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) row_top = fmaxf(row_top, warp_f32[w]);

  // what reaches the threshold, and the sum of exponentials
  const float at_least = from_order_bits(floor_bits);
  // the difference first: a rounded row_top * log2(e) would shift every term alike
  const float base = row_top == -INFINITY ? 0.0f : row_top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      part += ex2_approx((x[i][j] - base) * kLog2e);
      if (x[i][j] >= at_least && x[i][j] > -INFINITY) {
        const int place = atomicAdd(&count, 1);
        const int64_t v = v0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8 + j;
        if (place < kBuffer) buf[place] = make_key(x[i][j], static_cast<uint32_t>(v));
      }
    }
    sum += part;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();  // row_top has been read by all
  if ((threadIdx.x & 31) == 0) warp_f32[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += warp_f32[w];
    p.stats[out] = make_float2(row_top, s);
  }
  const int n = count;
  if (n <= kBuffer) {
    rank_keys(buf, n, p.m, [&](int rank, uint64_t key) { keys[rank] = key; });
    for (int i = n + threadIdx.x; i < p.m; i += kThreads) keys[i] = 0;
    return;
  }
  // more equal values than the buffer holds: one after the other
  uint64_t last = ~0ull;
  for (int r = 0; r < p.m; ++r) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t v = v0 + (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8 + j;
        const uint64_t key = make_key(x[i][j], static_cast<uint32_t>(v));
        if (x[i][j] > -INFINITY && key < last && key > best) best = key;
      }
    best = block_best(best, warp_key);
    if (threadIdx.x == 0) keys[r] = best;
    last = best;
  }
}

// The M best of one prompt from its beams' slices.
__global__ void __launch_bounds__(kThreads) beam_choose_kernel(const BeamSelectParams p) {
  __shared__ Scored buf[kBuffer];
  __shared__ Scored warp_best[kWarps];
  // lse = top + log_sum of each beam, kept apart: next to a large top the sum's
  // logarithm would be lost even in 64 bits
  __shared__ double log_sum[kBeamMaxSelectBeams];
  __shared__ float row_top[kBeamMaxSelectBeams];
  __shared__ int count;
  const int b = blockIdx.x;
  if (threadIdx.x == 0) count = 0;
  // log_sum is NaN for a beam that offers nothing, +infinity for a finished one
  int err = 0;
  for (int k = threadIdx.x; k < p.beams; k += kThreads) {
    const int64_t row = static_cast<int64_t>(b) * p.beams + k;
    const float score = p.beam_scores[row];
    double l = NAN;
    float top = -INFINITY;
    if (!(score < INFINITY)) {
      err |= FLCE_DEVERR_NOT_FINITE;
    } else if (score > -INFINITY) {
      if (p.finished != nullptr && p.finished[row] != 0) {
        l = INFINITY;
      } else {
        bool bad = false;
        for (int i = 0; i < p.splits; ++i) {
          const float m = p.stats[row * p.splits + i].x;
          bad |= !(m < INFINITY);
          top = fmaxf(top, m);
        }
        if (bad) {
          err |= FLCE_DEVERR_NOT_FINITE;
        } else if (top > -INFINITY) {
          double s = 0.0;
          for (int i = 0; i < p.splits; ++i) {
            const float2 st = p.stats[row * p.splits + i];
            if (st.x > -INFINITY)
              s += static_cast<double>(st.y) * exp(static_cast<double>(st.x) - static_cast<double>(top));
          }
          l = log(s);
        }
      }
    }
    log_sum[k] = l;
    row_top[k] = top;
  }
  if (err != 0 && p.err_word != nullptr) atomicOr(p.err_word, err);
  __syncthreads();

  const int per_beam = p.splits * p.m;
  const int64_t total = static_cast<int64_t>(p.beams) * per_beam;
  const Scored none{-INFINITY, ~0ull};
  auto candidate = [&](int64_t c) -> Scored {
    const int k = static_cast<int>(c / per_beam);
    const int64_t row = static_cast<int64_t>(b) * p.beams + k;
    const double l = log_sum[k];
    if (isnan(l)) return none;
    const double score = static_cast<double>(p.beam_scores[row]);
    if (isinf(l))
      return c == static_cast<int64_t>(k) * per_beam
                 ? Scored{score, static_cast<uint64_t>(k) * p.v + p.pad_token}
                 : none;
    const uint64_t key = p.keys[row * per_beam + (c - static_cast<int64_t>(k) * per_beam)];
    if (key == 0) return none;
    const double zv = static_cast<double>(from_order_bits(static_cast<uint32_t>(key >> 32)));
    const uint32_t v = 0xffffffffu - static_cast<uint32_t>(key);
    return Scored{score + ((zv - static_cast<double>(row_top[k])) - l), static_cast<uint64_t>(k) * p.v + v};
  };
  // the thread's candidates: a rotation, because the keys of a slice are in
  // order and the groups shall see all ranks alike
  auto place_of = [&](int64_t round) -> int64_t {
    return round * kThreads + ((threadIdx.x + static_cast<unsigned>(round) * 97u) & (kThreads - 1));
  };
  const int64_t rounds = (total + kThreads - 1) / kThreads;
  Scored best = none;
  for (int64_t r = 0; r < rounds; ++r) {
    const int64_t c = place_of(r);
    if (c >= total) continue;
    const Scored x = candidate(c);
    if (better(x, best)) best = x;
  }
  // the smallest of the groups' best
  const int width = kThreads / groups_for(p.m);
  for (int o = 1; o < 32 && o < width; o <<= 1) {
    const Scored y = shfl_xor(best, o);
    if (better(y, best)) best = y;
  }
  if (width <= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Scored y = shfl_xor(best, o);
      if (better(best, y)) best = y;
    }
  }
  if ((threadIdx.x & 31) == 0) warp_best[threadIdx.x >> 5] = best;
  __syncthreads();
  const int per = width > 32 ? width / 32 : 1;
  Scored floor_at = none;
  for (int a = 0; a < kWarps; a += per) {
    Scored m = warp_best[a];
    for (int w = a + 1; w < a + per; ++w)
      if (better(warp_best[w], m)) m = warp_best[w];
    if (a == 0 || better(floor_at, m)) floor_at = m;
  }
  for (int64_t r = 0; r < rounds; ++r) {
    const int64_t c = place_of(r);
    if (c >= total) continue;
    const Scored x = candidate(c);
    if (x.s > -INFINITY && !better(floor_at, x)) {
      const int place = atomicAdd(&count, 1);
      if (place < kBuffer) buf[place] = x;
    }
  }
  __syncthreads();
  const int64_t o0 = static_cast<int64_t>(b) * p.m;
  auto emit = [&](int rank, const Scored& x) {
    const uint64_t k = x.at / static_cast<uint64_t>(p.v);
    p.scores_out[o0 + rank] = static_cast<float>(x.s);
    p.parents_out[o0 + rank] = static_cast<int64_t>(k);
    p.tokens_out[o0 + rank] = static_cast<int64_t>(x.at - k * static_cast<uint64_t>(p.v));
  };
  auto emit_none = [&](int rank) {
    p.scores_out[o0 + rank] = -INFINITY;
    p.parents_out[o0 + rank] = 0;
    p.tokens_out[o0 + rank] = p.pad_token;
  };
  const int n = count;
  if (n <= kBuffer) {
    rank_keys(buf, n, p.m, emit);
    for (int i = n + threadIdx.x; i < p.m; i += kThreads) emit_none(i);
    return;
  }
  Scored last{INFINITY, 0};
  for (int r = 0; r < p.m; ++r) {
    Scored x = none;
    for (int64_t q = 0; q < rounds; ++q) {
      const int64_t c = place_of(q);
      if (c >= total) continue;
      const Scored y = candidate(c);
      if (better(last, y) && better(y, x)) x = y;
    }
    x = block_best(x, warp_best);
    if (threadIdx.x == 0) {
      if (x.s > -INFINITY)
        emit(r, x);
      else
        emit_none(r);
    }
    last = x;
  }
}

template <class T>
cudaError_t launch_select(const BeamSelectParams& p, bool large, cudaStream_t s) {
  const int64_t blocks = static_cast<int64_t>(p.batch) * p.beams * p.splits;
  if (large)
    beam_slices_kernel<T, kSliceLarge / (8 * kThreads)>
        <<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  else
    beam_slices_kernel<T, kSliceSmall / (8 * kThreads)>
        <<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  beam_choose_kernel<<<static_cast<unsigned>(p.batch), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------- reordering
template <int W>
struct Vec;
template <>
struct Vec<16> { using T = uint4; };
template <>
struct Vec<8> { using T = uint2; };
template <>
struct Vec<4> { using T = uint32_t; };
template <>
struct Vec<2> { using T = uint16_t; };
template <>
struct Vec<1> { using T = uint8_t; };

// KM: an upper bound of the beams; a thread holds one vector of each.
template <int W, int KM>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ ReorderTable t) {
  using V = typename Vec<W>::T;
  __shared__ int parent[KM];
  int lo = 0, hi = t.count;  // the state of this block
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid;
  }
  const ReorderEntry& e = t.e[lo];
  const uint32_t blocks_per_prompt = (e.total + kReorderBlock - 1) / kReorderBlock;
  const uint32_t u = blockIdx.x - t.first[lo];
  const uint32_t b = u / blocks_per_prompt;
  const uint32_t c = (u - b * blocks_per_prompt) * kReorderBlock + threadIdx.x;
  if (static_cast<int>(threadIdx.x) < t.beams) {
    const int j = static_cast<int>(threadIdx.x);
    const int64_t q = t.parents[static_cast<int64_t>(b) * t.beams + j];
    const bool valid = q >= 0 && q < t.beams;
    parent[j] = valid ? static_cast<int>(q) : j;
    if (!valid && t.err_word != nullptr) atomicOr(t.err_word, FLCE_DEVERR_PARENT_RANGE);
  }
  __syncthreads();
  if (c >= e.total) return;
  uint32_t outer = c / e.run;
  int64_t at = static_cast<int64_t>(c - outer * e.run) * W;
#pragma unroll
  for (int d = kReorderDims - 1; d >= 0; --d) {
    if (e.size[d] > 1) {
      const uint32_t up = outer / e.size[d];
      at += static_cast<int64_t>(outer - up * e.size[d]) * e.stride[d];
      outer = up;
    }
  }
  uint8_t* const base = e.data + static_cast<int64_t>(b) * t.beams * e.beam_stride + at;
  V v[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < t.beams && parent[j] != j)
      v[j] = *reinterpret_cast<const V*>(base + parent[j] * e.beam_stride);
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < t.beams && parent[j] != j) *reinterpret_cast<V*>(base + j * e.beam_stride) = v[j];
}

template <int W>
cudaError_t launch_reorder(const ReorderTable& t, unsigned blocks, cudaStream_t s) {
  if (t.beams <= 4)
    beam_reorder_kernel<W, 4><<<blocks, kThreads, 0, s>>>(t);
  else if (t.beams <= 8)
    beam_reorder_kernel<W, 8><<<blocks, kThreads, 0, s>>>(t);
  else if (t.beams <= 16)
    beam_reorder_kernel<W, 16><<<blocks, kThreads, 0, s>>>(t);
  else if (t.beams <= 32)
    beam_reorder_kernel<W, 32><<<blocks, kThreads, 0, s>>>(t);
  else if constexpr (W <= 8)
    beam_reorder_kernel<W, 64><<<blocks, kThreads, 0, s>>>(t);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, bool large,
                               cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_select<float>(p, large, s);
  if (dtype == FLCE_BF16) return launch_select<__nv_bfloat16>(p, large, s);
  return launch_select<__half>(p, large, s);
}

cudaError_t launch_beam_reorder(const ReorderTable& t, int width, int64_t blocks,
                                cudaStream_t s) {
  const unsigned n = static_cast<unsigned>(blocks);
  switch (width) {
    case 16: return launch_reorder<16>(t, n, s);
    case 8: return launch_reorder<8>(t, n, s);
    case 4: return launch_reorder<4>(t, n, s);
    case 2: return launch_reorder<2>(t, n, s);
    default: return launch_reorder<1>(t, n, s);
  }
}

}  // namespace flce
