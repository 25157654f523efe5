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
// K x slices x M survivors, and the M best of them.
//
// A slice's sum is made of ex2.approx values (2^-22 each) added in 32 bits, so
// that lse is right to some 1e-6 and candidates of two beams closer than 1e-5
// may change places. What follows is in 64 bits, where scores of different
// logits of one beam stay different: in 32 bits rounding would make them equal
// and hand the choice to the index.
//
// Finding the M best of a tile: the threads are put into G >= M groups; the
// smallest of the groups' maxima has at least M values at or above it, and
// about G ln G of them for values in no particular order. Those few go into a
// buffer and are sorted there: up to 128 by counting, for each key, the keys
// above it, more by a bitonic network. Keys hold the value's order and the
// complement of the index, so they are all different and ties go to the lowest
// index. A slice is several tiles; after 1, 2, 4, ... of them the threshold
// becomes the M-th best so far, so that about M values pass it between two
// such points. Where the buffer would overflow (thousands of equal logits at
// the top), the M best of the slice are taken one after the other.
//
// Bound: the logits are read once, each thread's 16-byte pieces of the next
// tile while it works on this one. Per logit there are two additions, a
// product, an exponential and a maximum; whether a value reaches the threshold
// is asked once for a piece. With half of the issue slots used, what bounds a
// large call is the CTAs' progress from tile to tile (more loads on their way,
// through registers or shared memory, gained nothing); a small one is bound by
// the chain from the loads through two launches.
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
constexpr int kBuffer = 4096;  // keys that may pass a slice's threshold
constexpr int kChoiceBuffer = 2048;
constexpr int kHeld = 4;       // candidates that a thread of the choice keeps in registers

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

// 16 bytes of logits as floats, and one logit.
template <class T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int kElems = 4;
  static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[4]) {
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
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
struct Piece<__half> {
  static constexpr int kElems = 8;
  static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
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

// A score with its place in the order of all candidates: larger scores first,
// then lower indices. Scores are kept as the order of their 64 bits (integer
// comparisons; this GPU compares few doubles a cycle).
struct Scored {
  uint64_t s;   // 0: nothing
  uint64_t at;  // beam in the upper 32 bits, token in the lower
};
__device__ __forceinline__ uint64_t order_bits64(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double from_order_bits64(uint64_t o) {
  return __longlong_as_double(
      static_cast<long long>(o ^ ((o >> 63) ? 0x8000000000000000ull : ~0ull)));
}
__device__ __forceinline__ bool better(const Scored& a, const Scored& b) {
  return a.s > b.s || (a.s == b.s && a.at < b.at);
}
__device__ __forceinline__ bool better(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ bool better(uint32_t a, uint32_t b) { return a > b; }
__device__ __forceinline__ Scored nothing(const Scored&) { return Scored{0, ~0ull}; }
__device__ __forceinline__ uint64_t nothing(uint64_t) { return 0; }

__device__ __forceinline__ Scored shfl_xor(const Scored& a, int o) {
  return Scored{__shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.at, o)};
}
__device__ __forceinline__ uint64_t shfl_xor(uint64_t a, int o) {
  return __shfl_xor_sync(0xffffffffu, a, o);
}
__device__ __forceinline__ uint32_t shfl_xor(uint32_t a, int o) {
  return __shfl_xor_sync(0xffffffffu, a, o);
}

// A place in a shared list. Few lanes come here at a time: an atomic of each
// is shorter than agreeing on one.
__device__ __forceinline__ uint32_t take_place(int* count) {
  uint32_t r;
  asm volatile("atom.shared.add.u32 %0, [%1], 1;" : "=r"(r) : "r"(smem_addr(count)) : "memory");
  return r;
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

// Sorts the n keys in buf, which has room for the next power of two: a bitonic
// network. All threads of the CTA.
template <class K>
__device__ __forceinline__ void sort_keys(K* buf, int n) {
  int len = 256;
  while (len < n) len <<= 1;
  for (int i = n + static_cast<int>(threadIdx.x); i < len; i += kThreads) buf[i] = nothing(buf[0]);
  for (int size = 2; size <= len; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      __syncthreads();
      for (int q = static_cast<int>(threadIdx.x); q < len / 2; q += kThreads) {
        const int i = 2 * q - (q & (step - 1)), j = i + step;
        const K x = buf[i], y = buf[j];
        if (better(y, x) == ((i & size) == 0)) {
          buf[i] = y;
          buf[j] = x;
        }
      }
    }
  __syncthreads();
}

// The first m of the n different keys in buf (with room for the next power of
// two), in order:
// out(rank, key) for the ranks below m and n.
template <class K, class Out>
__device__ __forceinline__ void rank_keys(K* buf, int n, int m, Out out) {
  if (n <= 128) {
    const int i = static_cast<int>(threadIdx.x);
    if (i < n) {
      const K mine = buf[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += better(buf[j], mine) ? 1 : 0;
      if (rank < m) out(rank, mine);
    }
    return;
  }
  sort_keys(buf, n);
  for (int i = static_cast<int>(threadIdx.x); i < m && i < n; i += kThreads) out(i, buf[i]);
}

// The smallest of the maxima of g groups of threads (g a power of two, at most
// 256), on every thread. Thread t is in group t mod g: threads without a value
// lie together, at the end of a short slice, and leave no group empty. `red`
// has a place for each lane of each warp.
template <class K>
__device__ __forceinline__ K group_floor(K x, int g, K (*red)[32]) {
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  for (int o = 16; o >= g; o >>= 1) {
    const K y = shfl_xor(x, o);
    if (better(y, x)) x = y;
  }
  __syncthreads();
  red[warp][lane] = x;
  __syncthreads();
  const int classes = g > 32 ? g / 32 : 1;  // warps w and w + classes share their groups
  K floor_at = x;
  for (int c = 0; c < classes; ++c) {
    K m = red[c][lane];
    for (int w = c + classes; w < kWarps; w += classes) {
      const K y = red[w][lane];
      if (better(y, m)) m = y;
    }
    if (c == 0 || better(floor_at, m)) floor_at = m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const K y = shfl_xor(floor_at, o);
    if (better(floor_at, y)) floor_at = y;
  }
  return floor_at;
}

// The 16 bytes that start `s` bytes (0 to 15) into the 32 of a and b.
__device__ __forceinline__ uint4 shift_bytes(const uint4& a, const uint4& b, uint32_t s) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = (s & 8u) ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = (s & 4u) ? w[j + 1] : w[j];
  const uint32_t bits = 8u * (s & 3u);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// One slice of a row as the threads of a CTA see it; places count from its start.
template <class T>
struct Slice {
  static constexpr int E = Piece<T>::kElems;
  const T* z;
  const uint8_t* ok;  // or null
  int len;
  bool z16, ok_vec;   // 16-byte (E-byte) loads are aligned
  uint32_t shift;     // bytes from a multiple of 16 to the slice's start; 0 without SHIFT

  // The aligned 16 bytes that hold the first of the logits from v on (v a
  // multiple of E).
  __device__ __forceinline__ const uint4* chunk(int v) const {
    return reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(z + v) - shift);
  }
  __device__ __forceinline__ uint4 raw(int v) const { return __ldcs(chunk(v)); }
  // What lies past the end, and where the mask says so, is -infinity.
  __device__ __forceinline__ void mask(int v, float (&x)[E]) const {
    if (ok_vec && v + E <= len) {
      uint32_t a[2];
      a[0] = __ldg(reinterpret_cast<const uint32_t*>(ok + v));
      a[1] = E == 8 ? __ldg(reinterpret_cast<const uint32_t*>(ok + v) + 1) : 0;
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (((a[j >> 2] >> (8 * (j & 3))) & 0xffu) == 0) x[j] = -INFINITY;
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (v + j < len && ok[v + j] == 0) x[j] = -INFINITY;
    }
  }
  __device__ __forceinline__ void load(int v, float (&x)[E]) const {
    if (z16 && v + E <= len) {
      Piece<T>::unpack(raw(v), x);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = v + j < len ? Piece<T>::one(z + v + j) : -INFINITY;
    }
    if (ok != nullptr) mask(v, x);
  }
};

// One slice of one row: its M best logits, maximum and sum of exponentials.
// A tile is N pieces of 16 bytes per thread; the next tile's are on their way
// while one is worked on. SHIFT: rows may start anywhere, and a thread's logits
// come from two aligned pieces (64 x 8 rows of 128255 bf16: 58 us, value by
// value 80; of 128256 as aligned ones 46, by the shifting kernel 50). Two
// 16-bit pieces at six CTAs an SM spill two bytes of the 40 registers; with
// five and 48, which spill nothing, those aligned rows take 49 us and 32 of
// them 19, with six 47 and 14.
template <class T, int N, bool SHIFT>
__global__ void __launch_bounds__(kThreads, N == 4 ? 4 : N == 2 && SHIFT ? 5 : 6)
    beam_slices_kernel(const BeamSelectParams p) {
  constexpr int E = Piece<T>::kElems;
  constexpr int kTile = kThreads * E * N;
  __shared__ uint64_t buf[kBuffer];
  __shared__ uint64_t kept[kBeamMaxCandidates];
  __shared__ uint64_t warp_key[kWarps];
  __shared__ uint32_t red[kWarps][32];
  __shared__ float2 warp_stat[kWarps];
  __shared__ int count;
  grid_launch_dependents();
  const uint32_t row = blockIdx.x / static_cast<uint32_t>(p.splits);
  const uint32_t slice = blockIdx.x - row * static_cast<uint32_t>(p.splits);
  const uint32_t b = row / static_cast<uint32_t>(p.beams);
  const uint32_t k = row - b * static_cast<uint32_t>(p.beams);
  const float score = p.beam_scores[row];
  // a finished beam and one that cannot be continued need none of their logits
  if (p.finished != nullptr && p.finished[row] != 0) return;
  if (score == -INFINITY) return;
  const int64_t v0 = static_cast<int64_t>(slice) * p.slice_len;
  const uint32_t v0_32 = static_cast<uint32_t>(v0);
  Slice<T> in;
  in.z = static_cast<const T*>(p.logits) + b * p.stride_b + k * p.stride_k + v0;
  in.ok = p.allowed != nullptr ? p.allowed + b * p.allowed_b + k * p.allowed_k + v0 : nullptr;
  in.len = static_cast<int>(v0 + p.slice_len < p.v ? p.slice_len : p.v - v0);
  in.z16 = !SHIFT || (reinterpret_cast<uintptr_t>(in.z) & 15u) == 0;
  in.ok_vec = (reinterpret_cast<uintptr_t>(in.ok) & 3u) == 0;
  in.shift = SHIFT ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(in.z) & 15u) : 0u;
  if (threadIdx.x == 0) count = 0;

  // the thread's maximum so far and its sum of e^(z - maximum); NaN and
  // +infinity make the sum NaN
  float top = -INFINITY, sum = 0.0f;
  uint32_t floor_bits = 0;  // below every value's order
  bool full = false;
  int tiles = 0;
  uint4 next[N];
  const int mine = static_cast<int>(threadIdx.x) * E;
  // Whether the tile at t0 is loaded in 16 bytes, ahead of time: it is whole,
  // and in a row that starts elsewhere than at a multiple of 16 bytes, where a
  // thread's logits come from two such pieces, neither reaches past the row.
  const int64_t rest = p.v - v0 - E;
  const int limit = !SHIFT || in.z16 || rest >= in.len ? in.len : static_cast<int>(rest);
  const int start = !SHIFT || in.z16 || v0 > 0 ? 0 : 1;
  auto ahead = [&](int t0) { return t0 >= start && t0 + kTile <= limit; };
  if (ahead(0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) next[i] = in.raw(mine + i * kThreads * E);
  }
  for (int t0 = 0; t0 < in.len; t0 += kTile) {
    float x[N][E];
    if (ahead(t0)) {
      if (SHIFT && !in.z16) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          next[i] = shift_bytes(next[i], __ldg(in.chunk(t0 + mine + i * kThreads * E) + 1),
                                in.shift);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) Piece<T>::unpack(next[i], x[i]);
      if (in.ok != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) in.mask(t0 + mine + i * kThreads * E, x[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) in.load(t0 + mine + i * kThreads * E, x[i]);
    }
    if (ahead(t0 + kTile)) {
#pragma unroll
      for (int i = 0; i < N; ++i) next[i] = in.raw(t0 + kTile + mine + i * kThreads * E);
    }
    float piece_top[N], tile_top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      piece_top[i] = x[i][0];
#pragma unroll
      for (int j = 1; j < E; ++j) piece_top[i] = fmaxf(piece_top[i], x[i][j]);
      tile_top = fmaxf(tile_top, piece_top[i]);
    }
    if (tile_top > top) {
      sum *= ex2_approx((top - tile_top) * kLog2e);  // 0 while top is -infinity
      top = tile_top;
    }
    {
      // the difference first: a rounded maximum times log2(e) would shift
      // every term alike
      const float base = top == -INFINITY ? 0.0f : top;
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) part[j & 1] += ex2_approx((x[i][j] - base) * kLog2e);
      sum += part[0] + part[1];
    }

    // what reaches the threshold: the M-th best so far, once there are M
    if (!full) floor_bits = max(floor_bits, group_floor(order_bits(tile_top), p.groups, red));
    const float at_least = floor_bits == 0 ? -INFINITY : from_order_bits(floor_bits);
    if (tile_top >= at_least && tile_top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (piece_top[i] >= at_least) {
          const uint32_t v = v0_32 + static_cast<uint32_t>(t0 + mine + i * kThreads * E);
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (x[i][j] >= at_least && x[i][j] > -INFINITY) {
              const uint32_t place = take_place(&count);
              if (place < kBuffer) buf[place] = make_key(x[i][j], v + j);
            }
        }
    }
    // after every tile until there are M, then after 2, 4, 8, ... of them
    ++tiles;
    if (t0 + kTile < in.len && (!full || (tiles & (tiles - 1)) == 0)) {
      __syncthreads();
      const int n = count;
      __syncthreads();
      if (n > kBuffer) {
        // taken one after the other below: the rest is only summed (this floor
        // stands for a NaN, which nothing reaches)
        floor_bits = 0xffffffffu;
        full = true;
      } else if (n >= p.m && (!full || n > p.m)) {
        rank_keys(buf, n, p.m, [&](int rank, uint64_t key) { kept[rank] = key; });
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < p.m) buf[threadIdx.x] = kept[threadIdx.x];
        floor_bits = static_cast<uint32_t>(kept[p.m - 1] >> 32);
        full = true;
        if (threadIdx.x == 0) count = p.m;
        __syncthreads();
      }
    }
  }

  // the slice's statistics
  const bool bad = sum != sum;
  float all_top = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    all_top = fmaxf(all_top, __shfl_xor_sync(0xffffffffu, all_top, o));
  if (all_top > -INFINITY && !bad) sum *= ex2_approx((top - all_top) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) warp_stat[threadIdx.x >> 5] = make_float2(all_top, sum);
  __syncthreads();
  const int64_t out = static_cast<int64_t>(row) * p.splits + slice;
  uint64_t* const keys = p.keys + out * p.m;
  const int n = count;
  if (threadIdx.x == 0) {
    float m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_stat[w].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      total += warp_stat[w].x > -INFINITY || warp_stat[w].y != warp_stat[w].y
                   ? warp_stat[w].y * ex2_approx((warp_stat[w].x - m) * kLog2e)
                   : 0.0f;
    p.stats[out] = total == total && m < INFINITY ? make_float2(m, total) : make_float2(NAN, 0.0f);
  }
  if (n <= kBuffer) {
    rank_keys(buf, n, p.m, [&](int rank, uint64_t key) { keys[rank] = key; });
    for (int i = n + static_cast<int>(threadIdx.x); i < p.m; i += kThreads) keys[i] = 0;
    return;
  }
  // more equal values than the buffer holds: one after the other
  uint64_t last = ~0ull;
  for (int r = 0; r < p.m; ++r) {
    uint64_t best = 0;
    for (int v = mine; v < in.len; v += kThreads * E) {
      float x[E];
      in.load(v, x);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const uint64_t key = make_key(x[j], v0_32 + static_cast<uint32_t>(v + j));
        if (x[j] > -INFINITY && key < last && key > best) best = key;
      }
    }
    best = block_best(best, warp_key);
    if (threadIdx.x == 0) keys[r] = best;
    last = best;
  }
}

// log(s / 2^31) within 2^-24: the exponent's part in 64 bits, and a 32-bit
// logarithm of what is within a factor of sqrt(2) of 1.
__device__ __forceinline__ double log_of(unsigned long long s) {
  const float f = __ull2float_rn(s);
  const float rest = static_cast<float>(static_cast<long long>(s - __float2ull_rn(f))) / f;
  int e = static_cast<int>(__float_as_uint(f) >> 23) - 127;
  float m = __uint_as_float((__float_as_uint(f) & 0x007fffffu) | 0x3f800000u);
  if (m > 1.41421356f) {
    m *= 0.5f;
    ++e;
  }
  return static_cast<double>(e - 31) * 0.693147180559945309 +
         static_cast<double>(logf(m) + rest);
}

// The M best of one prompt from its beams' slices.
__global__ void __launch_bounds__(kThreads) beam_choose_kernel(const BeamSelectParams p) {
  __shared__ Scored buf[kChoiceBuffer];
  __shared__ Scored warp_best[kWarps];
  // lse = top + log_sum of each beam, kept apart: next to a large top the sum's
  // logarithm would be lost even in 64 bits
  __shared__ double log_sum[kBeamMaxSelectBeams];
  __shared__ float row_top[kBeamMaxSelectBeams];
  __shared__ int count;
  const int b = blockIdx.x;
  const int lane = static_cast<int>(threadIdx.x & 31);
  if (threadIdx.x == 0) count = 0;
  grid_dependency_wait();
  // A warp takes a beam. log_sum is NaN for one that offers nothing, +infinity
  // for a finished one.
  int err = 0;
  for (int k = static_cast<int>(threadIdx.x >> 5); k < p.beams; k += kWarps) {
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
        for (int i = lane; i < p.splits; i += 32) {
          const float m = p.stats[row * p.splits + i].x;
          bad |= !(m < INFINITY);
          top = fmaxf(top, m);
        }
        bad = __any_sync(0xffffffffu, bad);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (bad) {
          err |= FLCE_DEVERR_NOT_FINITE;
        } else if (top > -INFINITY) {
          // At most 2^31 terms of at most 1, each rounded to a multiple of 2^-31:
          // adding those is exact, and in any order the same.
          unsigned long long s = 0;
          for (int i = lane; i < p.splits; i += 32) {
            const float2 st = p.stats[row * p.splits + i];
            s += __float2ull_rn(st.y * ex2_approx((st.x - top) * kLog2e) * 2147483648.0f);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          l = log_of(s);
        }
      }
    }
    if (lane == 0) {
      log_sum[k] = l;
      row_top[k] = top;
    }
  }
  if (err != 0 && lane == 0 && p.err_word != nullptr) atomicOr(p.err_word, err);
  __syncthreads();

  const int per_beam = p.splits * p.m;
  const int total = p.beams * per_beam;
  const Scored none{0, ~0ull};
  // The c-th candidate. Keys of beams that were not read are loaded and not used.
  auto candidate = [&](int c) -> Scored {
    const int k = c / per_beam;
    const int64_t row = static_cast<int64_t>(b) * p.beams + k;
    const uint64_t key = p.keys[row * per_beam + (c - k * per_beam)];
    const double l = log_sum[k];
    const double score = static_cast<double>(p.beam_scores[row]);
    const double zv = static_cast<double>(from_order_bits(static_cast<uint32_t>(key >> 32)));
    const uint32_t v = 0xffffffffu - static_cast<uint32_t>(key);
    Scored x{order_bits64(score + ((zv - static_cast<double>(row_top[k])) - l)),
             (static_cast<uint64_t>(k) << 32) | v};
    if (key == 0 || isnan(l)) x = none;
    if (isinf(l))
      x = c == k * per_beam
              ? Scored{order_bits64(score), (static_cast<uint64_t>(k) << 32) |
                                                static_cast<uint64_t>(p.pad_token)}
              : none;
    return x;
  };
  // the thread's candidates: rotated in each 16, because the keys of a slice
  // are in order and the groups shall see all ranks alike
  auto place_of = [&](int round) -> int {
    const int t = static_cast<int>(threadIdx.x);
    return round * kThreads + (t & ~15) + ((t + (t >> 4) + 5 * round) & 15);
  };
  const int rounds = (total + kThreads - 1) / kThreads;
  // the first of them stay in registers
  Scored mine[kHeld];
  Scored best = none;
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    mine[r] = none;
    if (r < rounds) {
      const int c = place_of(r);
      if (c < total) mine[r] = candidate(c);
      if (better(mine[r], best)) best = mine[r];
    }
  }
  for (int r = kHeld; r < rounds; ++r) {
    const int c = place_of(r);
    const Scored x = c < total ? candidate(c) : none;
    if (better(x, best)) best = x;
  }
  const Scored floor_at = group_floor(best, p.groups, reinterpret_cast<Scored(*)[32]>(buf));
  __syncthreads();  // its part of buf has been read
  auto push = [&](const Scored& x) {
    if (x.s == 0 || better(floor_at, x)) return;
    const uint32_t place = take_place(&count);
    if (place < kChoiceBuffer) buf[place] = x;
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r) push(mine[r]);
  for (int r = kHeld; r < rounds; ++r) {
    const int c = place_of(r);
    if (c < total) push(candidate(c));
  }
  __syncthreads();
  const int64_t o0 = static_cast<int64_t>(b) * p.m;
  auto emit = [&](int rank, const Scored& x) {
    p.scores_out[o0 + rank] = static_cast<float>(from_order_bits64(x.s));
    p.parents_out[o0 + rank] = static_cast<int64_t>(x.at >> 32);
    p.tokens_out[o0 + rank] = static_cast<int64_t>(x.at & 0xffffffffu);
  };
  auto emit_none = [&](int rank) {
    p.scores_out[o0 + rank] = -INFINITY;
    p.parents_out[o0 + rank] = 0;
    p.tokens_out[o0 + rank] = p.pad_token;
  };
  const int n = count;
  if (n <= kChoiceBuffer) {
    rank_keys(buf, n, p.m, emit);
    for (int i = n + static_cast<int>(threadIdx.x); i < p.m; i += kThreads) emit_none(i);
    return;
  }
  Scored last{~0ull, 0};
  for (int r = 0; r < p.m; ++r) {
    Scored x = none;
    for (int q = 0; q < rounds; ++q) {
      const int c = place_of(q);
      const Scored y = c < total ? candidate(c) : none;
      if (better(last, y) && better(y, x)) x = y;
    }
    x = block_best(x, warp_best);
    if (threadIdx.x == 0) {
      if (x.s != 0)
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
  const unsigned grid = static_cast<unsigned>(blocks);
  constexpr int kLarge = kTileLarge / (kThreads * Piece<T>::kElems);
  if (p.shifted) {
    if (large)
      beam_slices_kernel<T, kLarge, true><<<grid, kThreads, 0, s>>>(p);
    else
      beam_slices_kernel<T, 1, true><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (large)
      beam_slices_kernel<T, kLarge, false><<<grid, kThreads, 0, s>>>(p);
    else
      beam_slices_kernel<T, 1, false><<<grid, kThreads, 0, s>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // may be placed while the slices run, and waits for them
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, beam_choose_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
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

// One vector of W bytes of each of a prompt's beams, `at` bytes from base:
// all that moves is read before anything is written.
template <int W, int KM>
__device__ __forceinline__ void move_beams(uint8_t* base, int64_t beam_stride, int beams,
                                           const int* parent) {
  using V = typename Vec<W>::T;
  V v[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < beams && parent[j] != j)
      v[j] = *reinterpret_cast<const V*>(base + parent[j] * beam_stride);
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (j < beams && parent[j] != j) *reinterpret_cast<V*>(base + j * beam_stride) = v[j];
}

// KM: an upper bound of the beams; a thread holds one vector of each.
template <int KM, int CAP>
__global__ void __launch_bounds__(kThreads)
    beam_reorder_kernel(const __grid_constant__ ReorderTable<CAP> t) {
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
  int64_t at = static_cast<int64_t>(c - outer * e.run) * e.width;
#pragma unroll
  for (int d = kReorderDims - 1; d >= 0; --d) {
    if (e.size[d] > 1) {
      const uint32_t up = outer / e.size[d];
      at += static_cast<int64_t>(outer - up * e.size[d]) * e.stride[d];
      outer = up;
    }
  }
  uint8_t* const base = e.data + static_cast<int64_t>(b) * t.beams * e.beam_stride + at;
  if (e.width == 16) {
    if constexpr (KM <= 32) move_beams<16, KM>(base, e.beam_stride, t.beams, parent);
  } else if (e.width == 8) {
    move_beams<8, KM>(base, e.beam_stride, t.beams, parent);
  } else if (e.width == 4) {
    move_beams<4, KM>(base, e.beam_stride, t.beams, parent);
  } else if (e.width == 2) {
    move_beams<2, KM>(base, e.beam_stride, t.beams, parent);
  } else {
    move_beams<1, KM>(base, e.beam_stride, t.beams, parent);
  }
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectParams& p, int dtype, bool large,
                               cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_select<float>(p, large, s);
  if (dtype == FLCE_BF16) return launch_select<__nv_bfloat16>(p, large, s);
  return launch_select<__half>(p, large, s);
}

template <int CAP>
cudaError_t launch_beam_reorder(const ReorderTable<CAP>& t, int64_t blocks, cudaStream_t s) {
  const unsigned n = static_cast<unsigned>(blocks);
  if (t.beams <= 4)
    beam_reorder_kernel<4, CAP><<<n, kThreads, 0, s>>>(t);
  else if (t.beams <= 8)
    beam_reorder_kernel<8, CAP><<<n, kThreads, 0, s>>>(t);
  else if (t.beams <= 16)
    beam_reorder_kernel<16, CAP><<<n, kThreads, 0, s>>>(t);
  else if (t.beams <= 32)
    beam_reorder_kernel<32, CAP><<<n, kThreads, 0, s>>>(t);
  else
    beam_reorder_kernel<64, CAP><<<n, kThreads, 0, s>>>(t);
  return cudaGetLastError();
}

template cudaError_t launch_beam_reorder(const ReorderTable<kReorderSmall>&, int64_t, cudaStream_t);
template cudaError_t launch_beam_reorder(const ReorderTable<kReorderLarge>&, int64_t, cudaStream_t);

}  // namespace flce
