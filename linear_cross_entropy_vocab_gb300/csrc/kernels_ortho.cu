// Orthogonalising matrices by Newton-Schulz products, all matrices of a batch
// at once:
//
//   x_0 = g / (|g| + eps)            |g|: root of the sum of squares
//   x  <- p x,  p = a I + b A + c A A,  A = x x^T        a step
//
// in three products a step. A and p are symmetric: their tiles above the
// diagonal are computed and stored twice, once transposed.
//
// Bound by the tensor cores: m^2 n + m^3 + 2 m^2 n operations a step for an
// m x n matrix, m <= n, against a few passes over it. One persistent kernel
// runs all steps with CTA pairs on 256 x 256 tiles (tcgen05.mma over the pair,
// operands staged by TMA in a ring of six 32 KB stages, two accumulators in
// tensor memory, so that a tile is stored behind the next one's products).
// Products follow one another by counts in global memory, not by launches. Five
// steps of 4096 x 4096 take it 905 us (the tensor pipe is busy in 69 % of the
// cycles), of 14336 x 4096 1515 us (73 %), of eight 1024 x 4096 351 us (47 %: their
// small products have 80 tiles, and one follows the other after 13 us, of which
// 5.4 are the tensor cores').
//
// The operands are halves with a power-of-two scale for each product, chosen by
// the host from the bounds on the singular values, so that nothing leaves the
// range. Their 11 bits at the rate of bf16's 8 keep the result of noise within
// 1e-3 to 2.5e-3 of itself (five default steps, before its own rounding), where
// bf16 operands give 1e-2; sums are held in 32 bits. A rounding is noise of 2^-12
// of what is rounded, and the steps magnify it in the directions of small
// singular values by the product of their a (485) at most: a matrix of rank one
// gets noise of a 2-norm of 0.10 (measured; 0.02 from bf16, which is not rounded).
// The norm's factor is applied to the first step's products, in 32 bits: a
// 16-bit input is copied without rounding.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "norm_rows.cuh"
#include "ortho_internal.h"
#include "ortho_norm.cuh"
#include "tc_ptx.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------ norm and copy

// Sums of squares of a share of a matrix. Rows are read in spans of 4096
// values, in aligned 16-byte pieces wherever a row starts (a dense matrix is
// one long row), with a span's loads on their way while the one before is added
// up (67 MB take 19 us, 28 without); 16 values are summed in 32 bits, those sums
// in 64, and again in 64 where one leaves the 32-bit range.
constexpr int kSpan = 4096;
template <class T>
__global__ void __launch_bounds__(256, 5) ortho_norm_kernel(const OrthoCopyParams p) {
  __shared__ double buf[8];
  grid_launch_dependents();
  const T* const src = static_cast<const T*>(p.src) + blockIdx.y * p.batch_stride;
  const bool dense = p.row_pitch == p.cols;
  const int64_t rows = dense ? 1 : p.rows;
  const int64_t len = dense ? int64_t(p.rows) * p.cols : p.cols;
  const int64_t spans_row = (len + kSpan - 1 + 8) / kSpan;  // a row may start 7 values into its first
  const int64_t spans = rows * spans_row;
  const auto load = [&](int64_t i, Raw<T>(&raw)[2]) {
    const int64_t r = rows == 1 ? 0 : i / spans_row;
    const T* const row = src + r * p.row_pitch;
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7;
    const int64_t at = (i - r * spans_row) * kSpan - phase + threadIdx.x * 8;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = at + k * 2048;
      if (e >= 0 && e + 8 <= len) {
        raw[k].load(row + e);
      } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = e + j >= 0 && e + j < len ? to_f32(row[e + j]) : 0.0f;
        store8(reinterpret_cast<T*>(raw[k].q), v);
      }
    }
  };
  double total = 0.0;
  Raw<T> raw[2];
  if (blockIdx.x < spans) load(blockIdx.x, raw);
  for (int64_t i = blockIdx.x; i < spans; i += gridDim.x) {
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) raw[k].values(v[k]);
    if (i + gridDim.x < spans) load(i + gridDim.x, raw);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
    double wide = sum;
    if (!(sum < 3.0e38f && sum > 1.0e-30f)) {
      wide = 0.0;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) wide += static_cast<double>(v[k][j]) * v[k][j];
    }
    total += wide;
  }
  total = team_all<256>(total, buf, SumOp{});
  if (threadIdx.x == 0) p.partial[int64_t(blockIdx.y) * p.parts + blockIdx.x] = total;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.counts; i += 256) p.count[i] = 0;
}

// Where the halves of row i from column 8 * c on lie in a 64 x 64 part in
// shared memory: 16-byte pieces are swapped so that neither rows nor columns of
// pieces meet in a bank.
__device__ __forceinline__ int piece_at(int i, int c) { return i * 64 + ((c ^ (i >> 3)) & 7) * 8; }

// Halves of the padded matrix, 64 x 128 at a time. The transpose of a tall
// matrix, and rows that do not start at 16-byte boundaries, go through shared
// memory.
template <class T>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 3 : 4) ortho_copy_kernel(const OrthoCopyParams p) {
  __shared__ __align__(16) __half part[2][64 * 64];
  __shared__ double buf[8];
  grid_dependency_wait();
  const int b = blockIdx.y;
  const double* const partial = p.partial + int64_t(b) * p.parts;
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.parts; i += 256) sum += partial[i];
  sum = team_all<256>(sum, buf, SumOp{});
  // by one thread, as 64-bit arithmetic is slow
  __shared__ int exponent;
  __shared__ float factor;
  if (threadIdx.x == 0) {
    norm_factor(sum, p.eps, exponent, factor);
    if (blockIdx.x == 0) p.factor[b] = factor;
  }
  __syncthreads();
  const int e = exponent;
  // the power of two in two factors, as one could leave the 32-bit range
  const int shift = p.x_shift - e;
  const float scale0 = scalbnf(1.0f, shift / 2), scale1 = scalbnf(1.0f, shift - shift / 2);
  auto half_of = [&](float v) { return __float2half_rn(v * scale0 * scale1); };
  auto halves_of = [&](const float(&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i] * scale0 * scale1,
                                          v[2 * i + 1] * scale0 * scale1);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  const T* const src = static_cast<const T*>(p.src) + b * p.batch_stride;
  __half* const x = static_cast<__half*>(p.x) + int64_t(b) * p.m_pad * p.n_pad;
  const bool aligned = reinterpret_cast<uintptr_t>(src) % 16 == 0 &&
                       p.row_pitch * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  const int r8 = threadIdx.x >> 3, c8 = threadIdx.x & 7;
  const int tiles_n = (p.n_pad + 127) / 128, tiles = tiles_n * (p.m_rows / 64);
  for (int u = blockIdx.x; u < tiles; u += gridDim.x) {
    const int i0 = u / tiles_n * 64, j0 = u % tiles_n * 128;  // of x
    const int halves = j0 + 64 < p.n_pad ? 2 : 1;
    const int s0 = p.tall ? j0 : i0, t0 = p.tall ? i0 : j0;  // of src
    const bool whole = aligned && (p.tall ? t0 + 64 : t0 + 128) <= p.cols;
    if (!p.tall && whole) {
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = s0 + r8 + 32 * (k & 1), c = t0 + (k >> 1) * 64 + c8 * 8;
        float v[8] = {};
        if (r < p.rows) load8(src + int64_t(r) * p.row_pitch + c, v);
        w[k] = halves_of(v);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = s0 + r8 + 32 * (k & 1), c = t0 + (k >> 1) * 64 + c8 * 8;
        *reinterpret_cast<uint4*>(x + int64_t(r) * p.n_pad + c) = w[k];
      }
      continue;
    }
    __syncthreads();  // the last part has been taken
    if (whole) {  // tall
      float v[4][8] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = s0 + r8 + 32 * k;
        if (r < p.rows) load8(src + int64_t(r) * p.row_pitch + t0 + c8 * 8, v[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int dr = r8 + 32 * (k & 1);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          part[k >> 1][piece_at(c8 * 8 + j, dr >> 3) + (dr & 7)] = half_of(v[k][j]);
      }
    } else {
      // rows that start anywhere: the nine aligned pieces that hold 64 values,
      // all of a thread's loads before its stores
      constexpr int kEach = (2 * 64 * 9 + 255) / 256;
      Raw<T> raw[kEach];
      const auto place = [&](int k, int& g, int& dr, int& dc, const T*& row) {
        const int u9 = k * 256 + threadIdx.x, line = u9 / 9;
        g = line >> 6;
        dr = line & 63;
        const int r = s0 + dr + (p.tall ? 64 * g : 0), c0 = t0 + (p.tall ? 0 : 64 * g);
        row = src + int64_t(r) * p.row_pitch;
        const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7;
        dc = (u9 - line * 9) * 8 - ((c0 + phase) & 7);
        row += c0 + dc;
        return c0 + dc;
      };
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        int g, dr, dc;
        const T* at;
        const int c = place(k, g, dr, dc, at);
        const bool in = g < halves && s0 + dr + (p.tall ? 64 * g : 0) < p.rows;
        if (in && c >= 0 && c + 8 <= p.cols) {
          raw[k].load(at);
        } else {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = in && c + j >= 0 && c + j < p.cols ? to_f32(at[j]) : 0.0f;
          store8(reinterpret_cast<T*>(raw[k].q), v);
        }
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        int g, dr, dc;
        const T* at;
        place(k, g, dr, dc, at);
        if (g >= halves) continue;
        float v[8];
        raw[k].values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = dc + j;
          if (d < 0 || d >= 64) continue;
          const int i = p.tall ? d : dr, to = p.tall ? dr : d;
          part[g][piece_at(i, to >> 3) + (to & 7)] = half_of(v[j]);
        }
      }
    }
    __syncthreads();
    for (int g = 0; g < halves; ++g) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int di = r8 + 32 * k;
        *reinterpret_cast<uint4*>(x + int64_t(i0 + di) * p.n_pad + j0 + 64 * g + c8 * 8) =
            *reinterpret_cast<const uint4*>(part[g] + piece_at(di, c8));
      }
    }
  }
}

// ----------------------------------------------------------------- products

constexpr int kRows = 128;  // accumulator rows of a CTA
constexpr int kDepth = 64;  // of a stage: one 128-byte swizzle row of halves
constexpr int kStages = 6;
constexpr int kOperandBytes = kRows * kDepth * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kWarps = kOrthoWarps;  // of the epilogue: two a quarter of the rows, half of the columns each
constexpr int kThreads = 64 + 32 * kWarps;
constexpr int kBoxBytes = 32 * 32 * 2;

// CG = 2: a pair of CTAs on a tile of 256 x 256, each with 128 of its rows. CG =
// 1: a CTA on a tile of 128 x 128, for matrices that have too few tiles of 256
// for the SMs: a tile's products and its way out take half as long, and more
// SMs have one.
template <int CG>
struct Shape {
  static constexpr int kTile = kRows * CG;
  static constexpr int kPieces = kTile / 64;  // of 32 columns, for an epilogue warp
};

constexpr int kSlots = 4;  // items on their way to the roles

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t done;
  uint64_t item_full[kSlots], item_empty[kSlots];
  int item[kSlots];  // an item's number, or -1: none left
  uint32_t tmem;
  int abort;
};
constexpr int kSmemBytes =
    1024 + kStages * kStageBytes + kWarps * 2 * kBoxBytes + static_cast<int>(sizeof(Ctl));

template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y) {
  if constexpr (CG == 2)
    tma_load_2d_pair(dst, map, bar, x, y);
  else
    tma_load_2d(dst, map, bar, x, y);
}
template <int CG, bool ACROSS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int side, int depth) {
  if constexpr (!ACROSS) {
    load_box<CG>(dst, map, bar, depth, side);  // {64 deep, 128 rows}
  } else {
    load_box<CG>(dst, map, bar, side, depth);  // two boxes {64, 64 deep}
    load_box<CG>(dst + 8192, map, bar, side + 64, depth);
  }
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    umma_commit_pair(bar, 0x3);
  else
    umma_commit(bar);
}
template <int CG>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  return CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
template <bool ACROSS>
__device__ __forceinline__ uint64_t slice_desc(uint32_t base, int kk) {
  return ACROSS ? smem_desc_sw128(base + kk * 2048, 8192, 1024)
                : smem_desc_sw128(base + kk * 32, 16, 1024);
}

// Every wait has a limit: past it the CTA gives up, lets what is in flight
// finish and leaves, and the error word says so.
__device__ __forceinline__ bool give_up(uint64_t t0, volatile int* abort_flag,
                                        const OrthoRunParams& p) {
  if (*abort_flag) return true;
  if (globaltimer_ns() - t0 <= p.wait_ns) return false;
  *abort_flag = 1;
  if (p.err_word) atomicOr(p.err_word, FLCE_DEVERR_TIMEOUT);
  return true;
}
template <int CG>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         const OrthoRunParams& p) {
  if (try_wait<CG>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (try_wait<CG>(bar, parity)) return true;
    if ((it & 63u) == 0u && give_up(t0, abort_flag, p)) return false;
  }
}
template <int CG>
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!try_wait<CG>(bar, parity)) {
    if (globaltimer_ns() - t0 > 1000000000ull) break;
  }
}
__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Orders accesses of global memory by bulk copies and by ordinary instructions.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// One product of the sequence, as every role walks it.
struct Product {
  OrthoOp op;
  bool symmetric;
  int m_tiles, n_tiles, per;  // tiles of a matrix
  int k_iters;
  const OrthoProduct* with;
};
__device__ __forceinline__ Product product_of(const OrthoRunParams& p, int i) {
  Product q;
  q.with = &p.product[i];
  q.op = static_cast<OrthoOp>(q.with->op);
  q.symmetric = q.op <= OrthoOp::kPoly;
  q.m_tiles = q.op == OrthoOp::kOutTall ? p.n_tiles : p.m_tiles;
  q.n_tiles = q.symmetric || q.op == OrthoOp::kOutTall ? p.m_tiles : p.n_tiles;
  q.per = q.symmetric ? p.m_tiles * (p.m_tiles + 1) / 2 : p.m_tiles * p.n_tiles;
  q.k_iters = q.op == OrthoOp::kGram ? p.k_n : p.k_m;
  return q;
}

struct Tile {
  int b, m, n;
};
__device__ __forceinline__ Tile tile_of(const Product& q, int u) {
  Tile t;
  t.b = u / q.per;
  int r = u - t.b * q.per;
  if (q.symmetric) {  // the triangle above the diagonal
    t.m = 0;
    while (r >= q.m_tiles - t.m) {
      r -= q.m_tiles - t.m;
      ++t.m;
    }
    t.n = t.m + r;
  } else if (q.op == OrthoOp::kOutTall) {  // p stays in L2, x passes once
    t.m = r / q.n_tiles;
    t.n = r - t.m * q.n_tiles;
  } else {
    t.n = r / q.m_tiles;
    t.m = r - t.n * q.m_tiles;
  }
  return t;
}

// A stretch of a tile's contraction, [k0, k1).
struct Part {
  int tile, k0, k1;
};
// Where stretch `unit` of a product's cut tiles begins: they are laid end to end
// and divided into equal stretches.
__device__ __forceinline__ int stretch(const OrthoCut& c, int k_iters, int unit) {
  return unit * (c.cut * k_iters) / c.units;  // the host keeps this in 31 bits
}
// The stretch that has iteration x.
__device__ __forceinline__ int owner_of(const OrthoCut& c, int k_iters, int x) {
  return ((x + 1) * c.units - 1) / (c.cut * k_iters);
}
__device__ __forceinline__ void store_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// What a pair of CTAs (or a CTA) works on, as one of its roles meets it: items,
// numbered over all products, each a stretch or a whole tile, a product's
// stretches first (what joins their sums then runs behind whole tiles'
// products). Pairs draw the numbers from a counter: the loading thread (of the
// even CTA) draws when it has issued the loads of the item before, and hands the
// number to all roles through a ring of slots. (Drawn one item ahead, two tiles
// of one product went to a pair while others waited for the product: 2500 x 2500
// took 664 us instead of 404.) An item waits for items of smaller numbers
// only, and every pair takes its items in order, so that the smallest unfinished
// one never waits: pairs that have not started yet hold nobody up.
enum class Role { kDrawer, kThread, kWarp };
template <int CG, Role ROLE>
struct Feed {
  const OrthoRunParams& p;
  Ctl* const ctl;
  const int rank, lane;
  Product q;
  int i = 0;             // the product's number
  int base = 0, count;   // its first item, and how many it has
  int at = 0, end = 0;   // what is left of a stretch
  int unit = 0;          // the stretch
  int slot = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ int items_of(const Product& of) const {
    const OrthoCut& c = p.cut[of.with->cut];
    return c.cut > 0 ? c.units + c.whole : of.per * p.batch;
  }
  __device__ __forceinline__ Feed(const OrthoRunParams& p_, Ctl* ctl_, int rank_, int lane_)
      : p(p_), ctl(ctl_), rank(rank_), lane(lane_), q(product_of(p_, 0)) {
    count = items_of(q);
  }
  __device__ __forceinline__ void advance() {
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // Draws a number, or -1 past the last item, and puts it into the next slot of
  // all CTAs.
  __device__ __forceinline__ bool draw(int& u) {
    u = atomicAdd(p.ticket, 1);
    if (!wait_bar<CG>(smem_addr(&ctl->item_empty[slot]), phase ^ 1u, &ctl->abort, p))
      return false;
    if (u >= p.items) u = -1;
    const uint32_t to = smem_addr(&ctl->item[slot]), bar = smem_addr(&ctl->item_full[slot]);
    if constexpr (CG == 2) {
      store_cluster(map_to_rank(to, 1), u);
      mbar_arrive_cluster(map_to_rank(bar, 1));
    }
    *reinterpret_cast<volatile int*>(&ctl->item[slot]) = u;
    mbar_arrive(bar);
    advance();
    return true;
  }
  // The next part and its product `q`. False when none are left or a wait gave
  // up. All lanes of a Role::kWarp call it together.
  __device__ __forceinline__ bool next(Part& part) {
    if (at >= end) {
      int u;
      if constexpr (ROLE == Role::kDrawer) {
        if (!draw(u)) return false;
      } else {
        const bool here = wait_bar<CG>(smem_addr(&ctl->item_full[slot]), phase, &ctl->abort, p);
        if (ROLE == Role::kWarp ? !__all_sync(0xffffffffu, here) : !here) return false;
        u = *reinterpret_cast<volatile int*>(&ctl->item[slot]);
        if constexpr (ROLE == Role::kWarp) __syncwarp();
        if (lane == 0) {
          const uint32_t bar = smem_addr(&ctl->item_empty[slot]);
          if (CG == 1 || rank == 0)
            mbar_arrive(bar);
          else
            mbar_arrive_cluster(map_to_rank(bar, 0));
        }
        advance();
      }
      if (u < 0) return false;
      while (u >= base + count) {
        base += count;
        q = product_of(p, ++i);
        count = items_of(q);
      }
      u -= base;
      const OrthoCut& c = p.cut[q.with->cut];
      const int stretches = c.cut > 0 ? c.units : 0;
      if (u >= stretches) {
        part.tile = u - stretches;
        part.k0 = 0;
        part.k1 = q.k_iters;
        return true;
      }
      unit = u;
      at = stretch(c, q.k_iters, u);
      end = stretch(c, q.k_iters, u + 1);
    }
    const int t = at / q.k_iters;
    part.tile = p.cut[q.with->cut].whole + t;
    part.k0 = at - t * q.k_iters;
    part.k1 = min(q.k_iters, part.k0 + end - at);
    at += part.k1 - part.k0;
    return true;
  }
};

// What a product reads of a matrix is there once each epilogue warp of each
// tile of the products before has counted one up. Where tiles are cut, all
// matrices count together: the places of their sums are used again by the next
// product.
struct Need {
  const int* count;
  int least;
};
__device__ __forceinline__ int* count_of(const OrthoRunParams& p, int b) {
  return p.finished + (p.joint ? 0 : b);
}
__device__ __forceinline__ Need need_of(const OrthoRunParams& p, const Product& q, int b) {
  return {count_of(p, b), q.with->need};
}
__device__ __forceinline__ bool wait_need(const Need& need, volatile int* abort_flag,
                                          const OrthoRunParams& p) {
  if (load_acquire(need.count) >= need.least) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (load_acquire(need.count) >= need.least) return true;
    if ((it & 15u) == 0u && give_up(t0, abort_flag, p)) return false;
  }
}

// A box of 32 x 32 16-bit values, rows of 64 bytes: the 16-byte pieces of a row
// are swapped by its number as the store's map expects (64-byte swizzle), so
// that eight rows' pieces fall into different banks.
__device__ __forceinline__ int box_at(int row, int piece) {
  return row * 64 + ((piece ^ (row >> 1)) & 3) * 16;
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Until all but the last committed store have read shared memory.
__device__ __forceinline__ void tma_store_wait_read_but_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Where a pair leaves a warp's sums of a part: of the first part of a tile
// (which ends the pair's stretch) or of another (which begins it).
template <int CG>
__device__ __forceinline__ float4* share_of(const OrthoRunParams& p, int unit, bool first,
                                            int rank, int warp) {
  const int64_t slot = ((unit * 2 + (first ? 1 : 0)) * CG + rank) * kWarps + warp;
  return reinterpret_cast<float4*>(p.shares) + slot * (Shape<CG>::kPieces * 8 * 32);
}

// The loads of a part: each CTA its 128 rows of one operand and 128 of the 256
// of the other.
struct Ring {
  int stage;
  uint32_t phase, armed, last;
};
template <int CG, OrthoOp OP>
__device__ __forceinline__ bool load_part(const OrthoRunParams& p, const Product& q,
                                          const Part& part, const Tile& t, uint32_t base, int rank,
                                          Ctl* ctl, Ring& ring) {
  constexpr bool kAcrossA = OP == OrthoOp::kOutTall, kAcrossB = OP == OrthoOp::kMul || OP == OrthoOp::kOutWide;
  const CUtensorMap* const a = kAcrossA ? &p.across[q.with->a] : &p.along[q.with->a];
  const CUtensorMap* const b = kAcrossB ? &p.across[q.with->b] : &p.along[q.with->b];
  constexpr int kTile = Shape<CG>::kTile;
  const int a_side = t.m * kTile + rank * kRows, b_side = t.n * kTile + rank * kRows;
  const int row0 = t.b * p.m_pad;
  for (int k = part.k0; k < part.k1; ++k) {
    const int s = ring.stage;
    if (!wait_bar<CG>(smem_addr(&ctl->empty[s]), ring.phase ^ 1u, &ctl->abort, p))
      return false;
    const uint32_t full_local = smem_addr(&ctl->full[s]);
    const uint32_t full = CG == 2 ? map_to_rank(full_local, 0) : full_local;
    if (rank == 0) mbar_arrive_expect_tx(full_local, CG * kStageBytes);
    const uint32_t dst = base + s * kStageBytes;
    load_operand<CG, kAcrossA>(dst, a, full, kAcrossA ? a_side : row0 + a_side,
                           kAcrossA ? row0 + k * kDepth : k * kDepth);
    load_operand<CG, kAcrossB>(dst + kOperandBytes, b, full, kAcrossB ? b_side : row0 + b_side,
                           kAcrossB ? row0 + k * kDepth : k * kDepth);
    ring.armed |= 1u << s;
    ring.last = (ring.last & ~(1u << s)) | (ring.phase << s);
    if (++ring.stage == kStages) {
      ring.stage = 0;
      ring.phase ^= 1u;
    }
  }
  return true;
}

template <int CG, OrthoOp OP>
__device__ __forceinline__ bool multiply_part(const OrthoRunParams& p, const Part& part,
                                              uint32_t base, uint32_t d, Ctl* ctl, Ring& ring) {
  constexpr bool kAcrossA = OP == OrthoOp::kOutTall, kAcrossB = OP == OrthoOp::kMul || OP == OrthoOp::kOutWide;
  constexpr uint32_t idesc =
      idesc_f16kind_f32(Shape<CG>::kTile, Shape<CG>::kTile, kAcrossA ? 1 : 0, kAcrossB ? 1 : 0, 0);
  for (int k = part.k0; k < part.k1; ++k) {
    if (!wait_bar<CG>(smem_addr(&ctl->full[ring.stage]), ring.phase, &ctl->abort, p))
      return false;
    tc_fence_after_sync();
    const uint32_t a0 = base + ring.stage * kStageBytes, b0 = a0 + kOperandBytes;
#pragma unroll
    for (int kk = 0; kk < kDepth / 16; ++kk)
      if constexpr (CG == 2)
        umma_bf16_pair(d, slice_desc<kAcrossA>(a0, kk), slice_desc<kAcrossB>(b0, kk), idesc,
                       k != part.k0 || kk != 0 ? 1u : 0u);
      else
        umma_bf16(d, slice_desc<kAcrossA>(a0, kk), slice_desc<kAcrossB>(b0, kk), idesc,
                  k != part.k0 || kk != 0 ? 1u : 0u);
    commit<CG>(smem_addr(&ctl->empty[ring.stage]));
    if (++ring.stage == kStages) {
      ring.stage = 0;
      ring.phase ^= 1u;
    }
  }
  return true;
}

// A warp's 32 rows and 128 columns of a part's accumulator: stored, or left for
// the warp that joins the tile's sums. Returns whether the tile is stored.
template <int CG, OrthoOp OP, class T>
__device__ __forceinline__ bool finish_part(const OrthoRunParams& p, const Product& q,
                                            const Part& part, const Tile& t, uint32_t taddr,
                                            int unit, int rank, int warp, int quarter, int first,
                                            uint8_t* boxes, int lane) {
  constexpr int kTile = Shape<CG>::kTile, kPieces = Shape<CG>::kPieces;
  constexpr bool kOut = OP == OrthoOp::kOutWide || OP == OrthoOp::kOutTall;
  const int row0 = t.m * kTile + rank * kRows + quarter * 32;  // of the matrix
  const int row = row0 + lane;
  const bool mirrored = OP <= OrthoOp::kPoly && t.n > t.m;
  const OrthoProduct& with = *q.with;
  const int rows = kOut ? p.rows : p.m_rows;
  const int cols = kOut ? p.cols : OP == OrthoOp::kMul ? p.n_pad : p.m_rows;
  float scale = with.scale;
  if (with.power != 0) {
    // the norm's factor belongs to the first x
    const float f = p.factor[t.b];
    scale *= with.power == 2 ? f * f : f;
  }
  // Pieces of the tile that this warp keeps. Where the tile's contraction is
  // cut, each pair leaves its sums, and the warp that comes last adds all of
  // them, in the order of the contraction.
  const int pieces =
      row0 >= rows ? 0 : min(kPieces, (cols - t.n * kTile - first * 32 + 31) / 32);
  int from = unit, to = unit;
  if (part.k1 - part.k0 < q.k_iters) {
    const OrthoCut& c = p.cut[q.with->cut];
    const int x = (part.tile - c.whole) * q.k_iters;
    from = owner_of(c, q.k_iters, x);
    to = owner_of(c, q.k_iters, x + q.k_iters - 1);
    int* const counter = p.arrived + ((part.tile - c.whole) * CG + rank) * kWarps + warp;
    int before = 0;
    if (lane == 0) before = *reinterpret_cast<volatile int*>(counter);
    before = __shfl_sync(0xffffffffu, before, 0);
    if (before != to - from) {
      float4* const mine = share_of<CG>(p, unit, unit == from, rank, warp) + lane;
#pragma unroll 1
      for (int i = 0; i < pieces; ++i) {
        float v[32];
        tmem_load_32cols(taddr + static_cast<uint32_t>((first + i) * 32), v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mine[(i * 8 + j) * 32] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) before = atomicAdd(counter, 1);
      before = __shfl_sync(0xffffffffu, before, 0);
    }
    if (before == to - from && lane == 0) *counter = 0;  // for the next product
    __threadfence();
    __syncwarp();
    if (before != to - from) return false;
  }
  // The gram's values of this piece and the next: four lanes take 64 bytes of a
  // row, so that a load touches eight lines and not 32.
  uint4 held[2][4];
  const uint4* const old = reinterpret_cast<const uint4*>(
      static_cast<const __half*>(p.gram) +
      (int64_t(t.b) * p.m_pad + row0 + (lane >> 2)) * p.m_pad + t.n * kTile + first * 32 +
      (lane & 3) * 8);
  const auto fetch = [&](uint4(&g)[4], int i) {
    if (OP == OrthoOp::kPoly && i < pieces) {
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = __ldcg(old + 4 * i + j * p.m_pad);  // eight rows further
    }
  };
  fetch(held[0], 0);
  fetch(held[1], 1);
#pragma unroll 1
  for (int i = 0; i < pieces; ++i) {
    const int ch = first + i;
    const int col = t.n * kTile + ch * 32;
    float v[32];
    tmem_load_32cols(taddr + static_cast<uint32_t>(ch * 32), v);
    if (from < to) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // eight columns at a time
        float sum[8] = {};
        for (int u = from; u <= to; ++u) {
          if (u == unit) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[8 * g + j];
          } else {
            const float4* const other =
                share_of<CG>(p, u, u == from, rank, warp) + lane + (i * 8 + 2 * g) * 32;
            const float4 f = __ldcg(other), h = __ldcg(other + 32);
            sum[0] += f.x, sum[1] += f.y, sum[2] += f.z, sum[3] += f.w;
            sum[4] += h.x, sum[5] += h.y, sum[6] += h.z, sum[7] += h.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * g + j] = sum[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= scale;
    // The boxes' last contents have been taken: both boxes are a piece and its
    // mirror image, or two pieces in turn.
    if (lane == 0) {
      if (mirrored || i == 0)
        tma_store_wait_read();
      else
        tma_store_wait_read_but_one();
    }
    __syncwarp();
    uint8_t* const box = mirrored ? boxes : boxes + (i & 1) * kBoxBytes;
    uint8_t* const mirror = boxes + kBoxBytes;
    if constexpr (OP == OrthoOp::kPoly) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(box + box_at(8 * j + (lane >> 2), lane & 3)) = held[0][j];
#pragma unroll
      for (int j = 0; j < 4; ++j) held[0][j] = held[1][j];
      fetch(held[1], i + 2);
      __syncwarp();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 w = *reinterpret_cast<const uint4*>(box + box_at(lane, g));
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
          v[8 * g + 2 * j] = fmaf(f.x, with.old, v[8 * g + 2 * j]);
          v[8 * g + 2 * j + 1] = fmaf(f.y, with.old, v[8 * g + 2 * j + 1]);
        }
      }
      if (row0 == col) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += lane == j ? with.diag : 0.0f;
      }
    }
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(box + box_at(lane, j)) =
          make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    if (mirrored) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        *reinterpret_cast<uint16_t*>(mirror + box_at(j, lane >> 3) + (lane & 7) * 2) =
            static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
    if (kOut && !p.out_mapped) {
      // rows that no map can describe: 32 values of one after the other
      __syncwarp();
      T* const out =
          static_cast<T*>(p.out) + (int64_t(t.b) * rows + row0) * cols + col + lane;
      const int some = rows - row0 < 32 ? rows - row0 : 32;
      if (col + lane < cols) {
#pragma unroll 8
        for (int r = 0; r < some; ++r)
          out[int64_t(r) * cols] =
              *reinterpret_cast<const T*>(box + box_at(r, lane >> 3) + (lane & 7) * 2);
      }
      continue;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if constexpr (kOut) {
        tma_store_3d(&p.store[with.c], smem_addr(box), col, row0, t.b);
      } else {
        const CUtensorMap* const c = &p.store[with.c];
        tma_store_2d(c, smem_addr(box), col, t.b * p.m_pad + row0);
        if (mirrored) tma_store_2d(c, smem_addr(mirror), row0, t.b * p.m_pad + col);
      }
      tma_store_commit();
    }
  }
  return true;
}

// All products of all steps: pairs of CTAs (or CTAs), as many as there are SMs
// for, draw their tiles in order; a tile waits until the products before have
// finished its matrix, so that matrices of a batch pass one another and nothing
// but a matrix's own order holds a pair up.
template <int CG, class T>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_run_kernel(const __grid_constant__ OrthoRunParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const boxes = smem_raw + (base - raw) + kStages * kStageBytes;
  Ctl* const ctl = reinterpret_cast<Ctl*>(boxes + kWarps * 2 * kBoxBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTile = Shape<CG>::kTile, kPieces = Shape<CG>::kPieces;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  volatile int* const abort_flag = &ctl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&ctl->acc_full[b]), 1);
      mbar_init(smem_addr(&ctl->acc_empty[b]), CG * kWarps);  // of both CTAs
    }
    mbar_init(smem_addr(&ctl->done), 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_addr(&ctl->item_full[i]), 1);
      // the product thread, the odd CTA's loading thread, the epilogue warps
      mbar_init(smem_addr(&ctl->item_empty[i]), CG + CG * kWarps);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.along[kOrthoX0]);
    tma_prefetch_desc(&p.along[kOrthoGram]);
    tma_prefetch_desc(&p.along[kOrthoP0]);
    tma_prefetch_desc(&p.across[kOrthoX0]);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(smem_addr(&ctl->tmem), 2 * kTile);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(&ctl->tmem), 2 * kTile);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem;
  if (warp == 0) {
    if (lane == 0) {
      Ring ring{};
      bool ok = true;
      const auto load = [&](auto&& feed) {
        int product = 0, ready = -1;  // the matrix whose operands are known to be there
        for (Part part; ok && feed.next(part);) {
          const Product& q = feed.q;
          const Tile t = tile_of(q, part.tile);
          if (feed.i > 0 && (t.b != ready || feed.i != product)) {
            ok = wait_need(need_of(p, q, t.b), abort_flag, p);
            if (!ok) break;
            fence_proxy_async_global();
            ready = t.b;
            product = feed.i;
          }
          switch (q.op) {
            case OrthoOp::kGram:
            case OrthoOp::kSquare:
            case OrthoOp::kPoly:
              ok = load_part<CG, OrthoOp::kGram>(p, q, part, t, base, rank, ctl, ring);
              break;
            case OrthoOp::kMul:
            case OrthoOp::kOutWide:
              ok = load_part<CG, OrthoOp::kMul>(p, q, part, t, base, rank, ctl, ring);
              break;
            case OrthoOp::kOutTall:
              ok = load_part<CG, OrthoOp::kOutTall>(p, q, part, t, base, rank, ctl, ring);
              break;
          }
        }
      };
      if (rank == 0)
        load(Feed<CG, Role::kDrawer>(p, ctl, rank, 0));
      else
        load(Feed<CG, Role::kThread>(p, ctl, rank, 0));
      if (*abort_flag && rank == 0) {
        for (int s = 0; s < kStages; ++s)
          if (ring.armed & (1u << s))
            drain_bar<CG>(smem_addr(&ctl->full[s]), (ring.last >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      Ring ring{};
      Feed<CG, Role::kThread> feed(p, ctl, rank, 0);
      int it = 0;
      for (Part part; feed.next(part); ++it) {
        const int buf = it & 1;
        if (!wait_bar<CG>(smem_addr(&ctl->acc_empty[buf]), ((it >> 1) & 1u) ^ 1u, abort_flag,
                          p))
          break;
        tc_fence_after_sync();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kTile);
        bool ok = true;
        switch (feed.q.op) {
          case OrthoOp::kGram:
          case OrthoOp::kSquare:
          case OrthoOp::kPoly:
            ok = multiply_part<CG, OrthoOp::kGram>(p, part, base, d, ctl, ring);
            break;
          case OrthoOp::kMul:
          case OrthoOp::kOutWide:
            ok = multiply_part<CG, OrthoOp::kMul>(p, part, base, d, ctl, ring);
            break;
          case OrthoOp::kOutTall:
            ok = multiply_part<CG, OrthoOp::kOutTall>(p, part, base, d, ctl, ring);
            break;
        }
        if (!ok) break;
        commit<CG>(smem_addr(&ctl->acc_full[buf]));
      }
      commit<CG>(smem_addr(&ctl->done));
      drain_bar<CG>(smem_addr(&ctl->done), 0);
    } else if (lane == 0) {
      // the other CTA's products write this one's tensor memory
      drain_bar<CG>(smem_addr(&ctl->done), 0);
    }
  } else {
    const int quarter = warp & 3;
    const int first = (warp - 2) >> 2 ? kPieces : 0;
    uint32_t acc_empty = smem_addr(&ctl->acc_empty[0]);
    if constexpr (CG == 2) acc_empty = map_to_rank(acc_empty, 0);
    uint8_t* const box = boxes + (warp - 2) * 2 * kBoxBytes;
    Feed<CG, Role::kWarp> feed(p, ctl, rank, lane);
    int it = 0, product = 0, ready = -1;
    for (Part part; feed.next(part); ++it) {
      const Product& q = feed.q;
      const Tile t = tile_of(q, part.tile);
      if (q.op == OrthoOp::kPoly && (t.b != ready || feed.i != product)) {
        // the gram is read here too
        if (!__all_sync(0xffffffffu, lane != 0 || wait_need(need_of(p, q, t.b), abort_flag, p)))
          break;
        __threadfence();
        __syncwarp();
        ready = t.b;
        product = feed.i;
      }
      const int buf = it & 1;
      if (!__all_sync(0xffffffffu, wait_bar<CG>(smem_addr(&ctl->acc_full[buf]), (it >> 1) & 1u,
                                                abort_flag, p)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(buf * kTile);
      bool stored = false;
      switch (q.op) {
        case OrthoOp::kGram:
        case OrthoOp::kSquare:
          stored = finish_part<CG, OrthoOp::kGram, __half>(p, q, part, t, taddr, feed.unit, rank,
                                                           warp - 2, quarter, first, box, lane);
          break;
        case OrthoOp::kPoly:
          stored = finish_part<CG, OrthoOp::kPoly, __half>(p, q, part, t, taddr, feed.unit, rank,
                                                           warp - 2, quarter, first, box, lane);
          break;
        case OrthoOp::kMul:
          stored = finish_part<CG, OrthoOp::kMul, __half>(p, q, part, t, taddr, feed.unit, rank,
                                                          warp - 2, quarter, first, box, lane);
          break;
        case OrthoOp::kOutWide:
          finish_part<CG, OrthoOp::kOutWide, T>(p, q, part, t, taddr, feed.unit, rank, warp - 2,
                                                quarter, first, box, lane);
          break;
        case OrthoOp::kOutTall:
          finish_part<CG, OrthoOp::kOutTall, T>(p, q, part, t, taddr, feed.unit, rank, warp - 2,
                                                quarter, first, box, lane);
          break;
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        const uint32_t free = acc_empty + static_cast<uint32_t>(buf * sizeof(uint64_t));
        if constexpr (CG == 2)
          mbar_arrive_cluster(free);
        else
          mbar_arrive(free);
        if (stored) {
          tma_store_wait_all();
          fence_proxy_async_global();
          add_release(count_of(p, t.b), 1);
        }
      }
    }
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem, 2 * kTile);
    else
      tmem_dealloc(tmem, 2 * kTile);
  }
}

template <int CG, class T>
cudaError_t launch_run(const OrthoRunParams& p, cudaStream_t s) {
  const auto kernel = ortho_run_kernel<CG, T>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(CG * p.units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CG;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CG - 1;  // a cluster where there are pairs
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T>
cudaError_t launch_copy(const OrthoCopyParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  // CTAs that each find the norm once: six an SM over the batch
  const int64_t tiles = int64_t((p.n_pad + 127) / 128) * (p.m_rows / 64);
  const int64_t most = std::max<int64_t>(1, 6 * kOrthoPlanSms / p.batch);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(tiles, most)),
                     static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ortho_copy_kernel<T>, p);
}

}  // namespace

cudaError_t launch_ortho_norm(const OrthoCopyParams& p, int dtype, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.parts), static_cast<unsigned>(p.batch));
  if (dtype == FLCE_F32)
    ortho_norm_kernel<float><<<grid, 256, 0, s>>>(p);
  else if (dtype == FLCE_BF16)
    ortho_norm_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else
    ortho_norm_kernel<__half><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_ortho_copy(const OrthoCopyParams& p, int dtype, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_copy<float>(p, s);
  if (dtype == FLCE_BF16) return launch_copy<__nv_bfloat16>(p, s);
  return launch_copy<__half>(p, s);
}

cudaError_t launch_ortho_run(const OrthoRunParams& p, int out_dtype, cudaStream_t s) {
  if (p.pairs)
    return out_dtype == FLCE_BF16 ? launch_run<2, __nv_bfloat16>(p, s)
                                  : launch_run<2, __half>(p, s);
  return out_dtype == FLCE_BF16 ? launch_run<1, __nv_bfloat16>(p, s) : launch_run<1, __half>(p, s);
}

}  // namespace flce
