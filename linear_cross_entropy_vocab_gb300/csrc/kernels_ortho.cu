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
// m x n matrix, m <= n, against a few passes over it. A persistent kernel runs
// CTA pairs on 256 x 256 tiles (tcgen05.mma over the pair, operands staged by
// TMA in a ring of six 32 KB stages, two accumulators in tensor memory, so that
// a tile is stored behind the next one's products); launches overlap at their
// ends.
//
// The operands are halves with a power-of-two scale for each product, chosen by
// the host from the bounds on the singular values, so that nothing leaves the
// range. Their 11 bits at the rate of bf16's 8 keep the result within about
// 1.5e-3 of itself, where bf16 operands give 1e-2; sums are held in 32 bits.
// The norm's factor is applied to the first step's products, in 32 bits: a
// 16-bit input is copied without rounding.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "norm_rows.cuh"
#include "ortho_internal.h"
#include "tc_ptx.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------ norm and copy

// Sums of squares of a share of a matrix. Rows are read in spans of 8192
// values, in aligned 16-byte pieces wherever a row starts (a dense matrix is
// one long row); 32 values are summed in 32 bits, those sums in 64, and again
// in 64 where one leaves the 32-bit range.
template <class T>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const OrthoCopyParams p) {
  __shared__ double buf[8];
  grid_launch_dependents();
  const T* const src = static_cast<const T*>(p.src) + blockIdx.y * p.batch_stride;
  const bool dense = p.row_pitch == p.cols;
  const int64_t rows = dense ? 1 : p.rows;
  const int64_t len = dense ? int64_t(p.rows) * p.cols : p.cols;
  const int64_t spans_row = (len + 8191 + 8) / 8192;  // a row may start 7 values into its first
  double total = 0.0;
  for (int64_t i = blockIdx.x; i < rows * spans_row; i += gridDim.x) {
    const int64_t r = i / spans_row;
    const T* const row = src + r * p.row_pitch;
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7;
    const int64_t at = (i - r * spans_row) * 8192 - phase + threadIdx.x * 8;
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = at + k * 2048;
      if (e >= 0 && e + 8 <= len) {
        load8(row + e, v[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = e + j >= 0 && e + j < len ? to_f32(row[e + j]) : 0.0f;
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
    double wide = sum;
    if (!(sum < 3.0e38f && sum > 1.0e-30f)) {
      wide = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) wide += static_cast<double>(v[k][j]) * v[k][j];
    }
    total += wide;
  }
  total = team_all<256>(total, buf, SumOp{});
  if (threadIdx.x == 0) p.partial[int64_t(blockIdx.y) * p.parts + blockIdx.x] = total;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.arrived_count; i += 256) p.arrived[i] = 0;
}

// Where the halves of row i from column 8 * c on lie in a 64 x 64 part in
// shared memory: 16-byte pieces are swapped so that neither rows nor columns of
// pieces meet in a bank.
__device__ __forceinline__ int piece_at(int i, int c) { return i * 64 + ((c ^ (i >> 3)) & 7) * 8; }

// Halves of the padded matrix, 64 x 128 at a time. The transpose of a tall
// matrix, and rows that do not start at 16-byte boundaries, go through shared
// memory.
template <class T>
__global__ void __launch_bounds__(256) ortho_copy_kernel(const OrthoCopyParams p) {
  __shared__ __align__(16) __half part[2][64 * 64];
  __shared__ double buf[8];
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.y;
  const double* const partial = p.partial + int64_t(b) * p.parts;
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.parts; i += 256) sum += partial[i];
  sum = team_all<256>(sum, buf, SumOp{});
  const double norm = sqrt(sum) + static_cast<double>(p.eps);
  // x = src * 2^-e, so that 1/2 < factor <= 1; a norm that is not finite makes
  // every result NaN
  int e = 0;
  float factor = NAN;
  if (norm < INFINITY) {
    e = ilogb(norm);
    factor = static_cast<float>(scalbn(1.0 / norm, e));
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.factor[b] = factor;
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
      // rows that start anywhere: the nine aligned pieces that hold 64 values
      for (int u9 = threadIdx.x; u9 < halves * 64 * 9; u9 += 256) {
        const int line = u9 / 9, g = line >> 6, dr = line & 63;
        const int r = s0 + dr + (p.tall ? 64 * g : 0), c0 = t0 + (p.tall ? 0 : 64 * g);
        const T* const row = src + int64_t(r) * p.row_pitch;
        const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 7;
        const int c = c0 - ((c0 + phase) & 7) + (u9 - line * 9) * 8;
        float v[8] = {};
        if (r < p.rows) {
          if (c >= 0 && c + 8 <= p.cols) {
            load8(row + c, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j >= 0 && c + j < p.cols) v[j] = to_f32(row[c + j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int dc = c + j - c0;
          if (dc < 0 || dc >= 64) continue;
          const int i = p.tall ? dc : dr, at = p.tall ? dr : dc;
          part[g][piece_at(i, at >> 3) + (at & 7)] = half_of(v[j]);
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
constexpr int kCols = 256;
constexpr int kDepth = 64;  // of a stage: one 128-byte swizzle row of halves
constexpr int kStages = 6;
constexpr int kOperandBytes = kRows * kDepth * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = kOrthoWarps;  // two a quarter of the rows, with half of the columns each
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kBoxBytes = 32 * 32 * 2;

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t done;
  uint32_t tmem;
  int abort;
};
constexpr int kSmemBytes =
    1024 + kStages * kStageBytes + kEpilogueWarps * 2 * kBoxBytes +
    static_cast<int>(sizeof(Ctl));

template <bool ACROSS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                             int side, int depth) {
  if constexpr (!ACROSS) {
    tma_load_2d_pair(dst, map, bar, depth, side);  // {64 deep, 128 rows}
  } else {
    tma_load_2d_pair(dst, map, bar, side, depth);  // two boxes {64, 64 deep}
    tma_load_2d_pair(dst + 8192, map, bar, side + 64, depth);
  }
}
template <bool ACROSS>
__device__ __forceinline__ uint64_t slice_desc(uint32_t base, int kk) {
  return ACROSS ? smem_desc_sw128(base + kk * 2048, 8192, 1024)
                : smem_desc_sw128(base + kk * 32, 16, 1024);
}

__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* err_word) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitBudgetNs) {
        *abort_flag = 1;
        if (err_word) atomicOr(err_word, FLCE_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}
// Lets what is in flight finish, with a limit, whatever the abort flag says.
__device__ __forceinline__ void drain_pair(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (globaltimer_ns() - t0 > 1000000000ull) break;
  }
}

struct Tile {
  int b, m, n;
};
template <OrthoOp OP>
__device__ __forceinline__ Tile tile_of(const OrthoGemmParams& p, int u) {
  Tile t;
  if constexpr (OP == OrthoOp::kGram || OP == OrthoOp::kPoly) {
    const int per = p.m_tiles * (p.m_tiles + 1) / 2;
    t.b = u / per;
    int r = u - t.b * per;
    t.m = 0;
    while (r >= p.m_tiles - t.m) {
      r -= p.m_tiles - t.m;
      ++t.m;
    }
    t.n = t.m + r;
  } else {
    const int per = p.m_tiles * p.n_tiles;
    t.b = u / per;
    const int r = u - t.b * per;
    if constexpr (OP == OrthoOp::kOutTall) {  // p stays in L2, x passes once
      t.m = r / p.n_tiles;
      t.n = r - t.m * p.n_tiles;
    } else {
      t.n = r / p.m_tiles;
      t.m = r - t.n * p.m_tiles;
    }
  }
  return t;
}

// A stretch of a tile's contraction, [k0, k1).
struct Part {
  int tile, k0, k1;
};
// The parts of one pair of CTAs. The last `split_tiles` tiles are laid end to
// end and cut into as many equal stretches as there are pairs, so that all
// pairs end together; the tiles before them are taken whole, one pair after the
// other. The stretches come first: what joins their sums runs behind whole
// tiles' products.
struct Walk {
  int at, end, whole;
  static __device__ __forceinline__ int start(const OrthoGemmParams& p, int unit, int units) {
    return unit * (p.split_tiles * p.k_iters) / units;  // the host keeps this in 31 bits
  }
  __device__ __forceinline__ Walk(const OrthoGemmParams& p, int unit, int units)
      : at(start(p, unit, units)), end(start(p, unit + 1, units)), whole(unit) {}
  __device__ __forceinline__ bool next(const OrthoGemmParams& p, int units, Part& part) {
    if (at < end) {
      const int t = at / p.k_iters;
      part.tile = p.whole_tiles + t;
      part.k0 = at - t * p.k_iters;
      part.k1 = min(p.k_iters, part.k0 + end - at);
      at += part.k1 - part.k0;
      return true;
    }
    if (whole < p.whole_tiles) {
      part = {whole, 0, p.k_iters};
      whole += units;
      return true;
    }
    return false;
  }
};
// The pair that has iteration x of the stretches.
__device__ __forceinline__ int owner_of(const OrthoGemmParams& p, int x, int units) {
  return ((x + 1) * units - 1) / (p.split_tiles * p.k_iters);
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
// Where a pair leaves a warp's sums of a part: of the first part of a tile
// (which ends the pair's stretch) or of another (which begins it).
__device__ __forceinline__ float4* share_of(const OrthoGemmParams& p, int unit, bool first,
                                            int rank, int warp) {
  const int64_t slot = ((unit * 2 + (first ? 1 : 0)) * 2 + rank) * kEpilogueWarps + warp;
  return reinterpret_cast<float4*>(p.shares) + slot * (kCols / 64 * 8 * 32);
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (sizeof(T) == sizeof(__half) && !std::is_same_v<T, __half>) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <OrthoOp OP, class T>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_gemm_kernel(const __grid_constant__ OrthoGemmParams p) {
  constexpr bool kSymmetric = OP == OrthoOp::kGram || OP == OrthoOp::kPoly;
  constexpr bool kOut = OP == OrthoOp::kOutWide || OP == OrthoOp::kOutTall;
  constexpr bool kAcrossA = OP == OrthoOp::kOutTall;
  constexpr bool kAcrossB = OP == OrthoOp::kMul || OP == OrthoOp::kOutWide;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const boxes = smem_raw + (base - raw) + kStages * kStageBytes;
  Ctl* const ctl = reinterpret_cast<Ctl*>(boxes + kEpilogueWarps * 2 * kBoxBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int unit0 = blockIdx.x >> 1, units = gridDim.x >> 1;
  volatile int* const abort_flag = &ctl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&ctl->acc_full[b]), 1);
      mbar_init(smem_addr(&ctl->acc_empty[b]), 2 * kEpilogueWarps);  // of both CTAs
    }
    mbar_init(smem_addr(&ctl->done), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a_map);
    tma_prefetch_desc(&p.b_map);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&ctl->tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem;
  if (threadIdx.x == 0) grid_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      // ---- loads: each CTA its 128 rows of a and 128 of b's 256
      int stage = 0;
      uint32_t phase = 0, armed = 0, last = 0;
      bool ok = true;
      grid_dependency_wait();
      Walk walk(p, unit0, units);
      for (Part part; ok && walk.next(p, units, part);) {
        const Tile t = tile_of<OP>(p, part.tile);
        const int a_side = t.m * kOrthoTile + rank * kRows;
        const int b_side = t.n * kOrthoTile + rank * kRows;
        const int a_base = t.b * p.a_stride, b_base = t.b * p.b_stride;
        for (int k = part.k0; k < part.k1; ++k) {
          if (!wait_pair(smem_addr(&ctl->empty[stage]), phase ^ 1u, abort_flag, p.err_word)) {
            ok = false;
            break;
          }
          const uint32_t full_local = smem_addr(&ctl->full[stage]);
          const uint32_t full = map_to_rank(full_local, 0);
          if (leader) mbar_arrive_expect_tx(full_local, 2 * kStageBytes);
          const uint32_t dst = base + stage * kStageBytes;
          load_operand<kAcrossA>(dst, &p.a_map, full, kAcrossA ? a_side : a_base + a_side,
                                 kAcrossA ? a_base + k * kDepth : k * kDepth);
          load_operand<kAcrossB>(dst + kOperandBytes, &p.b_map, full,
                                 kAcrossB ? b_side : b_base + b_side,
                                 kAcrossB ? b_base + k * kDepth : k * kDepth);
          armed |= 1u << stage;
          last = (last & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        for (int s = 0; s < kStages; ++s)
          if (armed & (1u << s)) drain_pair(smem_addr(&ctl->full[s]), (last >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---- products
      constexpr uint32_t idesc =
          idesc_f16kind_f32(2 * kRows, kCols, kAcrossA ? 1 : 0, kAcrossB ? 1 : 0, 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;
      Walk walk(p, unit0, units);
      for (Part part; ok && walk.next(p, units, part); ++it) {
        const int buf = it & 1;
        if (!wait_pair(smem_addr(&ctl->acc_empty[buf]), ((it >> 1) & 1u) ^ 1u, abort_flag,
                       p.err_word))
          break;
        tc_fence_after_sync();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kCols);
        for (int k = part.k0; k < part.k1; ++k) {
          if (!wait_pair(smem_addr(&ctl->full[stage]), phase, abort_flag, p.err_word)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a0 = base + stage * kStageBytes, b0 = a0 + kOperandBytes;
#pragma unroll
          for (int kk = 0; kk < kDepth / 16; ++kk)
            umma_bf16_pair(d, slice_desc<kAcrossA>(a0, kk), slice_desc<kAcrossB>(b0, kk), idesc,
                           k != part.k0 || kk != 0 ? 1u : 0u);
          umma_commit_pair(smem_addr(&ctl->empty[stage]), 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit_pair(smem_addr(&ctl->acc_full[buf]), 0x3);
      }
      umma_commit_pair(smem_addr(&ctl->done), 0x3);
      drain_pair(smem_addr(&ctl->done), 0);
    } else if (lane == 0) {
      // the other CTA's products write this one's tensor memory
      drain_pair(smem_addr(&ctl->done), 0);
    }
  } else {
    // ---- results: a thread has a row of the tile, 32 columns at a time
    const int quarter = warp & 3;
    const uint32_t acc_empty = map_to_rank(smem_addr(&ctl->acc_empty[0]), 0);
    const int first = (warp - 2) >> 2 ? kCols / 64 : 0;  // of the eight pieces of 32 columns
    uint8_t* const box = boxes + (warp - 2) * 2 * kBoxBytes;
    uint8_t* const mirror = box + kBoxBytes;
    grid_dependency_wait();  // the gram and the factors
    int it = 0;
    Walk walk(p, unit0, units);
    for (Part part; walk.next(p, units, part); ++it) {
      const Tile t = tile_of<OP>(p, part.tile);
      const int buf = it & 1;
      const int row0 = t.m * kOrthoTile + rank * kRows + quarter * 32;  // of the matrix
      const int row = row0 + lane;
      const bool mirrored = kSymmetric && t.n > t.m;
      float scale = p.acc_scale;
      if (p.factor != nullptr) {
        const float f = p.factor[t.b];
        scale *= p.factor_square ? f * f : f;
      }
      const uint4* old = nullptr;
      uint4 held[4];
      if constexpr (OP == OrthoOp::kPoly) {
        old = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.old) +
                                             (int64_t(t.b) * p.m_pad + row) * p.m_pad +
                                             t.n * kOrthoTile);
#pragma unroll
        for (int i = 0; i < 4; ++i) held[i] = old[4 * first + i];
      }
      if (!__all_sync(0xffffffffu, wait_pair(smem_addr(&ctl->acc_full[buf]), (it >> 1) & 1u,
                                             abort_flag, p.err_word)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(buf * kCols);
      // Pieces of the tile that this warp keeps. Where the tile's contraction
      // is cut, each pair leaves its sums, and the warp that comes last adds
      // all of them, in the order of the contraction.
      const int pieces =
          row0 >= p.rows ? 0 : min(kCols / 64, (p.cols - t.n * kOrthoTile - first * 32 + 31) / 32);
      int from = unit0, to = unit0;
      if (part.k1 - part.k0 < p.k_iters && pieces > 0) {
        const int x = (part.tile - p.whole_tiles) * p.k_iters;
        from = owner_of(p, x, units);
        to = owner_of(p, x + p.k_iters - 1, units);
        int* const counter = p.arrived +
            ((part.tile - p.whole_tiles) * 2 + rank) * kEpilogueWarps + warp - 2;
        int before = 0;
        if (lane == 0) before = *reinterpret_cast<volatile int*>(counter);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before != to - from) {
          float4* const mine = share_of(p, unit0, unit0 == from, rank, warp - 2) + lane;
#pragma unroll 1
          for (int i = 0; i < pieces; ++i) {
            float v[32];
            tmem_load_32cols(taddr + static_cast<uint32_t>((first + i) * 32), v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              mine[(i * 8 + j) * 32] =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
          __threadfence();
          __syncwarp();
          if (lane == 0) before = atomicAdd(counter, 1);
          before = __shfl_sync(0xffffffffu, before, 0);
        }
        if (before == to - from && lane == 0) *counter = 0;  // for the next launch
        __threadfence();
        __syncwarp();
        if (before != to - from) from = to + 1;  // not the last
      }
#pragma unroll 1
      for (int i = 0; from <= to && i < pieces; ++i) {
        const int ch = first + i;
        const int col = t.n * kOrthoTile + ch * 32;
        float v[32];
        tmem_load_32cols(taddr + static_cast<uint32_t>(ch * 32), v);
        if (from < to) {
          float sum[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[j] = 0.0f;
          for (int q = from; q <= to; ++q) {
            if (q == unit0) {
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[j] += v[j];
            } else {
              const float4* const other = share_of(p, q, q == from, rank, warp - 2) + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 f = __ldcg(other + (i * 8 + j) * 32);
                sum[4 * j] += f.x;
                sum[4 * j + 1] += f.y;
                sum[4 * j + 2] += f.z;
                sum[4 * j + 3] += f.w;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[j];
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= scale;
        if constexpr (OP == OrthoOp::kPoly) {
          const uint32_t w[16] = {held[0].x, held[0].y, held[0].z, held[0].w,
                                  held[1].x, held[1].y, held[1].z, held[1].w,
                                  held[2].x, held[2].y, held[2].z, held[2].w,
                                  held[3].x, held[3].y, held[3].z, held[3].w};
          if (ch + 1 < first + kCols / 64) {
#pragma unroll
            for (int i = 0; i < 4; ++i) held[i] = old[4 * (ch + 1) + i];
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = fmaf(g.x, p.old_scale, v[2 * i]);
            v[2 * i + 1] = fmaf(g.y, p.old_scale, v[2 * i + 1]);
          }
          if (row - col >= 0 && row - col < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (row - col == j) v[j] += p.diag;
          }
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        // the boxes' last contents have been taken
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(box + box_at(lane, i)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        if (mirrored) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            *reinterpret_cast<uint16_t*>(mirror + box_at(i, lane >> 3) + (lane & 7) * 2) =
                static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
        if (kOut && !p.out_mapped) {
          // rows that no map can describe: 32 values of one after the other
          __syncwarp();
          T* const out = static_cast<T*>(p.out) +
                         (int64_t(t.b) * p.rows + row0) * p.cols + col + lane;
          const int rows = p.rows - row0 < 32 ? p.rows - row0 : 32;
          if (col + lane < p.cols) {
#pragma unroll 8
            for (int r = 0; r < rows; ++r)
              out[int64_t(r) * p.cols] = *reinterpret_cast<const T*>(
                  box + box_at(r, lane >> 3) + (lane & 7) * 2);
          }
          continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kOut)
            tma_store_3d(&p.c_map, smem_addr(box), col, row0, t.b);
          else
            tma_store_2d(&p.c_map, smem_addr(box), col, t.b * p.m_pad + row0);
          if (mirrored) tma_store_2d(&p.c_map, smem_addr(mirror), row0, t.b * p.m_pad + col);
          tma_store_commit();
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0)
        mbar_arrive_cluster(acc_empty + static_cast<uint32_t>(buf * sizeof(uint64_t)));
    }
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <OrthoOp OP, class T>
cudaError_t launch_op(const OrthoGemmParams& p, cudaStream_t s) {
  const auto kernel = ortho_gemm_kernel<OP, T>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T>
cudaError_t launch_copy(const OrthoCopyParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  // CTAs that each find the norm once: six an SM over the batch
  const int64_t tiles = int64_t((p.n_pad + 127) / 128) * (p.m_rows / 64);
  const int64_t most = std::max<int64_t>(1, 6 * 152 / p.batch);
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

cudaError_t launch_ortho_gemm(const OrthoGemmParams& p, OrthoOp op, int out_dtype,
                              cudaStream_t s) {
  switch (op) {
    case OrthoOp::kGram:
      return launch_op<OrthoOp::kGram, __half>(p, s);
    case OrthoOp::kPoly:
      return launch_op<OrthoOp::kPoly, __half>(p, s);
    case OrthoOp::kMul:
      return launch_op<OrthoOp::kMul, __half>(p, s);
    case OrthoOp::kOutWide:
      return out_dtype == FLCE_BF16 ? launch_op<OrthoOp::kOutWide, __nv_bfloat16>(p, s)
                                    : launch_op<OrthoOp::kOutWide, __half>(p, s);
    case OrthoOp::kOutTall:
      return out_dtype == FLCE_BF16 ? launch_op<OrthoOp::kOutTall, __nv_bfloat16>(p, s)
                                    : launch_op<OrthoOp::kOutTall, __half>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace flce
