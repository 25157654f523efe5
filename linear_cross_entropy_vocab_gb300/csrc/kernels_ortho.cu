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
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "norm_rows.cuh"
#include "ortho_internal.h"
#include "tc_ptx.cuh"

namespace flce {
namespace {

// ------------------------------------------------------------ norm and copy

// Sums of squares of a share of a matrix's rows: 32 values in 32 bits, those
// sums in 64, and again in 64 where a sum leaves the 32-bit range.
template <class T>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const OrthoCopyParams p) {
  __shared__ double buf[8];
  grid_launch_dependents();
  const T* const src = static_cast<const T*>(p.src) + blockIdx.y * p.batch_stride;
  // a share is a range of whole pieces of 32 columns x 256 threads
  const int64_t pieces_row = (p.cols + 31) / 32;
  const int64_t pieces = pieces_row * p.rows;
  double total = 0.0;
  for (int64_t i = blockIdx.x * int64_t(8) + (threadIdx.x >> 5); i * 32 < pieces;
       i += int64_t(gridDim.x) * 8) {
    // the warp's 32 pieces follow one another; its lanes read them side by side
    float sum = 0.0f;
    double wide = 0.0;
    float v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int64_t piece = i * 32 + k;
      v[k] = 0.0f;
      if (piece < pieces) {
        const int64_t r = piece / pieces_row, c = (piece - r * pieces_row) * 32 + (threadIdx.x & 31);
        if (c < p.cols) v[k] = to_f32(src[r * p.row_pitch + c]);
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) sum = fmaf(v[k], v[k], sum);
    wide = sum;
    if (!(sum < 3.0e38f && sum > 1.0e-30f)) {
      wide = 0.0;
#pragma unroll
      for (int k = 0; k < 32; ++k) wide += static_cast<double>(v[k]) * v[k];
    }
    total += wide;
  }
  total = team_all<256>(total, buf, SumOp{});
  if (threadIdx.x == 0) p.partial[int64_t(blockIdx.y) * p.parts + blockIdx.x] = total;
}

// Halves of a 64 x 64 part of the padded matrix, through shared memory where it
// is transposed.
template <class T>
__global__ void __launch_bounds__(256) ortho_copy_kernel(const OrthoCopyParams p) {
  __shared__ __half part[64][66];
  __shared__ double buf[8];
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.z;
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
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.factor[b] = factor;
  const int shift = -e;
  const T* const src = static_cast<const T*>(p.src) + b * p.batch_stride;
  __half* const x = static_cast<__half*>(p.x) + int64_t(b) * p.m_pad * p.n_pad;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;  // of x
  auto half_of = [&](float v) {
    return __float2half_rn(scalbnf(v, shift) * p.x_scale);
  };
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  if (p.tall) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = j0 + ty + 4 * k, c = i0 + tx;  // of src
      part[tx][ty + 4 * k] = r < p.rows && c < p.cols
                                 ? half_of(to_f32(src[int64_t(r) * p.row_pitch + c]))
                                 : __half(0.0f);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int i = i0 + ty + 4 * k, j = j0 + tx;
      x[int64_t(i) * p.n_pad + j] = part[ty + 4 * k][tx];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int i = i0 + ty + 4 * k, j = j0 + tx;
      x[int64_t(i) * p.n_pad + j] = i < p.rows && j < p.cols
                                        ? half_of(to_f32(src[int64_t(i) * p.row_pitch + j]))
                                        : __half(0.0f);
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
constexpr int kThreads = 192;
constexpr int kBoxBytes = 32 * 32 * 2;

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t done;
  uint32_t tmem;
  int abort;
};
constexpr int kSmemBytes =
    1024 + kStages * kStageBytes + 4 * 2 * kBoxBytes + static_cast<int>(sizeof(Ctl));

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
template <bool SYMMETRIC>
__device__ __forceinline__ Tile tile_of(const OrthoGemmParams& p, int u) {
  Tile t;
  if constexpr (SYMMETRIC) {
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
    t.n = r / p.m_tiles;
    t.m = r - t.n * p.m_tiles;
  }
  return t;
}

// 32 values of a row to a dense output row of `cols` columns.
template <class T>
__device__ __forceinline__ void store_row(T* row, int col, int cols, bool vec,
                                          const float (&v)[32]) {
  if (vec && col + 32 <= cols) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = v[8 * g + j];
      store8(row + col + 8 * g, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col + j < cols) row[col + j] = from_f32<T>(v[j]);
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
  Ctl* const ctl = reinterpret_cast<Ctl*>(boxes + 4 * 2 * kBoxBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = kSymmetric ? p.m_tiles * (p.m_tiles + 1) / 2 : p.m_tiles * p.n_tiles;
  const int total = per * p.batch;
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
      mbar_init(smem_addr(&ctl->acc_empty[b]), 8);  // the epilogue warps of both CTAs
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
      for (int u = unit0; u < total && ok; u += units) {
        const Tile t = tile_of<kSymmetric>(p, u);
        const int a_side = t.m * kOrthoTile + rank * kRows;
        const int b_side = t.n * kOrthoTile + rank * kRows;
        const int a_base = t.b * p.a_stride, b_base = t.b * p.b_stride;
        for (int k = 0; k < p.k_iters; ++k) {
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
      for (int u = unit0; u < total && ok; u += units, ++it) {
        const int buf = it & 1;
        if (!wait_pair(smem_addr(&ctl->acc_empty[buf]), ((it >> 1) & 1u) ^ 1u, abort_flag,
                       p.err_word))
          break;
        tc_fence_after_sync();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kCols);
        for (int k = 0; k < p.k_iters; ++k) {
          if (!wait_pair(smem_addr(&ctl->full[stage]), phase, abort_flag, p.err_word)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a0 = base + stage * kStageBytes, b0 = a0 + kOperandBytes;
#pragma unroll
          for (int kk = 0; kk < kDepth / 16; ++kk)
            umma_bf16_pair(d, slice_desc<kAcrossA>(a0, kk), slice_desc<kAcrossB>(b0, kk), idesc,
                           (k | kk) != 0 ? 1u : 0u);
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
    uint8_t* const box = boxes + quarter * 2 * kBoxBytes;
    uint8_t* const mirror = box + kBoxBytes;
    grid_dependency_wait();  // the gram and the factors
    int it = 0;
    for (int u = unit0; u < total; u += units, ++it) {
      const Tile t = tile_of<kSymmetric>(p, u);
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
        for (int i = 0; i < 4; ++i) held[i] = old[i];
      }
      if (!__all_sync(0xffffffffu, wait_pair(smem_addr(&ctl->acc_full[buf]), (it >> 1) & 1u,
                                             abort_flag, p.err_word)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(buf * kCols);
#pragma unroll 1
      for (int ch = 0; ch < kCols / 32; ++ch) {
        const int col = t.n * kOrthoTile + ch * 32;
        float v[32];
        tmem_load_32cols(taddr + static_cast<uint32_t>(ch * 32), v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= scale;
        if constexpr (OP == OrthoOp::kPoly) {
          const uint32_t w[16] = {held[0].x, held[0].y, held[0].z, held[0].w,
                                  held[1].x, held[1].y, held[1].z, held[1].w,
                                  held[2].x, held[2].y, held[2].z, held[2].w,
                                  held[3].x, held[3].y, held[3].z, held[3].w};
          if (ch + 1 < kCols / 32) {
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
        if constexpr (kOut) {
          if (row < p.rows) {
            T* const out = static_cast<T*>(p.out) + (int64_t(t.b) * p.rows + row) * p.cols;
            store_row(out, col, p.cols, (reinterpret_cast<uintptr_t>(out) & 15u) == 0, v);
          }
        } else if (col < p.cols) {  // boxes lie in c or outside it
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __half2 q = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&q);
          }
          // the boxes' last stores have read them
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
          uint4* const mine = reinterpret_cast<uint4*>(box + lane * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mine[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if (mirrored) {
            uint16_t* const to = reinterpret_cast<uint16_t*>(mirror) + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              to[64 * i] = static_cast<uint16_t>(w[i]);
              to[64 * i + 32] = static_cast<uint16_t>(w[i] >> 16);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.c_map, smem_addr(box), col, t.b * p.m_pad + row0);
            if (mirrored) tma_store_2d(&p.c_map, smem_addr(mirror), row0, t.b * p.m_pad + col);
            tma_store_commit();
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0)
        mbar_arrive_cluster(acc_empty + static_cast<uint32_t>(buf * sizeof(uint64_t)));
    }
    if (!kOut && lane == 0) tma_store_wait_all();
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
cudaError_t launch_op(const OrthoGemmParams& p, int sms, cudaStream_t s) {
  const auto kernel = ortho_gemm_kernel<OP, T>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t per = OP == OrthoOp::kGram || OP == OrthoOp::kPoly
                          ? int64_t(p.m_tiles) * (p.m_tiles + 1) / 2
                          : int64_t(p.m_tiles) * p.n_tiles;
  const int64_t tiles = per * p.batch;
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
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
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_pad / 64), static_cast<unsigned>(p.m_pad / 64),
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

cudaError_t launch_ortho_gemm(const OrthoGemmParams& p, OrthoOp op, int out_dtype, int sms,
                              cudaStream_t s) {
  switch (op) {
    case OrthoOp::kGram:
      return launch_op<OrthoOp::kGram, __half>(p, sms, s);
    case OrthoOp::kPoly:
      return launch_op<OrthoOp::kPoly, __half>(p, sms, s);
    case OrthoOp::kMul:
      return launch_op<OrthoOp::kMul, __half>(p, sms, s);
    case OrthoOp::kOutWide:
      return out_dtype == FLCE_BF16 ? launch_op<OrthoOp::kOutWide, __nv_bfloat16>(p, sms, s)
                                    : launch_op<OrthoOp::kOutWide, __half>(p, sms, s);
    case OrthoOp::kOutTall:
      return out_dtype == FLCE_BF16 ? launch_op<OrthoOp::kOutTall, __nv_bfloat16>(p, sms, s)
                                    : launch_op<OrthoOp::kOutTall, __half>(p, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace flce
