// Orthogonalising matrices with one side of at most 128 (see kernels_ortho.cu
// for the steps): a matrix stays in the shared memory of a cluster of CTAs for
// all steps.
//
// Bound by the length of a chain of small products: each CTA of a cluster has
// all m rows (padded to 128) of up to 512 columns in shared memory as halves,
// and each step is a gram (tcgen05.mma, 128 x 128 over its columns), summed over
// the cluster through distributed shared memory in the order of the CTAs, the
// polynomial, which every CTA computes, and the product on its own columns, in
// place. The same bytes are the gram's operand along the columns and the
// product's across them: both forms of the 128-byte swizzle put 64 values of a
// row into 128 bytes and rows 128 bytes apart.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "norm_rows.cuh"
#include "ortho_internal.h"
#include "tc_ptx.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSide = 128;
constexpr int kBlockBytes = kSide * 128;  // 64 columns of all rows
constexpr int kGramBytes = 2 * kBlockBytes;
constexpr int kExchangeBytes = kSide * kSide * 4;

struct Ctl {
  uint64_t done;
  double squares[kWarps];
  double total[kOrthoMaxCluster];
  uint32_t tmem;
  int abort;
};

// Byte offset of the 16-byte piece of columns 8c to 8c + 7 of row r.
__device__ __forceinline__ int piece_of(int r, int c) {
  return (c >> 3) * kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ void store_cluster4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void store_cluster2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void store_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// Eight values of x, row i from column j on, or for a tall matrix column j from
// row i on: `along` consecutive elements of src either way. Zeros outside.
template <class T>
__device__ __forceinline__ void load_piece(const T* row, int at, int len, bool vec, float (&v)[8]) {
  if (vec && at + 8 <= len) {
    load8(row + at, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = at + k < len ? to_f32(row[at + k]) : 0.0f;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_small_kernel(const __grid_constant__ OrthoSmallParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const x = smem_raw + (base - raw);
  uint8_t* const gram = x + p.slab / 64 * kBlockBytes;
  float* const exchange = reinterpret_cast<float*>(gram + kGramBytes);
  Ctl* const ctl = reinterpret_cast<Ctl*>(gram + kGramBytes + (p.cluster > 1 ? kExchangeBytes : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ranks = p.cluster;
  const int rank = static_cast<int>(blockIdx.x) % ranks, b = static_cast<int>(blockIdx.x) / ranks;
  if (tid == 0) {
    mbar_init(smem_addr(&ctl->done), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctl->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  cluster_sync();  // all CTAs have started: their shared memory can be written
  tc_fence_after_sync();
  // ---- the slab: columns [j0, j0 + slab) of x
  const T* const src = static_cast<const T*>(p.src) + b * p.batch_stride;
  const int m = p.tall ? p.cols : p.rows, n = p.tall ? p.rows : p.cols;
  const int j0 = rank * p.slab;
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 &&
                   p.row_pitch * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  const int m8 = (m + 7) / 8;
  double squares = 0.0;
  const auto count = [&](const float(&v)[8]) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
    double wide = sum;
    if (!(sum < 3.0e38f && sum > 1.0e-30f)) {
      wide = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) wide += static_cast<double>(v[k]) * v[k];
    }
    squares += wide;
  };
  // Both passes walk the source alike: the squares, and then the halves.
  const auto walk = [&](auto take) {
    if (p.tall) {  // a lane a row of src, eight of its columns
      for (int u = tid; u < p.slab * m8; u += kThreads) {
        const int i = u / p.slab * 8, j = u % p.slab;
        float v[8] = {};
        if (j0 + j < n) load_piece(src + int64_t(j0 + j) * p.row_pitch, i, m, vec, v);
        take(i, j, v);
      }
    } else {
      const int pieces = p.slab / 8;
      for (int u = tid; u < m * pieces; u += kThreads) {
        const int i = u / pieces, j = u % pieces * 8;
        float v[8];
        load_piece(src + int64_t(i) * p.row_pitch, j0 + j, n, vec, v);
        take(i, j, v);
      }
    }
  };
  walk([&](int, int, const float(&v)[8]) { count(v); });
  // zeros where no row is written
  for (int u = tid; u < (kSide - m8 * 8) * (p.slab / 8); u += kThreads)
    *reinterpret_cast<uint4*>(x + piece_of(m8 * 8 + u / (p.slab / 8), u % (p.slab / 8))) =
        make_uint4(0, 0, 0, 0);
  if (!p.tall)
    for (int u = tid; u < (m8 * 8 - m) * (p.slab / 8); u += kThreads)
      *reinterpret_cast<uint4*>(x + piece_of(m + u / (p.slab / 8), u % (p.slab / 8))) =
          make_uint4(0, 0, 0, 0);
  squares = team_all<kThreads>(squares, ctl->squares, SumOp{});
  if (tid < ranks)
    store_cluster_f64(map_to_rank(smem_addr(&ctl->total[rank]), tid), squares);
  cluster_sync();
  const uint32_t tmem = ctl->tmem;
  double total = 0.0;
  for (int k = 0; k < ranks; ++k) total += ctl->total[k];
  const double norm = sqrt(total) + static_cast<double>(p.eps);
  // as in the copy of larger matrices: x = src * 2^(x_shift - e), and a factor
  // in (1/2, 1] that is applied to the first step's sums
  int e = 0;
  float factor = NAN;
  if (norm < INFINITY) {
    e = ilogb(norm);
    factor = static_cast<float>(scalbn(1.0 / norm, e));
  }
  const int shift = p.x_shift - e;
  const float scale0 = scalbnf(1.0f, shift / 2), scale1 = scalbnf(1.0f, shift - shift / 2);
  walk([&](int i, int j, const float(&v)[8]) {
    if (p.tall) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<__half*>(x + piece_of(i + k, j >> 3) + (j & 7) * 2) =
            __float2half_rn(v[k] * scale0 * scale1);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = half2_bits(v[2 * k] * scale0 * scale1, v[2 * k + 1] * scale0 * scale1);
      *reinterpret_cast<uint4*>(x + piece_of(i, j >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  });
  fence_proxy_async_all();
  __syncthreads();

  // ---- the steps. A warp has a quarter of the rows and half of the columns.
  const int row = (warp & 3) * 32 + lane, half = warp >> 2;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t done = smem_addr(&ctl->done);
  const uint32_t x_at = base, gram_at = smem_addr(gram);
  uint32_t phase = 0;
  const auto finished = [&] {
    mbar_wait(done, phase, &ctl->abort, p.err_word);
    phase ^= 1u;
    tc_fence_after_sync();
  };
  // what all threads have written to shared memory is there for the products
  const auto written = [&] {
    fence_proxy_async_all();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  };
  // 32 halves of a row of the gram or the polynomial from column 64 half + 32 g
  const auto gram_piece = [&](int g, int k) { return gram + piece_of(row, half * 8 + g * 4 + k); };
  for (int s = 0; s < p.steps; ++s) {
    const OrthoStep& st = p.step[s];
    const float f = s == 0 ? factor : 1.0f;
    if (tid == 0) {
      constexpr uint32_t idesc = idesc_f16kind_f32(kSide, kSide, 0, 0, 0);
      for (int k = 0; k < p.slab / 16; ++k) {
        const uint64_t d = smem_desc_sw128(x_at + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(tmem, d, d, idesc, k != 0 ? 1u : 0u);
      }
      umma_commit(done);
    }
    finished();
    if (ranks == 1) {
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        float v[32];
        tmem_load_32cols(lanes + half * 64 + g * 32, v);
        const float scale = st.gram * f * f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = half2_bits(v[8 * k + 2 * q] * scale, v[8 * k + 2 * q + 1] * scale);
          *reinterpret_cast<uint4*>(gram_piece(g, k)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    } else {
      // each CTA adds up its share of the rows and sends the halves to all
      const int rows = kSide / ranks, owner = row / rows;
      const uint32_t to = map_to_rank(smem_addr(exchange), owner) +
                          static_cast<uint32_t>((rank * rows + row - owner * rows) * kSide * 4);
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        float v[32];
        tmem_load_32cols(lanes + half * 64 + g * 32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          // pieces of a row turned by its number: rows are 512 bytes apart
          store_cluster4(to + (((half * 16 + g * 8 + k) ^ (row & 7)) << 4),
                         make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
      }
      tc_fence_before_sync();
      cluster_sync();
      tc_fence_after_sync();
      const float scale = st.gram * f * f;
      for (int u = tid; u < rows * 32; u += kThreads) {
        const int r = u >> 5, c4 = u & 31, full = rank * rows + r;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < ranks; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(
              exchange + (k * rows + r) * kSide + ((c4 ^ (full & 7)) << 2));
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        const uint32_t w0 = half2_bits(sum.x * scale, sum.y * scale);
        const uint32_t w1 = half2_bits(sum.z * scale, sum.w * scale);
        const uint32_t at = gram_at + piece_of(full, c4 >> 1) + (c4 & 1) * 8;
        for (int k = 0; k < ranks; ++k) store_cluster2(map_to_rank(at, k), w0, w1);
      }
      fence_proxy_async_all();
      cluster_sync();
    }
    written();
    if (tid == 0) {
      constexpr uint32_t idesc = idesc_f16kind_f32(kSide, kSide, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kSide / 16; ++k) {
        const uint64_t d =
            smem_desc_sw128(gram_at + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(tmem + kSide, d, d, idesc, k != 0 ? 1u : 0u);
      }
      umma_commit(done);
    }
    finished();
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      float v[32];
      tmem_load_32cols(lanes + kSide + half * 64 + g * 32, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4* const at = reinterpret_cast<uint4*>(gram_piece(g, k));
        const uint4 old = *at;
        const uint32_t h[4] = {old.x, old.y, old.z, old.w};
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[q]));
          const int col = half * 64 + g * 32 + 8 * k + 2 * q;
          float lo = fmaf(v[8 * k + 2 * q], st.poly, a.x * st.old);
          float hi = fmaf(v[8 * k + 2 * q + 1], st.poly, a.y * st.old);
          lo += row == col ? st.diag : 0.0f;
          hi += row == col + 1 ? st.diag : 0.0f;
          w[q] = half2_bits(lo, hi);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    written();
    if (tid == 0) {
      for (int c = 0; c < p.slab; c += 256) {
        const int cols = p.slab - c < 256 ? p.slab - c : 256;
        const uint32_t idesc = idesc_f16kind_f32(kSide, cols, 0, 1, 0);
#pragma unroll
        for (int k = 0; k < kSide / 16; ++k)
          umma_bf16(tmem + c,
                    smem_desc_sw128(gram_at + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024),
                    smem_desc_sw128(x_at + (c / 64) * kBlockBytes + k * 2048, kBlockBytes, 1024),
                    idesc, k != 0 ? 1u : 0u);
      }
      umma_commit(done);
    }
    finished();
    const float scale = st.product * f;
    const bool last = s + 1 == p.steps;
    const int groups = p.slab / 32;
#pragma unroll 1
    for (int g = half; g < groups; g += 2) {
      float v[32];
      tmem_load_32cols(lanes + g * 32, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float lo = v[8 * k + 2 * q] * scale, hi = v[8 * k + 2 * q + 1] * scale;
          if (last && p.out_bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[q] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            w[q] = half2_bits(lo, hi);
          }
        }
        *reinterpret_cast<uint4*>(x + piece_of(row, g * 4 + k)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    written();
  }

  // ---- the result, from shared memory
  uint16_t* const out = static_cast<uint16_t*>(p.out) + int64_t(b) * p.rows * p.cols;
  if (p.tall) {
    for (int u = tid; u < p.slab * m; u += kThreads) {
      const int i = u % m, j = u / m;
      if (j0 + j < n)
        out[int64_t(j0 + j) * p.cols + i] =
            *reinterpret_cast<const uint16_t*>(x + piece_of(i, j >> 3) + (j & 7) * 2);
    }
  } else if (p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0) {
    const int pieces = p.slab / 8;
    for (int u = tid; u < m * pieces; u += kThreads) {
      const int i = u / pieces, c = u % pieces;
      if (j0 + c * 8 < n)
        *reinterpret_cast<uint4*>(out + int64_t(i) * p.cols + j0 + c * 8) =
            *reinterpret_cast<const uint4*>(x + piece_of(i, c));
    }
  } else {
    for (int u = tid; u < m * p.slab; u += kThreads) {
      const int i = u / p.slab, j = u % p.slab;
      if (j0 + j < n)
        out[int64_t(i) * p.cols + j0 + j] =
            *reinterpret_cast<const uint16_t*>(x + piece_of(i, j >> 3) + (j & 7) * 2);
    }
  }
  tc_fence_before_sync();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <class T>
cudaError_t launch_small(const OrthoSmallParams& p, cudaStream_t s) {
  const int need = 1024 + p.slab / 64 * kBlockBytes + kGramBytes +
                   (p.cluster > 1 ? kExchangeBytes : 0) + static_cast<int>(sizeof(Ctl));
  // One CTA an SM: CTAs of two clusters that waited for each other's tensor
  // memory would never end.
  const int bytes = need > 120 * 1024 ? need : 120 * 1024;
  const auto kernel = ortho_small_kernel<T>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_ortho_small(const OrthoSmallParams& p, int dtype, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_small<float>(p, s);
  if (dtype == FLCE_BF16) return launch_small<__nv_bfloat16>(p, s);
  return launch_small<__half>(p, s);
}

}  // namespace flce
