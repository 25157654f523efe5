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
// row into 128 bytes and rows 128 bytes apart. Five steps of 128 x 256 take 28 us
// (one after the other in a graph; 35 with cold caches): 3.6 a step, and 10 to come
// and go. In a cluster a step takes 10, most of which is the exchange: 100 x 2048
// takes 59 us, 128 x 4096 64.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "norm_rows.cuh"
#include "ortho_internal.h"
#include "ortho_norm.cuh"
#include "tc_ptx.cuh"

namespace flce {
namespace {

constexpr int kThreads = 512;
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
  int abort, exponent;
  float factor;
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

// Eight values of a row of src from `at` on, zeros past its end.
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
  double squares = 0.0;
  // Both passes walk the source alike, 64 columns of x at a time and two pieces
  // a thread: the squares, and then the halves. A tall matrix gives a thread a
  // row of src and eight of its columns. (With divisions for the places, 128 x
  // 512 values took a CTA 29 us to come and go, 13 now.)
  const auto walk = [&](auto all, auto take) {
    for (int at = 0; at < p.slab; at += 64) {
      float v[2][8];
      const int j = p.tall ? at + (tid & 63) : at + (tid & 7) * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = p.tall ? ((tid >> 6) + 8 * q) * 8 : (tid >> 3) + 64 * q;
        const int r = p.tall ? j0 + j : i, c = p.tall ? i : j0 + j;  // of src
        if (r < p.rows && c < p.cols) {
          load_piece(src + int64_t(r) * p.row_pitch, c, p.cols, vec, v[q]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[q][k] = 0.0f;
        }
      }
      all(v);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        take(p.tall ? ((tid >> 6) + 8 * q) * 8 : (tid >> 3) + 64 * q, j, v[q]);
    }
  };
  const auto count = [&](const float(&v)[2][8]) {
    // 16 squares in 32 bits, or in 64 where those do not hold them
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(v[q][k], v[q][k], sum);
    double wide = sum;
    if (!(sum < 3.0e38f && sum > 1.0e-30f)) {
      wide = 0.0;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < 8; ++k) wide += static_cast<double>(v[q][k]) * v[q][k];
    }
    squares += wide;
  };
  // Whole aligned pieces that the registers hold are loaded at once and once.
  constexpr int kHeld = sizeof(T) == 4 ? 4 : 8;  // of 64 columns
  const bool held = vec && p.cols % 8 == 0 && p.slab <= kHeld * 64;
  Raw<T> raws[kHeld][2];
  if (held) {
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      const int j = p.tall ? g * 64 + (tid & 63) : g * 64 + (tid & 7) * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = p.tall ? ((tid >> 6) + 8 * q) * 8 : (tid >> 3) + 64 * q;
        const int r = p.tall ? j0 + j : i, c = p.tall ? i : j0 + j;
        if (g * 64 < p.slab && r < p.rows && c < p.cols)
          raws[g][q].load(src + int64_t(r) * p.row_pitch + c);
        else
          raws[g][q].clear();
      }
    }
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      float v[2][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) raws[g][q].values(v[q]);
      if (g * 64 < p.slab) count(v);
    }
  } else {
    walk(count, [](int, int, const float(&)[8]) {});
  }
  squares = team_all<kThreads>(squares, ctl->squares, SumOp{});
  if (tid < ranks)
    store_cluster_f64(map_to_rank(smem_addr(&ctl->total[rank]), tid), squares);
  cluster_sync();
  const uint32_t tmem = ctl->tmem;
  // As in the copy of larger matrices: x = src * 2^(x_shift - e), and a factor
  // in (1/2, 1] that is applied to the first step's sums. By one thread, as
  // 64-bit arithmetic is slow.
  if (tid == 0) {
    double total = 0.0;
    for (int k = 0; k < ranks; ++k) total += ctl->total[k];
    norm_factor(total, p.eps, ctl->exponent, ctl->factor);
  }
  __syncthreads();
  const int e = ctl->exponent;
  const float factor = ctl->factor;
  const int shift = p.x_shift - e;
  const float scale0 = scalbnf(1.0f, shift / 2), scale1 = scalbnf(1.0f, shift - shift / 2);
  const auto put = [&](int i, int j, const float(&v)[8]) {
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
  };
  if (held) {
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      const int j = p.tall ? g * 64 + (tid & 63) : g * 64 + (tid & 7) * 8;
      if (g * 64 < p.slab) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float v[8];
          raws[g][q].values(v);
          put(p.tall ? ((tid >> 6) + 8 * q) * 8 : (tid >> 3) + 64 * q, j, v);
        }
      }
    }
  } else {
    walk([](const float(&)[2][8]) {}, put);
  }
  fence_proxy_async_all();
  __syncthreads();

  // ---- the steps. A warp has a quarter of the rows and of the columns.
  const int row = (warp & 3) * 32 + lane, part = warp >> 2;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t done = smem_addr(&ctl->done);
  const uint32_t x_at = base, gram_at = smem_addr(gram);
  uint32_t phase = 0;
  const auto finished = [&] {
    mbar_wait(done, phase, &ctl->abort, p.err_word);
    phase ^= 1u;
    tc_fence_after_sync();
  };
  // Once a wait has given up no more products are issued, and what is left of
  // the steps is walked through with whatever is there: every CTA of the cluster
  // has to come to all of its barriers.
  const auto issues = [&] {
    return tid == 0 && *static_cast<volatile int*>(&ctl->abort) == 0;
  };
  uint32_t issued = 0;  // groups of products, by thread 0
  // what all threads have written to shared memory is there for the products
  const auto written = [&] {
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  };
  // of the thread's 32 halves of the gram or the polynomial
  const auto gram_piece = [&](int k) { return gram + piece_of(row, part * 4 + k); };
  for (int s = 0; s < p.steps; ++s) {
    const OrthoStep& st = p.step[s];
    const float f = s == 0 ? factor : 1.0f;
    if (issues()) {
      constexpr uint32_t idesc = idesc_f16kind_f32(kSide, kSide, 0, 0, 0);
      for (int k = 0; k < p.slab / 16; ++k) {
        const uint64_t d = smem_desc_sw128(x_at + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(tmem, d, d, idesc, k != 0 ? 1u : 0u);
      }
      umma_commit(done);
      ++issued;
    }
    finished();
    if (ranks == 1) {
      float v[32];
      tmem_load_32cols(lanes + part * 32, v);
      const float scale = st.gram * f * f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = half2_bits(v[8 * k + 2 * q] * scale, v[8 * k + 2 * q + 1] * scale);
        *reinterpret_cast<uint4*>(gram_piece(k)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      // each CTA adds up its share of the rows and sends the halves to all
      const int rows = kSide / ranks, owner = row / rows;
      const uint32_t to = map_to_rank(smem_addr(exchange), owner) +
                          static_cast<uint32_t>((rank * rows + row - owner * rows) * kSide * 4);
      float v[32];
      tmem_load_32cols(lanes + part * 32, v);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        // pieces of a row turned by its number: rows are 512 bytes apart
        store_cluster4(to + (((part * 8 + k) ^ (row & 7)) << 4),
                       make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
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
    if (issues()) {
      constexpr uint32_t idesc = idesc_f16kind_f32(kSide, kSide, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kSide / 16; ++k) {
        const uint64_t d =
            smem_desc_sw128(gram_at + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(tmem + kSide, d, d, idesc, k != 0 ? 1u : 0u);
      }
      umma_commit(done);
      ++issued;
    }
    finished();
    {
      float v[32];
      tmem_load_32cols(lanes + kSide + part * 32, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4* const at = reinterpret_cast<uint4*>(gram_piece(k));
        const uint4 old = *at;
        const uint32_t h[4] = {old.x, old.y, old.z, old.w};
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[q]));
          const int col = part * 32 + 8 * k + 2 * q;
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
    if (issues()) {
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
      ++issued;
    }
    finished();
    const float scale = st.product * f;
    const bool last = s + 1 == p.steps;
    const int groups = p.slab / 32;
#pragma unroll 1
    for (int g = part; g < groups; g += 4) {
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
  const auto value = [&](int i, int j) {
    return *reinterpret_cast<const uint16_t*>(x + piece_of(i, j >> 3) + (j & 7) * 2);
  };
  const bool whole = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  for (int at = 0; at < p.slab && j0 + at < n; at += 64) {
    if (p.tall) {  // a row of out is a column of x
      const int i = tid & 127;
#pragma unroll 8
      for (int q = 0; q < 16; ++q) {
        const int j = at + (tid >> 7) + 4 * q;
        if (i < m && j0 + j < n) out[int64_t(j0 + j) * p.cols + i] = value(i, j);
      }
    } else if (whole) {
      const int j = at + (tid & 7) * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = (tid >> 3) + 64 * q;
        if (i < m && j0 + j < n)
          *reinterpret_cast<uint4*>(out + int64_t(i) * p.cols + j0 + j) =
              *reinterpret_cast<const uint4*>(x + piece_of(i, j >> 3));
      }
    } else {
      const int j = at + (tid & 63);
#pragma unroll 8
      for (int q = 0; q < 16; ++q) {
        const int i = (tid >> 6) + 8 * q;
        if (i < m && j0 + j < n) out[int64_t(i) * p.cols + j0 + j] = value(i, j);
      }
    }
  }
  if (tid == 0 && ctl->abort != 0 && issued > 0) {
    // the last products, which may still write to tensor memory
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(done, (issued - 1) & 1u) && globaltimer_ns() - t0 < 1000000000ull) {
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
  // All of an SM's shared memory: where two CTAs share an SM's tensor memory,
  // those of two clusters could wait for each other's and never end.
  constexpr int kBytes = 227 * 1024;
  static_assert(1024 + 512 / 64 * kBlockBytes + kGramBytes + kExchangeBytes +
                        static_cast<int>(sizeof(Ctl)) <= kBytes,
                "the widest slab does not fit");
  const auto kernel = ortho_small_kernel<T>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
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
