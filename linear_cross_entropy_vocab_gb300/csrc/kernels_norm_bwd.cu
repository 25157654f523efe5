// Gradients of the root-mean-square norm with the residual's addition. With
// unit = s * rstd and u = grad_y * w:
//
//   grad_s = grad_sum + rstd * (u - unit * mean(u * unit))
//   grad_w = sum over the rows of grad_y * unit
//
// grad_s is the gradient of x and of the residual alike.
//
// Bound by memory: one pass over the rows. A CTA's team holds a row in
// registers between the mean and the output, takes rows one after the other
// and adds up its share of grad_w in registers too, in 32 bits; a second kernel
// adds the CTAs' shares in their order, so that every run gives the same bits.
// Rows of more than 16384 values take two passes: the means, and then columns
// by blocks. 32768 x 4096 bf16 with both gradients: 171 us (6.3 TB/s), and 6 us
// for the second kernel.
//
// Both kernels, by the library's call in turn: 8192 x 8192 bf16 98 us (5.5 TB/s),
// with an fp32 sum 164 (6.6), fp32 195 (5.5). Above 8192 values 1024 threads
// have two groups of eight each, which 64 registers do not hold (180 to 260 bytes
// of spills), and two rows with an fp32 sum do not fit into shared memory, so
// that those go value by value: 4096 x 16384 bf16 139 us (3.9), with an fp32 sum
// 281 (3.8), fp32 239 (4.5). Value by value for other reasons: 16384 x 2049 fp32 128
// (4.2) and bf16 216 (1.3), 4096 x 20000 bf16 415 (1.6).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "norm_internal.h"
#include "norm_rows.cuh"
#include "tc_ptx.cuh"

namespace flce {
namespace {

template <class T, int TEAM, int VECS, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rms_norm_bwd_kernel(const NormBwdParams p) {
  static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the CTA");
  using Cols = Columns<TEAM>;
  constexpr int kTeams = THREADS / TEAM;
  __shared__ float sum_buf[2][THREADS / 32];
  __shared__ float share[kTeams > 1 ? kTeams : 1][kTeams > 1 ? TEAM * VECS * 8 : 1];
  const int t = static_cast<int>(threadIdx.x) % TEAM;
  const int team = static_cast<int>(threadIdx.x) / TEAM;
  const int64_t h = p.h;
  float acc[VECS][8];
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(h));
  int turn = 0;
  grid_launch_dependents();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team; row < p.n;
       row += static_cast<int64_t>(gridDim.x) * kTeams) {
    float unit[VECS][8], u[VECS][8], g[VECS][8];
#pragma unroll
    for (int i = 0; i < VECS; ++i)
      Cols::template load_either<T>(p.total, row * p.total_pitch, p.wide, Cols::first(0, i, t), h,
                                    unit[i]);
#pragma unroll
    for (int i = 0; i < VECS; ++i)
      Cols::load(static_cast<const T*>(p.grad_y) + row * h, Cols::first(0, i, t), h, u[i]);
    const float rstd = p.rstd[row];
    if (p.grad_sum != nullptr) {
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        Cols::template load_either<T>(p.grad_sum, row * h, p.wide, Cols::first(0, i, t), h, g[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        unit[i][j] *= rstd;
        acc[i][j] = fmaf(u[i][j], unit[i][j], acc[i][j]);
      }
      if (p.weight != nullptr) {
        float w[8];
        Cols::template load_either<T>(p.weight, 0, p.weight_wide, Cols::first(0, i, t), h, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] *= w[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fmaf(u[i][j], unit[i][j], dot);
    }
    // rows in turn use two buffers: a warp that is a row ahead has passed the
    // barrier of the row before
    const float mean = team_all<TEAM>(dot, sum_buf[turn], SumOp{}) * inv_h;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[i][j] = fmaf(rstd, fmaf(-unit[i][j], mean, u[i][j]), g[i][j]);
      const int64_t e = Cols::first(0, i, t);
      if (p.grad_x != nullptr) Cols::store(static_cast<T*>(p.grad_x) + row * h, e, h, g[i]);
      if (p.grad_residual != nullptr)
        Cols::store(static_cast<float*>(p.grad_residual) + row * h, e, h, g[i]);
    }
  }
  if (p.grad_weight == nullptr) return;
  if constexpr (kTeams > 1) {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) share[team][Cols::first(0, i, t) + j * TEAM] = acc[i][j];
    __syncthreads();
    for (int64_t c = threadIdx.x; c < h; c += THREADS) {
      float v = share[0][c];
      for (int k = 1; k < kTeams; ++k) v += share[k][c];
      p.partial[static_cast<int64_t>(blockIdx.x) * h + c] = v;
    }
  } else {
    float* const out = p.partial + static_cast<int64_t>(blockIdx.x) * h;
#pragma unroll
    for (int i = 0; i < VECS; ++i) Cols::store(out, Cols::first(0, i, t), h, acc[i]);
  }
}

// Through L1: the two halves of eight fp32 values lie in the same sectors for
// both of their copies (past it, 16384 x 4096 fp32 takes 262 us instead of 171).
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// The same for rows of whole groups at 16-byte boundaries, copied to shared
// memory some rows ahead. Each thread copies what it reads itself, so that
// nothing but its own copies has to be waited for. R: the type of the sum.
// 32768 x 4096 bf16: 174 us (6.1 TB/s) with up to 192 KB an SM on their way,
// 226 with a row ahead in registers, 396 without.
template <class T, class R, int THREADS, int VECS>
struct Ring {
  static constexpr int kT = sizeof(T) == 4 ? 2 : 1, kR = sizeof(R) == 4 ? 2 : 1;  // of 16 bytes
  static constexpr int kPieces = VECS * (2 * kR + kT);
  static constexpr int kStage = kPieces * THREADS * 16;
};
template <class T, class R, int TEAM, int VECS, int THREADS, int CTAS, int DEPTH>
__global__ void __launch_bounds__(THREADS, CTAS) rms_norm_bwd_rows_kernel(const NormBwdParams p) {
  static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the CTA");
  using Stage = Ring<T, R, THREADS, VECS>;
  constexpr int kT = Stage::kT, kR = Stage::kR, kPieces = Stage::kPieces;
  constexpr int kTeams = THREADS / TEAM;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float sum_buf[2][THREADS / 32];
  __shared__ float share[kTeams > 1 ? kTeams : 1][kTeams > 1 ? TEAM * VECS * 8 : 1];
  const int t = static_cast<int>(threadIdx.x) % TEAM;
  const int team = static_cast<int>(threadIdx.x) / TEAM;
  const int64_t h = p.h, step = static_cast<int64_t>(gridDim.x) * kTeams;
  const int e = t * 8;
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(h));
  const bool adds = p.grad_sum != nullptr, weighs = p.weight != nullptr;
  float acc[VECS][8];
  Raw<T> w[VECS];
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  grid_launch_dependents();
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    w[i].clear();
    if (weighs && !p.weight_wide && e + i * TEAM * 8 < h)
      w[i].load(static_cast<const T*>(p.weight) + e + i * TEAM * 8);
  }
  // piece k of this thread in a stage: of the sum, its gradient and grad_y
  const auto slot = [&](int stage, int k) {
    return ring + (stage * kPieces + k) * THREADS + threadIdx.x;
  };
  const auto copy = [&](int64_t at, int stage) {
    if (at < p.n) {
      const R* const pt = static_cast<const R*>(p.total) + at * p.total_pitch + e;
      const R* const ps = static_cast<const R*>(p.grad_sum) + at * h + e;
      const T* const py = static_cast<const T*>(p.grad_y) + at * h + e;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        if (e + i * TEAM * 8 >= h) continue;
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          copy_async16(smem_addr(slot(stage, i * kR + k)),
                       reinterpret_cast<const uint4*>(pt + i * TEAM * 8) + k);
          if (adds)
            copy_async16(smem_addr(slot(stage, (VECS + i) * kR + k)),
                         reinterpret_cast<const uint4*>(ps + i * TEAM * 8) + k);
        }
#pragma unroll
        for (int k = 0; k < kT; ++k)
          copy_async16(smem_addr(slot(stage, 2 * VECS * kR + i * kT + k)),
                       reinterpret_cast<const uint4*>(py + i * TEAM * 8) + k);
      }
    }
    copy_async_commit();
  };
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) copy(row + d * step, d);
  float next_rstd = row < p.n ? p.rstd[row] : 0.0f;
  int stage = 0;
  for (int turn = 0; row < p.n; row += step, turn ^= 1) {
    float unit[VECS][8], u[VECS][8];
    float dot = 0.0f;
    const float inv = next_rstd;
    copy_async_wait<DEPTH - 2>();
    if (row + step < p.n) next_rstd = p.rstd[row + step];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      Raw<R> total;
      Raw<T> dy;
      total.clear();
      dy.clear();
      if (e + i * TEAM * 8 < h) {
#pragma unroll
        for (int k = 0; k < kR; ++k) total.q[k] = *slot(stage, i * kR + k);
#pragma unroll
        for (int k = 0; k < kT; ++k) dy.q[k] = *slot(stage, 2 * VECS * kR + i * kT + k);
      }
      total.values(unit[i]);
      dy.values(u[i]);
      float v[8];
      if (weighs) {
        if (p.weight_wide)
          load_weights(p.weight, e + i * TEAM * 8, h, v);
        else
          w[i].values(v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        unit[i][j] *= inv;
        acc[i][j] = fmaf(u[i][j], unit[i][j], acc[i][j]);
        if (weighs) u[i][j] *= v[j];
        dot = fmaf(u[i][j], unit[i][j], dot);
      }
    }
    // into the stage that the row before has left
    copy(row + (DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
    // rows in turn use two buffers: a warp that is a row ahead has passed the
    // barrier of the row before
    const float mean = team_all<TEAM>(dot, sum_buf[turn], SumOp{}) * inv_h;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = e + i * TEAM * 8;
      if (c >= h) continue;
      float g[8] = {};
      if (adds) {
        Raw<R> gs;
#pragma unroll
        for (int k = 0; k < kR; ++k) gs.q[k] = *slot(stage, (VECS + i) * kR + k);
        gs.values(g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[j] = fmaf(inv, fmaf(-unit[i][j], mean, u[i][j]), g[j]);
      if (p.grad_x != nullptr) store8(static_cast<T*>(p.grad_x) + row * h + c, g);
      if (p.grad_residual != nullptr) store8(static_cast<float*>(p.grad_residual) + row * h + c, g);
    }
    if (++stage == DEPTH) stage = 0;
  }
  if (p.grad_weight == nullptr) return;
  if constexpr (kTeams > 1) {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) share[team][e + i * TEAM * 8 + j] = acc[i][j];
    __syncthreads();
    for (int64_t c = threadIdx.x; c < h; c += THREADS) {
      float v = share[0][c];
      for (int k = 1; k < kTeams; ++k) v += share[k][c];
      p.partial[static_cast<int64_t>(blockIdx.x) * h + c] = v;
    }
  } else {
    float* const out = p.partial + static_cast<int64_t>(blockIdx.x) * h + e;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
      if (e + i * TEAM * 8 < h) store8(out + i * TEAM * 8, acc[i]);
  }
}

// grad_w of 32 columns a CTA: its 32 warps take the shares in turn, and their
// sums are added in order.
template <class W>
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partial, int64_t parts,
                                                           int64_t h, W* out) {
  __shared__ float buf[32][33];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float v = 0.0f;
  if (c < h) {
#pragma unroll 8
    for (int64_t k = warp; k < parts; k += 32) v += partial[k * h + c];
  }
  buf[warp][lane] = v;
  __syncthreads();
  v = buf[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && col < h) out[col] = from_f32<W>(v);
}

// Rows too long for one CTA's registers: mean(u * unit) of each, and then
// columns by blocks of 256 with a share of the rows each.
template <class T>
__global__ void __launch_bounds__(1024) norm_along_kernel(const NormBwdParams p) {
  __shared__ float buf[32];
  const int64_t row = blockIdx.x, h = p.h;
  const float rstd = p.rstd[row];
  const T* const grad_y = static_cast<const T*>(p.grad_y) + row * h;
  float dot = 0.0f;
  for (int64_t e0 = threadIdx.x; e0 < h; e0 += 32 * 1024) {
    float part = 0.0f;
    for (int64_t e = e0; e < h && e < e0 + 32 * 1024; e += 1024) {
      const float s = sizeof(T) == 4 || p.wide
                          ? static_cast<const float*>(p.total)[row * p.total_pitch + e]
                          : to_f32(static_cast<const T*>(p.total)[row * p.total_pitch + e]);
      float u = to_f32(grad_y[e]);
      if (p.weight != nullptr)
        u *= sizeof(T) == 4 || p.weight_wide ? static_cast<const float*>(p.weight)[e]
                                             : to_f32(static_cast<const T*>(p.weight)[e]);
      part = fmaf(u, s * rstd, part);
    }
    dot += part;
  }
  dot = team_all<1024>(dot, buf, SumOp{});
  if (threadIdx.x == 0) p.along[row] = __fdiv_rn(dot, static_cast<float>(h));
}

template <class T>
__global__ void __launch_bounds__(256) norm_bwd_columns_kernel(const NormBwdParams p,
                                                               int64_t parts) {
  const int64_t h = p.h, c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= h) return;
  const float w = p.weight == nullptr ? 1.0f
                  : sizeof(T) == 4 || p.weight_wide
                      ? static_cast<const float*>(p.weight)[c]
                      : to_f32(static_cast<const T*>(p.weight)[c]);
  for (int64_t part = blockIdx.y; part < parts; part += gridDim.y) {
    float acc = 0.0f;
    for (int64_t row = part; row < p.n; row += parts) {
      const int64_t at = row * h + c;
      const float s = sizeof(T) == 4 || p.wide
                          ? static_cast<const float*>(p.total)[row * p.total_pitch + c]
                          : to_f32(static_cast<const T*>(p.total)[row * p.total_pitch + c]);
      const float dy = to_f32(static_cast<const T*>(p.grad_y)[at]);
      const float rstd = p.rstd[row], unit = s * rstd;
      acc = fmaf(dy, unit, acc);
      float g = 0.0f;
      if (p.grad_sum != nullptr)
        g = sizeof(T) == 4 || p.wide ? static_cast<const float*>(p.grad_sum)[at]
                                     : to_f32(static_cast<const T*>(p.grad_sum)[at]);
      g = fmaf(rstd, fmaf(-unit, p.along[row], dy * w), g);
      if (p.grad_x != nullptr) static_cast<T*>(p.grad_x)[at] = from_f32<T>(g);
      if (p.grad_residual != nullptr) static_cast<float*>(p.grad_residual)[at] = g;
    }
    if (p.grad_weight != nullptr) p.partial[part * h + c] = acc;
  }
}

// How rows are dealt out: threads of a CTA, groups of eight values a thread,
// rows of a CTA at a time and CTAs an SM, by the length of a row and the
// kernel: value by value, groups with a 16-bit sum, groups with an fp32 sum.
// One group a thread where the sum is fp32 leaves 64 registers a thread and
// twice the threads: 16384 x 4096 with a bf16 x 220 us, 244 with half of them
// (both before their copies went through L1; 163 now).
struct Shape {
  int threads, vecs, rows, ctas;
};
constexpr Shape shape_of(int64_t h, int kind) {
  if (h <= 256) return {128, 1, 4, kind == 0 ? 4 : 5};
  if (h <= 512) return {64, 1, 1, kind == 0 ? 8 : 10};
  if (h <= 1024) return {128, 1, 1, kind == 0 ? 4 : 5};
  if (kind == 2) {
    if (h <= 2048) return {256, 1, 1, 4};
    if (h <= 4096) return {512, 1, 1, 2};
    if (h <= 8192) return {1024, 1, 1, 1};
    return {1024, 2, 1, 1};
  }
  if (h <= 2048) return {128, 2, 1, 4};
  if (h <= 4096) return {256, 2, 1, 2};
  if (h <= 8192) return {512, 2, 1, 1};
  return {1024, 2, 1, 1};
}

// Value by value, with the shape for rows of H values.
template <class T, int H>
cudaError_t launch_bwd_values(const NormBwdParams& p, int64_t parts, cudaStream_t s) {
  constexpr Shape k = shape_of(H, 0);
  constexpr int kTeam = k.rows > 1 ? 32 : k.threads;
  rms_norm_bwd_kernel<T, kTeam, k.vecs, k.threads, k.ctas>
      <<<static_cast<unsigned>(parts), k.threads, 0, s>>>(p);
  return cudaGetLastError();
}
template <class T, class R, int H>
cudaError_t launch_bwd_groups(const NormBwdParams& p, int64_t parts, cudaStream_t s) {
  constexpr Shape k = shape_of(H, sizeof(R) == 4 ? 2 : 1);
  constexpr int kTeam = k.rows > 1 ? 32 : k.threads;
  constexpr int kStage = Ring<T, R, k.threads, k.vecs>::kStage;
  constexpr int kFit = 200 * 1024 / k.ctas / kStage;
  constexpr int kDepth = kFit > 4 ? 4 : kFit;
  if constexpr (kDepth < 2) {  // no two rows in shared memory: above 8192 values, an fp32 sum
    return launch_bwd_values<T, H>(p, parts, s);
  } else {
    const auto kernel = rms_norm_bwd_rows_kernel<T, R, kTeam, k.vecs, k.threads, k.ctas, kDepth>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kDepth * kStage);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(parts), k.threads, kDepth * kStage, s>>>(p);
    return cudaGetLastError();
  }
}

template <class T, class R>
cudaError_t launch_bwd_rows(const NormBwdParams& p, bool groups, int64_t parts, cudaStream_t s) {
  const auto by_length = [&](auto h) {
    constexpr int H = decltype(h)::value;
    return groups ? launch_bwd_groups<T, R, H>(p, parts, s) : launch_bwd_values<T, H>(p, parts, s);
  };
  if (p.h <= 256) return by_length(std::integral_constant<int, 256>{});
  if (p.h <= 512) return by_length(std::integral_constant<int, 512>{});
  if (p.h <= 1024) return by_length(std::integral_constant<int, 1024>{});
  if (p.h <= 2048) return by_length(std::integral_constant<int, 2048>{});
  if (p.h <= 4096) return by_length(std::integral_constant<int, 4096>{});
  if (p.h <= 8192) return by_length(std::integral_constant<int, 8192>{});
  return by_length(std::integral_constant<int, 16384>{});
}

// CTAs that take n rows.
int64_t parts_of(int64_t n, int64_t h, int kind, int sms) {
  if (n < 1) return 0;
  if (h > kNormBwdMaxH) return n < 16 ? n : 16;
  const Shape k = shape_of(h, kind);
  const int64_t most = static_cast<int64_t>(sms) * k.ctas;
  const int64_t need = (n + k.rows - 1) / k.rows;
  return need < most ? need : most;
}

template <class W>
cudaError_t launch_weight(const NormBwdParams& p, int64_t parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.h + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const float* const partial = p.partial;
  return cudaLaunchKernelEx(&cfg, norm_weight_kernel<W>, partial, parts, p.h,
                            static_cast<W*>(p.grad_weight));
}

template <class T>
cudaError_t launch_bwd_typed(const NormBwdParams& p, int sms, cudaStream_t s) {
  constexpr int e = sizeof(T);
  int64_t parts = parts_of(p.n, p.h, 0, sms);
  cudaError_t err;
  if (p.h > kNormBwdMaxH) {
    norm_along_kernel<T><<<static_cast<unsigned>(p.n), 1024, 0, s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const dim3 grid(static_cast<unsigned>((p.h + 255) / 256), static_cast<unsigned>(parts));
    norm_bwd_columns_kernel<T><<<grid, 256, 0, s>>>(p, parts);
    err = cudaGetLastError();
  } else {
    const int wide = p.wide ? 4 : e;
    const bool groups = p.h % 8 == 0 && rows_of_16(p.grad_y, p.h, e) &&
                     rows_of_16(p.grad_sum, p.h, wide) &&
                     rows_of_16(p.total, p.total_pitch, wide) && rows_of_16(p.weight, 0, e) &&
                     rows_of_16(p.grad_x, p.h, e) && rows_of_16(p.grad_residual, p.h, 4);
    if (groups) parts = parts_of(p.n, p.h, wide == 4 ? 2 : 1, sms);
    err = sizeof(T) < 4 && p.wide ? launch_bwd_rows<T, float>(p, groups, parts, s)
                                  : launch_bwd_rows<T, T>(p, groups, parts, s);
  }
  if (err != cudaSuccess || p.grad_weight == nullptr) return err;
  return e == 4 || p.weight_wide ? launch_weight<float>(p, parts, s)
                                 : launch_weight<T>(p, parts, s);
}

}  // namespace

int64_t norm_bwd_parts(int64_t n, int64_t h, int sms) {
  return std::max({parts_of(n, h, 0, sms), parts_of(n, h, 1, sms), parts_of(n, h, 2, sms)});
}

cudaError_t launch_rms_norm_bwd(const NormBwdParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_bwd_typed<float>(p, sms, s);
  if (dtype == FLCE_BF16) return launch_bwd_typed<__nv_bfloat16>(p, sms, s);
  return launch_bwd_typed<__half>(p, sms, s);
}

}  // namespace flce
