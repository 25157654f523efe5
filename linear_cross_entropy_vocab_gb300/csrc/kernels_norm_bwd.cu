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
// by blocks.
#include <cstdint>

#include "norm_internal.h"
#include "norm_rows.cuh"
#include "tc_ptx.cuh"

namespace flce {
namespace {

template <class T, bool VEC, int TEAM, int VECS, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rms_norm_bwd_kernel(const NormBwdParams p) {
  static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the CTA");
  using Cols = Columns<TEAM, VEC>;
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
      for (int j = 0; j < 8; ++j) share[team][Cols::first(0, i, t) + j * Cols::kStep] = acc[i][j];
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
  if (c < h)
    for (int64_t k = warp; k < parts; k += 32) v += partial[k * h + c];
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

// CTAs an SM that the row kernel is compiled for.
constexpr int ctas_of(int threads) { return threads >= 1024 ? 1 : threads >= 512 ? 1 : 512 / threads; }

template <class T, bool VEC, int TEAM, int VECS, int THREADS = TEAM>
cudaError_t launch_bwd_team(const NormBwdParams& p, int64_t parts, cudaStream_t s) {
  rms_norm_bwd_kernel<T, VEC, TEAM, VECS, THREADS, ctas_of(THREADS)>
      <<<static_cast<unsigned>(parts), THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

struct Shape {
  int threads, rows;  // of a CTA
};
Shape shape_of(int64_t h) {
  if (h <= 256) return {128, 4};
  if (h <= 2048) return {128, 1};
  if (h <= 4096) return {256, 1};
  if (h <= 8192) return {512, 1};
  return {1024, 1};
}

template <class T, bool VEC>
cudaError_t launch_bwd_rows(const NormBwdParams& p, int64_t parts, cudaStream_t s) {
  if (p.h <= 256) return launch_bwd_team<T, VEC, 32, 1, 128>(p, parts, s);
  if (p.h <= 1024) return launch_bwd_team<T, VEC, 128, 1>(p, parts, s);
  if (p.h <= 2048) return launch_bwd_team<T, VEC, 128, 2>(p, parts, s);
  if (p.h <= 4096) return launch_bwd_team<T, VEC, 256, 2>(p, parts, s);
  if (p.h <= 8192) return launch_bwd_team<T, VEC, 512, 2>(p, parts, s);
  return launch_bwd_team<T, VEC, 1024, 2>(p, parts, s);
}

bool rows_of_16(const void* p, int64_t pitch, int size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch * size % 16 == 0);
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
  const int64_t parts = norm_bwd_parts(p.n, p.h, sms);
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
    const bool vec = p.h % 8 == 0 && rows_of_16(p.grad_y, p.h, e) &&
                     rows_of_16(p.grad_sum, p.h, wide) &&
                     rows_of_16(p.total, p.total_pitch, wide) && rows_of_16(p.weight, 0, e) &&
                     rows_of_16(p.grad_x, p.h, e) && rows_of_16(p.grad_residual, p.h, 4);
    err = vec ? launch_bwd_rows<T, true>(p, parts, s) : launch_bwd_rows<T, false>(p, parts, s);
  }
  if (err != cudaSuccess || p.grad_weight == nullptr) return err;
  return e == 4 || p.weight_wide ? launch_weight<float>(p, parts, s)
                                 : launch_weight<T>(p, parts, s);
}

}  // namespace

int64_t norm_bwd_parts(int64_t n, int64_t h, int sms) {
  if (n < 1) return 0;
  if (h > kNormBwdMaxH) return n < 16 ? n : 16;
  const Shape shape = shape_of(h);
  const int64_t most = static_cast<int64_t>(sms) * ctas_of(shape.threads);
  const int64_t need = (n + shape.rows - 1) / shape.rows;
  return need < most ? need : most;
}

cudaError_t launch_rms_norm_bwd(const NormBwdParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_bwd_typed<float>(p, sms, s);
  if (dtype == FLCE_BF16) return launch_bwd_typed<__nv_bfloat16>(p, sms, s);
  return launch_bwd_typed<__half>(p, sms, s);
}

}  // namespace flce
