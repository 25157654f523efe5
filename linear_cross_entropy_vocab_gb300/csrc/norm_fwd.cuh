// The forward kernel of the root-mean-square norm, with its output in the
// input's type (kernels_norm.cu) or in 8-bit integers (kernels_norm_q.cu):
//
//   s = x + r,  y = s * w / sqrt(mean(s^2) + eps)
//   scale = max|y| * (1/127),  q = round(y / scale)
//
// Bound by memory: one pass. A team of threads (a warp, or a CTA of 128 to 1024
// threads) takes a row and keeps its sums in registers, in 32 bits and not
// rounded, between the mean and the output; rows of more than 16384 values are
// read a second time. The squares are summed in 32 bits, over at most 32 values
// a thread in each sweep of up to 16384 values, over a thread's sweeps one after
// the other (1024 for the longest row), and then by a tree.
//
// With a residual, by the library's call in turn: 16384 x 3584 fp16 73 us (6.4 TB/s),
// 8192 x 8192 bf16 90 (6.0), 4096 x 16384 bf16 89 (6.0) and fp32 232 (4.6: 1024
// threads hold 64 registers each, and the fp32 form spills 264 bytes of them, the
// 8-bit one 304); to 8 bits 8192 x 4096 bf16 42 us (5.6), 8192 x 8192 116
// (4.0), 4096 x 16384 103 (4.6). Rows of more than 16384 values and rows that are not at
// 16-byte boundaries go value by value: 4096 x 20000 bf16 347 us (1.9) and fp32
// 347 (3.8), 16384 x 2049 bf16 142 (1.9) and fp32 97 (5.6). The two ways add
// squares and divide by h in different orders: a row's last bit may differ
// between them.
#pragma once

#include <cstdint>

#include "int8_round.cuh"
#include "norm_internal.h"
#include "norm_rows.cuh"

namespace flce {

template <class T, bool QUANT, int TEAM, int VECS, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_kernel(const NormParams p) {
  static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the CTA");
  using Cols = Columns<TEAM>;
  constexpr int kWarps = THREADS / 32;
  constexpr int kSweep = TEAM * VECS * 8;
  __shared__ float sum_buf[kWarps];
  __shared__ double wide_buf[kWarps];
  __shared__ uint32_t max_buf[kWarps];
  const int t = static_cast<int>(threadIdx.x) % TEAM;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / TEAM) +
                      static_cast<int>(threadIdx.x) / TEAM;
  if (TEAM == 32 && row >= p.n) return;  // whole warps
  const int64_t h = p.h;
  const T* const x = static_cast<const T*>(p.x) + row * p.x_pitch;
  float s[VECS][8];
  auto load = [&](int64_t e0, bool keep) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) Cols::load(x, Cols::first(e0, i, t), h, s[i]);
    if (p.residual != nullptr) {
      float r[VECS][8];
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        Cols::template load_either<T>(p.residual, row * p.residual_pitch, p.wide,
                                      Cols::first(e0, i, t), h, r[i]);
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[i][j];
        if (keep)
          Cols::template store_either<T>(p.sum, row * h, p.wide, Cols::first(e0, i, t), h, s[i]);
      }
    }
  };
  float part = 0.0f;
  for (int64_t e0 = 0; e0 < h; e0 += kSweep) {
    load(e0, true);
    float sweep = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sweep = fmaf(s[i][j], s[i][j], sweep);
    part += sweep;
  }
  const bool again = h > kSweep;  // the registers hold the last sweep alone
  float square = team_all<TEAM>(part, sum_buf, SumOp{});
  float rstd;
  if (square < 3.0e38f && (square > 1.0e-24f || p.eps > 1.0e-24f)) {
    rstd = __frsqrt_rn(__fdiv_rn(square, static_cast<float>(h)) + p.eps);
  } else {
    // squares that leave the 32-bit range, or are not finite: the same in 64 bits
    double wide = 0.0;
    for (int64_t e0 = 0; e0 < h; e0 += kSweep) {
      if (again) load(e0, false);
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) wide += static_cast<double>(s[i][j]) * s[i][j];
    }
    wide = team_all<TEAM>(wide, wide_buf, SumOp{});
    rstd = static_cast<float>(1.0 / sqrt(wide / static_cast<double>(h) + p.eps));
  }
  if (p.rstd != nullptr && t == 0) p.rstd[row] = rstd;
  // s becomes y in 32 bits
  auto finish = [&](int64_t e0) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] *= rstd;
      if (p.weight != nullptr) {
        float w[8];
        Cols::template load_either<T>(p.weight, 0, p.weight_wide, Cols::first(e0, i, t), h, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] *= w[j];
      }
    }
  };
  if constexpr (!QUANT) {
    for (int64_t e0 = 0; e0 < h; e0 += kSweep) {
      if (again) load(e0, false);
      finish(e0);
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        Cols::store(static_cast<T*>(p.y) + row * h, Cols::first(e0, i, t), h, s[i]);
    }
  } else {
    uint32_t peak = 0;  // of the bits without the sign: NaN is above infinity
    for (int64_t e0 = 0; e0 < h; e0 += kSweep) {
      if (again) load(e0, false);
      finish(e0);
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // columns past the end hold 0 * rstd, which is NaN where rstd is
          const uint32_t bits = __float_as_uint(s[i][j]) & 0x7fffffffu;
          peak = bits > peak ? bits : peak;
        }
    }
    const float top = __uint_as_float(team_all<TEAM>(peak, max_buf, MaxOp{}));
    const float scale = top < INFINITY ? top * (1.0f / 127.0f) : NAN;
    const float inv = __fdiv_rn(1.0f, scale);
    if (t == 0) p.scale[row] = scale;
    int8_t* const q = p.q + row * p.q_pitch;
    for (int64_t e0 = 0; e0 < h; e0 += kSweep) {
      if (again) {
        load(e0, false);
        finish(e0);
      }
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int64_t e = Cols::first(e0, i, t);
        if (e >= h) continue;
        round8(s[i], scale, inv);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e + j * TEAM < h)
            q[e + j * TEAM] = static_cast<int8_t>(__float_as_uint(s[i][j]) & 0xffu);
      }
    }
  }
}

// The same for rows of whole groups at 16-byte boundaries that fit the
// registers: as many CTAs as an SM holds take rows one after the other, and a
// row's loads are on their way while the row before is worked on. R: the type
// of the residual and the sum.
template <class T, class R, bool QUANT, int TEAM, int VECS, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rms_norm_rows_kernel(const NormParams p) {
  static_assert(TEAM == 32 || TEAM == THREADS, "a team is a warp or the CTA");
  constexpr int kWarps = THREADS / 32, kTeams = THREADS / TEAM;
  // rows in turn use two buffers: a warp that is a row ahead has passed the
  // barriers of the row before
  __shared__ float sum_buf[2][kWarps];
  __shared__ double wide_buf[2][kWarps];
  __shared__ uint32_t max_buf[2][kWarps];
  const int t = static_cast<int>(threadIdx.x) % TEAM;
  const int64_t h = p.h, step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + static_cast<int>(threadIdx.x) / TEAM;
  if (row >= p.n) return;  // whole teams
  const int e = t * 8;  // of the thread's first group; TEAM * 8 further the next
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(h));
  const bool sums = p.residual != nullptr, weighs = p.weight != nullptr;
  Raw<T> x[VECS], w[VECS];
  Raw<R> r[VECS];
  const auto load = [&](int64_t at) {
    const T* const px = static_cast<const T*>(p.x) + at * p.x_pitch + e;
    const R* const pr = static_cast<const R*>(p.residual) + at * p.residual_pitch + e;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      if (e + i * TEAM * 8 < h) {
        x[i].load(px + i * TEAM * 8);
        if (sums) r[i].load(pr + i * TEAM * 8);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    x[i].clear();
    r[i].clear();
    w[i].clear();
    if (weighs && !p.weight_wide && e + i * TEAM * 8 < h)
      w[i].load(static_cast<const T*>(p.weight) + e + i * TEAM * 8);
  }
  load(row);
  for (int turn = 0; row < p.n; row += step, turn ^= 1) {
    float s[VECS][8];
    float square = 0.0f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      float v[8];
      x[i].values(s[i]);
      r[i].values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[i][j] += v[j];
        square = fmaf(s[i][j], s[i][j], square);
      }
    }
    if (row + step < p.n) load(row + step);
    if (sums) {
      R* const out = static_cast<R*>(p.sum) + row * h + e;
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        if (e + i * TEAM * 8 < h) store8(out + i * TEAM * 8, s[i]);
    }
    square = team_all<TEAM>(square, sum_buf[turn], SumOp{});
    float rstd;
    if (square < 3.0e38f && (square > 1.0e-24f || p.eps > 1.0e-24f)) {
      rstd = __frsqrt_rn(fmaf(square, inv_h, p.eps));
    } else {
      double wide = 0.0;
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) wide += static_cast<double>(s[i][j]) * s[i][j];
      wide = team_all<TEAM>(wide, wide_buf[turn], SumOp{});
      rstd = static_cast<float>(1.0 / sqrt(wide / static_cast<double>(h) + p.eps));
    }
    if (p.rstd != nullptr && t == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] *= rstd;
      if (weighs) {
        float v[8];
        if (p.weight_wide)
          load_weights(p.weight, e + i * TEAM * 8, h, v);
        else
          w[i].values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] *= v[j];
      }
    }
    if constexpr (!QUANT) {
      T* const out = static_cast<T*>(p.y) + row * h + e;
#pragma unroll
      for (int i = 0; i < VECS; ++i)
        if (e + i * TEAM * 8 < h) store8(out + i * TEAM * 8, s[i]);
    } else {
      uint32_t peak = 0;  // of the bits without the sign: NaN is above infinity
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t bits = __float_as_uint(s[i][j]) & 0x7fffffffu;
          peak = bits > peak ? bits : peak;
        }
      const float top = __uint_as_float(team_all<TEAM>(peak, max_buf[turn], MaxOp{}));
      const float scale = top < INFINITY ? top * (1.0f / 127.0f) : NAN;
      const float inv = __fdiv_rn(1.0f, scale);
      if (t == 0) p.scale[row] = scale;
      int8_t* const q = p.q + row * p.q_pitch;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        if (e + i * TEAM * 8 >= h) continue;
        round8(s[i], scale, inv);
        put_bytes(q, e + i * TEAM * 8, h, true, s[i]);
      }
    }
  }
}

template <class T, bool QUANT, int TEAM, int VECS, int THREADS = TEAM>
cudaError_t launch_norm_team(const NormParams& p, cudaStream_t s) {
  constexpr int64_t rows = THREADS / TEAM;  // of a CTA
  const unsigned grid = static_cast<unsigned>((p.n + rows - 1) / rows);
  rms_norm_kernel<T, QUANT, TEAM, VECS, THREADS><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <class T, class R, bool QUANT, int TEAM, int VECS, int THREADS = TEAM>
cudaError_t launch_norm_stream(const NormParams& p, cudaStream_t s) {
  constexpr int64_t rows = THREADS / TEAM;
  // as many threads an SM as the registers of a row allow
  constexpr int kHold = VECS == 1 ? 1024 : sizeof(R) == 4 ? 512 : 768;
  constexpr int kCtas = THREADS >= kHold ? 1 : kHold / THREADS;
  const int64_t need = (p.n + rows - 1) / rows, most = int64_t(p.sms) * kCtas;
  const unsigned grid = static_cast<unsigned>(need < most ? need : most);
  rms_norm_rows_kernel<T, R, QUANT, TEAM, VECS, THREADS, kCtas><<<grid, THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

template <class T, bool QUANT>
cudaError_t launch_norm_any(const NormParams& p, cudaStream_t s) {
  if (p.h <= 256) return launch_norm_team<T, QUANT, 32, 1, 128>(p, s);
  if (p.h <= 1024) return launch_norm_team<T, QUANT, 32, 4, 128>(p, s);
  if (p.h <= 2048) return launch_norm_team<T, QUANT, 128, 2>(p, s);
  if (p.h <= 4096) return launch_norm_team<T, QUANT, 256, 2>(p, s);
  if (p.h <= 8192) return launch_norm_team<T, QUANT, 512, 2>(p, s);
  return launch_norm_team<T, QUANT, 1024, 2>(p, s);
}
template <class T, class R, bool QUANT>
cudaError_t launch_norm_groups(const NormParams& p, cudaStream_t s) {
  if (p.h <= 256) return launch_norm_stream<T, R, QUANT, 32, 1, 128>(p, s);
  if (p.h <= 512) return launch_norm_stream<T, R, QUANT, 32, 2, 128>(p, s);
  if (p.h <= 1024) return launch_norm_stream<T, R, QUANT, 128, 1>(p, s);
  if (p.h <= 2048) return launch_norm_stream<T, R, QUANT, 256, 1>(p, s);
  if (p.h <= 4096) return launch_norm_stream<T, R, QUANT, 256, 2>(p, s);
  if (p.h <= 8192) return launch_norm_stream<T, R, QUANT, 512, 2>(p, s);
  return launch_norm_stream<T, R, QUANT, 1024, 2>(p, s);
}

template <class T, bool QUANT>
cudaError_t launch_norm_typed(const NormParams& p, cudaStream_t s) {
  constexpr int e = sizeof(T);
  const bool groups = p.h % 8 == 0 && p.h <= 16384 && rows_of_16(p.x, p.x_pitch, e) &&
                   rows_of_16(p.residual, p.residual_pitch, p.wide ? 4 : e) &&
                   rows_of_16(p.sum, p.h, p.wide ? 4 : e) && rows_of_16(p.weight, 0, e) &&
                   rows_of_16(p.y, p.h, e) && rows_of_16(p.q, p.q_pitch, 1);
  if (!groups) return launch_norm_any<T, QUANT>(p, s);
  if (sizeof(T) < 4 && p.wide && p.residual != nullptr)
    return launch_norm_groups<T, float, QUANT>(p, s);
  return launch_norm_groups<T, T, QUANT>(p, s);
}

template <bool QUANT>
cudaError_t launch_norm(const NormParams& p, int dtype, cudaStream_t s) {
  if (dtype == FLCE_F32) return launch_norm_typed<float, QUANT>(p, s);
  if (dtype == FLCE_BF16) return launch_norm_typed<__nv_bfloat16, QUANT>(p, s);
  return launch_norm_typed<__half, QUANT>(p, s);
}

}  // namespace flce
