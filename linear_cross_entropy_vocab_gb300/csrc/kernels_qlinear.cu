// The linear layer on 8-bit integer rows, on the tensor cores:
//
//   out_ij = f(x_scale_i * weight_scale_j * sum_h q_ih w_jh + bias_j)
//
// The tensor cores of this GPU have no 8-bit integer rate worth using, but a
// half-precision number holds every 8-bit integer, its products are exact and
// the accumulators are 32 bits wide: sums up to 2^24 are exact too. So the
// weight travels from memory to the SM in 8 bits, which is what bounds a call
// with few rows, and is widened on the way into the MMA; the few rows of x are
// widened once, by a kernel of their own.
//
// The weight is the A operand (its rows are the accumulator's lanes) and is
// read by the MMA from tensor memory: widening warps take the bytes from the
// shared memory that TMA filled, turn each into a half and store them with
// tcgen05.st. Shared memory then carries the weight in 8 bits only, and
// the MMA reads only x from it. A byte b becomes a half by b xor 0x6480, which is
// 1024 + 128 + b, minus 1152. Bytes 0 and 2 of a word make one pair and 1 and
// 3 the other, without a permutation: x is laid out in that order
// (k = 0, 2, 1, 3 in each four) by the kernel that widens it.
//
// Tiles are 128 weight rows (CG = 1) or 256 over a pair of CTAs (CG = 2) by
// `nt` rows of x, a multiple of 16 (32) that the launch chooses so that the
// last tile is not mostly empty. A CTA stays on its SM and takes tile after
// tile. Tensor memory: columns [0, 256) the accumulators (two when nt <= 128,
// so that one drains while the other fills), [256, 512) four 128-deep slices
// of widened weight.
//
// Roles (23 warps): 0 loads the weight, 1 issues the MMAs, 2 loads x, 3-14
// widen (three groups of four that take 128-byte stages in turn; 8192 rows of
// the Llama-3 head take 4.26 ms with three groups, 4.31 with two and 4.32 with
// four), 15-22 run the epilogue (two per lane quarter, half of the columns
// each).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int8_internal.h"
#include "tc_gemm.cuh"

namespace flce {
namespace {

constexpr int kWStageBytes = 128 * 128;  // 128 weight rows x 128 bytes
constexpr int kMaxWStages = 12;
constexpr int kMaxXStages = kMaxWStages;
constexpr int kASlots = 4;
constexpr int kACols = 64;        // tensor-memory columns of a 128-deep slice
constexpr int kABase = 256;       // first of them
constexpr int kWidenGroups = 3;
constexpr int kWidenWarps = 4 * kWidenGroups;
constexpr int kEpilogueWarps = 8;
constexpr int kFirstWiden = 3;
constexpr int kFirstEpilogue = kFirstWiden + kWidenWarps;
constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogueWarps);
constexpr int kSmemBudget = 224 * 1024;

struct Ctl {
  uint64_t w_full[kMaxWStages], w_empty[kMaxWStages];
  uint64_t x_full[kMaxXStages], x_empty[kMaxXStages];
  uint64_t a_full[kASlots], a_empty[kASlots];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

// D (+)= A * B^T with A in tensor memory, fp16 inputs, fp32 accumulators.
template <int CG>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_store_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Bytes (0, 2) and (1, 3) of a word of four signed 8-bit integers as halves.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& even, uint32_t& odd) {
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  uint32_t e = (w & 0x00ff00ffu) ^ 0x64806480u;
  uint32_t o = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
  const __half2 eh = __hsub2(*reinterpret_cast<__half2*>(&e), bias);
  const __half2 oh = __hsub2(*reinterpret_cast<__half2*>(&o), bias);
  even = *reinterpret_cast<const uint32_t*>(&eh);
  odd = *reinterpret_cast<const uint32_t*>(&oh);
}

// True on one lane of a converged warp, which the compiler knows to be one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// An mbarrier arrive on the pair's even CTA. What the arrival announces lies in
// tensor memory, written or read by tcgen05 instructions that have completed
// and are ordered by tcgen05.fence; no other memory is handed over. So the
// arrival needs no release at cluster scope, and the waits below no acquire
// there: each costs hundreds of nanoseconds, once for a stage.
template <int CG>
__device__ __forceinline__ void arrive_leader(uint32_t bar, bool leader) {
  if (CG == 1 || leader)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, 0))
                 : "memory");
}

template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    umma_commit_pair(bar, 0x3);
}

// tanh of a pair, within 10 * 2^-24 of its value: x P(t) / Q(t) with t = x^2,
// P and Q of degree 4 fitted to tanh itself for the least relative error (below
// 2^-26; all coefficients are positive, so that nothing cancels). The form by
// exponentials, (e^2x - 1) / (e^2x + 1), is right to some 1e-7 absolute only: a
// logit of a millionth of the cap loses all its bits. Beyond 8.3 tanh is 1
// within 2^-23. The clamp keeps a NaN, which fminf and fmaxf would not.
__device__ __forceinline__ uint64_t tanh_pair(float a, float b) {
  constexpr float kEnd = 8.3f;
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(kEnd));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(kEnd));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(-kEnd));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(-kEnd));
  auto both = [](float c) { return f2_pack(c, c); };
  const uint64_t x = f2_pack(a, b);
  const uint64_t t = f2_mul(x, x);
  uint64_t p = f2_fma(t, both(1.4648282e-8f), both(2.1508517e-5f));
  uint64_t q = f2_fma(t, both(8.295119e-7f), both(3.3739527e-4f));
  p = f2_fma(p, t, both(3.5491704e-3f));
  q = f2_fma(q, t, both(2.6079955e-2f));
  p = f2_fma(p, t, both(0.13425872f));
  q = f2_fma(q, t, both(0.46759197f));
  p = f2_fma(p, t, both(1.0f));
  q = f2_fma(q, t, both(1.0f));
  float r_a, r_b;
  f2_unpack(q, r_a, r_b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r_a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r_b));
  return f2_mul(f2_mul(p, x), f2_pack(r_a, r_b));
}

__device__ __forceinline__ float bias_at(const void* p, int dtype, int64_t i) {
  if (dtype == FLCE_F32) return static_cast<const float*>(p)[i];
  if (dtype == FLCE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }
__device__ __forceinline__ void store(__half* p, float x) { *p = __float2half(x); }

// Tile u of a launch: its place along x and along the weight. Tiles of x run
// fastest, `band` of them at a time, so that what the tiles in flight share of
// x stays in L2 over the whole weight.
__device__ __forceinline__ void tile_place(const QLinearTcParams& p, int u, int& n, int& v) {
  const int per_band = p.band * p.v_tiles;
  const int first = (u / per_band) * p.band;
  const int wide = p.n_tiles - first < p.band ? p.n_tiles - first : p.band;
  const int r = u % per_band;
  n = first + r % wide;
  v = r / wide;
}

template <int CG, class T>
__global__ void __launch_bounds__(kThreads, 1)
    qlinear_kernel(const __grid_constant__ QLinearTcParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t x_base = base + static_cast<uint32_t>(p.w_stages) * kWStageBytes;
  const uint32_t x_bytes = static_cast<uint32_t>(p.nt / CG) * 128u;  // of one 64-deep box
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit0 = static_cast<int>(blockIdx.x) / CG;
  const int units = static_cast<int>(gridDim.x) / CG;
  const int total = p.n_tiles * p.v_tiles;
  volatile int* const abort_flag = &ctl.abort;
  int* const err_word = p.err_word;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.w_stages; ++s) {
      mbar_init(smem_addr(&ctl.w_full[s]), 1);
      mbar_init(smem_addr(&ctl.w_empty[s]), 4);
    }
    for (int s = 0; s < p.x_stages; ++s) {
      mbar_init(smem_addr(&ctl.x_full[s]), 1);
      mbar_init(smem_addr(&ctl.x_empty[s]), 1);
    }
    for (int s = 0; s < kASlots; ++s) {
      mbar_init(smem_addr(&ctl.a_full[s]), 4 * CG);
      mbar_init(smem_addr(&ctl.a_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.acc_full[s]), 1);
      mbar_init(smem_addr(&ctl.acc_empty[s]), kEpilogueWarps * CG);
    }
    mbar_init(smem_addr(&ctl.mma_done), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.w_map);
    tma_prefetch_desc(&p.x_map);
  }
  if (warp == 1) {
    if constexpr (CG == 1) {
      tmem_alloc(smem_addr(&ctl.tmem_base), 512);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(smem_addr(&ctl.tmem_base), 512);
      tmem_relinquish_pair();
    }
  }
  tc_fence_before_sync();
  if constexpr (CG == 1)
    __syncthreads();
  else
    cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  const int bufs = p.nt <= 128 ? 2 : 1;
  const int k_iters = (p.k_blocks + 1) / 2;  // 128-deep stages of a tile; the last may be half

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ weight loads
      int s = 0;
      uint32_t phase = 0, armed = 0, last_phase = 0;
      bool ok = true;
      for (int u = unit0; ok && u < total; u += units) {
        int n, v;
        tile_place(p, u, n, v);
        const int row = v * (128 * CG) + static_cast<int>(rank) * 128;
        for (int i = 0; i < k_iters; ++i) {
          if (!mbar_wait(smem_addr(&ctl.w_empty[s]), phase ^ 1u, abort_flag, err_word)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_addr(&ctl.w_full[s]);
          mbar_arrive_expect_tx(full, kWStageBytes);
          tma_load_2d(base + static_cast<uint32_t>(s) * kWStageBytes, &p.w_map, full, i * 128, row);
          armed |= 1u << s;
          last_phase = (last_phase & ~(1u << s)) | (phase << s);
          if (++s == p.w_stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok)  // copies in flight land before the CTA leaves
        for (int q = 0; q < p.w_stages; ++q)
          if (armed & (1u << q)) drain_wait(smem_addr(&ctl.w_full[q]), (last_phase >> q) & 1u);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // ------------------------------------------------ loads of x
      grid_dependency_wait();  // x is widened by the kernel before this one
      int s = 0;
      uint32_t phase = 0, armed = 0, last_phase = 0;
      bool ok = true;
      for (int u = unit0; ok && u < total; u += units) {
        int n, v;
        tile_place(p, u, n, v);
        const int row = n * p.nt + static_cast<int>(rank) * (p.nt / CG);
        for (int i = 0; i < k_iters; ++i) {
          if (!mbar_wait(smem_addr(&ctl.x_empty[s]), phase ^ 1u, abort_flag, err_word)) {
            ok = false;
            break;
          }
          const uint32_t local = smem_addr(&ctl.x_full[s]);
          const int boxes = 2 * i + 1 < p.k_blocks ? 2 : 1;
          if (leader) mbar_arrive_expect_tx(local, static_cast<uint32_t>(boxes) * CG * x_bytes);
          for (int j = 0; j < boxes; ++j) {
            const uint32_t dst = x_base + static_cast<uint32_t>(2 * s + j) * x_bytes;
            if constexpr (CG == 1)
              tma_load_2d(dst, &p.x_map, local, (2 * i + j) * 64, row);
            else
              tma_load_2d_pair(dst, &p.x_map, map_to_rank(local, 0), (2 * i + j) * 64, row);
          }
          armed |= 1u << s;
          last_phase = (last_phase & ~(1u << s)) | (phase << s);
          if (++s == p.x_stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader)
        for (int q = 0; q < p.x_stages; ++q)
          if (armed & (1u << q)) drain_wait(smem_addr(&ctl.x_full[q]), (last_phase >> q) & 1u);
    }
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------------ MMA issuer
      // The whole warp walks the stages and one elected lane issues: the
      // operands are then uniform registers, and an MMA takes 9 cycles to
      // issue. From code that one lane runs alone it takes 46, more than a
      // product with few rows of x.
      const uint32_t idesc = idesc_f16kind_f32(128 * CG, p.nt, 0, 0, 0u);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t desc0 = smem_desc_sw128(__shfl_sync(0xffffffffu, x_base, 0), 16, 1024);
      const uint32_t box = x_bytes >> 4;  // of a 64-deep box, in descriptor units
      int xs = 0, as = 0;
      uint32_t x_phase = 0, a_phase = 0;
      bool ok = true;
      int it = 0;
      for (int u = unit0; ok && u < total; u += units, ++it) {
        const int buf = bufs == 2 ? it & 1 : 0;
        const uint32_t use = static_cast<uint32_t>(bufs == 2 ? it >> 1 : it) & 1u;
        ok = mbar_wait(smem_addr(&ctl.acc_empty[buf]), use ^ 1u, abort_flag, err_word);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tm + static_cast<uint32_t>(buf * 128);
        for (int i = 0; i < k_iters; ++i) {
          ok = mbar_wait(smem_addr(&ctl.x_full[xs]), x_phase, abort_flag, err_word) &&
               mbar_wait(smem_addr(&ctl.a_full[as]), a_phase, abort_flag, err_word);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t a = tm + static_cast<uint32_t>(kABase + as * kACols);
            const uint64_t b = desc0 + static_cast<uint64_t>(static_cast<uint32_t>(2 * xs) * box);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_ts<CG>(d, a + static_cast<uint32_t>(kk * 8), b + static_cast<uint64_t>(kk * 2),
                          idesc, (i | kk) != 0 ? 1u : 0u);
            if (2 * i + 1 < p.k_blocks) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ts<CG>(d, a + static_cast<uint32_t>(32 + kk * 8),
                            b + static_cast<uint64_t>(box + static_cast<uint32_t>(kk * 2)), idesc,
                            1u);
            }
            commit<CG>(smem_addr(&ctl.x_empty[xs]));
            commit<CG>(smem_addr(&ctl.a_empty[as]));
            if (i == k_iters - 1) commit<CG>(smem_addr(&ctl.acc_full[buf]));
          }
          __syncwarp();
          if (++xs == p.x_stages) {
            xs = 0;
            x_phase ^= 1u;
          }
          if (++as == kASlots) {
            as = 0;
            a_phase ^= 1u;
          }
        }
      }
      if (elect_one()) {
        commit<CG>(smem_addr(&ctl.mma_done));
        drain_wait(smem_addr(&ctl.mma_done), 0);
      }
    } else if (lane == 0 && CG == 2) {
      drain_wait(smem_addr(&ctl.mma_done), 0);  // the even CTA's MMAs write this CTA's TMEM
    }
  } else if (warp < kFirstEpilogue) {
    // -------------------------------------------------- widening warps
    const int quarter = warp & 3;
    const int group = (warp - kFirstWiden) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    bool ok = true;
    // stages of all this CTA's tiles, counted through; group g takes g,
    // g + kWidenGroups, ...
    const int64_t stages =
        static_cast<int64_t>(total > unit0 ? (total - unit0 - 1) / units + 1 : 0) * k_iters;
    int s = group, as = group;
    uint32_t phase = 0, a_phase = 1;
    for (int64_t i = group; i < stages; i += kWidenGroups) {
      ok = mbar_wait(smem_addr(&ctl.w_full[s]), phase, abort_flag, err_word);
      if (!__all_sync(0xffffffffu, ok)) break;
      // 16-byte piece c of a row lies at c xor (row mod 8): TMA's 128-byte swizzle
      const uint32_t at = base + static_cast<uint32_t>(s) * kWStageBytes +
                          static_cast<uint32_t>(row) * 128u;
      uint32_t w[32];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                     : "r"(at + static_cast<uint32_t>((c ^ (row & 7)) * 16))
                     : "memory");
      uint32_t h[32];
#pragma unroll
      for (int j = 0; j < 16; ++j) widen(w[j], h[2 * j], h[2 * j + 1]);
      ok = mbar_wait(smem_addr(&ctl.a_empty[as]), a_phase, abort_flag, err_word);
      if (!__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.w_empty[s]));  // all lanes have read their bytes
      tc_fence_after_sync();
      const uint32_t dst = tmem + lanes + static_cast<uint32_t>(kABase + as * kACols);
      tmem_store_32cols(dst, h);
#pragma unroll
      for (int j = 0; j < 16; ++j) widen(w[16 + j], h[2 * j], h[2 * j + 1]);
      tmem_store_32cols(dst + 32, h);
      tmem_store_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_leader<CG>(smem_addr(&ctl.a_full[as]), leader);
      s += kWidenGroups;
      if (s >= p.w_stages) {
        s -= p.w_stages;
        phase ^= 1u;
      }
      as += kWidenGroups;
      if (as >= kASlots) {
        as -= kASlots;
        a_phase ^= 1u;
      }
    }
  } else {
    // -------------------------------------------------- epilogue warps
    const int quarter = warp & 3;
    const int half = (warp - kFirstEpilogue) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // an address is a uniform pointer to a row of the tile plus this lane's offset
    const uint32_t in_tile = rank * 128u + static_cast<uint32_t>(quarter * 32 + lane);
    const int64_t pitch = p.out_pitch * static_cast<int64_t>(sizeof(T));
    grid_dependency_wait();  // x_scale may come from the kernel before this one
    int it = 0;
    for (int u = unit0; u < total; u += units, ++it) {
      const int buf = bufs == 2 ? it & 1 : 0;
      const uint32_t use = static_cast<uint32_t>(bufs == 2 ? it >> 1 : it) & 1u;
      int tile_n, tile_v;
      tile_place(p, u, tile_n, tile_v);
      const int64_t v0 = static_cast<int64_t>(tile_v) * (128 * CG);
      const int64_t n0 = static_cast<int64_t>(tile_n) * p.nt;
      const bool mine = v0 + in_tile < p.v;
      // u_ij = acc * x_scale * (weight_scale * logit_scale) + bias * logit_scale
      const float ws = (mine ? __ldg(p.weight_scale + v0 + in_tile) : 0.0f) * p.xf.scale;
      const float b = mine && p.bias != nullptr
                          ? bias_at(p.bias, p.bias_dtype, v0 + in_tile) * p.xf.scale
                          : 0.0f;
      const int cols = static_cast<int>(p.n - n0 < p.nt ? p.n - n0 : p.nt);
      const int chunks = (cols + 31) / 32;
      // this warp's 32-column chunks: the first or the second half of them
      const int c0 = half == 0 ? 0 : (chunks + 1) / 2;
      const int c1 = half == 0 ? (chunks + 1) / 2 : chunks;
      // an ordinary load: the kernel before this one, which wrote the scales, may
      // have run beside it until the wait above
      auto scales = [&](int c) {
        return c * 32 + lane < cols ? p.x_scale[n0 + c * 32 + lane] : 0.0f;
      };
      float xs_next = scales(c0);
      const bool ok = mbar_wait(smem_addr(&ctl.acc_full[buf]), use, abort_flag, err_word);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after_sync();
      auto release = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_leader<CG>(smem_addr(&ctl.acc_empty[buf]), leader);
      };
      if (c0 >= c1) release();
      for (int c = c0; c < c1; ++c) {
        float z[32];
        tmem_load_32cols(tmem + lanes + static_cast<uint32_t>(buf * 128 + c * 32), z);
        if (c == c1 - 1) release();  // the accumulator has been read
        const float xs = xs_next;
        if (c + 1 < c1) xs_next = scales(c + 1);
        const int m = cols - c * 32;
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = fmaf(z[j] * __shfl_sync(0xffffffffu, xs, j), ws, b);
        if (p.xf.has_cap) {
          const uint64_t inv = f2_pack(p.xf.inv_softcap, p.xf.inv_softcap);
          const uint64_t cap = f2_pack(p.xf.softcap, p.xf.softcap);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            f2_unpack(f2_mul(f2_pack(z[j], z[j + 1]), inv), z[j], z[j + 1]);
            f2_unpack(f2_mul(tanh_pair(z[j], z[j + 1]), cap), z[j], z[j + 1]);
          }
        }
        uint8_t* const row0 = static_cast<uint8_t*>(p.out) +
                              ((n0 + c * 32) * p.out_pitch + v0) * static_cast<int64_t>(sizeof(T));
        const uint32_t off = in_tile * static_cast<uint32_t>(sizeof(T));
        if (mine) {
          if (m >= 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) store(reinterpret_cast<T*>(row0 + j * pitch + off), z[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < m) store(reinterpret_cast<T*>(row0 + j * pitch + off), z[j]);
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncwarp();
  if constexpr (CG == 1)
    __syncthreads();
  else
    cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    if constexpr (CG == 1)
      tmem_dealloc(tmem, 512);
    else
      tmem_dealloc_pair(tmem, 512);
  }
}

template <int CG, class T>
cudaError_t launch_typed(QLinearTcParams p, int sms, cudaStream_t s) {
  const int x_bytes = 2 * (p.nt / CG * 128);
  // The most weight stages that leave room for four of x and that are safe.
  // A widening group that waits for stage j has to find stage j - w of the
  // same buffer landed, or the parity that it waits for is the one before
  // last. Copies land in any order, so this holds where j - w was the group's
  // own (w a multiple of the groups), or where an MMA on a later stage is done:
  // the group's last stage, j - groups, had its slot freed by the MMAs up to
  // j - groups - slots.
  int w = kMaxWStages;
  while (w > kWidenGroups &&
         ((w % kWidenGroups != 0 && w < kWidenGroups + kASlots) ||
          kSmemBudget - w * kWStageBytes < 4 * x_bytes))
    --w;
  p.w_stages = w;
  p.x_stages = (kSmemBudget - w * kWStageBytes) / x_bytes;
  if (p.x_stages > kMaxXStages) p.x_stages = kMaxXStages;
  const int smem = w * kWStageBytes + p.x_stages * x_bytes + 1024;
  auto kern = qlinear_kernel<CG, T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBudget + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  // the kernel that widens x lets this one start: it loads weights meanwhile
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if constexpr (CG == 2) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const int64_t tiles = static_cast<int64_t>(p.n_tiles) * p.v_tiles;
  const int64_t units = sms / CG;
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < units ? tiles : units) * CG), 1, 1);
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int CG>
cudaError_t launch_cg(const QLinearTcParams& p, int out_dtype, int sms, cudaStream_t s) {
  if (out_dtype == FLCE_F32) return launch_typed<CG, float>(p, sms, s);
  if (out_dtype == FLCE_BF16) return launch_typed<CG, __nv_bfloat16>(p, sms, s);
  return launch_typed<CG, __half>(p, sms, s);
}

}  // namespace

cudaError_t launch_qlinear_tc(const QLinearTcParams& p, int cg, int out_dtype, int sms,
                              cudaStream_t s) {
  return cg == 1 ? launch_cg<1>(p, out_dtype, sms, s) : launch_cg<2>(p, out_dtype, sms, s);
}

}  // namespace flce
