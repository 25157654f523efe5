// C entry points that orthogonalise matrices (include/flce.h): argument checks,
// scales, workspace and launches. Nothing is allocated on the device and
// nothing waits for it.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <utility>

#include "flce.h"
#include "host_common.h"
#include "ortho_internal.h"

namespace {

using namespace flce::host;

constexpr int64_t kMaxSide = 1 << 20;
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxSteps = flce::kOrthoMaxSteps;

bool float_type(int32_t d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }
size_t size_of(int32_t d) { return d == FLCE_F32 ? 4 : 2; }

// The largest |a + b t + c t^2| for 0 <= t <= top.
double poly_bound(double a, double b, double c, double top) {
  double best = std::max(std::fabs(a), std::fabs(a + b * top + c * top * top));
  const double t = c != 0.0 ? -b / (2.0 * c) : -1.0;
  if (t > 0.0 && t < top) best = std::max(best, std::fabs(a + b * t + c * t * t));
  return best;
}
// The largest |s (a + b s^2 + c s^4)| for 0 <= s <= top: at the end, or where
// a + 3 b t + 5 c t^2 = 0 with t = s^2.
double step_bound(double a, double b, double c, double top) {
  const auto at = [&](double t) { return std::sqrt(t) * std::fabs(a + b * t + c * t * t); };
  double best = at(top * top);
  const auto root = [&](double t) {
    if (t > 0.0 && t < top * top) best = std::max(best, at(t));
  };
  if (c != 0.0) {
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0) {
      root((-3.0 * b + std::sqrt(d)) / (10.0 * c));
      root((-3.0 * b - std::sqrt(d)) / (10.0 * c));
    }
  } else if (b != 0.0) {
    root(-a / (3.0 * b));
  }
  return best;
}

// The power of two that takes values up to `bound` to at most 2^14: halves
// reach 65504, which leaves what roundings add to a bound a factor of four.
int shift_for(double bound) {
  int e = 0;
  std::frexp(bound, &e);  // bound < 2^e
  return 14 - std::max(e, -40);
}
double scale_for(double bound) { return std::ldexp(1.0, shift_for(bound)); }

// What the steps do to singular values, from which everything else is planned:
// bounds on them before each step (and after the last), and on the step's
// polynomial of their squares, both of the formula without roundings.
struct Bounds {
  double top[kMaxSteps + 1], poly[kMaxSteps];
};
// Roundings move a singular value: by up to 2^-11 of it where x is rounded, and
// up to four times as much where the gram and a polynomial are that is larger
// elsewhere than for this value. The steps that follow must not make much of it.
// Above the largest value that a schedule is made for, its polynomials may rise
// twelve times as fast as the value itself, and five such steps turn 2^-11 into
// anything (64-bit arithmetic with every operand rounded to halves: noise of 12 x
// 20 values off by up to 93 %, a constant matrix NaN). So schedules have to bear
// kMoved before every step, as those with the usual safety factor of 1.01 do.
constexpr double kMoved = 1.0 / 512;
constexpr double kMost = 1.5;  // times a bound, by moved values: 1.5^3 stays below 4
// Fills `b`. The step whose bounds do not hold, or -1; `moved` says whether
// that is by moved values alone.
int find_bounds(const flce_ortho_problem* p, Bounds* b, bool* moved) {
  b->top[0] = 1.0;
  *moved = false;
  double with = 1.0;  // top[k], moved
  for (int k = 0; k < p->steps; ++k) {
    const float* const abc = p->coefficients + 3 * k;
    const double top = b->top[k];
    const double poly = poly_bound(abc[0], abc[1], abc[2], top * top);
    const double next = step_bound(abc[0], abc[1], abc[2], top);
    b->poly[k] = poly;
    b->top[k + 1] = next;
    if (!(poly <= 1.0e4) || !(next <= 16.0) || !(next >= 1.0e-4)) return k;
    with *= 1.0 + kMoved;
    const double poly_with = poly_bound(abc[0], abc[1], abc[2], with * with);
    with = step_bound(abc[0], abc[1], abc[2], with);
    if (!(poly_with <= kMost * poly) || !(with <= kMost * next)) {
      *moved = true;
      return k;
    }
  }
  return -1;
}

// The scales of each step's operands, and what turns sums into them.
void fill_steps(const flce_ortho_problem* p, const Bounds& b, flce::OrthoStep* step) {
  double x_scale = scale_for(b.top[0]);
  for (int k = 0; k < p->steps; ++k) {
    const float* const abc = p->coefficients + 3 * k;
    const double g_scale = scale_for(b.top[k] * b.top[k]);
    const double p_scale = scale_for(b.poly[k]);
    const double next_scale = k + 1 == p->steps ? 1.0 : scale_for(b.top[k + 1]);
    flce::OrthoStep& t = step[k];
    t.gram = static_cast<float>(g_scale / (x_scale * x_scale));
    t.poly = static_cast<float>(abc[2] * p_scale / (g_scale * g_scale));
    t.old = static_cast<float>(abc[1] * p_scale / g_scale);
    t.diag = static_cast<float>(abc[0] * p_scale);
    t.product = static_cast<float>(next_scale / (x_scale * p_scale));
    x_scale = next_scale;
  }
}

// The products of all steps. A group of steps s, s + 1, ... multiplies x by the
// polynomials of its steps all at once: with the gram A of the group's x, and
// P = p_s(A), the next step's gram is P A P and its x P x, and all of these
// commute. So each step after a group's first takes two products for its gram,
// one for its polynomial and one to gather the polynomials, all m x m.
//
// Roundings of a gram, of 2^-12 of it, are noise in the directions of small
// singular values too, and there P on both sides magnifies them by the square of
// its largest value. A group goes on while that is below 12^2 (11.9 before the
// third of the default steps): with the published tuned steps, of 8.2, 4.1 and 3.9,
// three in a group put noise of 0.3 to 1.0 (the 2-norm, for singular values as
// 1 / k^2) where steps by themselves and groups of two put 0.2.
constexpr double kCarried = 12.0;

// The gram's values are below the squares of the singular values' bound, and a
// gathered polynomial's below the product of the bounds of its parts. Each is
// held with a power of two of its own.
int list_products(const flce_ortho_problem* p, const Bounds& b, bool grouped, bool tall,
                  flce::OrthoProduct* out) {
  using flce::OrthoOp;
  int count = 0;
  const auto add = [&](OrthoOp op, int a, int b, int c, double scale, int power = 0,
                       double old = 0.0, double diag = 0.0) {
    flce::OrthoProduct& t = out[count++];
    t.op = static_cast<int8_t>(op);
    t.a = static_cast<int8_t>(a);
    t.b = static_cast<int8_t>(b);
    t.c = static_cast<int8_t>(c);
    t.cut = op == OrthoOp::kGram ? 0 : op <= OrthoOp::kPoly ? 1 : 2;
    t.power = static_cast<int8_t>(power);
    t.scale = static_cast<float>(scale);
    t.old = static_cast<float>(old);
    t.diag = static_cast<float>(diag);
  };
  double x_scale = scale_for(b.top[0]);
  int from = flce::kOrthoX0;
  for (int k = 0; k < p->steps;) {
    // groups of three, of two at the end
    const int left = p->steps - k;
    const int most = !grouped ? 1 : left == 4 ? 2 : std::min(3, left);
    int group = 1;
    for (double carried = b.poly[k]; group < most && carried <= kCarried; ++group)
      carried *= b.poly[k + group];
    const int first = k;
    double g_scale = scale_for(b.top[k] * b.top[k]);
    add(OrthoOp::kGram, from, from, flce::kOrthoGram, g_scale / (x_scale * x_scale),
        k == 0 ? 2 : 0);
    // the buffers of the gathered polynomial, of a step's own, and a free one
    int gathered = flce::kOrthoP0, own = flce::kOrthoP1, spare = flce::kOrthoP2;
    double all = 1.0, all_scale = 1.0;  // its bound and scale
    for (int s = 0; s < group; ++s, ++k) {
      const float* const abc = p->coefficients + 3 * k;
      const double most = b.poly[k], top = b.top[k], next = b.top[k + 1];
      const double p_scale = scale_for(most);
      const int mine = s == 0 ? gathered : own;
      add(OrthoOp::kPoly, flce::kOrthoGram, flce::kOrthoGram, mine,
          abc[2] * p_scale / (g_scale * g_scale), 0, abc[1] * p_scale / g_scale,
          abc[0] * p_scale);
      if (s + 1 < group) {  // the gram of the next step
        const double half_scale = scale_for(most * top * top);
        const double next_scale = scale_for(next * next);
        add(OrthoOp::kSquare, mine, flce::kOrthoGram, spare, half_scale / (p_scale * g_scale));
        add(OrthoOp::kSquare, spare, mine, flce::kOrthoGram,
            next_scale / (half_scale * p_scale));
        g_scale = next_scale;
      }
      if (s == 0) {
        all = most;
        all_scale = p_scale;
      } else {
        all *= most;
        const double scale = scale_for(all);
        add(OrthoOp::kSquare, mine, gathered, spare, scale / (p_scale * all_scale));
        std::swap(gathered, spare);
        all_scale = scale;
      }
    }
    const bool last = k == p->steps;
    const double next_scale = last ? 1.0 : scale_for(b.top[k]);
    const double scale = next_scale / (x_scale * all_scale);
    const int power = first == 0 ? 1 : 0;
    if (last && tall) {
      add(OrthoOp::kOutTall, from, gathered, flce::kOrthoOut, scale, power);
    } else if (last) {
      add(OrthoOp::kOutWide, gathered, from, flce::kOrthoOut, scale, power);
    } else {
      const int to = from == flce::kOrthoX0 ? flce::kOrthoX1 : flce::kOrthoX0;
      add(OrthoOp::kMul, gathered, from, to, scale, power);
      from = to;
    }
    x_scale = next_scale;
  }
  return count;
}

// Fills `b` where it returns FLCE_OK.
flce_status check_problem(const flce_ortho_problem* p, Bounds* b) {
  if (p == nullptr) return fail(FLCE_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0 || p->rows < 0 || p->cols < 0)
    return fail(FLCE_ERR_INVALID_ARG, "batch = %lld, rows = %lld, cols = %lld",
                (long long)p->batch, (long long)p->rows, (long long)p->cols);
  if (p->batch > kMaxBatch || p->rows > kMaxSide || p->cols > kMaxSide)
    return fail(FLCE_ERR_UNSUPPORTED, "at most %lld matrices of at most %lld rows and columns",
                (long long)kMaxBatch, (long long)kMaxSide);
  if (!float_type(p->dtype))
    return fail(FLCE_ERR_INVALID_ARG, "dtype %d is not an flce_dtype", p->dtype);
  if (p->out_dtype != FLCE_BF16 && p->out_dtype != FLCE_F16)
    return fail(FLCE_ERR_INVALID_ARG, "out_dtype must be FLCE_BF16 or FLCE_F16");
  if (p->row_pitch < p->cols || p->batch_stride < 0 || p->row_pitch > (int64_t(1) << 40) ||
      p->batch_stride > (int64_t(1) << 46))
    return fail(FLCE_ERR_INVALID_ARG, "row_pitch = %lld, batch_stride = %lld",
                (long long)p->row_pitch, (long long)p->batch_stride);
  if (!(p->eps >= FLT_MIN) || !std::isfinite(p->eps))
    return fail(FLCE_ERR_INVALID_ARG, "eps must be finite and at least %g", (double)FLT_MIN);
  if (p->steps < 1 || p->steps > kMaxSteps || p->coefficients == nullptr)
    return fail(FLCE_ERR_INVALID_ARG, "1 to %lld steps, with coefficients for each",
                (long long)kMaxSteps);
  bool moved = false;
  const int bad = find_bounds(p, b, &moved);
  if (bad >= 0 && moved)
    return fail(FLCE_ERR_UNSUPPORTED,
                "step %d magnifies roundings of the largest singular values past its range: give "
                "the steps a safety factor, as a / 1.01, b / 1.01^3, c / 1.01^5", bad);
  if (bad >= 0)
    return fail(FLCE_ERR_UNSUPPORTED,
                "the coefficients of step %d take singular values up to %g", bad, b->top[bad + 1]);
  if (p->reserved != 0) return fail(FLCE_ERR_INVALID_ARG, "reserved is not 0");
  return FLCE_OK;
}

// How many pairs of CTAs take a product's tiles, and how many of the tiles are
// cut between pairs.
struct Split {
  int64_t units, whole, cut;
};
constexpr int64_t kPlanPairs = 80;  // that a workspace is planned for
constexpr int64_t kMaxParts = 4;    // of a tile where there are fewer tiles than pairs

// A step of 64 along the contraction takes a pair 0.27 us (a CTA on 128 x 128
// 0.14). Cutting costs a tile some 3 us and 1.1 (0.6) more for each further part, as the sums go through L2, and
// pairs that no longer walk the contraction together share fewer loads. So
// tiles are cut where the last round would leave most pairs idle for long:
// eight grams of 1024 x 4096 (80 tiles, 64 steps) take 38 us cut and 49 whole,
// the product of 4096 x 4096 (256 tiles) 82 and 89, but its gram (136 tiles)
// 54 and 50, and that of 4096 x 14336 169 and 152.
Split split_of(int64_t tiles, int64_t k_iters, int64_t pairs, bool large) {
  const double each = large ? 0.27 : 0.14, join = large ? 1.1 : 0.6;
  if (tiles >= pairs) {
    const int64_t left = tiles % pairs;
    // the last round would run with `left` pairs
    if (left == 0 || 2 * left > pairs || (pairs - left) * k_iters < 24 * pairs)
      return {pairs, tiles, 0};
    return {pairs, tiles - pairs - left, pairs + left};
  }
  int64_t parts = 1;
  double best = each * k_iters;
  for (int64_t s = 2; s <= kMaxParts && s * tiles <= pairs && 4 * s <= k_iters; ++s) {
    const double t = each * k_iters / s + 1.9 + join * s;
    if (t < best) {
      best = t;
      parts = s;
    }
  }
  return parts > 1 ? Split{parts * tiles, 0, tiles} : Split{tiles, tiles, 0};
}

constexpr int32_t kArrived = 2 * (2 * kPlanPairs) * 2 * flce::kOrthoWarps;

struct Plan {
  int64_t cluster, slab;  // of matrices that stay in shared memory, else 0
  int64_t m, n, m_pad, n_pad, parts;
  size_t buffer[flce::kOrthoBuffers], partial, factor, counts, shares, total;
  bool grouped;  // several steps on one gram
};
Plan plan_of(const flce_ortho_problem* p) {
  Plan q{};
  q.m = std::min(p->rows, p->cols);
  q.n = std::max(p->rows, p->cols);
  if (q.m <= 128 && q.n <= 512 * flce::kOrthoMaxCluster) {
    q.cluster = 1;
    while (q.n > 512 * q.cluster) q.cluster *= 2;
    q.slab = std::max<int64_t>(64, ceil_div(ceil_div(q.n, q.cluster), 64) * 64);
    return q;
  }
  q.m_pad = ceil_div(q.m, flce::kOrthoTile) * flce::kOrthoTile;
  q.n_pad = ceil_div(q.n, 64) * 64;
  // Shares of 4096 values while the batch has two or fewer for an SM, of 8192 to
  // five CTAs an SM.
  q.parts = q.m * q.n / 4096;
  if (q.parts * p->batch > 2 * flce::kOrthoPlanSms)
    q.parts = std::min<int64_t>(q.m * q.n / 8192,
                                5 * flce::kOrthoPlanSms / std::max<int64_t>(1, p->batch));
  q.parts = std::max<int64_t>(1, q.parts);
  const size_t b = static_cast<size_t>(p->batch);
  const size_t x_bytes = align_256(b * static_cast<size_t>(q.m_pad * q.n_pad) * 2);
  const size_t g_bytes = align_256(b * static_cast<size_t>(q.m_pad * q.m_pad) * 2);
  // Steps of one group take one gram and one product with x, 3 m^2 n operations
  // together, instead of one each, and 3 m^3 more for each step after the first.
  // Two groups of five steps are three products more than five steps by
  // themselves, each of which waits some 8 us for the one before.
  q.grouped = p->steps > 1 &&
              static_cast<double>(p->batch) * q.m * q.m * (q.n - q.m) > 4.0e9;
  q.buffer[flce::kOrthoX0] = 0;
  q.buffer[flce::kOrthoX1] = x_bytes;
  q.buffer[flce::kOrthoGram] = q.buffer[flce::kOrthoX1] + (p->steps > 1 ? x_bytes : 0);
  q.buffer[flce::kOrthoP0] = q.buffer[flce::kOrthoGram] + g_bytes;
  q.buffer[flce::kOrthoP1] = q.buffer[flce::kOrthoP0] + g_bytes;
  q.buffer[flce::kOrthoP2] = q.buffer[flce::kOrthoP1] + (q.grouped ? g_bytes : 0);
  q.partial = q.buffer[flce::kOrthoP2] + (q.grouped ? g_bytes : 0);
  q.factor = q.partial + align_256(b * static_cast<size_t>(q.parts) * 8);
  q.counts = q.factor + align_256(b * 4);
  q.shares = q.counts + align_256((kArrived + b + 1) * 4);
  const int64_t side = q.m_pad / flce::kOrthoTile;
  const int64_t tiles = p->batch * side * ceil_div(q.n, flce::kOrthoTile);
  q.total = q.shares + static_cast<size_t>(2 * std::min(kPlanPairs, kMaxParts * tiles)) *
                           flce::kOrthoShareBytes;
  return q;
}

// A map of [batch][outer][inner] 16-bit values (batch 0: two dimensions).
bool make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer,
              uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle,
              int64_t batch = 0) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) {
    fail(FLCE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2,
                                 static_cast<cuuint64_t>(inner) * outer * 2};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, batch > 0 ? 3 : 2, const_cast<void*>(base), dims,
          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fail(FLCE_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d (%lld x %lld)",
         static_cast<int>(r), (long long)inner, (long long)outer);
    return false;
  }
  return true;
}

constexpr CUtensorMapSwizzle kLoad = CU_TENSOR_MAP_SWIZZLE_128B;
constexpr CUtensorMapSwizzle kStore = CU_TENSOR_MAP_SWIZZLE_64B;

// After which a wait gives up. The longest one is for some tiles' products.
constexpr uint64_t kWaitNs = 4000000000ull;  // 4 s

// `lost`: each product after the first waits for one count that never comes.
flce_status orthogonalize(const flce_ortho_problem* p, const void* src, void* out,
                          int32_t* err_word, void* workspace, size_t workspace_bytes,
                          void* stream, uint64_t wait_ns, bool lost) {
  Bounds bounds;
  flce_status st = check_problem(p, &bounds);
  if (st != FLCE_OK) return st;
  const bool empty = p->batch == 0 || p->rows == 0 || p->cols == 0;
  if (!empty && (src == nullptr || out == nullptr))
    return fail(FLCE_ERR_INVALID_ARG, "src and out are required");
  if (!aligned_to(src, size_of(p->dtype)) || !aligned_to(out, 2) || !aligned_to(err_word, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "a pointer is misaligned for its type");
  const Plan plan = plan_of(p);
  // coordinates and the numbers of tiles are 32-bit
  if (p->batch * plan.m_pad > (int64_t(1) << 30) ||
      p->batch * ceil_div(plan.n, 256) * (plan.m_pad / 256) > (int64_t(1) << 28))
    return fail(FLCE_ERR_UNSUPPORTED, "the batch has too many rows");
  st = check_workspace(workspace, workspace_bytes, plan.total);
  if (st != FLCE_OK) return st;
  int sms = 0;
  st = check_device(&sms);
  if (st != FLCE_OK || empty) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const bool tall = p->rows > p->cols;

  if (lost && plan.cluster > 0)
    return fail(FLCE_ERR_UNSUPPORTED, "the matrices stay in shared memory");
  if (plan.cluster > 0) {
    flce::OrthoSmallParams k{};
    fill_steps(p, bounds, k.step);
    k.src = src;
    k.batch_stride = p->batch_stride;
    k.row_pitch = p->row_pitch;
    k.out = out;
    k.batch = static_cast<int32_t>(p->batch);
    k.rows = static_cast<int32_t>(p->rows);
    k.cols = static_cast<int32_t>(p->cols);
    k.tall = tall ? 1 : 0;
    k.steps = p->steps;
    k.cluster = static_cast<int32_t>(plan.cluster);
    k.slab = static_cast<int32_t>(plan.slab);
    k.x_shift = shift_for(1.0);
    k.out_bf16 = p->out_dtype == FLCE_BF16 ? 1 : 0;
    k.eps = p->eps;
    k.err_word = err_word;
    const cudaError_t e = flce::launch_ortho_small(k, p->dtype, s);
    return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "orthogonalising kernel");
  }
  flce::OrthoCopyParams c{};
  c.src = src;
  c.batch_stride = p->batch_stride;
  c.row_pitch = p->row_pitch;
  c.batch = static_cast<int32_t>(p->batch);
  c.rows = static_cast<int32_t>(p->rows);
  c.cols = static_cast<int32_t>(p->cols);
  c.tall = tall ? 1 : 0;
  c.m = static_cast<int32_t>(plan.m);
  c.n = static_cast<int32_t>(plan.n);
  c.m_pad = static_cast<int32_t>(plan.m_pad);
  c.n_pad = static_cast<int32_t>(plan.n_pad);
  c.x = ws + plan.buffer[flce::kOrthoX0];
  c.partial = reinterpret_cast<double*>(ws + plan.partial);
  c.parts = static_cast<int32_t>(plan.parts);
  c.eps = p->eps;
  c.x_shift = shift_for(1.0);
  c.m_rows = static_cast<int32_t>(ceil_div(plan.m, 64) * 64);
  c.factor = reinterpret_cast<float*>(ws + plan.factor);
  c.count = reinterpret_cast<int32_t*>(ws + plan.counts);
  c.counts = kArrived + c.batch + 1;
  flce::OrthoRunParams r{};
  const int64_t x_rows = p->batch * plan.m_pad;
  for (int i = 0; i < flce::kOrthoBuffers; ++i) {
    if ((i == flce::kOrthoX1 && p->steps == 1) || (i > flce::kOrthoP0 && !plan.grouped)) continue;
    const bool is_x = i <= flce::kOrthoX1;
    const int64_t cols = is_x ? plan.n_pad : plan.m_pad;
    uint8_t* const base = ws + plan.buffer[i];
    if (!make_map(&r.along[i], base, cols, x_rows, 64, 128, kLoad) ||
        !make_map(&r.store[i], base, cols, x_rows, 32, 32, kStore) ||
        (is_x && !make_map(&r.across[i], base, cols, x_rows, 64, 64, kLoad)))
      return FLCE_ERR_CUDA;
  }
  // maps take rows of whole 16 bytes
  const bool out_mapped = p->cols % 8 == 0 && aligned_to(out, 16);
  if (out_mapped && !make_map(&r.store[flce::kOrthoOut], out, p->cols, p->rows, 32, 32, kStore,
                              p->batch))
    return FLCE_ERR_CUDA;
  r.products = list_products(p, bounds, plan.grouped, tall, r.product);
  r.batch = c.batch;
  // Tiles of 128, one to an SM, or of 256, one to a pair of SMs. The small ones
  // take half as long to come and go, which counts where products are short and
  // wait for each other, and pad less; the large ones load half as much for an
  // operation, which counts over many rounds. So small ones are taken
  // - where a product with x has two rounds of them: 2048 x 2048 takes 278 us,
  //   with large ones 333;
  // - where a symmetric product has one round (a quarter more in a batch, whose
  //   matrices fill each other's rounds) and the product with x not too many: 2048
  //   x 4096 356 and 474, 1024 x 8192 242 and 297, four of 1024 x 4096 293 and 318,
  //   six of 777 x 1555 226 and 242 (but 1536 x 16384, 10 rounds, 519 and 458; 2304
  //   x 2304 389 and 368; three of 2049 x 1365 312 and 299);
  // - for short contractions: 100 of 384 x 384 278 and 380, 128 of 256 x 512 225
  //   and 253;
  // - in a batch where they pad to five sixths at most: ten of 640 x 900 167 and 197,
  //   fourteen of 640 x 640 165 and 192 (but eight of 1000 x 1000 254 and 237).
  const int64_t side = ceil_div(plan.m, 128);
  const int64_t gram_tiles = p->batch * side * (side + 1) / 2;
  const int64_t x_tiles = p->batch * side * ceil_div(plan.n, 128);
  const int64_t x_large = p->batch * ceil_div(plan.m, 256) * ceil_div(plan.n, 256);
  const bool small =
      plan.m <= 384 || x_tiles <= 2 * sms || (gram_tiles <= sms && x_tiles <= 7 * sms) ||
      (p->batch > 1 && ((4 * gram_tiles <= 5 * sms && x_tiles <= 4 * sms) ||
                        (6 * x_tiles <= 5 * 4 * x_large && x_tiles <= 7 * sms)));
  r.pairs = small ? 0 : 1;
  const int64_t tile = r.pairs ? flce::kOrthoTile : flce::kOrthoTile / 2;
  const int64_t ctas = r.pairs ? 2 : 1;  // of a tile
  r.m_tiles = static_cast<int32_t>(ceil_div(plan.m, tile));
  r.n_tiles = static_cast<int32_t>(ceil_div(plan.n, tile));
  r.k_n = static_cast<int32_t>(plan.n_pad / 64);
  r.k_m = static_cast<int32_t>(ceil_div(plan.m, 64));
  r.m_pad = c.m_pad;
  r.m_rows = c.m_rows;
  r.n_pad = c.n_pad;
  r.out_mapped = out_mapped ? 1 : 0;
  r.rows = c.rows;
  r.cols = c.cols;
  r.factor = c.factor;
  r.gram = ws + plan.buffer[flce::kOrthoGram];
  r.out = out;
  r.shares = ws + plan.shares;
  r.arrived = c.count;
  r.finished = c.count + kArrived;
  r.ticket = r.finished + c.batch;
  r.wait_ns = wait_ns;
  r.err_word = err_word;
  const int64_t pairs = std::min<int64_t>(2 * kPlanPairs, sms) / ctas;
  const int64_t triangle = p->batch * r.m_tiles * (r.m_tiles + 1) / 2;
  const int64_t all = p->batch * r.m_tiles * r.n_tiles;
  // Matrices of a batch fill each other's rounds: their tiles stay whole, unless
  // there are too few of them all the same.
  const bool whole = p->batch > 1 && all >= pairs;
  for (int i = 0; i < 3; ++i) {
    const int64_t tiles = i < 2 ? triangle : all;
    const Split split = whole ? Split{std::min(tiles, pairs), tiles, 0}
                              : split_of(tiles, i == 0 ? r.k_n : r.k_m, pairs, r.pairs != 0);
    r.cut[i].units = static_cast<int32_t>(split.units);
    r.cut[i].whole = static_cast<int32_t>(split.whole);
    r.cut[i].cut = static_cast<int32_t>(split.cut);
    r.units = std::max(r.units, r.cut[i].units);
    if (split.cut > 0) r.joint = 1;
  }
  int64_t need = 0, items = 0;
  for (int i = 0; i < r.products; ++i) {
    const flce::OrthoCut& c = r.cut[r.product[i].cut];
    items += c.cut > 0 ? c.units + c.whole : r.product[i].cut < 2 ? triangle : all;
    r.product[i].need = static_cast<int32_t>(need) + (lost && i > 0 ? 1 << 30 : 0);
    need += (r.product[i].cut < 2 ? triangle : all) / (r.joint ? 1 : p->batch) * ctas *
            flce::kOrthoWarps;
  }
  r.items = static_cast<int32_t>(items);
  if (need > (lost ? 1 << 30 : 0x7fffffff) || items > 0x7fff0000)
    return fail(FLCE_ERR_UNSUPPORTED, "too many tiles and steps to count");
  cudaError_t e = flce::launch_ortho_norm(c, p->dtype, s);
  if (e != cudaSuccess) return cuda_fail(e, "matrix norm kernel");
  e = flce::launch_ortho_copy(c, p->dtype, s);
  if (e != cudaSuccess) return cuda_fail(e, "matrix copy kernel");
  e = flce::launch_ortho_run(r, p->out_dtype, s);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e, "orthogonalising kernel");
}

}  // namespace

extern "C" {

size_t flce_orthogonalize_workspace_size(const flce_ortho_problem* p) {
  Bounds bounds;
  if (check_problem(p, &bounds) != FLCE_OK) return 0;
  return plan_of(p).total;
}

flce_status flce_orthogonalize(const flce_ortho_problem* p, const void* src, void* out,
                               int32_t* err_word, void* workspace, size_t workspace_bytes,
                               void* stream) {
  clear_error();
  return orthogonalize(p, src, out, err_word, workspace, workspace_bytes, stream, kWaitNs, false);
}

flce_status flce_selftest_orthogonalize_timeout(const flce_ortho_problem* p, const void* src,
                                                void* out, int32_t* err_word, void* workspace,
                                                size_t workspace_bytes, double budget_s,
                                                void* stream) {
  clear_error();
  if (err_word == nullptr) return fail(FLCE_ERR_INVALID_ARG, "err_word is required");
  if (!(budget_s > 0.0) || budget_s > 1.0)
    return fail(FLCE_ERR_INVALID_ARG, "budget_s must be in (0, 1] seconds");
  return orthogonalize(p, src, out, err_word, workspace, workspace_bytes, stream,
                       static_cast<uint64_t>(budget_s * 1e9), true);
}

}  // extern "C"
