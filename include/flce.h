/*
 * flce.h -- C ABI of libflce.so: fused linear cross-entropy on one GB300
 * (sm_103a) GPU.
 *
 * The operation ("fused-linear-ce" model card, trl-lib: §Full signature,
 * §Metrics for free, §Algorithm):
 *
 *   lin_ij  = hidden_i . weight_j + bias_j                 (i < N, j < V)
 *   u_ij    = logit_scale * lin_ij
 *   z_ij    = softcap * tanh(u_ij / softcap)   if softcap > 0, else u_ij
 *   lse_i   = log sum_j exp(z_ij),   p_ij = exp(z_ij - lse_i)
 *   loss_i  = lse_i - z_{i,t_i}      (0 when t_i == ignore_index)
 *   loss    = sum_i loss_i / n_valid ("mean") | sum_i loss_i ("sum") | loss_i ("none")
 *   mean_token_accuracy = #{valid i : argmax_j z_ij == t_i} / n_valid
 *   entropy             = sum_{valid i} (lse_i - sum_j p_ij z_ij) / n_valid   (nats)
 *
 * and its backward (§Algorithm: the logits are recomputed and the logit
 * gradient is the softmax minus the one-hot target):
 *
 *   D_ij          = g_i (p_ij - [j == t_i]) * logit_scale * (1 - tanh^2(u_ij/softcap))
 *   grad_hidden   = D @ weight,  grad_weight = D^T @ hidden,  grad_bias = sum_i D_ij
 *
 * with g_i = grad_out/n_valid ("mean"), grad_out ("sum") or grad_out[i]
 * ("none"), and g_i = 0 on ignored rows. n_valid counts rows whose target is
 * not ignore_index. The N x V logit matrix is never stored: the forward keeps
 * per-(row, vocabulary tile) softmax statistics, the backward recomputes the
 * logits one vocabulary chunk at a time.
 *
 * Conventions shared by every entry point:
 *   - Every pointer argument except `p` is a DEVICE pointer on the current
 *     CUDA device; `p` is a host pointer read during the call only.
 *   - The caller owns all memory, including the workspace. The library never
 *     allocates or frees device memory and never synchronises the stream:
 *     every kernel is enqueued on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and the call returns before the work completes.
 *   - Tensors are dense row-major: hidden [N,H], weight [V,H], bias [V],
 *     targets int64 [N]. hidden, weight and bias share `p->dtype`.
 *   - FLCE_BF16 and FLCE_F16 need H % 8 == 0 and 16-byte aligned
 *     hidden/weight/bias pointers (tensor-memory-accelerator row pitch rule);
 *     FLCE_F32 needs 4-byte alignment. Violations return FLCE_ERR_UNSUPPORTED
 *     before any launch.
 *   - Dtypes: FLCE_BF16 and FLCE_F16 run on the tensor cores (bf16 or fp16
 *     products, fp32 accumulation). FLCE_F32 runs on the tensor cores too,
 *     each operand split into three bf16 parts that sum to it exactly and each
 *     product formed from six part products (within about 2^-23 of it), when
 *     H % 8 == 0 and the parts' workspace stays under 40 % of one fp32 N x V
 *     matrix; otherwise on fp32 FFMA kernels. Both meet the same fp32 bars.
 *   - Argument errors are detected on the host, before any launch, and
 *     return a non-OK status; flce_last_error() then describes the problem.
 *     A failed launch returns FLCE_ERR_CUDA.
 *   - Errors that only the device can see are ORed into `*err_word` (when it
 *     is non-NULL) asynchronously: FLCE_DEVERR_TARGET_RANGE for a target
 *     outside [0,V) that is not ignore_index (that row's loss is NaN and it
 *     gets no gradient), FLCE_DEVERR_TIMEOUT when a kernel's bounded wait
 *     expired (results are then invalid). The caller zeroes the word and
 *     reads it after its own synchronisation.
 *   - No C++ exception crosses this interface. Entry points are thread-safe;
 *     calls that share a workspace must be ordered on one stream.
 */
#ifndef FLCE_H
#define FLCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum flce_status {
  FLCE_OK = 0,
  FLCE_ERR_INVALID_ARG = 1,   /* bad shape, option, or NULL required pointer */
  FLCE_ERR_UNSUPPORTED = 2,   /* valid but not supported (alignment, GPU arch) */
  FLCE_ERR_WORKSPACE = 3,     /* workspace smaller than *_workspace_size() or misaligned */
  FLCE_ERR_CUDA = 4,          /* a CUDA runtime/driver call or launch failed */
  FLCE_ERR_DEVICE_TIMEOUT = 5 /* reserved for callers that translate FLCE_DEVERR_TIMEOUT */
} flce_status;

typedef enum flce_dtype { FLCE_F32 = 0, FLCE_BF16 = 1, FLCE_F16 = 2 } flce_dtype;

typedef enum flce_reduction {
  FLCE_RED_NONE = 0,
  FLCE_RED_SUM = 1,
  FLCE_RED_MEAN = 2
} flce_reduction;

/* Bits of the device error word. */
#define FLCE_DEVERR_TARGET_RANGE 1
#define FLCE_DEVERR_TIMEOUT 2

/* Problem description (host struct, copied during the call).
 *   n, h, v            tokens, hidden size, vocabulary size (n >= 0, h >= 1, v >= 1)
 *   dtype              flce_dtype of hidden, weight and bias
 *   has_bias           0 or 1
 *   ignore_index       target value that marks an ignored row (default -100)
 *   logit_scale        multiplies the linear logits (finite)
 *   softcap            > 0 enables z = softcap*tanh(u/softcap); <= 0 disables
 *   reduction          flce_reduction
 *   grad_weight_dtype  dtype of grad_weight: FLCE_F32, or equal to dtype
 *   vocab_chunk        backward vocabulary chunk width; 0 picks the default:
 *                      equal chunks of whole 256-column tiles, at least five
 *                      of them (one per tile for a vocabulary of fewer than
 *                      five tiles), more where an N x chunk dlogits buffer
 *                      would exceed 512 MiB. The buffer is the largest
 *                      workspace item, so a smaller chunk lowers peak memory
 *                      at some cost in speed. Rounded up to a multiple of 256
 *   flags              OR of FLCE_SKIP_IGNORED_ROWS; 0 for none
 *   label_smoothing    eps in [0, 1]: cross-entropy against the target
 *                      distribution (1-eps)*onehot + eps/V, i.e.
 *                      loss_i = (1-eps)(lse_i - z_{i,t_i}) + eps(lse_i - mean_j z_ij)
 *   z_loss             lam >= 0: lam * lse_i^2 is added to each non-ignored row
 *   reserved           must be 0
 * With label smoothing and z-loss the logit gradient is
 *   g_i (p_ij (1 + 2 lam lse_i) - (1-eps)[j == t_i] - eps/V).
 * Both options are named in the CuTe-DSL FLCE pull request's feature list
 * (Liger-Kernel #1287, Summary); the forms above are the plain readings.
 */
typedef struct flce_problem {
  int64_t n, h, v;
  int32_t dtype;
  int32_t has_bias;
  int64_t ignore_index;
  float logit_scale;
  float softcap;
  int32_t reduction;
  int32_t grad_weight_dtype;
  int64_t vocab_chunk;
  int32_t flags;
  float label_smoothing;
  float z_loss;
  int32_t reserved;
} flce_problem;

/* Leave rows whose target is ignore_index out of every contraction (bf16 and
 * fp16 paths; the fp32 path computes every row either way). The non-ignored rows are
 * gathered, in their original order, into the workspace, and the GEMMs run
 * over them alone: ignored rows contribute nothing to the loss or to any
 * gradient, so their logits are never needed. Loss, metrics and gradients are
 * unchanged; loss_rows and correct_rows of ignored rows are 0 as without the
 * flag, but lse_rows and entropy_rows of ignored rows are not computed (NaN).
 * Grad_hidden rows of ignored rows are written as 0. */
#define FLCE_SKIP_IGNORED_ROWS 1

/* Bytes of device workspace flce_forward() needs for `p` (0 if `p` is
 * invalid). Following §Algorithm (the vocabulary is swept in tiles, each
 * folded into a running log-sum-exp), the workspace holds the per-(row,
 * vocabulary tile) statistics that the merge combines: about
 * N * ceil(V/256) * 16 bytes (20 with label smoothing). */
size_t flce_forward_workspace_size(const flce_problem* p);

/* Forward pass. Cite: §Algorithm (forward), §Metrics for free.
 *   hidden [N,H], weight [V,H], bias [V] (NULL unless p->has_bias), targets [N]
 *   loss_rows    [N] fp32 out: per-row loss (0 on ignored rows)       required
 *   lse_rows     [N] fp32 out: per-row log-sum-exp, kept for backward required
 *   correct_rows [N] int32 out: 1 where argmax == target (valid rows) nullable
 *   entropy_rows [N] fp32 out: per-row softmax entropy in nats       nullable
 *   loss_out     scalar fp32 out: the reduced loss; required for "sum" and
 *                "mean", ignored (may be NULL) for "none"
 *   metrics_out  [2] fp32 out: {mean_token_accuracy, entropy}; NULL skips
 *                them. Loss outputs are bit-identical either way.
 *   n_valid      scalar int32 out: rows whose target != ignore_index  required
 *   err_word     scalar int32, ORed with FLCE_DEVERR_* bits           nullable
 *   workspace    >= flce_forward_workspace_size(p) bytes, 256-byte aligned
 * With n_valid = 0, "mean" gives NaN loss and NaN metrics. */
flce_status flce_forward(const flce_problem* p, const void* hidden,
                         const void* weight, const void* bias,
                         const int64_t* targets, float* loss_rows,
                         float* lse_rows, int32_t* correct_rows,
                         float* entropy_rows, float* loss_out,
                         float* metrics_out, int32_t* n_valid,
                         int32_t* err_word, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Forward pass that allocates nothing and takes no workspace. The method's
 * pages have no counterpart to it; it exists for callers that cannot call
 * cudaMalloc and have no workspace to hand in: for example a host framework
 * whose memory pool owns the whole device and refuses allocations from
 * libraries, or a latency-bound loop where a cudaMalloc (which may
 * synchronise the device) is not allowed.
 *   Arguments and outputs are those of flce_forward() without `workspace`
 *   and `workspace_bytes`; results are the same as flce_forward's.
 *   Scratch: a fixed 16 MiB array inside the library, held by every GPU that
 *   loads the library until the process exits. A problem is accepted when
 *   flce_forward_workspace_size(p) <= 16 MiB, and otherwise rejected with
 *   FLCE_ERR_UNSUPPORTED before any launch. For bf16 at H = 4096,
 *   V = 128256 that is N <= 2089 tokens; with FLCE_SKIP_IGNORED_ROWS, whose
 *   gathered copy of the kept hidden rows adds N * H * 2 bytes, N <= 1033
 *   (N <= 919 with label smoothing as well).
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current, and so does the first
 *   call after the device's context was destroyed and re-created (for
 *   example by cudaDeviceReset); make that first call before any stream
 *   capture.
 *   All calls share the one array, which keeps the last call's contents:
 *   calls whose work overlaps on the GPU (for example on two streams without
 *   ordering between them) race and corrupt each other's results. Order them
 *   on one stream. */
flce_status flce_forward_noalloc(const flce_problem* p, const void* hidden,
                                 const void* weight, const void* bias,
                                 const int64_t* targets, float* loss_rows,
                                 float* lse_rows, int32_t* correct_rows,
                                 float* entropy_rows, float* loss_out,
                                 float* metrics_out, int32_t* n_valid,
                                 int32_t* err_word, void* stream);

/* Bytes of device workspace flce_backward() needs for `p` (0 if invalid):
 * the dlogits buffer of one vocabulary chunk (N x chunk, in the input type for
 * FLCE_BF16 / FLCE_F16; fp32 for FLCE_F32 on FFMA kernels, or three bf16 parts
 * on the tensor cores, which also hold the bf16 parts of hidden and of the
 * chunk's weight rows), an fp32 [N,H] grad_hidden accumulator when there is
 * more than one chunk on the tensor-core path, and fp32 grad_bias partial sums
 * when has_bias. */
size_t flce_backward_workspace_size(const flce_problem* p);

/* Backward pass: all three gradients. Cite: §Algorithm (backward: recompute
 * each logit tile, form p - onehot, grad_hidden = (p - onehot) @ weight,
 * grad_weight = (p - onehot)^T @ hidden); §Full signature ("hidden, weight
 * and bias all receive gradients").
 *   hidden, weight, bias, targets   as for flce_forward (same values)
 *   lse_rows    [N] fp32 in: from flce_forward on the same inputs   required
 *   n_valid     scalar int32 in: from flce_forward                   required
 *   grad_out    fp32 in: scalar d(objective)/d(loss) for "sum"/"mean",
 *               [N] per-row upstream gradients for "none"            required
 *   grad_hidden [N,H] out, dtype p->dtype                            required
 *   grad_weight [V,H] out, dtype p->grad_weight_dtype                required
 *   grad_bias   [V] out, dtype p->dtype; required iff p->has_bias
 *   err_word    as for flce_forward                                  nullable
 *   workspace   >= flce_backward_workspace_size(p) bytes, 256-byte aligned
 * Outputs are overwritten, not accumulated into. */
flce_status flce_backward(const flce_problem* p, const void* hidden,
                          const void* weight, const void* bias,
                          const int64_t* targets, const float* lse_rows,
                          const int32_t* n_valid, const float* grad_out,
                          void* grad_hidden, void* grad_weight,
                          void* grad_bias, int32_t* err_word, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Fused linear KL divergence (FusedLinearKLDivLoss pull request, Liger-Kernel
 * #1423, Summary and Details): the vocabulary projection followed by
 * KL(Q || P) against an explicit target distribution Q (teacher
 * probabilities), without materialising the N x V logits:
 *
 *   z_ij   = (hidden_i . weight_j + bias_j) / temperature
 *   loss_i = sum_j q_ij (log max(q_ij, eps) - (z_ij - lse_i))     (counted rows)
 *          = sum_j q_ij (log max(q_ij, eps) - z_ij) + lse_i * sum_j q_ij
 *   D_ij   = g_i (p_ij * sum_k q_ik - q_ij) / temperature          (d loss / d lin)
 *
 * Rows whose label equals ignore_index are not counted (labels may be NULL:
 * every row counts). Reductions follow torch.nn.KLDivLoss: batchmean divides
 * the sum by the counted rows, mean by counted rows * V; none returns the
 * per-row losses and takes per-row upstream gradients. The same kernels as
 * the cross-entropy run underneath; conventions are those of flce_forward /
 * flce_backward above.
 */
typedef enum flce_kl_reduction {
  FLCE_KL_NONE = 0,
  FLCE_KL_SUM = 1,
  FLCE_KL_BATCHMEAN = 2,
  FLCE_KL_MEAN = 3
} flce_kl_reduction;

/*   n, h, v, dtype, has_bias, grad_weight_dtype, vocab_chunk, flags
 *                      as in flce_problem (target_probs has the input dtype)
 *   ignore_index       label value of rows left out (used only with labels)
 *   temperature        > 0: the student logits are divided by it
 *   eps                > 0: clamp inside log q (so that 0 * log 0 adds 0)
 *   reduction          flce_kl_reduction
 *   reserved           must be 0 */
typedef struct flce_kl_problem {
  int64_t n, h, v;
  int32_t dtype;
  int32_t has_bias;
  int64_t ignore_index;
  float temperature;
  float eps;
  int32_t reduction;
  int32_t grad_weight_dtype;
  int64_t vocab_chunk;
  int32_t flags;
  int32_t reserved;
} flce_kl_problem;

/* Bytes of device workspace flce_kl_forward() needs (0 if `p` is invalid). */
size_t flce_kl_forward_workspace_size(const flce_kl_problem* p);

/* KL forward. target_probs [N,V] (input dtype), labels [N] int64 (nullable).
 *   loss_rows [N] fp32 out (0 on uncounted rows)                     required
 *   lse_rows  [N] fp32 out: log-sum-exp of z, kept for the backward   required
 *   qsum_rows [N] fp32 out: sum_j q_ij, kept for the backward         required
 *   loss_out  scalar fp32 out (not written for FLCE_KL_NONE)
 *   n_counted scalar int32 out: rows counted                          required
 * With FLCE_SKIP_IGNORED_ROWS and labels, uncounted rows are left out of
 * the contractions (their lse and qsum are then NaN). */
flce_status flce_kl_forward(const flce_kl_problem* p, const void* hidden,
                            const void* weight, const void* bias,
                            const void* target_probs, const int64_t* labels,
                            float* loss_rows, float* lse_rows, float* qsum_rows,
                            float* loss_out, int32_t* n_counted,
                            int32_t* err_word, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of device workspace flce_kl_backward() needs (0 if `p` is invalid). */
size_t flce_kl_backward_workspace_size(const flce_kl_problem* p);

/* KL backward: grad_hidden, grad_weight, grad_bias as in flce_backward, from
 * the forward's lse_rows, qsum_rows and n_counted; grad_out is a scalar, or
 * [N] for FLCE_KL_NONE. */
flce_status flce_kl_backward(const flce_kl_problem* p, const void* hidden,
                             const void* weight, const void* bias,
                             const void* target_probs, const int64_t* labels,
                             const float* lse_rows, const float* qsum_rows,
                             const int32_t* n_counted, const float* grad_out,
                             void* grad_hidden, void* grad_weight,
                             void* grad_bias, int32_t* err_word,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * Self-test of the bounded waits (not part of the method; the pages describe
 * no such check). Every pipeline wait of the kernels gives up after a time
 * budget, records FLCE_DEVERR_TIMEOUT in the error word and returns instead
 * of spinning forever. This call exercises exactly those wait routines on an
 * mbarrier that nothing arrives on, with a budget of budget_s seconds
 * (0 < budget_s <= 1): once in a single CTA and once in a pair of CTAs (the
 * cluster-scope wait). On completion of the stream's work, *err_word has
 * FLCE_DEVERR_TIMEOUT set and result[0..2] (int32, device) are 0: each wait
 * gave up. Nothing faults; the context stays usable.
 *   err_word  int32 device scalar, ORed into (not cleared)
 *   result    int32 device [3]                                           */
flce_status flce_selftest_wait_timeout(int32_t* err_word, int32_t* result,
                                       double budget_s, void* stream);

/* ------------------------------------------------------------------------
 * The norm of a set of gradients taken together, and clipping by it: what a
 * training step does with the gradients of the losses above and of the rest
 * of its model.
 *
 *   norm = (sum |g|^p)^(1/p) over every element of every gradient (p = 1, 2),
 *          or max |g| (inf)
 *   dst  = g * min(1, max_norm / (norm + eps))        (a NaN norm gives NaN;
 *                                                      0 / 0 counts as 1)
 *
 * Sums are held in 64 bits above 64-element parts, with no 32-bit overflow or
 * underflow in between; the result is the same in every run. Products are
 * rounded to fp32 and then to dst's type. Each gradient is `rows` runs of `cols`
 * contiguous elements, `src_pitch` (`dst_pitch`) elements from run to run; a
 * dense tensor of any shape is one run. Tensors may start at any address that
 * their element type allows; 16-byte aligned runs are fastest.
 */
typedef enum flce_norm { FLCE_NORM_L1 = 1, FLCE_NORM_L2 = 2, FLCE_NORM_INF = 3 } flce_norm;

typedef struct flce_grad {
  const void* src;
  void* dst;           /* may be src; ignored by flce_grad_norm */
  int64_t rows, cols;  /* either may be 0: nothing there */
  int64_t src_pitch, dst_pitch;
  int32_t src_dtype;   /* flce_dtype */
  int32_t dst_dtype;   /* src_dtype or FLCE_F32 */
} flce_grad;

/* Bytes of device workspace that both calls need for `count` gradients. */
size_t flce_grad_workspace_size(int64_t count);

/* norm_out: fp32 device scalar. `grads` is a host array, read during the call
 * only, of any length. No gradients: the norm is 0. */
flce_status flce_grad_norm(const flce_grad* grads, int64_t count, int32_t norm,
                           float* norm_out, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The same, and dst = clipped src for every gradient. Where the factor is 1
 * and every dst is its src, nothing is written. Memory that the call writes
 * must not overlap what it reads or writes for another gradient
 * (FLCE_ERR_INVALID_ARG). max_norm and eps are finite and >= 0. */
flce_status flce_grad_clip(const flce_grad* grads, int64_t count, int32_t norm,
                           float max_norm, float eps, float* norm_out,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * One step of a beam search over the vocabulary.
 *
 *   s_bkv = beam_scores_bk + z_bkv - log sum_u e^{z_bku}
 *
 * and, for each prompt b, the `candidates` largest of its K * V scores, best
 * first; equal scores in the order of k * V + v. The comparison is in 64 bits
 * on row sums of 32-bit exponentials, which leave a beam's scores within 8e-6:
 * candidates of two beams closer than twice that may change places, those of
 * one beam do not. The scores are rounded to fp32. The result is the same in
 * every run of one shape and type.
 *   - allowed (bytes, nullable): a token whose byte is 0 counts as z = -inf,
 *     whatever its logit holds: it is neither offered nor in the sum.
 *   - finished (bytes, nullable): a beam whose byte is not 0 offers itself
 *     alone, with its score unchanged, under pad_token; its logits are not read.
 *   - A beam with score -inf, or with no token left, offers nothing.
 *   - Places that nothing fills hold score -inf, parent 0 and pad_token.
 *   - An allowed logit that is NaN or +inf, or a beam score that is, sets
 *     FLCE_DEVERR_NOT_FINITE, and that beam offers nothing.
 * Rows of logits are V contiguous elements; strides are in elements (bytes of
 * `allowed`), 0 where an axis shares one row.
 */
#define FLCE_DEVERR_NOT_FINITE 4
#define FLCE_DEVERR_PARENT_RANGE 8

typedef struct flce_beam_problem {
  int64_t batch, beams, v;     /* batch >= 0; 1 <= beams <= 1024; 1 <= v < 2^31 - 8192 */
  int64_t candidates;          /* 1 to 256 */
  int64_t stride_batch, stride_beam;
  int64_t allowed_stride_batch, allowed_stride_beam;
  int64_t pad_token;           /* in [0, v) */
  int32_t dtype;               /* of the logits */
  int32_t reserved;            /* 0 */
} flce_beam_problem;

/* Bytes of device workspace flce_beam_select() needs (0 if `p` is invalid). */
size_t flce_beam_select_workspace_size(const flce_beam_problem* p);

/* beam_scores [batch][beams]; finished [batch][beams]; the outputs
 * [batch][candidates]. */
flce_status flce_beam_select(const flce_beam_problem* p, const void* logits,
                             const float* beam_scores, const uint8_t* finished,
                             const uint8_t* allowed, float* scores_out,
                             int64_t* parents_out, int64_t* tokens_out,
                             int32_t* err_word, void* workspace,
                             size_t workspace_bytes, void* stream);

/* In-place reordering of what a beam search keeps for each beam (caches,
 * token histories, scores):
 *
 *   state[b * beams + j] = state[b * beams + parents[b * beams + j]]
 *
 * for every state, as if all were read before any is written. A state is
 * batch * beams beams, beam_stride bytes apart, each of size[0] x ... x
 * size[3] runs of run_bytes contiguous bytes, stride[d] bytes apart. Its
 * elements do not overlap, and no two states do (two that start at one address
 * are refused, FLCE_ERR_INVALID_ARG; other sharing is not looked for). 16-byte aligned runs and
 * strides are fastest. A parent outside [0, beams) sets
 * FLCE_DEVERR_PARENT_RANGE and leaves its beam as it is. beams <= 64. */
typedef struct flce_beam_state {
  void* data;
  int64_t beam_stride;
  int64_t size[4];   /* 1 where unused */
  int64_t stride[4];
  int64_t run_bytes;
} flce_beam_state;

flce_status flce_beam_reorder(const flce_beam_state* states, int64_t count,
                              const int64_t* parents, int64_t batch,
                              int64_t beams, int32_t* err_word, void* stream);

/* ------------------------------------------------------------------------
 * A linear layer in 8-bit integers (a head for answering, not for training).
 *
 *   scale_i = max_h |x_ih| * (1/127)   (both rounded to fp32)
 *   q_ih    = round(x_ih / scale_i)    (the quotient rounded to fp32, halves to even)
 *   lin_ij  = scale_i * weight_scale_j * sum_h q_ih * w_jh + bias_j
 *   u_ij    = logit_scale * lin_ij
 *   out_ij  = softcap * tanh(u_ij / softcap)   if softcap > 0, else u_ij
 *             (tanh within 10 * 2^-24 of its value)
 *
 * A row of zeros has scale 0; a row that holds a NaN or an infinity gives
 * NaN. Products are exact and sums are held in 32-bit floating point: they are
 * exact up to 2^24, and beyond it rounded at each of the h / 16 steps of the
 * tensor core. Rows lie `pitch` elements apart.
 */
typedef enum flce_qdtype { FLCE_Q_I8 = 3 } flce_qdtype; /* beside flce_dtype, for x */

/* x [n][h] -> q [n][h] (int8) and scale [n] (fp32). */
flce_status flce_quantize_rows(const void* x, int32_t dtype, int64_t n, int64_t h,
                               int64_t x_pitch, int8_t* q, int64_t q_pitch,
                               float* scale, void* stream);

typedef struct flce_qproblem {
  int64_t n, h, v;                      /* n, v >= 0; 1 <= h <= 131071 */
  int64_t x_pitch, weight_pitch, out_pitch;
  int32_t x_dtype;     /* an flce_dtype (quantised within the call), or FLCE_Q_I8 */
  int32_t out_dtype;   /* flce_dtype of out */
  int32_t bias_dtype;  /* flce_dtype of bias */
  int32_t has_bias;    /* 0 or 1 */
  float logit_scale;   /* finite */
  float softcap;       /* > 0 enables it; 1 / softcap is finite */
  int32_t flags;       /* OR of FLCE_Q_LAY_OUT_WEIGHT; 0 for none */
  int32_t reserved;    /* 0 */
} flce_qproblem;

/* Lay the weight out in the workspace first, one more pass over it. It is
 * implied by a weight_pitch that is no multiple of 16, and a caller sets it
 * for a weight that does not start at a multiple of 16 bytes (such a call is
 * FLCE_ERR_UNSUPPORTED without it). */
#define FLCE_Q_LAY_OUT_WEIGHT 1

/* Bytes of device workspace flce_qlinear() needs (0 if `p` is invalid). */
size_t flce_qlinear_workspace_size(const flce_qproblem* p);

/* x_scale [n]: with FLCE_Q_I8 only, else NULL. weight int8 [v][h] with
 * weight_scale fp32 [v]. Weight rows that start at multiples of 16 bytes are
 * read where they are (see FLCE_Q_LAY_OUT_WEIGHT for others). */
flce_status flce_qlinear(const flce_qproblem* p, const void* x, const float* x_scale,
                         const int8_t* weight, const float* weight_scale,
                         const void* bias, void* out, int32_t* err_word,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Per-kernel timing, for measurement tools (not part of the method; the
 * pages describe no profiler). While enabled, every kernel launch made by
 * flce_forward / flce_backward on the calling process is bracketed by two
 * CUDA events recorded on the caller's stream, so the launch sequence and
 * its stream ordering are unchanged. Up to FLCE_PROFILE_MAX_RECORDS launches
 * are recorded; later ones are counted in `dropped`. The events are created
 * on the current device the first time profiling is enabled.
 */
#define FLCE_PROFILE_MAX_RECORDS 8192
#define FLCE_PROFILE_NAME_LEN 40

typedef struct flce_kernel_time {
  char name[FLCE_PROFILE_NAME_LEN]; /* kernel role, e.g. "fwd_stats" */
  int32_t launches;                 /* launches recorded since the last collect */
  double total_ms;                  /* summed event-to-event time of those launches */
} flce_kernel_time;

/* Turn recording on (1) or off (0). Enabling clears earlier records. */
flce_status flce_profile_enable(int enable);

/* Synchronise on the recorded events, write up to `max_entries` per-kernel
 * totals (one entry per kernel role, in first-launch order) and clear the
 * record. Returns the number of entries written, or -1 on a CUDA error.
 * `*dropped` (nullable) receives the launches not recorded. */
int flce_profile_collect(flce_kernel_time* out, int max_entries, int32_t* dropped);

/* Static text for a status code. */
const char* flce_status_string(flce_status s);

/* Description of the last non-OK status returned on the calling thread
 * (empty string if none). Valid until the next call on that thread. */
const char* flce_last_error(void);

/* 1 if the current CUDA device can run this library's kernels (compute
 * capability 10.3, i.e. sm_103a), else 0. */
int flce_device_supported(void);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_H */
