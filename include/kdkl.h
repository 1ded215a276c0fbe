/*
 * kdkl.h — C ABI of the fused chunked KL distillation loss for GB300 (sm_103a).
 *
 * The operation is the one the pages state ("Making knowledge distillation
 * cheap enough to run at scale", section "Two system changes"): a student's
 * output projection z = H W^T over the full vocabulary, compared by a KL
 * divergence with an offline cache of the teacher's top-K (id, logit) pairs
 * per token, without ever storing the tokens x vocabulary logit grid. The
 * backward computes each chunk's projection a second time instead of keeping
 * it (same section, the fused-chunked bullet; "Efficient knowledge
 * distillation for LLMs: offline top-K logits and a fused chunked KL loss",
 * section "Two systemic changes for scalable distillation", item 2).
 *
 * Definitions (the pages name a closed-form gradient but do not print it):
 *   p[t,k]   = softmax_k(topk_logit[t,k] / tau)        teacher, renormalised over K
 *   lse[t]   = log sum_v exp(z[t,v] / tau)             full vocabulary
 *   KL[t]    = sum_k p[t,k] (log p[t,k] - z[t,idx[t,k]]/tau + lse[t])
 *   loss     = sum_t m[t] KL[t] / N,  N = sum_t m[t]   (0 when N = 0)
 *   dL/dz    = m[t] (softmax(z[t]/tau) - P[t]) / (tau N), P = p scattered at idx
 *   dH = g dL/dz . W,  dW = g (dL/dz)^T . H            (g = upstream gradient)
 *
 * Conventions for every call:
 *   - All arrays are DEVICE pointers, row-major and contiguous, owned by the
 *     caller. The library never allocates device memory: scratch lives in a
 *     caller-provided workspace of kd_kl_workspace_size() bytes.
 *   - bf16 arrays are passed as uint16_t bit patterns.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream). Calls are
 *     asynchronous on it and never synchronise the device, except
 *     kd_kl_check_status() and kd_timing_end(), which say so.
 *   - Argument errors are returned synchronously and launch nothing.
 *     Errors found on the device (a topk index outside [0, V), a teacher row
 *     with no finite logit, a pipeline wait that ran out) are recorded in the
 *     workspace and read with kd_kl_check_status().
 *   - Calls sharing one workspace must be ordered on one stream.
 */
#ifndef KDKL_H
#define KDKL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDKL_MAX_K 512 /* largest K the teacher-prep sort handles */

typedef enum {
  KD_OK = 0,
  KD_ERR_INVALID_ARG = 1,  /* null pointer, tau <= 0 or not finite, chunk < 1,
                              or (device) a teacher row without a finite logit */
  KD_ERR_SHAPE = 2,        /* T < 0, d < 8, V < 1, K < 1, K > V, K > KDKL_MAX_K,
                              or a size >= 2^31 */
  KD_ERR_ALIGNMENT = 3,    /* d % 8 != 0, or H/W/dH/dW/workspace not 16-byte aligned */
  KD_ERR_INDEX_RANGE = 4,  /* (device) a topk_idx entry outside [0, V) */
  KD_ERR_WORKSPACE = 5,    /* workspace NULL or smaller than kd_kl_workspace_size() */
  KD_ERR_CUDA = 6,         /* a CUDA runtime or driver call failed */
  KD_ERR_TIMEOUT = 7,      /* (device) a bounded pipeline wait ran out; outputs undefined */
  KD_ERR_UNSUPPORTED = 8   /* the current device is not compute capability 10.3 */
} kd_status;

typedef struct {
  int64_t T;          /* tokens (rows of H) */
  int64_t d;          /* hidden size (columns of H and W); multiple of 8 */
  int64_t V;          /* vocabulary size (rows of W) */
  int32_t K;          /* cached teacher entries per token, 1..min(V, KDKL_MAX_K) */
  float temperature;  /* tau > 0; divides both student and teacher logits */
  int64_t chunk;      /* token-chunk size of the pages' method: bounds the
                         backward's gradient-of-logits buffer to chunk x V
                         bf16 elements, plus tile padding (the scheduler may
                         tile that budget as fewer tokens x more vocabulary,
                         in whole 256-wide vocabulary tiles; results are the
                         same) */
} kd_kl_problem;

/* Workspace bytes for kd_kl_forward (which = 0), kd_kl_backward (which = 1),
 * kd_kl_forward_ex (which = 2), kd_kl_backward_ex (which = 3) or
 * kd_kl_backward_reuse (which = 4).
 * Linear in T (no T x V term). Returns 0 if the problem is invalid. */
size_t kd_kl_workspace_size(const kd_kl_problem* prob, int which);

/* Forward: mean KL loss over unmasked tokens and the per-token logsumexp.
 *   H          [T, d] bf16        student hidden states
 *   W          [V, d] bf16        student output projection (LM head)
 *   topk_idx   [T, K] int32       teacher's cached ids, any order, in [0, V)
 *   topk_logit [T, K] fp32        teacher's cached logits (-inf allowed, not all)
 *   mask       [T] uint8 or NULL  nonzero = token counts (NULL: all count)
 *   loss       [1] fp32 out       sum_t m[t] KL[t] / N (0 when N = 0)
 *   lse        [T] fp32 out       log sum_v exp(z[t,v]/tau) of every counted token
 *   token_kl   [T] fp32 out or NULL   KL[t] of every counted token
 * The logits z are produced tile by tile inside the SMs and never written to
 * memory. With a mask, the counted tokens are compacted first (in order) and
 * every later step runs on them alone: a masked token costs no tensor-core
 * work, and its lse and token_kl read 0 (they are not computed). With a NULL
 * mask every token counts. */
kd_status kd_kl_forward(const kd_kl_problem* prob, const uint16_t* H, const uint16_t* W,
                        const int32_t* topk_idx, const float* topk_logit, const uint8_t* mask,
                        float* loss, float* lse, float* token_kl,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Backward: gradients of g * loss. Masked tokens are skipped as in the
 * forward (their dH rows are exact zeros).
 *   lse        [T] fp32           from kd_kl_forward on the same inputs
 *   grad_loss  g                  upstream dL_outer/dloss (host scalar)
 *   dH         [T, d] bf16 out    overwritten; fp32 accumulation inside, masked rows = 0
 *   dW         [V, d] fp32 out    overwritten, or added to when accumulate_dW != 0
 * Each logit tile is recomputed and turned into (softmax - P) in the GEMM
 * epilogue; the result is kept in a bf16 buffer of about chunk x V elements
 * (the block's vocabulary rounded up to whole 256-wide tiles) that feeds the
 * dH and dW tensor-core GEMMs. */
kd_status kd_kl_backward(const kd_kl_problem* prob, const uint16_t* H, const uint16_t* W,
                         const int32_t* topk_idx, const float* topk_logit, const uint8_t* mask,
                         const float* lse, float grad_loss,
                         uint16_t* dH, float* dW, int accumulate_dW,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Loss variant. The pages report ablations over the choice of loss without
 * printing one ("Making knowledge distillation cheap enough to run at scale",
 * closing section); this is the standard distillation mix:
 *   loss_t = alpha * c * KL_t(tau) + (1 - alpha) * CE_t,  c = tau^2 or 1,
 *   CE_t   = log sum_v exp(z[t,v]) - z[t, labels[t]]      (temperature 1),
 *   loss   = sum_t m[t] loss_t / N.
 * dL/dz[t,v] = m[t]/N * (alpha c (softmax(z/tau) - P)/tau + (1-alpha)(softmax(z) - onehot)).
 * Same kernels as the calls above, with the temperature-1 sum and the label
 * logit added to the GEMM epilogues. */
typedef struct {
  float alpha;            /* weight of the soft term, in [0, 1]; 1 = KL only */
  int32_t scale_tau_sq;   /* nonzero: the soft term and its gradient are scaled by tau^2 */
  const int32_t* labels;  /* [T] device, hard labels in [0, V); may be NULL when alpha == 1 */
} kd_kl_options;

/* Workspace: kd_kl_workspace_size(prob, 2) for the forward, (prob, 3) for the backward.
 *   lse        [T] fp32 out   logsumexp of z / tau (counted tokens; masked ones read 0)
 *   lse1       [T] fp32 out   logsumexp of z (temperature 1; equals lse when tau == 1)
 *   token_loss [T] fp32 out or NULL   alpha c KL_t + (1 - alpha) CE_t (counted tokens)
 * A counted token's label outside [0, V) is reported as KD_ERR_INDEX_RANGE by
 * kd_kl_check_status (masked tokens' labels and teacher ids are not read). */
kd_status kd_kl_forward_ex(const kd_kl_problem* prob, const kd_kl_options* opts,
                           const uint16_t* H, const uint16_t* W, const int32_t* topk_idx,
                           const float* topk_logit, const uint8_t* mask, float* loss, float* lse,
                           float* lse1, float* token_loss, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Backward of grad_loss * loss. lse1 may be NULL when tau == 1 or alpha == 1. */
kd_status kd_kl_backward_ex(const kd_kl_problem* prob, const kd_kl_options* opts,
                            const uint16_t* H, const uint16_t* W, const int32_t* topk_idx,
                            const float* topk_logit, const uint8_t* mask, const float* lse,
                            const float* lse1, float grad_loss, uint16_t* dH, float* dW,
                            int accumulate_dW, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Backward that reuses the teacher cache the forward already prepared. The
 * forward turns the cache into sorted (id, p) rows and counts the mask
 * (N) in its workspace; the pages compute the teacher side once and keep it
 * ("Making knowledge distillation cheap enough to run at scale", section "Two
 * system changes"), so the backward can read those rows instead of preparing
 * them again. Same results as kd_kl_backward / kd_kl_backward_ex.
 *   opts           NULL for the plain KL loss, else as kd_kl_backward_ex
 *   mask, lse, lse1  as kd_kl_backward(_ex); mask must be the forward's
 *   fwd_workspace  the workspace of the latest kd_kl_forward or
 *                  kd_kl_forward_ex call on the same problem (T, d, V, K and
 *                  temperature; chunk may differ), queued earlier on the same
 *                  stream and not reused since; read only
 *   workspace      kd_kl_workspace_size(prob, 4) bytes (no teacher region)
 * The library remembers, on the host, which problem each forward workspace
 * was last filled for, until any call is given that workspace as its own; a
 * fwd_workspace it does not know for this problem, or that is also `workspace`,
 * or fwd_workspace_bytes smaller than that call's, returns KD_ERR_INVALID_ARG
 * synchronously. The teacher cache was validated by the forward: its
 * device-detected errors are read from fwd_workspace, this call's (wait
 * timeouts) from workspace. */
kd_status kd_kl_backward_reuse(const kd_kl_problem* prob, const kd_kl_options* opts,
                               const uint16_t* H, const uint16_t* W, const uint8_t* mask,
                               const float* lse, const float* lse1, const void* fwd_workspace,
                               size_t fwd_workspace_bytes, float grad_loss, uint16_t* dH,
                               float* dW, int accumulate_dW, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Allocation-free forward. The paper has no counterpart to this call; it
 * exists for callers that cannot allocate device memory for a workspace: code
 * inside a host framework whose memory pool owns (and has typically reserved)
 * all free HBM, and loops with a latency budget that rules out cudaMalloc,
 * which can synchronise the device.
 * Same arguments, results and errors as kd_kl_forward, minus the workspace:
 * the scratch is a fixed array of KDKL_NOALLOC_SCRATCH_BYTES compiled into the
 * library, held on every GPU where the library's device code is loaded until
 * the process exits. Problems whose kd_kl_workspace_size(prob, 0) exceeds it
 * return KD_ERR_WORKSPACE before anything is queued.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current), and so does the first
 *     call after a device reset; make that first call before any stream
 *     capture.
 *   - It calls no cudaMalloc, cudaFree or other allocating routine (with
 *     per-kernel timing off, the default).
 *   - Every call on a device shares the one array and clears its header when
 *     it starts. Calls whose GPU work overlaps (other streams, other host
 *     threads) race on it: order them on one stream.
 *   - Device-detected errors (an id outside [0, V), a teacher row with no
 *     finite logit, a wait that ran out) go to the array's status word and are
 *     read with kd_kl_noalloc_check_status(); outputs are then undefined. */
#define KDKL_NOALLOC_SCRATCH_BYTES (64u << 20)
kd_status kd_kl_forward_noalloc(const kd_kl_problem* prob, const uint16_t* H, const uint16_t* W,
                                const int32_t* topk_idx, const float* topk_logit,
                                const uint8_t* mask, float* loss, float* lse, float* token_kl,
                                void* stream);

/* BLOCKING: synchronises `stream`, then returns the first device-detected
 * error recorded by the latest kd_kl_forward_noalloc call on the current
 * device (KD_OK if none), like kd_kl_check_status does for a workspace. */
kd_status kd_kl_noalloc_check_status(void* stream);

/* ---------------------------------------------------------------------------
 * Second loss variant: reverse KL restricted to the cached ids. The pages
 * report ablations over the choice of loss without printing one ("Making
 * knowledge distillation cheap enough to run at scale", closing section);
 * this is the mode-seeking direction, taken over the same support as the
 * teacher cache (entries whose teacher logit is not finite are dropped from
 * both distributions):
 *   qt[t,k]  = softmax_k(z[t,idx[t,k]] / tau)      student, renormalised over the ids
 *   p[t,k]   = softmax_k(topk_logit[t,k] / tau)    teacher, as above
 *   RKL[t]   = sum_k qt[t,k] (log qt[t,k] - log p[t,k])
 *   loss     = sum_t m[t] RKL[t] / N              (0 when N = 0)
 *   grad_z[t,k] = dloss/dz[t,idx[t,k]] = m[t]/N * qt (log qt - log p - RKL[t]) / tau
 *               (0 for dropped entries)
 * Only the K cached logits of each token enter, so there is no vocabulary-wide
 * contraction: the kernels stream rows of W and H per (token, id) pair, on CUDA
 * cores, over the pairs sorted by id (forward, dW) or per token (dH). The problem struct
 * is kd_kl_problem; `chunk` is not used (any value >= 1); T * K < 2^31.
 * Both calls take a workspace of kd_rkl_workspace_size() bytes: linear in T,
 * plus 8 bytes per vocabulary row. */
size_t kd_rkl_workspace_size(const kd_kl_problem* prob);

/*   loss       [1] fp32 out           sum_t m[t] RKL[t] / N
 *   token_rkl  [T] fp32 out or NULL   RKL[t] before masking
 *   grad_z     [T, K] fp32 out or NULL   dloss/dz at the cached ids (upstream
 *                                     gradient 1); passing it to kd_rkl_backward
 *                                     saves the backward its logit recompute
 * Other arguments and errors as kd_kl_forward. */
kd_status kd_rkl_forward(const kd_kl_problem* prob, const uint16_t* H, const uint16_t* W,
                         const int32_t* topk_idx, const float* topk_logit, const uint8_t* mask,
                         float* loss, float* token_rkl, float* grad_z, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Gradients of grad_loss * loss.
 *   grad_z  [T, K] fp32 or NULL   from kd_rkl_forward on the same inputs; NULL:
 *                                 the backward recomputes it (the forward's z pass)
 *   dH      [T, d] bf16 out       overwritten (fp32 sums inside; masked rows = 0)
 *   dW      [V, d] fp32 out       overwritten, or added to when accumulate_dW != 0
 * The (id, token) pairs are sorted by id inside the call so that each dW row is
 * summed by one warp in token order: no atomics, and both outputs are bitwise
 * reproducible from run to run. An id outside [0, V) contributes nothing and is
 * reported as KD_ERR_INDEX_RANGE by kd_kl_check_status. */
kd_status kd_rkl_backward(const kd_kl_problem* prob, const uint16_t* H, const uint16_t* W,
                          const int32_t* topk_idx, const float* topk_logit, const uint8_t* mask,
                          const float* grad_z, float grad_loss, uint16_t* dH, float* dW,
                          int accumulate_dW, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ---------------------------------------------------------------------------
 * Offline teacher cache producer: for every row t of H, the K largest logits
 * z[t,v] = H[t] . W[v] over the full vocabulary, with their ids. This is the
 * cache the loss above consumes ("Making knowledge distillation cheap enough
 * to run at scale", section "Two system changes": compute the teacher's
 * output once and cache the 100 most likely tokens per position). The same
 * tensor-core GEMM produces each logit tile; its epilogue keeps per-row
 * candidate lists above a running threshold, so the logits are never stored.
 */
#define KDKL_TOPK_MAX_K 512

typedef struct {
  int64_t T;   /* rows of H (tokens) */
  int64_t d;   /* hidden size; multiple of 8 */
  int64_t V;   /* vocabulary (rows of W) */
  int32_t K;   /* entries kept per row, 1..min(V, KDKL_TOPK_MAX_K) */
  int32_t reserved;  /* set to 0 */
} kd_topk_problem;

/* Workspace bytes for kd_lmhead_topk; linear in T; 0 if the problem is invalid. */
size_t kd_lmhead_topk_workspace_size(const kd_topk_problem* prob);

/*   H          [T, d] bf16      hidden states (device)
 *   W          [V, d] bf16      output projection (device)
 *   topk_idx   [T, K] int32 out ids, per row by logit descending, ties to the smaller id
 *   topk_logit [T, K] fp32 out  the logits z (fp32 accumulation of the bf16 products)
 * Errors: KD_ERR_SHAPE (T < 0, d < 8, V < 1, K outside 1..min(V, KDKL_TOPK_MAX_K)),
 * KD_ERR_ALIGNMENT (d % 8 != 0 or misaligned pointers), KD_ERR_INVALID_ARG (null
 * pointers), KD_ERR_WORKSPACE, KD_ERR_CUDA, KD_ERR_UNSUPPORTED; device-detected
 * errors via kd_kl_check_status(workspace). */
kd_status kd_lmhead_topk(const kd_topk_problem* prob, const uint16_t* H, const uint16_t* W,
                         int32_t* topk_idx, float* topk_logit, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Tuning the head by preferences or by a policy. Four calls, in the order in
 * which a training step makes them: the log-probabilities of given tokens, a
 * loss over them with its gradient, the way back to dH and dW, and the
 * optimizer's step. As above: device pointers, no allocation, asynchronous on
 * `stream`, device-detected errors through kd_kl_check_status(workspace).
 *
 * Token log-probabilities of the LM head, the logits never stored (the backward holds
 * the gradient of up to chunk * V of them at a time):
 *   z = H W^T / tau,  lse[t] = log sum_v exp(z[t,v]),  logp[t] = z[t,ids[t]] - lse[t]
 *   dL/dz[t,v] = g[t] (onehot(ids[t])[v] - softmax(z[t])[v]),  g = dL/dlogp
 *   dH = dL/dz . W / tau,  dW = (dL/dz)^T . H / tau */
typedef struct {
  int64_t T;          /* tokens (rows of H) */
  int64_t d;          /* hidden size; multiple of 8 */
  int64_t V;          /* vocabulary (rows of W) */
  float temperature;  /* tau > 0 */
  int32_t dw_bf16;    /* backward: dW is bf16 [V, d] instead of fp32 (not accumulated) */
  int64_t chunk;      /* backward: the gradient-of-logits buffer holds chunk * V bf16 values (of
                         fewer tokens: T * V), as in kd_kl_problem */
} kd_logprob_problem;

/* Workspace bytes of the forward (which = 0) or the backward (which = 1);
 * linear in T; 0 if the problem is invalid. At d = 2880, V = 201,088, in MiB: forward of
 * 6000 tokens 41, of 32,768 tokens 218; backward (fp32 / bf16 dW) of 6000 tokens
 * 486 / 552 at chunk 1024 and 1256 / 1322 at 4096, of 32,768 tokens 929 / 1302 and
 * 2126 / 2486. The losses take kilobytes. */
size_t kd_logprob_workspace_size(const kd_logprob_problem* prob, int which);

/*   ids   [T] int32            the token whose log-probability is wanted, in [0, V)
 *   mask  [T] uint8 or NULL    nonzero = wanted; the others' logp and lse read 0,
 *                              their ids are not read and no product is computed
 *   logp  [T] fp32 out,  lse [T] fp32 out
 * A wanted id outside [0, V) is reported as KD_ERR_INDEX_RANGE by
 * kd_kl_check_status. */
kd_status kd_logprob_forward(const kd_logprob_problem* prob, const uint16_t* H, const uint16_t* W,
                             const int32_t* ids, const uint8_t* mask, float* logp, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream);

/*   lse        [T] fp32        from kd_logprob_forward on the same inputs
 *   grad_logp  [T] fp32        dL/dlogp. A token whose gradient is zero (masked,
 *                              clipped) contributes nothing: it is left out of every
 *                              product, its id and lse are not read, its dH row is zero
 *   dH         [T, d] bf16 out
 *   dW         [V, d] out      fp32, overwritten or (accumulate_dW) added to; or bf16
 *                              when prob->dw_bf16 (accumulate_dW must be 0)
 * The entry of each token's own id, g (1 - p) / tau, is taken from its logit and lse
 * and added in fp32, from first to last: it is off by lse's rounding (g / tau times
 * 2^-24 |lse|, which is what 1 - p of a confident token is told by) and a few fp32
 * roundings. The other entries of the logits' gradient, -g p / tau, are rounded to bf16
 * before they enter the two products: dH and dW carry that relative 2^-8 of those terms. */
kd_status kd_logprob_backward(const kd_logprob_problem* prob, const uint16_t* H, const uint16_t* W,
                              const int32_t* ids, const float* lse, const float* grad_logp,
                              uint16_t* dH, void* dW, int accumulate_dW, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Clipped policy loss with a KL term. Per counted token, with r =
 * exp(logp - old_logp), A its advantage, x = ref_logp - logp:
 *   surrogate  s = min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *              and, when A < 0 and dual_clip > 0, s = max(s, dual_clip A)
 *   penalty    k = e^x - 1 - x
 *   loss = sum_t w[t] (-s[t] + kl_coef k[t])
 * with w = 1 / N (KD_REDUCE_TOKEN; N counted tokens), 1 / (S' n_s)
 * (KD_REDUCE_SEQUENCE: the mean over the S' sequences that have counted
 * tokens, of each one's mean over its n_s), or 1 / norm (KD_REDUCE_SUM).
 *   dloss/dlogp = w (-A r [r not clipped] + kl_coef (1 - e^x))
 * On which side of a border a ratio is, is decided in 48 bits of logp - old_logp. */
enum { KD_REDUCE_TOKEN = 0, KD_REDUCE_SEQUENCE = 1, KD_REDUCE_SUM = 2 };

typedef struct {
  int64_t T;         /* tokens, below 2^31 - 4096 */
  int64_t S;         /* sequences, up to 2^30; 0 without cu_seqlens */
  double clip_low;   /* in [0, 1] */
  double clip_high;  /* >= 0 */
  double dual_clip;  /* > 1, or 0: off */
  double kl_coef;    /* finite in 32 bits; 0 without ref_logp */
  double norm;       /* KD_REDUCE_SUM: > 0, and 1 / norm finite in 32 bits */
  int32_t reduction;
  int32_t advantage_per_sequence; /* advantages are [S], else [T] */
} kd_policy_problem;

size_t kd_policy_workspace_size(const kd_policy_problem* prob);

/*   logp, old_logp, ref_logp  [T] fp32; old_logp NULL: ratio 1 (on-policy);
 *                             ref_logp NULL: no penalty
 *   advantages  [T] or [S] fp32
 *   mask        [T] uint8 or NULL   what lies in uncounted places is never used
 *   cu_seqlens  [S+1] int32 or NULL  sequence s is tokens [cu[s], cu[s+1]): from 0 to T,
 *               never falling (empty sequences allowed); needed, and read, for
 *               KD_REDUCE_SEQUENCE and advantages per sequence only.
 *               Otherwise KD_ERR_INVALID_ARG through kd_kl_check_status
 *   grad_loss   upstream gradient (host scalar), and grad_loss / norm finite in 32 bits
 *   loss        [1] fp32 out (0 when nothing counts)
 *   stats       [3] fp32 out or NULL   sum w (-s), sum w k, and the share of counted tokens
 *               that are clipped: whose ratio is past the border that bounds it, the upper
 *               one for A >= 0 (a token of advantage 0 too, though nothing depends on its
 *               ratio), the lower one or the dual one for A < 0
 *   grad_logp   [T] fp32 out or NULL   grad_loss * dloss/dlogp (0 where not counted)
 * Ratios and penalties are formed in fp32 (e^x to 2 ulp and 2^-24 |x|), sums in 48 bits.
 * Sums have a fixed order: results are the same from run to run. */
kd_status kd_policy_loss(const kd_policy_problem* prob, const float* logp, const float* old_logp,
                         const float* ref_logp, const float* advantages, const uint8_t* mask,
                         const int32_t* cu_seqlens, float grad_loss, float* loss, float* stats,
                         float* grad_logp, void* workspace, size_t workspace_bytes, void* stream);

/* Preference loss over pairs (chosen, rejected) of sequences:
 *   q_s = sum over s's counted tokens of (logp - ref_logp), divided by their
 *         number when average != 0 (an empty sequence has q = 0)
 *   h = q_chosen - q_rejected - margin
 *   KD_PREF_SIGMOID  -(1 - e) log sigma(beta h) - e log sigma(-beta h), e = label_smoothing
 *   KD_PREF_IPO      (h - 1 / (2 beta))^2
 *   KD_PREF_HINGE    max(0, 1 - beta h)
 *   loss = mean over the P pairs */
enum { KD_PREF_SIGMOID = 0, KD_PREF_IPO = 1, KD_PREF_HINGE = 2 };

typedef struct {
  int64_t T;               /* tokens, below 2^31 - 4096 */
  int64_t P;               /* pairs: 2 P sequences, up to 2^30 */
  double beta;             /* > 0, in 32 bits too; 1 / (2 beta) and margin finite there */
  double label_smoothing;  /* in [0, 1) */
  double margin;
  int32_t kind;
  int32_t average;
  int32_t halves;          /* 0: sequences 2i (chosen) and 2i+1; else i and P + i */
  int32_t reserved;        /* set to 0 */
} kd_pref_problem;

size_t kd_pref_workspace_size(const kd_pref_problem* prob);

/*   logp, ref_logp [T] fp32 (ref_logp NULL: 0), mask [T] uint8 or NULL,
 *   cu_seqlens [2P+1] int32 as in kd_policy_loss
 *   loss      [1] fp32 out
 *   rewards   [P, 2] fp32 out       beta q of the chosen and of the rejected sequence
 *   grad_logp [T] fp32 out or NULL  grad_loss * dloss/dlogp */
kd_status kd_pref_loss(const kd_pref_problem* prob, const float* logp, const float* ref_logp,
                       const uint8_t* mask, const int32_t* cu_seqlens, float grad_loss, float* loss,
                       float* rewards, float* grad_logp, void* workspace, size_t workspace_bytes,
                       void* stream);

/* One AdamW step over a list of tensors, in one launch for up to 384 of them:
 *   m = beta1 m + (1 - beta1) g s,  v = beta2 v + (1 - beta2) (g s)^2
 *   p = p (1 - lr weight_decay [decay]) - lr / (1 - beta1^step)
 *         * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * with s = grad_scale (times *grad_scale_dev). All tensors of a call have the
 * same types. With state_8bit, exp_avg holds m and exp_avg_sq holds sqrt(v) as
 * e4m3 bytes, and every 256 consecutive elements of a tensor share one fp32
 * power of two in m_scale / v_scale (ceil(n / 256) of them): value = code *
 * scale. Zero bytes and scales of 1 are the state of a first step. */
typedef struct {
  void* param;       /* [n] fp32 or bf16, updated */
  const void* grad;  /* [n] fp32 or bf16 */
  void* exp_avg;     /* [n] fp32, or e4m3 bytes */
  void* exp_avg_sq;  /* [n] fp32 (v), or e4m3 bytes (sqrt(v)) */
  uint16_t* copy;    /* [n] bf16 out: the new parameters rounded; or NULL */
  float* m_scale;    /* state_8bit: [ceil(n/256)] */
  float* v_scale;
  int64_t n;         /* elements, >= 0 */
  int32_t decay;     /* nonzero: weight_decay applies */
  int32_t reserved;  /* set to 0 */
} kd_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;                  /* this step's number, from 1 */
  const float* grad_scale_dev;   /* device scalar or NULL (a clip coefficient) */
  float grad_scale;
  int32_t param_bf16, grad_bf16, state_8bit;
} kd_adamw_options;

/* `tensors` is a host array; it is read before the call returns. */
kd_status kd_adamw_step(const kd_adamw_tensor* tensors, int32_t n_tensors,
                        const kd_adamw_options* opts, void* stream);

/* BLOCKING: synchronises `stream`, then returns the first device-detected
 * error recorded in `workspace` by the latest call that used it (KD_OK if
 * none). Each forward/backward call clears the record when it starts. */
kd_status kd_kl_check_status(void* workspace, void* stream);

/* Human-readable name of a status code (static storage). */
const char* kd_status_string(kd_status status);

/* Number of kernels this library has launched in this process (all calls,
 * all devices). Lets a caller count launches inside a timed region. */
int64_t kd_launch_count(void);

/* Per-kernel timing. After kd_timing_begin(), every kernel the library
 * launches is bracketed by CUDA events recorded on its launch stream.
 * kd_timing_end() is BLOCKING: it synchronises those events, fills up to
 * `max_entries` rows (one per kernel name, in first-launch order), stores
 * the row count in *n_entries, and stops recording. */
typedef struct {
  char name[32];
  int64_t launches;
  double total_ms;
} kd_kernel_time;

kd_status kd_timing_begin(void);
kd_status kd_timing_end(kd_kernel_time* out, int max_entries, int* n_entries);

#ifdef __cplusplus
}
#endif

#endif /* KDKL_H */
