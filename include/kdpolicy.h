/*
 * libkdloss, policy and preference training over the output head: what a
 * program trains with after, or beside, distillation.
 *
 *  - token log-probabilities: log q(y_t) of one token per row, and the
 *    entropy of its distribution, through the output projection Z = H.W,
 *    forward and backward, without the [T, V] logits;
 *  - the clipped policy loss on such log-probabilities, with a KL term
 *    against a reference and an entropy bonus;
 *  - the preference loss of pairs of sequences, from the log-probability
 *    ratios against a reference;
 *  - the global L2 norm of many gradient tensors, and clipping by it.
 *
 * Conventions (layouts, alignment, ownership, streams, status codes, error
 * text, KD_BF16 / KD_F32) are those of kdloss.h: dense row-major arrays,
 * caller-allocated buffers and workspace, every argument checked on the host
 * before anything is enqueued, no synchronisation, no state between calls,
 * the same bits for the same call.  Values on the device are not checked;
 * what each call does with values outside their range is said there, and no
 * value leads to a read or write outside the arrays.  An output may not
 * overlap an input or another output, except where a call says so.
 */
#ifndef KDPOLICY_H
#define KDPOLICY_H

#include "kdloss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- token log-probabilities
 * Per valid row t, with s = (H_t . W) / tau, L_t = logsumexp(s), q = softmax(s):
 *   logp[t]    = s[tokens[t]] - L_t
 *   entropy[t] = L_t - sum_v q_v s_v
 *   dZ_t       = (1/tau) ( g_t [v = tokens[t]] - q_v (g_t + e_t (entropy[t] + log q_v)) )
 * for the upstream gradients g = grad_logp and e = grad_entropy; dH = dZ . W^T, dW = H^T . dZ.
 * tokens [T] int32; logp, lse, entropy, grad_logp, grad_entropy [T] float32.
 * The rules for H, W, d, V, mask and tau are those of kd_topk_kl_fwd; d and V
 * must be below 2^25 (KD_ERR_UNSUPPORTED).
 * Masked rows get logp = lse = entropy = 0 and dH = 0, add nothing to dW and
 * are never read beyond mask[t].  A token of a valid row outside [0, V) gives
 * logp = NaN; its dZ has no token term.  Columns masked by large negative
 * logits, down to the type's lowest value (in a row of W that every hidden
 * state meets with 1, say), have probability 0 and add nothing; a row with
 * nothing but such columns may be NaN.  Infinite and NaN entries of H and W are
 * no such mask: the results that they enter may be NaN.
 * Speed: bf16 heads below 4 GiB with d a multiple of 32 and V >= 256 run at the
 * matrix cores' rate from a few hundred rows on, other bf16 heads at about 0.4
 * of it.
 */

/* Bytes of the optional buffer `logits` in which the forward call leaves the
 * valid rows' logits (float32, packed in row order, rows of roundup(V, 256)):
 * with it the backward call reads them instead of computing the projection
 * again. */
kd_status kd_token_logp_logits_size(int64_t T, int64_t V, size_t* bytes);
/* Workspace bytes for a forward call alone (kd_token_logp_fwd, its shard
 * form): the tiles' records and up to a default chunk's rows of H. */
kd_status kd_token_logp_fwd_workspace_size(int64_t T, int64_t d, int64_t V, kd_dtype dt, size_t* bytes);
/* Workspace bytes for kd_token_logp_fwd and kd_token_logp_bwd (one size
 * serves both, and the shard calls; it holds a chunk's dZ).  dw_dtype: the
 * type of dW below.
 * chunk_rows as in kd_topk_kl_workspace_size. */
kd_status kd_token_logp_workspace_size(int64_t T, int64_t d, int64_t V, kd_dtype dt, kd_dtype dw_dtype,
                                       int64_t chunk_rows, size_t* bytes);
/* logp [T] and lse [T] (L_t, kept for the backward call); entropy [T] and
 * logits are optional (NULL to skip). */
kd_status kd_token_logp_fwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                            int64_t T, int64_t d, int64_t V, kd_dtype dt, float* logp, float* lse, float* entropy,
                            float* logits, void* workspace, size_t workspace_bytes, void* stream);
/* dH [T,d] (dtype dt) and dW [d,V] (dw_dtype: KD_F32, or KD_BF16 for bf16
 * inputs), both overwritten; either may be NULL where it is not needed (a
 * frozen head), not both.  dZ is rounded to the inputs' type before its two
 * products, as for the other losses.  grad_logp or grad_entropy may be NULL (zero),
 * not both.  grad_entropy needs entropy, the forward's output.  logits: the
 * forward's, or NULL.  A bf16 dW is the rounded float32 sum over all rows
 * (several chunks add up in a float32 buffer of the workspace).
 * T = 0 sets dW to zero. */
kd_status kd_token_logp_bwd(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                            int64_t T, int64_t d, int64_t V, kd_dtype dt, const float* lse, const float* entropy,
                            const float* logits, const float* grad_logp, const float* grad_entropy, void* dH,
                            void* dW, kd_dtype dw_dtype, int64_t chunk_rows, void* workspace,
                            size_t workspace_bytes, void* stream);
/* A head split by vocabulary columns over R ranks, W = columns [v0, v0 + V):
 * each rank's forward gives rec [T,4] (16-byte aligned); all-gathered in rank
 * order, kd_token_logp_shard_combine gives the whole head's logp, lse and
 * (optional) entropy on every rank; each rank's backward, with those, gives
 * its columns of dW and a float32 partial of dH [T,d] to be summed over the
 * ranks.  rec = (m, l, e, x): with y = s log2(e) over the shard's columns
 * m = max y (-infinity, with l = e = 0, where all are below the 32-bit range;
 * beyond 2^24 in size at most two steps above), l = sum 2^(y - m), e = sum
 * 2^(y - m) (y - m), and x the raw logit at the token, or 0 in the shards that
 * do not hold it.  A token that no shard holds is not told from one whose logit
 * is 0. */
kd_status kd_token_logp_fwd_shard(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                                  int64_t T, int64_t d, int64_t V, int64_t v0, kd_dtype dt, float* rec, float* logits,
                                  void* workspace, size_t workspace_bytes, void* stream);
kd_status kd_token_logp_shard_combine(const float* rec, int64_t R, const uint8_t* mask, float tau, int64_t T,
                                      float* logp, float* lse, float* entropy, void* stream);
kd_status kd_token_logp_bwd_shard(const void* H, const void* W, const int32_t* tokens, const uint8_t* mask, float tau,
                                  int64_t T, int64_t d, int64_t V, int64_t v0, kd_dtype dt, const float* lse,
                                  const float* entropy, const float* logits, const float* grad_logp,
                                  const float* grad_entropy, float* dH, void* dW, kd_dtype dw_dtype,
                                  int64_t chunk_rows, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- clipped policy loss
 * Per valid token t, with r = exp(logp - old_logp), A the token's advantage
 * and d = ref_logp - logp:
 *   policy_t = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A); with
 *              dual_clip = c > 1, where A < 0 at most -c A
 *   kl_t     = -d (KD_KL_1), d^2 / 2 (KD_KL_2) or exp(d) - d - 1 (KD_KL_3)
 *   loss_t   = policy_t + kl_weight kl_t - entropy_weight entropy_t
 *   total    = sum_t w_t loss_t
 * w_t: 1 (KD_SUM), 1 / N with N valid tokens (KD_TOKEN_MEAN), or
 * 1 / (S' n_s) with n_s valid tokens in t's sequence s and S' sequences that
 * have any (KD_SEQUENCE_MEAN).  No valid token at all: total 0, gradients 0.
 * The gradient of policy_t is -A r, and 0 where the clip is what counts:
 * A > 0 and r > 1 + clip_high, A < 0 and r < 1 - clip_low, or A < 0 and
 * r > c; at the borders themselves it is -A r.
 *
 * Sequences: cu_seqlens [S+1] int32, ascending; sequence s is tokens
 * [cu_seqlens[s], cu_seqlens[s+1]).  Needed for KD_SEQUENCE_MEAN and for one
 * advantage per sequence; then a token in no sequence counts as masked.
 * (cu_seqlens that do not ascend give unspecified results, but no access
 * outside the arrays: entries are taken into [0, T].)
 * Masked tokens' values are read but never used (NaN there is fine); their
 * gradients are 0.
 *
 * All arithmetic is in 64 bits, so a ratio falls on the side of a border on
 * which the given log-probabilities put it; results are rounded once. */
typedef enum kd_reduction { KD_SUM = 0, KD_TOKEN_MEAN = 1, KD_SEQUENCE_MEAN = 2, KD_REDUCTION_MAX_ENUM = 0x7fffffff } kd_reduction;
typedef enum kd_kl_kind { KD_KL_1 = 1, KD_KL_2 = 2, KD_KL_3 = 3, KD_KL_KIND_MAX_ENUM = 0x7fffffff } kd_kl_kind;
typedef struct kd_policy_opts {
  const float* ref_logp;      /* [T]; needed with kl_weight != 0, else kl_t = 0 where NULL */
  const float* entropy;       /* [T]; needed with entropy_weight != 0, else 0 where NULL */
  const int32_t* cu_seqlens;  /* [S+1] or NULL */
  int64_t S;                  /* number of sequences (>= 1 with cu_seqlens) */
  int32_t per_sequence;       /* nonzero: advantages is [S], not [T] */
  kd_reduction reduction;
  kd_kl_kind kl_kind;
  double clip_low, clip_high; /* in [0, 1] and >= 0 */
  double dual_clip;           /* 0 (none) or > 1 */
  double kl_weight, entropy_weight; /* finite */
} kd_policy_opts;
kd_status kd_policy_loss_workspace_size(int64_t T, int64_t S, size_t* bytes);
/* stats [6] float32: total, sum w policy, sum w kl, sum w entropy, sum w over
 * the clipped tokens, N.  total: the same as stats[0], in a place of its own
 * (NULL to skip).  weights [max(S, 1)] float64 (8-byte aligned): w of
 * each sequence's valid tokens (one entry without cu_seqlens), kept for the
 * backward. */
kd_status kd_policy_loss_fwd(const float* logp, const float* old_logp, const float* advantages, const uint8_t* mask,
                             const kd_policy_opts* opts, int64_t T, float* total, float* stats, double* weights,
                             void* workspace, size_t workspace_bytes, void* stream);
/* grad_logp [T] and, if not NULL, grad_entropy [T], for the upstream gradient
 * *grad_total (one float32 on the device). */
kd_status kd_policy_loss_bwd(const float* logp, const float* old_logp, const float* advantages, const uint8_t* mask,
                             const kd_policy_opts* opts, int64_t T, const double* weights, const float* grad_total,
                             float* grad_logp, float* grad_entropy, void* stream);
/* Both in one call, for an upstream gradient of 1. */
kd_status kd_policy_loss_fwd_bwd(const float* logp, const float* old_logp, const float* advantages,
                                 const uint8_t* mask, const kd_policy_opts* opts, int64_t T, float* stats,
                                 double* weights, float* grad_logp, float* grad_entropy, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- preference loss
 * 2 P packed sequences (cu_seqlens [2P+1], as above): 0 .. P-1 are the
 * chosen ones of the pairs, P .. 2P-1 the rejected ones in the same order.
 * Over the valid tokens of sequence s, R_s = sum (logp - ref_logp) (ref_logp
 * NULL: 0), or with `average` that sum over their number (0 if there is
 * none); D_p = R_p - R_(P+p), h = beta D_p - margin:
 *   KD_PREF_SIGMOID  -(1 - e) log sigmoid(h) - e log sigmoid(-h), e = label_smoothing
 *   KD_PREF_HINGE    max(0, 1 - h)
 *   KD_PREF_IPO      (D_p - 1 / (2 beta))^2   (margin must be 0)
 * loss [P]; rewards [2P] = beta R_s.  Sums and the loss are computed in 64 bits. */
typedef enum kd_pref_kind { KD_PREF_SIGMOID = 0, KD_PREF_HINGE = 1, KD_PREF_IPO = 2, KD_PREF_KIND_MAX_ENUM = 0x7fffffff } kd_pref_kind;
typedef struct kd_pref_opts {
  const float* ref_logp;   /* [T] or NULL */
  kd_pref_kind kind;
  int32_t average;
  double beta;             /* > 0, finite */
  double label_smoothing;  /* in [0, 1/2); 0 except for KD_PREF_SIGMOID */
  double margin;           /* finite */
} kd_pref_opts;
kd_status kd_preference_loss_workspace_size(int64_t T, int64_t P, size_t* bytes);
/* sums [2P,2] float64 (8-byte aligned): R_s and the number of valid tokens of
 * each sequence, kept for the backward. */
kd_status kd_preference_loss_fwd(const float* logp, const int32_t* cu_seqlens, const uint8_t* mask,
                                 const kd_pref_opts* opts, int64_t T, int64_t P, float* loss, float* rewards,
                                 double* sums, void* workspace, size_t workspace_bytes, void* stream);
/* grad_logp [T] for the upstream gradient grad_loss [P]; 0 at masked tokens and outside all sequences. */
kd_status kd_preference_loss_bwd(const int32_t* cu_seqlens, const uint8_t* mask, const kd_pref_opts* opts, int64_t T,
                                 int64_t P, const double* sums, const float* grad_loss, float* grad_logp,
                                 void* stream);
kd_status kd_preference_loss_fwd_bwd(const float* logp, const int32_t* cu_seqlens, const uint8_t* mask,
                                     const kd_pref_opts* opts, int64_t T, int64_t P, const float* grad_loss,
                                     float* loss, float* rewards, double* sums, float* grad_logp, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- gradient norm and clipping
 * n tensors given by host arrays: device pointers (aligned to their element),
 * element counts (0 is fine, the pointer is then not looked at) and types.
 * Any order and alignment; the tensors' elements are dense in memory. */
#define KD_F16 2 /* a third element type, for the calls of this section only */
kd_status kd_grad_norm_workspace_size(const int64_t* numel, int64_t n, size_t* bytes);
/* sumsq: one float64 on the device, the sum of the squares of all elements
 * (each squared and added in 64 bits).  Ranks that hold parts of the
 * gradients add theirs up before the next call. */
kd_status kd_grad_sumsq(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                        double* sumsq, void* workspace, size_t workspace_bytes, void* stream);
/* norm (one float32 on the device) = sqrt(*sumsq); every output element =
 * input element * min(1, max_norm / (norm + 1e-6)), the product in float32,
 * rounded to the output's type.  outs[i] may be grads[i] (in place, the same
 * type); otherwise outputs overlap nothing (KD_ERR_INVALID_ARG).  In place
 * nothing is written when the factor is 1.  A NaN in the norm makes every
 * output NaN, an infinite norm makes the finite ones 0.  n = 0 gives the
 * norm alone.  max_norm >= 0; infinity: factor 1 whatever the norm. */
kd_status kd_grad_clip(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                       void* const* outs, const int32_t* out_dtypes, const double* sumsq, double max_norm,
                       float* norm, void* stream);

/* Both at once, over the same tensors: sumsq and norm as above.  Up to 2^16
 * elements in at most 8 tensors that have any are one launch. */
kd_status kd_grad_clip_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n,
                            void* const* outs, const int32_t* out_dtypes, double max_norm, double* sumsq,
                            float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDPOLICY_H */
