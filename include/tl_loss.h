/*
 * tl_loss.h - C ABI of the training objectives over vocabulary logits whose
 * gradients feed the optimizer step of tl.h.
 *
 * The optimizer step takes the gradient of a micro-batch's MEAN loss times the
 * loss scale S ("Practical LLM in Rust", chapter 13 "Weight each mean by the
 * targets it represents"; "Mixed precision, loss scaling, gradient
 * accumulation, and activation checkpointing", section 4 "The interface":
 * scale(loss) = loss * S).  The functions here are the point where such a
 * gradient begins: one call takes the logits of a micro-batch and gives its
 * loss and the gradient of the logits, already multiplied by a scale that is
 * read on the device (tl_scale_ptr, or the seed tl_loss_seed wrote), so that
 * neither needs a host read.
 *
 *   tl_token_logprob     log-probability of one token per row (the forward that
 *                        yields the old and reference log-probabilities below)
 *   tl_policy_loss       clipped policy objective with a KL penalty
 *   tl_preference_loss   paired preference objective (log-ratio of a chosen and a
 *                        rejected sequence)
 *   tl_distill_loss      distillation from a teacher's top-k logits, with or
 *                        without the cross-entropy of the labels
 *   tl_token_stats       log-probabilities of given tokens with the entropies and
 *                        the likeliest alternatives of their rows (among them a
 *                        teacher's entries for tl_distill_loss)
 *   tl_token_grad        the gradient of the logits for an objective of the
 *                        caller's own over those log-probabilities and entropies
 *
 * Rows.  Row t of the logits is scored against target[t].  A row with
 * target[t] < 0 is ignored: it adds nothing to any sum, its gradient row is
 * zero, its per-row outputs are zero, and neither its logits nor its other
 * per-row inputs are used, whatever they hold (NaN included).  A target of vocab or more is not an
 * id: the row's loss and gradient are NaN (no memory outside the row is read),
 * so the optimizer's finite check skips the update.  n is the divisor of the
 * mean: the number of valid targets (of pairs, for tl_preference_loss), as
 * given to tl_accumulate; result->count returns how many the device saw.
 *
 * Numbers.  z = logits / temperature; softmax statistics, losses and sums are
 * held in fp32 or fp64 whatever the logits' type; a gradient element is
 * computed in fp32 and rounded once to the logits' type.  Entries of -inf
 * (excluded tokens) have probability and gradient 0.  A row with a +inf or NaN
 * entry, or with nothing but -inf, has no softmax: its loss and all of its
 * gradient are NaN, whatever the weights (also for a +inf or NaN among the teacher
 * entries that a row uses).  Results do not depend on timing: every sum has a fixed order for given
 * sizes on a given device.
 *
 * Memory.  The caller owns every tensor.  Rows are contiguous, row t starting
 * at element t * ld; any ld >= vocab and any element-aligned address is
 * accepted.  Rows that start at equal offsets modulo 16 bytes in logits and
 * dlogits take vector accesses; others take element accesses (correct, slower).
 * dlogits may be the logits' own memory (same address and ld): the gradient
 * then replaces them.  Any other overlap of an output with another argument is
 * an error.  A context owns the scratch that its calls share.
 *
 * Calls are asynchronous on the given stream and never wait for the device
 * (tl_loss_create and tl_loss_destroy do).  They can be captured in a CUDA
 * graph; make one call of each kind, with the sizes to be captured, before the
 * capture, so that its kernel is loaded.  A context is not thread-safe, and its calls must be ordered on the
 * device (one stream, or events between streams), since they share its scratch.
 * Status codes are those of tl.h; a call that returns TL_EINVAL or TL_ESTATE
 * has launched nothing.
 */
#ifndef TL_LOSS_H
#define TL_LOSS_H

#include "tl.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tl_loss_ctx tl_loss_ctx;

/* The logits of a micro-batch: rows x vocab elements of dtype (TL_F32, TL_BF16
 * or TL_F16), row t at data + t * ld elements; z = logits / temperature. */
typedef struct {
    const void* data;
    int64_t rows;       /* >= 0 */
    int64_t vocab;      /* 1 .. 2^30; rows * vocab at most 2^40 */
    int64_t ld;         /* >= vocab, < 2^40 */
    int32_t dtype;
    float temperature;  /* > 0, normal; 1 for plain logits */
} tl_logits;

/* Scalars of one call, written by the device (16 bytes, 4-byte aligned). */
typedef struct {
    float loss;    /* sum of the row (pair) losses / n */
    float first;   /* policy: mean clipped surrogate; preference: mean margin beta*h; distill: mean KD term */
    float second;  /* policy: mean KL; preference: share of pairs with h > 0; distill: mean cross-entropy */
    float count;   /* valid rows (pairs) seen */
} tl_loss_result;

/* What a loss gives.  dlogits = NULL computes the forward alone. */
typedef struct {
    int64_t n;               /* divisor of the mean, 1 .. 2^53 */
    const float* seed;       /* device float that multiplies the gradient (S); NULL: 1 */
    void* dlogits;           /* gradient, logits' dtype, row t at t * ld_dlogits; NULL: none */
    int64_t ld_dlogits;      /* >= vocab, < 2^40 */
    float* logp;             /* rows floats, or NULL: log-probability of the target (not tl_distill_loss) */
    float* loss;             /* rows floats (preference: one per pair), or NULL: each one's loss */
    tl_loss_result* result;  /* device memory, required */
} tl_loss_out;

/* A context for calls of at most max_rows rows and max_pairs preference pairs
 * (max_pairs = 0: none) on the current device: it allocates their scratch.  Errors: TL_EINVAL (sizes: 0 <= max_rows <= 2^31 - 1,
 * 0 <= max_pairs <= 2^28), TL_ENOMEM, TL_ECUDA. */
int tl_loss_create(tl_loss_ctx** out, int64_t max_rows, int64_t max_pairs, tl_stream stream);

/* Release it (waits for the device first, so not while a stream of it is being
 * captured).  NULL is accepted. */
int tl_loss_destroy(tl_loss_ctx* ctx);

/* logp[t] = z_t[target[t]] - log sum_j exp(z_t[j]); 0 for ignored rows.
 * Errors of this and the following: TL_EINVAL (arguments), TL_ESTATE (another
 * device is current), TL_ECUDA. */
int tl_token_logprob(tl_loss_ctx* ctx, const tl_logits* logits, const int64_t* target, float* logp,
                     tl_stream stream);

/* Clipped policy objective.  Per valid row, with lp the log-probability of the
 * target, r = exp(lp - old_logp) and A the advantage:
 *   surrogate = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *   kl        = exp(ref_logp - lp) - (ref_logp - lp) - 1      (0 without ref_logp)
 *   loss      = surrogate + kl_weight * kl
 * The surrogate's gradient is -r A where r A is the smaller (or equal) of the
 * two, else 0; old_logp, ref_logp and the advantages are constants. */
typedef struct {
    const int64_t* target;
    const float* old_logp;
    const float* ref_logp;   /* NULL: no KL term (kl_weight must be 0) */
    const float* advantage;
    float clip_low;          /* 0 .. 1 */
    float clip_high;         /* >= 0 */
    float kl_weight;         /* >= 0 */
} tl_policy_args;

int tl_policy_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_policy_args* args, const tl_loss_out* out,
                   tl_stream stream);

/* Paired preference objective.  seq holds 2 * pairs + 1 non-decreasing row
 * offsets: rows [seq[2p], seq[2p+1]) are the chosen sequence of pair p, rows
 * [seq[2p+1], seq[2p+2]) the rejected one (a prompt's rows are ignored through
 * target < 0; a row outside every sequence has no part in any sum and a zero
 * gradient, and its logp is still its log-probability; offsets are held to
 * [0, rows] on the device).  With s(.) the sum over a sequence's valid rows of
 * lp - ref_logp (of lp without ref_logp), reward = beta * s, h = s(chosen) -
 * s(rejected) and sg the logistic function:
 *   loss = -(1 - label_smoothing) log sg(beta h) - label_smoothing log sg(-beta h)
 * A sequence without valid rows has s = 0. */
typedef struct {
    const int64_t* target;
    const int64_t* seq;      /* device, 2 * pairs + 1 offsets */
    int64_t pairs;           /* 0 .. max_pairs */
    const float* ref_logp;   /* NULL: without a reference model */
    float beta;              /* > 0 */
    float label_smoothing;   /* 0 .. 0.5 */
    float* reward;           /* 2 * pairs floats, or NULL: beta * s of each sequence */
} tl_preference_args;

int tl_preference_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_preference_args* args,
                       const tl_loss_out* out, tl_stream stream);

/* Distillation from a teacher's top-k logits.  Row t has k teacher entries: ids
 * teacher_id[t * ld_teacher + i] (int32 or int64) and logits teacher[t *
 * ld_teacher + i].  The teacher's distribution is p = softmax(teacher /
 * temperature) over the row's entries with id >= 0 (a negative id pads; equal
 * ids add up), q = softmax(logits / temperature) over the vocabulary:
 *   kd   = temperature^2 * sum_i p_i (log p_i - log q_id_i)   (0 for a row without entries, or when kd_weight = 0)
 *   ce   = -log softmax(logits)_target     (temperature 1; 0 when ce_weight = 0)
 *   loss = kd_weight * kd + ce_weight * ce
 * Entries of teacher logit -inf have p = 0; a row whose entries are all -inf
 * has kd = 0, as one without entries.  An id of vocab or more makes the row NaN.
 * With k = 0 the call is the plain cross-entropy of the labels. */
typedef struct {
    const int64_t* target;    /* NULL: every row is valid (ce_weight must be 0) */
    const void* teacher;      /* rows x k logits of teacher_dtype */
    const void* teacher_id;
    int64_t ld_teacher;       /* >= k */
    int32_t k;                /* 0 .. 1024 */
    int32_t teacher_dtype;    /* TL_F32, TL_BF16 or TL_F16 */
    int32_t id_bytes;         /* 4 or 8 */
    float kd_weight;          /* >= 0 */
    float ce_weight;          /* >= 0 */
} tl_distill_args;

int tl_distill_loss(tl_loss_ctx* ctx, const tl_logits* logits, const tl_distill_args* args, const tl_loss_out* out,
                    tl_stream stream);

/* What the forward keeps of a row for the backward: log q_j = (x_j - max) /
 * temperature - log_sum, so max / temperature + log_sum is the logarithm of the
 * row's sum of exponentials. */
typedef struct {
    float max;       /* largest logit */
    float log_sum;   /* log sum_j exp((x_j - max) / temperature) */
    float entropy;
} tl_token_saved;

/* Log-probabilities, entropies and alternatives.  Per valid row, with log q the
 * log-softmax of the logits / temperature (for log-probabilities alone there is
 * tl_token_logprob, which takes about as long):
 *   logp     = log q_target
 *   entropy  = -sum_j q_j log q_j
 *   top      the k largest logits, the largest first and the lower id first among
 *            equal ones: their ids and log q.  Excluded tokens (-inf) are never
 *            among them; places without an entry (k above the number of others)
 *            hold id -1 and -inf.
 * Every output may be NULL, not all of them.  Of an ignored row the outputs are 0
 * and its ids -1.  A target of vocab or more makes logp NaN and nothing else; a row
 * without a softmax has NaN outputs and ids of -1.  Ids and their log-probabilities
 * are what tl_distill_loss takes as a teacher's entries: a common offset of the
 * logits leaves its softmax as it is, at temperature 1 here and any there.  (A row
 * without a softmax, as an ignored one, is a row without entries there: kd 0.) */
typedef struct {
    const int64_t* target;   /* NULL: every row is valid (logp must be NULL) */
    float* logp;             /* rows floats, or NULL */
    float* entropy;          /* rows floats, or NULL */
    tl_token_saved* saved;   /* rows entries, or NULL */
    void* top_id;            /* rows x k ids, row t at t * ld_top; NULL where k = 0 */
    float* top_logp;         /* rows x k floats, row t at t * ld_top; NULL where k = 0 */
    int64_t ld_top;          /* >= k */
    int32_t k;               /* 0 .. 256 */
    int32_t id_bytes;        /* 4 or 8 (k > 0) */
} tl_token_stats_args;

int tl_token_stats(tl_loss_ctx* ctx, const tl_logits* logits, const tl_token_stats_args* args, tl_stream stream);

/* dlogits = d/dlogits of seed * sum_t (grad_logp[t] * logp[t] + grad_entropy[t] *
 * entropy[t]): per valid row
 *   seed / temperature * (grad_logp (1[j = target] - q_j) - grad_entropy q_j (log q_j + entropy))
 * saved is what tl_token_stats wrote for these logits at this temperature; the
 * gradients are those of the caller's objective (its own 1 / n included).  Rows
 * whose softmax is missing, or whose target is vocab or more, are NaN. */
typedef struct {
    const int64_t* target;        /* NULL: every row is valid (grad_logp must be NULL) */
    const tl_token_saved* saved;
    const float* grad_logp;       /* rows floats, or NULL: 0 */
    const float* grad_entropy;    /* rows floats, or NULL: 0; not both NULL */
    const float* seed;            /* device float (S); NULL: 1 */
    void* dlogits;                /* logits' dtype, row t at t * ld_dlogits */
    int64_t ld_dlogits;           /* >= vocab, < 2^40 */
} tl_token_grad_args;

int tl_token_grad(tl_loss_ctx* ctx, const tl_logits* logits, const tl_token_grad_args* args, tl_stream stream);

/* Kernels launched so far, and the text of the last error. */
int64_t tl_loss_launch_count(const tl_loss_ctx* ctx);
const char* tl_loss_last_error(const tl_loss_ctx* ctx);

#ifdef __cplusplus
}
#endif

#endif /* TL_LOSS_H */
