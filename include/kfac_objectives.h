/*
 * kfac_objectives.h -- C ABI of the operators on either side of an optimizer
 * step: the training objectives that make the output-gradient rows kfac.h's
 * factors are built from, and the dropout that makes a layer's input rows.
 *
 *   kfac_token_logp       log-probability of each row's label
 *   kfac_policy_loss      clipped policy loss with a KL term, logit gradients
 *   kfac_preference_loss  loss over pairs of sequences, logit gradients
 *   kfac_balance_loss     router balance loss with per-expert counts, gradients
 *   kfac_dropout          dropout from a counter-based generator, no mask stored
 *
 * Conventions, as in kfac.h: device pointers owned by the caller, `stream` a
 * hipStream_t the calls only enqueue on, `workspace` 256-byte aligned with a
 * sticky flag word at its start (kfac_read_flags reads it), zeroed whole
 * once by the caller, one workspace for one call at a time; arguments are validated
 * before anything is enqueued.  The objectives may take turns on one workspace of
 * the largest size that they ask for; a step of kfac.h needs one of its own (the
 * policy loss keeps counters behind the flag word that have to be 0 between its
 * calls, and a step would write over them: its statistics would then not be
 * written).  Differences: matrices are row-major with a
 * row stride in elements (`ld` >= the width), and a pointer needs the
 * alignment of its element type only.  Nothing is allocated and no host
 * synchronisation is made, so every call may be captured into a graph.
 * Results do not depend on the order in which workgroups run.
 *
 * Element types (dtype): KFAC_F32 or KFAC_BF16 for logits, gradients and the
 * tensors of dropout; everything else is float32 or an integer.  Gradients
 * are those of the objective times grad_scale: with a mean over rows and
 * grad_scale = rows they are per-row gradients, the rows g that
 * kfac_layer_t expects.  That descriptor has no row stride: write them with
 * grad_ld = the width, into the layer's buffer.
 */
#ifndef KFAC_OBJECTIVES_H
#define KFAC_OBJECTIVES_H

#include "kfac.h"

#ifdef __cplusplus
extern "C" {
#endif

/* integer types of labels and expert numbers */
enum { KFAC_I32 = 0, KFAC_I64 = 1 };
/* sticky flag, beside those of kfac.h: a label, an expert number or a
 * sequence offset beyond its range (that row, slot or sequence is then left
 * out, nothing is read or written out of bounds).  KFAC_FLAG_NONFINITE: a row
 * that counts has a loss or a gradient that is not finite, or the losses' sum
 * is not, in float32. */
enum { KFAC_FLAG_BAD_INDEX = 4u };
/* kfac_objective_workspace_size objectives */
enum { KFAC_OBJ_LOGP = 0, KFAC_OBJ_POLICY = 1, KFAC_OBJ_PREFERENCE = 2, KFAC_OBJ_BALANCE = 3 };
/* kfac_preference_t.kind */
enum { KFAC_PREF_SIGMOID = 0, KFAC_PREF_SQUARED = 1 };

/*
 * Logits and labels of `rows` tokens.  For row r with label l >= 0
 *     logp[r] = s x[r, l] - log sum_j exp(s x[r, j]),   s = logit_scale > 0;
 * a negative label marks a row to leave out: logp[r] = 0, its gradient is 0,
 * its logits are not looked at.  Logits of minus infinity, or of the type's
 * lowest value, are columns of probability 0.
 */
typedef struct kfac_token_rows {
  const void* logits;   /* [rows, vocab], row stride ld */
  const void* labels;   /* [rows], int32 or int64 (label_type) */
  float* logp;          /* [rows], written */
  void* grad;           /* losses: [rows, vocab] of dtype, row stride grad_ld, written; may be `logits`
                           itself with grad_ld == ld, must not overlap it otherwise */
  int64_t rows;         /* >= 0 (0: pointers of [rows, ...] arrays may be NULL; the policy's stats
                           are then 0, a preference pair counts with h = 0) */
  int64_t ld;
  int64_t grad_ld;
  int32_t vocab;        /* >= 1 */
  int32_t dtype;
  int32_t label_type;
  float logit_scale;
  float grad_scale;
  int32_t reserved;     /* must be 0 */
} kfac_token_rows_t;

/*
 * Clipped policy loss.  With a = advantage, w = weight, and per row
 *     ratio = exp(logp - old_logp)
 *     A = -min(ratio a, clamp(ratio, 1 - clip_low, 1 + clip_high) a)
 *     K = exp(d) - d - 1,  d = ref_logp - logp
 *     loss = sum w (A + kl_coef K)
 * The gradient of a row is coef (onehot(label) - softmax) with
 *     coef = w s grad_scale ([unclipped] (-a ratio) + kl_coef (1 - exp(d))).
 * Rows with a negative label or weight 0 count for nothing, whatever their
 * other values; their gradient is 0.
 */
typedef struct kfac_policy {
  const float* advantage;  /* [rows] */
  const float* weight;     /* [rows], NULL: 1 / rows */
  const float* old_logp;   /* [rows], NULL: the policy's own, held fixed (ratio 1).  One that
                              kfac_token_logp gave for the same logits makes a ratio that is 1
                              up to float32 roundings of logp */
  const float* ref_logp;   /* [rows], NULL: no KL term (kl_coef must be 0) */
  float* stats;            /* [4], written: loss, sum w A, sum w K, sum w [clipped] */
  float clip_low;          /* 0 <= clip_low <= 1 */
  float clip_high;         /* >= 0 */
  float kl_coef;           /* >= 0 */
  int32_t reserved;        /* must be 0 */
} kfac_policy_t;

/*
 * Preference loss over pairs of sequences.  Sequence i holds the rows
 * offsets[i] .. offsets[i + 1] - 1; pair i < pairs prefers sequence i to
 * sequence pairs + i.  Per sequence
 *     R = sum over its rows with a label of (logp - ref_logp), divided by
 *         their number when average is set (0 for a sequence without any)
 * and with h = R[i] - R[pairs + i], w = pair_weight[i], e = label_smoothing
 *     sigmoid: L = -(1 - e) log sigma(beta h) - e log sigma(-beta h)
 *     squared: L = (h - 1 / (2 beta))^2
 *     loss = sum w L
 * A pair of weight 0 counts for nothing.  Rows outside every sequence have
 * gradient 0.  Where decreasing offsets (flagged) leave rows to two sequences,
 * they have the gradient of one of them.
 */
typedef struct kfac_preference {
  const int32_t* offsets;    /* [2 pairs + 1], device, not decreasing, within [0, rows] */
  const float* ref_logp;     /* [rows], NULL: 0 */
  const float* pair_weight;  /* [pairs], NULL: 1 / pairs */
  float* seq;                /* [2 pairs], written: R */
  float* stats;              /* [4], written: loss, sum w [h > 0], sum w beta h, sum w */
  int32_t pairs;             /* 1 .. 2^22 - 1; rows <= 2^31 - 1 */
  int32_t kind;              /* KFAC_PREF_SIGMOID | KFAC_PREF_SQUARED */
  float beta;                /* > 0 */
  float label_smoothing;     /* 0 <= e < 0.5 (sigmoid) */
  int32_t average;           /* 0 | 1 */
  int32_t reserved;          /* must be 0 */
} kfac_preference_t;

/*
 * Router balance loss.  With p = softmax of a token's logits over E experts,
 * the n tokens whose mask is set and experts[t, 0 .. top_k) the experts each
 * token was sent to (negative: a slot that was dropped)
 *     counts[e] = slots of the n tokens that name e
 *     prob[e]   = sum over the n tokens of p[t, e] / n
 *     balance   = coef E sum_e counts[e] / (top_k n) prob[e]
 *     z         = z_coef sum over the n tokens of (log sum_e exp logits)^2 / n
 * The gradient is that of balance + z, with counts held fixed.  Masked tokens
 * have gradient 0 and their logits are not looked at; n = 0 gives zeros.
 */
typedef struct kfac_balance {
  const void* logits;      /* [tokens, experts], row stride ld */
  const void* chosen;      /* [tokens, top_k] contiguous, int32 or int64 (index_type) */
  const uint8_t* mask;     /* [tokens], 0 or 1, NULL: all set */
  int32_t* counts;         /* [experts], written */
  float* prob;             /* [experts], written */
  float* stats;            /* [4], written: balance + z, balance, z, n */
  void* grad;              /* [tokens, experts], row stride grad_ld, written; may be `logits` itself
                              with grad_ld == ld, must not overlap it otherwise */
  int64_t tokens;          /* >= 0 (0: pointers of [tokens, ...] arrays may be NULL) */
  int64_t ld;
  int64_t grad_ld;
  int32_t experts;         /* 1 .. 1024 */
  int32_t top_k;           /* 1 .. experts */
  int32_t dtype;
  int32_t index_type;
  float coef;
  float z_coef;
  float grad_scale;
  int32_t reserved;        /* must be 0 */
} kfac_balance_t;

/*
 * Dropout with a mask that is computed, never stored:
 *     y[r, c] = keep[r, c] ? x[r, c] 65536 / (65536 - T) : 0, plus residual[r, c],
 * T = p 65536 rounded to the nearest integer (p = 1: nothing is kept).  The
 * mask comes from the counter-based generator Philox 4x32 with 10 rounds
 * (Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3"):
 * key = seed, counter = (block, offset) with block = r ceil(cols / 8) + c / 8;
 * the 128 bits are eight 16-bit draws, low half of the first word first, for
 * the block's eight columns, and an element is kept when its draw is at least
 * T.  The same seed, offset and shape give the same mask in any call, so the
 * backward pass is the same call on the output gradient, without residual.
 * A dropped value is 0 whatever x holds there.  At most 2^32 - 1024 blocks
 * (2^35 elements) a call.
 */
typedef struct kfac_dropout {
  const void* x;           /* [rows, cols], row stride ld */
  const void* residual;    /* [rows, cols], row stride residual_ld, or NULL */
  void* y;                 /* [rows, cols], row stride y_ld, written; may be x or residual itself with
                              the same stride, must not overlap them otherwise */
  const int64_t* offset_dev;  /* NULL, or a device word whose value is added to offset when the kernel
                              runs (a captured graph then draws a new mask at every replay) */
  int64_t rows;            /* >= 0 */
  int64_t cols;            /* >= 1 */
  int64_t ld, residual_ld, y_ld;
  uint64_t seed;
  uint64_t offset;
  double p;                /* 0 .. 1 */
  int32_t dtype;
  int32_t reserved;        /* must be 0 */
} kfac_dropout_t;

/* Bytes of workspace (host only): rows = rows or tokens; groups = pairs
 * (preference), experts (balance), not used otherwise.  Dropout needs none. */
kfac_status_t kfac_objective_workspace_size(int32_t objective, int64_t rows, int32_t groups, size_t* bytes);

kfac_status_t kfac_token_logp(const kfac_token_rows_t* rows, void* workspace, size_t ws_bytes, void* stream);
kfac_status_t kfac_policy_loss(const kfac_token_rows_t* rows, const kfac_policy_t* policy, void* workspace,
                               size_t ws_bytes, void* stream);
kfac_status_t kfac_preference_loss(const kfac_token_rows_t* rows, const kfac_preference_t* pref, void* workspace,
                                   size_t ws_bytes, void* stream);
kfac_status_t kfac_balance_loss(const kfac_balance_t* balance, void* workspace, size_t ws_bytes, void* stream);
kfac_status_t kfac_dropout(const kfac_dropout_t* dropout, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KFAC_OBJECTIVES_H */
