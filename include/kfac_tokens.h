/*
 * kfac_tokens.h -- C ABI of the operators between tokens and the rows that the
 * rest of the library works on.
 *
 *   kfac_sample_tokens     a token of each row of logits, from given random numbers
 *   kfac_embedding_lookup  rows of a table by token, scaled
 *   kfac_embedding_grad    the table's gradient and the tokens' counts
 *
 * A sampled token is the label, and its log-probability the old_logp, that
 * kfac_policy_loss of kfac_objectives.h takes; a negative token is a row left
 * out there and a row of zeros here.
 *
 * Conventions, as in kfac_objectives.h: device pointers owned by the caller,
 * `stream` a hipStream_t the calls only enqueue on, `workspace` 256-byte
 * aligned with a sticky flag word at its start (kfac_read_flags reads it),
 * zeroed whole once by the caller, one workspace for one call at a time;
 * arguments are validated before anything is enqueued.  These operators may
 * take turns on one workspace of the largest size that they ask for.  Matrices
 * are row-major with a row stride in elements, and a pointer needs the
 * alignment of its element type only.  Nothing is allocated and no host
 * synchronisation is made, so every call may be captured into a graph.
 * Results do not depend on the order in which workgroups run.
 */
#ifndef KFAC_TOKENS_H
#define KFAC_TOKENS_H

#include "kfac_objectives.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kfac_token_workspace_size operators */
enum { KFAC_TOK_SAMPLE = 0, KFAC_TOK_EMBEDDING = 1 };

/*
 * Sampling.  For a row x of logits with maximum M and temperature T
 *     w[i] = exp((x[i] - M) / T)
 * and the columns in order of falling x, equal ones by rising number, the row
 * keeps the first min(n_k, n_p, n_m) of them, at least one:
 *     n_k   top_k (0: all),
 *     n_p   the least n whose w add up to at least top_p times those of the
 *           first n_k (1: all),
 *     n_m   those with w >= min_p.
 * The token is the first column, by number, at which the running sum of the
 * kept w exceeds u times their whole sum.  T = 0 (any T below 1e-6) keeps the
 * first of the order alone; a T above 1e30 counts as 1e30.  logp is the token's
 * log-probability in the whole row, (x[token] - M) / T - log sum w (at T = 0 that
 * of T = 1): what kfac_token_logp gives at logit_scale = 1 / T.  Columns of minus infinity are
 * never kept; a row of nothing else has token -1, logp 0 and kept 0.
 *
 * A row with a NaN or plus infinity among its logits raises
 * KFAC_FLAG_NONFINITE, one whose u lies outside [0, 1) or whose own settings
 * are no numbers (or a negative temperature) KFAC_FLAG_BAD_INDEX; both have
 * token -1, logp 0 and kept 0.
 *
 * w is formed to 2^-44 of M's, in whole multiples of it, and summed exactly: a
 * draw or a border of top_p is decided as in 64-bit arithmetic.
 */
typedef struct kfac_sample {
  const void* logits;         /* [rows, vocab], row stride ld */
  const float* u;             /* [rows], in [0, 1) */
  const float* row_temperature;  /* [rows], in place of the value below; NULL: that value in every row */
  const int32_t* row_top_k;   /* likewise (values below 1: all) */
  const float* row_top_p;     /* likewise (values of at least 1: all; at most 0: the first) */
  const float* row_min_p;     /* likewise (at most 0: all; over 1 counts as 1) */
  int64_t* token;             /* [rows], written */
  float* logp;                /* [rows], written */
  int32_t* kept;              /* [rows], written: the number of columns kept */
  int64_t rows;               /* >= 0 (0: the pointers may be NULL) */
  int64_t ld;
  double temperature;         /* >= 0, finite */
  double top_p;               /* 0 .. 1 */
  double min_p;               /* 0 .. 1 */
  int32_t top_k;              /* >= 0 */
  int32_t vocab;              /* 1 .. 2^20 - 1 */
  int32_t dtype;              /* KFAC_F32 | KFAC_BF16 */
  int32_t reserved;           /* must be 0 */
} kfac_sample_t;

/*
 * Embedding.  y[t] = scale table[ids[t]], rounded once; a negative id gives a
 * row of zeros, and one of at least vocab as well, with KFAC_FLAG_BAD_INDEX.
 * The gradient of sum_t <dy[t], y[t]> by the table is
 *     grad[v]   = scale (sum of dy[t] over the t with ids[t] = v)
 *     counts[v] = the number of those t
 * with the t in rising order, added in 32 bits and rounded once; tokens that do
 * not occur have zeros.  With accumulate set, the sum is added to what grad
 * holds, and rows of tokens that do not occur are not touched.  counts /
 * tokens is the diagonal of the factor A of a layer whose inputs are one-hot
 * rows.  What is written must not share memory with what is read, but for
 * accumulate (between the rows of it is beside it): KFAC_ERR_ARG.
 */
typedef struct kfac_embedding {
  void* table;             /* [vocab, width] of table_dtype, row stride table_ld: read by lookup, and
                              the gradient, written by grad */
  void* y;                 /* [tokens, width] of dtype, row stride y_ld: written by lookup, and dy,
                              read by grad */
  const void* ids;         /* [tokens], int32 or int64 (id_type) */
  int32_t* counts;         /* [vocab], written by grad; NULL: not wanted */
  int64_t tokens;          /* 0 .. 2^30 (0: y and ids may be NULL) */
  int64_t table_ld;
  int64_t y_ld;
  int32_t vocab;           /* 1 .. 2^29 */
  int32_t width;           /* 1 .. 2^24 */
  int32_t dtype;           /* KFAC_F32 | KFAC_BF16 */
  int32_t table_dtype;
  int32_t id_type;
  float scale;             /* finite */
  int32_t accumulate;      /* 0 | 1 (grad) */
  int32_t reserved;        /* must be 0 */
} kfac_embedding_t;

/* Bytes of workspace (host only).  vocab and width as in the operator's
 * descriptor (sampling: width is not used); rows = rows or tokens. */
kfac_status_t kfac_token_workspace_size(int32_t op, int64_t rows, int32_t vocab, int32_t width, size_t* bytes);

kfac_status_t kfac_sample_tokens(const kfac_sample_t* sample, void* workspace, size_t ws_bytes, void* stream);
kfac_status_t kfac_embedding_lookup(const kfac_embedding_t* e, void* workspace, size_t ws_bytes, void* stream);
kfac_status_t kfac_embedding_grad(const kfac_embedding_t* e, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KFAC_TOKENS_H */
