/*
 * kfac_orthogonal.h -- C ABI of the orthogonalised update: a third way, beside
 * kfac.h's two methods, to turn a layer's gradient into a step.  It needs
 * neither the layer's input nor its output-gradient rows, keeps no factors, and
 * costs products of the weight's own size only.
 *
 *   kfac_orthogonalize    O(x) of a matrix, or of a batch of one shape
 *   kfac_step_orthogonal  momentum, O, weight decay and the parameter write for
 *                         a stack of layers
 *
 * For x [m, n], d = min(m, n), X = x (m <= n) or x^T, with d rows:
 *     X <- X / (||X||_F + eps)
 *     X <- a X + (b A + c A A) X,  A = X X^T      for each step's (a, b, c)
 * and O(x) is the last X, turned back.  Every singular value s goes through
 * a s + b s^3 + c s^5 once a step, the singular vectors stay: with the usual
 * coefficients (3.4445, -4.7750, 2.0315; published by K. Jordan and others in 2024
 * for updates like these) five steps bring values from 0.01 to 1
 * of the norm to between 0.68 and 1.13, near the orthogonal factor of x (Newton-
 * Schulz iteration for the polar factor).
 *
 * Conventions as in kfac.h: device pointers owned by the caller, `stream` a
 * hipStream_t the calls only enqueue on, `workspace` 256-byte aligned with a
 * sticky flag word at its start, zeroed whole once by the caller, one workspace
 * for one call at a time; arguments are validated before anything is enqueued.
 * Nothing is allocated and no host synchronisation is made, so every call may
 * be captured into a graph.  Results do not depend on the order in which
 * workgroups run.  A norm that is not finite raises KFAC_FLAG_NONFINITE; the
 * update is then no number either.  A matrix of zeros has O = 0.
 */
#ifndef KFAC_ORTHOGONAL_H
#define KFAC_ORTHOGONAL_H

#include "kfac.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kfac_orthogonal_t.products: what the iteration's matrices are held in
 * between its products, whose sums are float32 either way.  O is then off that
 * of 64 bits by (2-norm, relative):
 *   HALF  11 bits (IEEE half, scaled).  5e-4 to 1.2e-3 for noise with or without
 *         strong directions over it (bfloat16's own rounding is 1.7e-3); up to
 *         4e-3 for sparse matrices, 1e-2 for equal singular values (an
 *         identity), whose roundings are all the same, and 1.2e-2 where a few
 *         directions make up all of x and its shorter side is below 300: of the
 *         others there are then hardly any but roundings, and they are what grows
 *   FULL  22 bits (two halves, three products each).  What float32 products are
 *         off: 1e-6 to 5e-6 (sides of more than 4096: to 1e-5), and where a few
 *         directions make up nearly all of x up to 3e-4 (shorter sides up to 1024)
 * Matrices with a side of at most 64 take neither: they are iterated in 64 bits. */
enum { KFAC_PRODUCTS_HALF = 0, KFAC_PRODUCTS_FULL = 1 };
/* kfac_orthogonal_t.scale: the factor s of a layer's step, W [d_out, d_in]
 *   NONE 1, ASPECT sqrt(max(1, d_out / d_in)), RMS 0.2 sqrt(max(d_out, d_in)) */
enum { KFAC_SCALE_NONE = 0, KFAC_SCALE_ASPECT = 1, KFAC_SCALE_RMS = 2 };

#define KFAC_ORTHOGONAL_MAX_STEPS 16

typedef struct kfac_orthogonal {
  const float* coefs;   /* host, [steps][3]: a, b, c, each within [-64, 64].  KFAC_ERR_UNSUPPORTED where
                           they let a singular value of at most 1 grow past 10^4 */
  double eps;           /* >= 0 */
  int32_t steps;        /* 1 .. KFAC_ORTHOGONAL_MAX_STEPS */
  int32_t products;     /* KFAC_PRODUCTS_* */
  int32_t nesterov;     /* step: 0 | 1 */
  int32_t scale;        /* step: KFAC_SCALE_* */
} kfac_orthogonal_t;

/* A batch of matrices, row-major, rows `ld` elements and matrices `stride`
 * elements apart.  y may be x itself with the same strides, and must not
 * share memory with it otherwise: KFAC_ERR_ARG.  Pointers need the alignment of
 * their element. */
typedef struct kfac_orthogonal_matrix {
  const void* x;        /* [batch, rows, cols] of dtype */
  void* y;              /* likewise, written */
  int64_t ld, stride;
  int64_t y_ld, y_stride;
  int32_t rows, cols;   /* 1 .. 65536 */
  int32_t batch;        /* >= 0 (0: x and y may be NULL), at most 65535 */
  int32_t dtype;        /* KFAC_F32 | KFAC_BF16 */
} kfac_orthogonal_matrix_t;

/* Bytes of workspace (host only; pointers of tensors are not inspected). */
kfac_status_t kfac_orthogonal_workspace_size(const kfac_orthogonal_matrix_t* m, const kfac_orthogonal_t* how,
                                             size_t* bytes);
kfac_status_t kfac_orthogonal_step_workspace_size(const kfac_layer_t* layers, int32_t n_layers,
                                                  const kfac_orthogonal_t* how, size_t* bytes);

kfac_status_t kfac_orthogonalize(const kfac_orthogonal_matrix_t* m, const kfac_orthogonal_t* how, void* workspace,
                                 size_t ws_bytes, void* stream);

/*
 * One step of every layer, with hp's lr, momentum (mu) and weight_decay (wd),
 * hp's other fields not looked at but `reserved`, `options` and `phase_mask`,
 * which must be 0:
 *     V <- mu V + grad_w;   U = grad_w + mu V (nesterov) or V
 *     W <- (1 - lr wd) W - lr s O(U)
 * Of a layer's descriptor kind (linear or conv2d, whose weights are a matrix
 * [d_out, c_in kh kw]), d_in, d_out, has_bias and the pointers w, mom_w,
 * grad_w, b, mom_b and grad_b are used (all float32, contiguous, aligned to
 * their element).  A bias has no matrix to orthogonalise and takes the step
 * that it takes in kfac.h with D its gradient:
 *     V <- mu V + (grad_b + wd b);   b <- b - lr V
 * What is written must not share memory, with itself or with a gradient: KFAC_ERR_ARG.
 */
kfac_status_t kfac_step_orthogonal(const kfac_layer_t* layers, int32_t n_layers, const kfac_hparams_t* hp,
                                   const kfac_orthogonal_t* how, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KFAC_ORTHOGONAL_H */
