// Declarations shared by the orthogonalisation kernels and their C entry points
// (include/kfac_orthogonal.h).
#pragma once

#include <algorithm>
#include <cmath>

#include "common.h"
#include "../../include/kfac_orthogonal.h"

namespace kfac {

constexpr int32_t kOrthMaxDim = 65536;
constexpr int32_t kOrthMaxBatch = 65535;

// A matrix to orthogonalise, or a batch of them, with what becomes of it.
struct OrthTask {
  int32_t rows, cols, batch;
  int32_t dtype;                       // of x and y
  const void* x;                       // the matrix, or a layer's gradient (with mom)
  int64_t ld, stride;
  float* mom;                          // a layer: its momentum, [rows, cols] contiguous
  void* y;                             // the update, where there is no weight
  int64_t y_ld, y_stride;
  float* w;                            // a layer's weight, [rows, cols] contiguous
  float factor;                        // w <- decay w - factor O
  float* bias;                         // [rows], with its momentum and gradient; NULL: none
  float* bias_mom;
  const float* bias_grad;
};
struct OrthStep {
  float lr, momentum, weight_decay;
};

// Of a step's polynomials over the singular values up to rho: the norm of
// B = b A + c A A, and that of the next X, each with 2% for rounding.  Extremes
// lie at rho or where the derivative vanishes.
struct PolyBound {
  double b, next;
};
inline PolyBound poly_of(const float* coef, double rho) {
  const double a = coef[0], b = coef[1], c = coef[2], top = rho * rho;
  PolyBound r{0.0, 0.0};
  auto see = [&](double u) {           // u: the value's square
    if (!(u >= 0.0 && u <= top)) return;
    r.b = std::max(r.b, std::fabs(u * (b + c * u)));
    r.next = std::max(r.next, std::fabs(std::sqrt(u) * (a + u * (b + c * u))));
  };
  see(top);
  if (c != 0.0) {
    see(-b / (2.0 * c));
    const double q = 9.0 * b * b - 20.0 * a * c;       // a + 3 b u + 5 c u^2 = 0
    if (q >= 0.0) {
      see((-3.0 * b + std::sqrt(q)) / (10.0 * c));
      see((-3.0 * b - std::sqrt(q)) / (10.0 * c));
    }
  } else if (b != 0.0) {
    see(-a / (3.0 * b));
  }
  r.b *= 1.02;
  r.next *= 1.02;
  return r;
}

// Matrices with a side of at most this run on d x d matrices in one workgroup each.
constexpr int kOrthSmall = 64;
inline bool orth_is_small(const OrthTask& t) { return std::min(t.rows, t.cols) <= kOrthSmall; }
size_t orth_small_bytes(const std::vector<OrthTask>& tasks);
kfac_status_t launch_orth_small(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how, const OrthStep& step,
                                char* regions, uint32_t* flags, hipStream_t st);

size_t orth_workspace_bytes(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how);
kfac_status_t launch_orthogonal(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how, const OrthStep& step,
                                char* ws, hipStream_t st);

}  // namespace kfac
