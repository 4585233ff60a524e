// The extern "C" entry points of include/kfac_orthogonal.h: host-side
// validation and dispatch.
#include "orthogonal.h"
#include "overlap.h"
#include "validate.h"

#include <algorithm>
#include <cmath>

namespace kfac {

namespace {

// 64 x 64 tiles of all matrices together: one launch covers 2^32 - 1 threads, 256 a tile.
constexpr int64_t kMaxTiles = 1 << 23;

kfac_status_t check_how(const kfac_orthogonal_t* how) {
  if (!how || !how->coefs || how->steps < 1 || how->steps > KFAC_ORTHOGONAL_MAX_STEPS) return KFAC_ERR_ARG;
  if (!(how->eps >= 0.0) || !std::isfinite(how->eps)) return KFAC_ERR_ARG;
  if (how->products != KFAC_PRODUCTS_HALF && how->products != KFAC_PRODUCTS_FULL) return KFAC_ERR_ARG;
  if (how->nesterov != 0 && how->nesterov != 1) return KFAC_ERR_ARG;
  if (how->scale != KFAC_SCALE_NONE && how->scale != KFAC_SCALE_ASPECT && how->scale != KFAC_SCALE_RMS) return KFAC_ERR_ARG;
  // coefficients that keep every power of two of the planes within float32
  for (int i = 0; i < 3 * how->steps; ++i)
    if (!(std::fabs(how->coefs[i]) <= 64.f)) return KFAC_ERR_ARG;
  double rho = 1.0;
  for (int k = 0; k < how->steps; ++k) {
    rho = poly_of(how->coefs + 3 * k, rho).next;
    if (!(rho <= 1e4)) return KFAC_ERR_UNSUPPORTED;
  }
  return KFAC_OK;
}

int64_t tiles_of(int32_t rows, int32_t cols) {
  auto side = [](int32_t v) { return (static_cast<int64_t>(v) + 255) / 256 * 4; };
  return side(rows) * side(cols);
}

kfac_status_t check_matrix(const kfac_orthogonal_matrix_t* m) {
  if (!m) return KFAC_ERR_ARG;
  if (!dtype_ok(m->dtype)) return KFAC_ERR_DTYPE;
  if (m->rows < 1 || m->cols < 1 || m->batch < 0) return KFAC_ERR_ARG;
  if (m->rows > kOrthMaxDim || m->cols > kOrthMaxDim || m->batch > kOrthMaxBatch) return KFAC_ERR_UNSUPPORTED;
  if (tiles_of(m->rows, m->cols) * m->batch > kMaxTiles) return KFAC_ERR_UNSUPPORTED;
  return KFAC_OK;
}

OrthTask task_of(const kfac_orthogonal_matrix_t& m) {
  OrthTask t{};
  t.rows = m.rows;
  t.cols = m.cols;
  t.batch = m.batch;
  t.dtype = m.dtype;
  t.x = m.x;
  t.ld = m.ld;
  t.stride = m.stride;
  t.y = m.y;
  t.y_ld = m.y_ld;
  t.y_stride = m.y_stride;
  return t;
}

kfac_status_t tasks_of(const kfac_layer_t* layers, int32_t n, const kfac_orthogonal_t& how, float lr, std::vector<OrthTask>* out) {
  if (n < 1 || !layers) return KFAC_ERR_ARG;
  int64_t tiles = 0;
  for (int32_t i = 0; i < n; ++i) {
    const kfac_layer_t& L = layers[i];
    if (L.reserved != 0 || (L.has_bias != 0 && L.has_bias != 1) || L.d_in < 1 || L.d_out < 1) return KFAC_ERR_ARG;
    if (L.kind == KFAC_BATCHNORM) return KFAC_ERR_UNSUPPORTED;
    if (L.kind != KFAC_LINEAR && L.kind != KFAC_CONV2D) return KFAC_ERR_ARG;
    if (L.d_in > kOrthMaxDim || L.d_out > kOrthMaxDim) return KFAC_ERR_UNSUPPORTED;
    tiles += tiles_of(L.d_out, L.d_in);
    if (tiles > kMaxTiles) return KFAC_ERR_UNSUPPORTED;
    OrthTask t{};
    t.rows = L.d_out;
    t.cols = L.d_in;
    t.batch = 1;
    t.dtype = KFAC_F32;
    t.x = L.grad_w;
    t.ld = L.d_in;
    t.mom = L.mom_w;
    t.w = L.w;
    double s = 1.0;
    if (how.scale == KFAC_SCALE_ASPECT) s = std::sqrt(std::max(1.0, static_cast<double>(L.d_out) / L.d_in));
    if (how.scale == KFAC_SCALE_RMS) s = 0.2 * std::sqrt(static_cast<double>(std::max(L.d_out, L.d_in)));
    t.factor = static_cast<float>(lr * s);
    if (L.has_bias) {
      t.bias = L.b;
      t.bias_mom = L.mom_b;
      t.bias_grad = L.grad_b;
    }
    out->push_back(t);
  }
  return KFAC_OK;
}

}  // namespace
}  // namespace kfac

extern "C" {

kfac_status_t kfac_orthogonal_workspace_size(const kfac_orthogonal_matrix_t* m, const kfac_orthogonal_t* how, size_t* bytes) {
  if (!bytes) return KFAC_ERR_ARG;
  kfac_status_t s = kfac::check_matrix(m);
  if (s == KFAC_OK) s = kfac::check_how(how);
  if (s != KFAC_OK) return s;
  *bytes = kfac::orth_workspace_bytes({kfac::task_of(*m)}, *how);
  return KFAC_OK;
}

kfac_status_t kfac_orthogonal_step_workspace_size(const kfac_layer_t* layers, int32_t n_layers, const kfac_orthogonal_t* how,
                                                  size_t* bytes) {
  if (!bytes) return KFAC_ERR_ARG;
  kfac_status_t s = kfac::check_how(how);
  if (s != KFAC_OK) return s;
  std::vector<kfac::OrthTask> tasks;
  s = kfac::tasks_of(layers, n_layers, *how, 0.f, &tasks);
  if (s != KFAC_OK) return s;
  *bytes = kfac::orth_workspace_bytes(tasks, *how);
  return KFAC_OK;
}

kfac_status_t kfac_orthogonalize(const kfac_orthogonal_matrix_t* m, const kfac_orthogonal_t* how, void* workspace,
                                 size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_matrix(m);
  if (s == KFAC_OK) s = kfac::check_how(how);
  if (s != KFAC_OK) return s;
  if (m->ld < m->cols || m->y_ld < m->cols) return KFAC_ERR_ARG;
  if (!kfac::extent_ok(m->rows, m->ld) || !kfac::extent_ok(m->rows, m->y_ld)) return KFAC_ERR_UNSUPPORTED;
  const int64_t span = (m->rows - 1) * m->ld + m->cols, y_span = (m->rows - 1) * m->y_ld + m->cols;
  if (m->batch > 1) {
    if (m->stride < span || m->y_stride < y_span) return KFAC_ERR_ARG;
    if (!kfac::extent_ok(m->batch, m->stride) || !kfac::extent_ok(m->batch, m->y_stride)) return KFAC_ERR_UNSUPPORTED;
  }
  if (m->batch > 0) {
    kfac::Ptrs p;
    p.need(m->x, kfac::elem_size(m->dtype));
    p.need(m->y, kfac::elem_size(m->dtype));
    if (p.s != KFAC_OK) return p.s;
    if (m->x == m->y && (m->ld != m->y_ld || (m->batch > 1 && m->stride != m->y_stride))) return KFAC_ERR_ARG;
  }
  const std::vector<kfac::OrthTask> tasks{kfac::task_of(*m)};
  s = kfac::check_workspace(workspace, ws_bytes, kfac::orth_workspace_bytes(tasks, *how));
  if (s != KFAC_OK || m->batch == 0) return s;
  const int64_t el = static_cast<int64_t>(kfac::elem_size(m->dtype));
  const kfac::Lines x = kfac::lines_of(m->x, m->cols * el, m->rows, m->ld * el, m->batch, m->stride * el);
  const kfac::Lines y = kfac::lines_of(m->y, m->cols * el, m->rows, m->y_ld * el, m->batch, m->y_stride * el);
  if (m->x != m->y && kfac::overlap(x, y)) return KFAC_ERR_ARG;
  return kfac::launch_orthogonal(tasks, *how, kfac::OrthStep{}, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_step_orthogonal(const kfac_layer_t* layers, int32_t n_layers, const kfac_hparams_t* hp,
                                   const kfac_orthogonal_t* how, void* workspace, size_t ws_bytes, void* stream) {
  if (!hp || hp->reserved != 0) return KFAC_ERR_ARG;
  if (hp->options != 0 || hp->phase_mask != 0) return KFAC_ERR_UNSUPPORTED;
  if (!std::isfinite(hp->lr) || !std::isfinite(hp->momentum) || !std::isfinite(hp->weight_decay)) return KFAC_ERR_ARG;
  kfac_status_t s = kfac::check_how(how);
  if (s != KFAC_OK) return s;
  std::vector<kfac::OrthTask> tasks;
  s = kfac::tasks_of(layers, n_layers, *how, hp->lr, &tasks);
  if (s != KFAC_OK) return s;
  kfac::Ptrs p;
  for (int32_t i = 0; i < n_layers; ++i) {
    const kfac_layer_t& L = layers[i];
    p.need(L.grad_w, 4);
    p.need(L.w, 4);
    p.need(L.mom_w, 4);
    if (L.has_bias) {
      p.need(L.grad_b, 4);
      p.need(L.b, 4);
      p.need(L.mom_b, 4);
    }
  }
  if (p.s != KFAC_OK) return p.s;
  s = kfac::check_workspace(workspace, ws_bytes, kfac::orth_workspace_bytes(tasks, *how));
  if (s != KFAC_OK) return s;
  if (kfac::step_shares_memory(layers, n_layers)) return KFAC_ERR_ARG;
  return kfac::launch_orthogonal(tasks, *how, kfac::OrthStep{hp->lr, hp->momentum, hp->weight_decay},
                                 static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

}  // extern "C"
