// The extern "C" entry points of include/kfac_objectives.h: host-side
// validation and dispatch.
#include "objectives.h"
#include "validate.h"

#include <cmath>

namespace kfac {

namespace {

kfac_status_t check_rows(const kfac_token_rows_t* t, bool grad) {
  if (!t || t->reserved != 0) return KFAC_ERR_ARG;
  if (!dtype_ok(t->dtype) || !index_ok(t->label_type)) return KFAC_ERR_DTYPE;
  if (t->rows < 0 || t->vocab < 1 || t->ld < t->vocab) return KFAC_ERR_ARG;
  if (!(t->logit_scale > 0.f) || !std::isfinite(t->logit_scale)) return KFAC_ERR_ARG;
  if (!extent_ok(t->rows, t->ld)) return KFAC_ERR_UNSUPPORTED;
  if (grad) {
    if (t->grad_ld < t->vocab || !std::isfinite(t->grad_scale)) return KFAC_ERR_ARG;
    if (t->grad == t->logits && t->grad && t->grad_ld != t->ld) return KFAC_ERR_ARG;
    if (!extent_ok(t->rows, t->grad_ld)) return KFAC_ERR_UNSUPPORTED;
  }
  if (t->rows == 0) return KFAC_OK;
  Ptrs p;
  p.need(t->logits, elem_size(t->dtype));
  p.need(t->labels, index_size(t->label_type));
  p.need(t->logp, 4);
  if (grad) p.need(t->grad, elem_size(t->dtype));
  return p.s;
}

}  // namespace
}  // namespace kfac

extern "C" {

kfac_status_t kfac_objective_workspace_size(int32_t objective, int64_t rows, int32_t groups, size_t* bytes) {
  if (!bytes || rows < 0) return KFAC_ERR_ARG;
  switch (objective) {
    case KFAC_OBJ_LOGP:
    case KFAC_OBJ_POLICY: break;
    case KFAC_OBJ_PREFERENCE:
      if (groups < 1) return KFAC_ERR_ARG;
      // one launch covers 2^32 - 1 threads
      if (static_cast<int64_t>(groups) * kfac::kPairThreads > UINT32_MAX || rows > INT32_MAX) return KFAC_ERR_UNSUPPORTED;
      break;
    case KFAC_OBJ_BALANCE:
      if (groups < 1) return KFAC_ERR_ARG;
      if (groups > kfac::kBalanceMaxExperts) return KFAC_ERR_UNSUPPORTED;
      if (rows > INT32_MAX) return KFAC_ERR_UNSUPPORTED;
      *bytes = kfac::balance_workspace_bytes(rows, groups);
      return KFAC_OK;
    default: return KFAC_ERR_ARG;
  }
  *bytes = kfac::token_workspace_bytes(objective, rows, groups);
  return KFAC_OK;
}

kfac_status_t kfac_token_logp(const kfac_token_rows_t* rows, void* workspace, size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_rows(rows, false);
  if (s != KFAC_OK) return s;
  s = kfac::check_workspace(workspace, ws_bytes, kfac::token_workspace_bytes(KFAC_OBJ_LOGP, rows->rows, 0));
  if (s != KFAC_OK) return s;
  return kfac::launch_token_logp(*rows, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_policy_loss(const kfac_token_rows_t* rows, const kfac_policy_t* policy, void* workspace,
                               size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_rows(rows, true);
  if (s != KFAC_OK) return s;
  if (!policy || policy->reserved != 0) return KFAC_ERR_ARG;
  if (!(policy->clip_low >= 0.f && policy->clip_low <= 1.f)) return KFAC_ERR_ARG;
  if (!(policy->clip_high >= 0.f) || !std::isfinite(policy->clip_high)) return KFAC_ERR_ARG;
  if (!(policy->kl_coef >= 0.f) || !std::isfinite(policy->kl_coef)) return KFAC_ERR_ARG;
  if (policy->kl_coef > 0.f && !policy->ref_logp && rows->rows > 0) return KFAC_ERR_ARG;
  kfac::Ptrs p;
  p.need(policy->stats, 4);
  if (rows->rows > 0) p.need(policy->advantage, 4);
  p.may(policy->weight, 4);
  p.may(policy->old_logp, 4);
  p.may(policy->ref_logp, 4);
  if (p.s != KFAC_OK) return p.s;
  s = kfac::check_workspace(workspace, ws_bytes, kfac::token_workspace_bytes(KFAC_OBJ_POLICY, rows->rows, 0));
  if (s != KFAC_OK) return s;
  return kfac::launch_policy(*rows, *policy, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_preference_loss(const kfac_token_rows_t* rows, const kfac_preference_t* pref, void* workspace,
                                   size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_rows(rows, true);
  if (s != KFAC_OK) return s;
  if (!pref || pref->reserved != 0) return KFAC_ERR_ARG;
  if (pref->pairs < 1 || (pref->average != 0 && pref->average != 1)) return KFAC_ERR_ARG;
  if (pref->kind != KFAC_PREF_SIGMOID && pref->kind != KFAC_PREF_SQUARED) return KFAC_ERR_ARG;
  if (!(pref->beta > 0.f) || !std::isfinite(pref->beta)) return KFAC_ERR_ARG;
  if (!(pref->label_smoothing >= 0.f && pref->label_smoothing < 0.5f)) return KFAC_ERR_ARG;
  if (pref->kind == KFAC_PREF_SQUARED && pref->label_smoothing != 0.f) return KFAC_ERR_ARG;
  kfac::Ptrs p;
  p.need(pref->offsets, 4);
  p.need(pref->seq, 4);
  p.need(pref->stats, 4);
  p.may(pref->ref_logp, 4);
  p.may(pref->pair_weight, 4);
  if (p.s != KFAC_OK) return p.s;
  size_t need = 0;
  s = kfac_objective_workspace_size(KFAC_OBJ_PREFERENCE, rows->rows, pref->pairs, &need);
  if (s != KFAC_OK) return s;
  s = kfac::check_workspace(workspace, ws_bytes, need);
  if (s != KFAC_OK) return s;
  return kfac::launch_preference(*rows, *pref, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_balance_loss(const kfac_balance_t* b, void* workspace, size_t ws_bytes, void* stream) {
  if (!b || b->reserved != 0) return KFAC_ERR_ARG;
  if (!kfac::dtype_ok(b->dtype) || !kfac::index_ok(b->index_type)) return KFAC_ERR_DTYPE;
  if (b->tokens < 0 || b->experts < 1 || b->top_k < 1 || b->top_k > b->experts) return KFAC_ERR_ARG;
  if (b->experts > kfac::kBalanceMaxExperts) return KFAC_ERR_UNSUPPORTED;
  if (b->ld < b->experts || b->grad_ld < b->experts) return KFAC_ERR_ARG;
  if (b->grad == b->logits && b->grad && b->grad_ld != b->ld) return KFAC_ERR_ARG;
  if (!std::isfinite(b->coef) || !std::isfinite(b->z_coef) || !std::isfinite(b->grad_scale)) return KFAC_ERR_ARG;
  if (!kfac::extent_ok(b->tokens, b->ld) || !kfac::extent_ok(b->tokens, b->grad_ld)) return KFAC_ERR_UNSUPPORTED;
  // counts are 32-bit
  if (b->tokens > INT32_MAX) return KFAC_ERR_UNSUPPORTED;
  kfac::Ptrs p;
  p.need(b->counts, 4);
  p.need(b->prob, 4);
  p.need(b->stats, 4);
  if (b->tokens > 0) {
    p.need(b->logits, kfac::elem_size(b->dtype));
    p.need(b->grad, kfac::elem_size(b->dtype));
    p.need(b->chosen, kfac::index_size(b->index_type));
  }
  if (p.s != KFAC_OK) return p.s;
  kfac_status_t s = kfac::check_workspace(workspace, ws_bytes, kfac::balance_workspace_bytes(b->tokens, b->experts));
  if (s != KFAC_OK) return s;
  return kfac::launch_balance(*b, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_dropout(const kfac_dropout_t* d, void* stream) {
  if (!d || d->reserved != 0) return KFAC_ERR_ARG;
  if (!kfac::dtype_ok(d->dtype)) return KFAC_ERR_DTYPE;
  if (d->rows < 0 || d->cols < 1 || d->ld < d->cols || d->y_ld < d->cols) return KFAC_ERR_ARG;
  if (d->residual && d->residual_ld < d->cols) return KFAC_ERR_ARG;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return KFAC_ERR_ARG;
  if (d->y == d->x && d->y && d->y_ld != d->ld) return KFAC_ERR_ARG;
  if (d->y == d->residual && d->y && d->y_ld != d->residual_ld) return KFAC_ERR_ARG;
  if (!kfac::extent_ok(d->rows, d->ld) || !kfac::extent_ok(d->rows, d->y_ld) ||
      (d->residual && !kfac::extent_ok(d->rows, d->residual_ld)))
    return KFAC_ERR_UNSUPPORTED;
  // one launch covers 2^32 - 1 threads, a thread one generator block of eight columns at least
  if (d->rows > 0 && (d->cols > kfac::kDropoutMaxBlocks * 8 || (d->cols + 7) / 8 > kfac::kDropoutMaxBlocks / d->rows))
    return KFAC_ERR_UNSUPPORTED;
  if (d->rows == 0) return KFAC_OK;
  kfac::Ptrs p;
  p.need(d->x, kfac::elem_size(d->dtype));
  p.need(d->y, kfac::elem_size(d->dtype));
  p.may(d->residual, kfac::elem_size(d->dtype));
  p.may(d->offset_dev, 8);
  if (p.s != KFAC_OK) return p.s;
  return kfac::launch_dropout(*d, static_cast<hipStream_t>(stream));
}

}  // extern "C"
