// The extern "C" entry points of include/kfac_tokens.h: host-side validation
// and dispatch.
#include "overlap.h"
#include "tokens.h"
#include "validate.h"

#include <cmath>

namespace kfac {

namespace {

kfac_status_t check_embedding(const kfac_embedding_t* e) {
  if (!e || e->reserved != 0 || (e->accumulate != 0 && e->accumulate != 1)) return KFAC_ERR_ARG;
  if (!dtype_ok(e->dtype) || !dtype_ok(e->table_dtype) || !index_ok(e->id_type)) return KFAC_ERR_DTYPE;
  if (e->tokens < 0 || e->vocab < 1 || e->width < 1 || e->table_ld < e->width || e->y_ld < e->width) return KFAC_ERR_ARG;
  if (!std::isfinite(e->scale)) return KFAC_ERR_ARG;
  if (e->vocab > kEmbeddingMaxVocab || e->width > kEmbeddingMaxWidth || e->tokens > kEmbeddingMaxTokens) return KFAC_ERR_UNSUPPORTED;
  if (!extent_ok(e->vocab, e->table_ld) || !extent_ok(e->tokens, e->y_ld)) return KFAC_ERR_UNSUPPORTED;
  return KFAC_OK;
}

Lines table_lines(const kfac_embedding_t* e) {
  const int64_t el = elem_size(e->table_dtype);
  return lines_of(e->table, e->width * el, e->vocab, e->table_ld * el);
}
Lines row_lines(const kfac_embedding_t* e) {
  const int64_t el = elem_size(e->dtype);
  return lines_of(e->y, e->width * el, e->tokens, e->y_ld * el);
}
Lines id_lines(const kfac_embedding_t* e) { return lines_of(e->ids, e->tokens * static_cast<int64_t>(index_size(e->id_type))); }

}  // namespace
}  // namespace kfac

extern "C" {

kfac_status_t kfac_token_workspace_size(int32_t op, int64_t rows, int32_t vocab, int32_t width, size_t* bytes) {
  if (!bytes || rows < 0 || vocab < 1) return KFAC_ERR_ARG;
  switch (op) {
    case KFAC_TOK_SAMPLE:
      if (vocab > kfac::kSampleMaxVocab) return KFAC_ERR_UNSUPPORTED;
      *bytes = kfac::sample_workspace_bytes(rows, vocab);
      return KFAC_OK;
    case KFAC_TOK_EMBEDDING:
      if (width < 1) return KFAC_ERR_ARG;
      if (vocab > kfac::kEmbeddingMaxVocab || width > kfac::kEmbeddingMaxWidth || rows > kfac::kEmbeddingMaxTokens)
        return KFAC_ERR_UNSUPPORTED;
      *bytes = kfac::embedding_workspace_bytes(rows, vocab, width);
      return KFAC_OK;
    default: return KFAC_ERR_ARG;
  }
}

kfac_status_t kfac_sample_tokens(const kfac_sample_t* s, void* workspace, size_t ws_bytes, void* stream) {
  if (!s || s->reserved != 0) return KFAC_ERR_ARG;
  if (!kfac::dtype_ok(s->dtype)) return KFAC_ERR_DTYPE;
  if (s->rows < 0 || s->vocab < 1 || s->ld < s->vocab || s->top_k < 0) return KFAC_ERR_ARG;
  if (!(s->temperature >= 0.0) || !std::isfinite(s->temperature)) return KFAC_ERR_ARG;
  if (!(s->top_p >= 0.0 && s->top_p <= 1.0) || !(s->min_p >= 0.0 && s->min_p <= 1.0)) return KFAC_ERR_ARG;
  if (s->vocab > kfac::kSampleMaxVocab || !kfac::extent_ok(s->rows, s->ld)) return KFAC_ERR_UNSUPPORTED;
  if (s->rows > 0) {
    kfac::Ptrs p;
    p.need(s->logits, kfac::elem_size(s->dtype));
    p.need(s->u, 4);
    p.may(s->row_temperature, 4);
    p.may(s->row_top_k, 4);
    p.may(s->row_top_p, 4);
    p.may(s->row_min_p, 4);
    p.need(s->token, 8);
    p.need(s->logp, 4);
    p.need(s->kept, 4);
    if (p.s != KFAC_OK) return p.s;
  }
  const kfac_status_t st = kfac::check_workspace(workspace, ws_bytes, kfac::sample_workspace_bytes(s->rows, s->vocab));
  if (st != KFAC_OK) return st;
  return kfac::launch_sample(*s, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_embedding_lookup(const kfac_embedding_t* e, void* workspace, size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_embedding(e);
  if (s != KFAC_OK) return s;
  if (e->tokens > 0) {
    kfac::Ptrs p;
    p.need(e->table, kfac::elem_size(e->table_dtype));
    p.need(e->y, kfac::elem_size(e->dtype));
    p.need(e->ids, kfac::index_size(e->id_type));
    if (p.s != KFAC_OK) return p.s;
  }
  s = kfac::check_workspace(workspace, ws_bytes, kfac::kRegions);
  if (s != KFAC_OK) return s;
  if (kfac::overlap(kfac::row_lines(e), kfac::table_lines(e)) || kfac::overlap(kfac::row_lines(e), kfac::id_lines(e))) return KFAC_ERR_ARG;
  return kfac::launch_embedding_lookup(*e, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

kfac_status_t kfac_embedding_grad(const kfac_embedding_t* e, void* workspace, size_t ws_bytes, void* stream) {
  kfac_status_t s = kfac::check_embedding(e);
  if (s != KFAC_OK) return s;
  kfac::Ptrs p;
  p.need(e->table, kfac::elem_size(e->table_dtype));
  p.may(e->counts, 4);
  if (e->tokens > 0) {
    p.need(e->y, kfac::elem_size(e->dtype));
    p.need(e->ids, kfac::index_size(e->id_type));
  }
  if (p.s != KFAC_OK) return p.s;
  s = kfac::check_workspace(workspace, ws_bytes, kfac::embedding_workspace_bytes(e->tokens, e->vocab, e->width));
  if (s != KFAC_OK) return s;
  const kfac::Lines table = kfac::table_lines(e), counts = kfac::lines_of(e->counts, e->counts ? 4 * static_cast<int64_t>(e->vocab) : 0);
  for (const kfac::Lines& read : {kfac::row_lines(e), kfac::id_lines(e)})
    if (kfac::overlap(table, read) || kfac::overlap(counts, read)) return KFAC_ERR_ARG;
  if (kfac::overlap(table, counts)) return KFAC_ERR_ARG;
  return kfac::launch_embedding_grad(*e, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

}  // extern "C"
