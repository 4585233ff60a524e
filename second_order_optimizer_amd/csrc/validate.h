// Host-side checks of arguments, shared by the C entry points whose pointers need
// their element's alignment only.
#pragma once

#include "common.h"
#include "../../include/kfac_objectives.h"

namespace kfac {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Pointers that are dereferenced: present, and aligned to their element.
struct Ptrs {
  kfac_status_t s = KFAC_OK;
  void need(const void* p, size_t align) {
    if (s == KFAC_OK && !p) s = KFAC_ERR_ARG;
    else may(p, align);
  }
  void may(const void* p, size_t align) {
    if (s == KFAC_OK && p && !aligned(p, align)) s = KFAC_ERR_ALIGN;
  }
};

inline bool dtype_ok(int32_t d) { return d == KFAC_F32 || d == KFAC_BF16; }
inline size_t elem_size(int32_t d) { return d == KFAC_BF16 ? 2 : 4; }
inline bool index_ok(int32_t t) { return t == KFAC_I32 || t == KFAC_I64; }
inline size_t index_size(int32_t t) { return t == KFAC_I64 ? 8 : 4; }

// rows x ld elements must have byte offsets of at most 62 bits.
inline bool extent_ok(int64_t rows, int64_t ld) { return rows == 0 || ld <= (INT64_MAX / 8) / rows; }

inline kfac_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return KFAC_ERR_WORKSPACE;
  return aligned(ws, 256) ? KFAC_OK : KFAC_ERR_ALIGN;
}

}  // namespace kfac
