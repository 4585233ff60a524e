// Loads shared by the orthogonalisation kernels.
#pragma once

#include "objectives.h"
#include "orthogonal.h"

namespace kfac {

// 8 values of a row from column c on, those past its `cols` columns 0.
__device__ inline void load8(float (&f)[8], const void* row, int c, int cols, int bf16) {
  if (c + 8 <= cols) {
    if (bf16) {
      const u32x4 v = load16(static_cast<const unsigned short*>(row) + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = Elem<__bf16>::get(v, e);
    } else {
      const u32x4 v0 = load16(static_cast<const float*>(row) + c), v1 = load16(static_cast<const float*>(row) + c + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(e < 4 ? v0[e & 3] : v1[e & 3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[e] = c + e >= cols ? 0.f
             : bf16        ? bf16_bits_to_float(static_cast<const unsigned short*>(row)[c + e])
                           : static_cast<const float*>(row)[c + e];
  }
}

}  // namespace kfac
