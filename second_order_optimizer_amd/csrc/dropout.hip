// Dropout from a counter-based generator (include/kfac_objectives.h): the
// mask is computed where it is needed, forward and backward, and never
// stored.  One thread makes one Philox 4x32-10 block, eight 16-bit draws, for
// eight neighbours of a row: 16 bytes of bf16, 32 of float32.  Bound by HBM:
// x (and the residual) in, y out.
#include "objectives.h"

#include <algorithm>
#include <cmath>

namespace kfac {

namespace {

constexpr int kThreads = 256;
constexpr int kBlockCols = 8;     // draws of one generator block

struct DropArgs {
  const char* x;
  const char* res;
  char* y;
  const int64_t* offset_dev;
  int64_t blocks;            // generator blocks in all
  int64_t ldx, ldr, ldy;     // bytes
  uint64_t offset;
  uint32_t k0, k1;           // key
  uint32_t per_row;          // generator blocks a row
  uint32_t tail;             // columns of a row's last block (1 .. 8)
  uint32_t threshold;
  float scale;
};

// x of eight neighbours as floats, from whole vectors or (n < 8) one by one.
template <typename T, bool NT>
__device__ inline void load8(float (&f)[8], const char* p, int n) {
  if (n == 8) {
    constexpr int VE = Elem<T>::VE;
#pragma unroll
    for (int q = 0; q < 8 / VE; ++q) {
      const u32x4 v = load16<NT>(p + q * 16);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[q * VE + i] = Elem<T>::get(v, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? Elem<T>::load(p, i) : 0.f;
  }
}

template <typename T, bool RES, bool NT, int U>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropArgs a) {
  constexpr int VE = Elem<T>::VE;
  const uint64_t off = a.offset + (a.offset_dev ? static_cast<uint64_t>(*a.offset_dev) : 0);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * U) + threadIdx.x;
  float x[U][8], r[U][8];
  int n[U];
  char* out[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b = first + u * kThreads;
    n[u] = 0;
    if (b < a.blocks) {
      int64_t row;
      uint32_t col;
      if (a.blocks <= UINT32_MAX) {
        const uint32_t q = static_cast<uint32_t>(b) / a.per_row;
        row = q;
        col = static_cast<uint32_t>(b) - q * a.per_row;
      } else {
        row = b / a.per_row;
        col = static_cast<uint32_t>(b - row * a.per_row);
      }
      const int64_t at = static_cast<int64_t>(col) * (kBlockCols * sizeof(T));
      n[u] = col == a.per_row - 1 ? a.tail : kBlockCols;
      load8<T, NT>(x[u], a.x + row * a.ldx + at, n[u]);
      if constexpr (RES) load8<T, NT>(r[u], a.res + row * a.ldr + at, n[u]);
      out[u] = a.y + row * a.ldy + at;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (n[u] == 0) continue;
    const uint64_t b = static_cast<uint64_t>(first + u * kThreads);
    uint32_t c0 = static_cast<uint32_t>(b), c1 = static_cast<uint32_t>(b >> 32);
    uint32_t c2 = static_cast<uint32_t>(off), c3 = static_cast<uint32_t>(off >> 32);
    uint32_t k0 = a.k0, k1 = a.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
      c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
      c1 = static_cast<uint32_t>(p1);
      c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
      c3 = static_cast<uint32_t>(p0);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    const uint32_t c[4] = {c0, c1, c2, c3};
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t draw = (i & 1) ? c[i >> 1] >> 16 : c[i >> 1] & 0xFFFFu;
      o[i] = draw >= a.threshold ? x[u][i] * a.scale : 0.f;
      if constexpr (RES) o[i] += r[u][i];
    }
    if (n[u] == 8) {
#pragma unroll
      for (int q = 0; q < 8 / VE; ++q) store16<NT>(out[u] + q * 16, pack16<T>(o + q * VE));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n[u]) Elem<T>::store(out[u], i, o[i]);
    }
  }
}

template <typename T, bool RES>
void run(const DropArgs& a, hipStream_t st) {
  constexpr int U = 2;
  const int64_t per = static_cast<int64_t>(kThreads) * U;
  const dim3 grid(static_cast<uint32_t>((a.blocks + per - 1) / per));
  const bool nt = a.blocks * static_cast<int64_t>(kBlockCols * sizeof(T)) * (RES ? 3 : 2) > kCacheBytes;
  if (nt) hipLaunchKernelGGL((dropout_kernel<T, RES, true, U>), grid, dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((dropout_kernel<T, RES, false, U>), grid, dim3(kThreads), 0, st, a);
}

}  // namespace

kfac_status_t launch_dropout(const kfac_dropout_t& d, hipStream_t st) {
  if (d.rows == 0) return KFAC_OK;
  const int64_t el = d.dtype == KFAC_BF16 ? 2 : 4;
  DropArgs a{};
  a.x = static_cast<const char*>(d.x);
  a.res = static_cast<const char*>(d.residual);
  a.y = static_cast<char*>(d.y);
  a.offset_dev = d.offset_dev;
  a.per_row = static_cast<uint32_t>((d.cols + kBlockCols - 1) / kBlockCols);
  a.blocks = d.rows * static_cast<int64_t>(a.per_row);
  a.ldx = d.ld * el;
  a.ldr = d.residual_ld * el;
  a.ldy = d.y_ld * el;
  a.offset = d.offset;
  a.k0 = static_cast<uint32_t>(d.seed);
  a.k1 = static_cast<uint32_t>(d.seed >> 32);
  a.tail = static_cast<uint32_t>(d.cols - (static_cast<int64_t>(a.per_row) - 1) * kBlockCols);
  a.threshold = static_cast<uint32_t>(std::nearbyint(d.p * 65536.0));
  a.scale = a.threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - a.threshold)) : 0.f;
  const bool half = d.dtype == KFAC_BF16;
  if (a.res) half ? run<__bf16, true>(a, st) : run<float, true>(a, st);
  else half ? run<__bf16, false>(a, st) : run<float, false>(a, st);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

}  // namespace kfac
