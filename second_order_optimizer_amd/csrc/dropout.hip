// Dropout from a counter-based generator (include/kfac_objectives.h): the
// mask is computed where it is needed, forward and backward, and never
// stored.  One Philox 4x32-10 block is eight 16-bit draws for eight
// neighbours of a row: 16 bytes of bf16, 32 of float32.  Bound by HBM: x (and
// the residual) in, y out.  8192 x 4096 bf16 with its residual 35 us forward, 25
// us backward, 5.6 TB/s together; 16384 x 1025 f32 25 us each way, 5.3 TB/s (a
// copy past the cache: 6.2).  One row: 2.4 us, all of it launch and latency.
#include "objectives.h"

#include <algorithm>
#include <cmath>

namespace kfac {

namespace {

constexpr int kThreads = 256;
constexpr int kBlockCols = 8;     // draws of one generator block
// Passes of more than this go past the cache: 8192 x 4096 bf16 forward with
// residual and backward 69 -> 59 us (U = 4 chunks a thread: 76 -> 62).
constexpr int64_t kStreamBytes = kCacheBytes / 4;

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

// Four words of the generator for one block.
__device__ inline void philox(uint64_t block, uint64_t off, uint32_t k0, uint32_t k1, uint32_t (&c)[4]) {
  c[0] = static_cast<uint32_t>(block);
  c[1] = static_cast<uint32_t>(block >> 32);
  c[2] = static_cast<uint32_t>(off);
  c[3] = static_cast<uint32_t>(off >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c[0], p1 = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
    c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ k0;
    c[1] = static_cast<uint32_t>(p1);
    c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ k1;
    c[3] = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}
__device__ inline uint32_t swap_pair(uint32_t v) { return __builtin_amdgcn_update_dpp(0, v, kXor1, 0xF, 0xF, true); }

// VE neighbours as floats: one vector, or (n < VE) one by one.
template <typename T, bool NT>
__device__ inline void load_some(float (&f)[Elem<T>::VE], const char* p, int n) {
  constexpr int VE = Elem<T>::VE;
  if (n == VE) {
    const u32x4 v = load16<NT>(p);
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = Elem<T>::get(v, i);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = i < n ? Elem<T>::load(p, i) : 0.f;
  }
}

// A thread works on U chunks of 16 bytes.  bf16: a chunk is a generator block.
// float32: a chunk is half of one, and to keep a wavefront's accesses in one
// run the two halves of a block sit in neighbouring lanes; each lane of such a
// pair makes one block for two chunks, 32 blocks apart, and they exchange the
// halves.
template <typename T, bool RES, bool NT, int U>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropArgs a) {
  constexpr int VE = Elem<T>::VE;
  constexpr bool HALVES = VE < kBlockCols;
  constexpr int GROUPS = HALVES ? U / 2 : U;      // generator blocks a thread makes
  const uint64_t off = a.offset + (a.offset_dev ? static_cast<uint64_t>(*a.offset_dev) : 0);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * GROUPS);
  const int lane = threadIdx.x & (kWave - 1), odd = lane & 1;
  const int64_t wave = first + (threadIdx.x & ~(kWave - 1));
  float x[U][VE], r[U][VE];
  int n[U];
  char* out[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b = HALVES ? wave + (u / 2) * kThreads + (u & 1) * 32 + (lane >> 1) : first + u * kThreads + threadIdx.x;
    n[u] = 0;
    if (b < a.blocks) {
      const uint32_t q = static_cast<uint32_t>(b) / a.per_row;      // at most kDropoutMaxBlocks in all
      const uint32_t col = static_cast<uint32_t>(b) - q * a.per_row;
      const int64_t row = q;
      const int lead = HALVES ? odd * VE : 0;
      const int64_t at = (static_cast<int64_t>(col) * kBlockCols + lead) * static_cast<int64_t>(sizeof(T));
      n[u] = col == a.per_row - 1 ? max(0, min(VE, static_cast<int>(a.tail) - lead)) : VE;
      load_some<T, NT>(x[u], a.x + row * a.ldx + at, n[u]);
      if constexpr (RES) load_some<T, NT>(r[u], a.res + row * a.ldr + at, n[u]);
      out[u] = a.y + row * a.ldy + at;
    }
  }
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) {
    uint32_t c[4];
    const int64_t b = HALVES ? wave + k * kThreads + odd * 32 + (lane >> 1) : first + k * kThreads + threadIdx.x;
    philox(static_cast<uint64_t>(b), off, a.k0, a.k1, c);
    uint32_t words[HALVES ? 2 : 1][VE / 2];       // the draws of this group's chunks
    if constexpr (HALVES) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t own = odd ? c[2 + i] : c[i];
        const uint32_t got = swap_pair(odd ? c[i] : c[2 + i]);
        words[0][i] = odd ? got : own;
        words[1][i] = odd ? own : got;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) words[0][i] = c[i];
    }
#pragma unroll
    for (int h = 0; h < (HALVES ? 2 : 1); ++h) {
      const int u = HALVES ? 2 * k + h : k;
      if (n[u] == 0) continue;
      float o[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const uint32_t draw = (i & 1) ? words[h][i >> 1] >> 16 : words[h][i >> 1] & 0xFFFFu;
        o[i] = draw >= a.threshold ? x[u][i] * a.scale : 0.f;
        if constexpr (RES) o[i] += r[u][i];
      }
      if (n[u] == VE) {
        store16<NT>(out[u], pack16<T>(o));
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (i < n[u]) Elem<T>::store(out[u], i, o[i]);
      }
    }
  }
}

template <typename T, bool RES>
void run(const DropArgs& a, hipStream_t st) {
  constexpr int U = 2;
  const int64_t per = static_cast<int64_t>(kThreads) * U * Elem<T>::VE / kBlockCols;
  const dim3 grid(static_cast<uint32_t>((a.blocks + per - 1) / per));
  const bool nt = a.blocks * static_cast<int64_t>(kBlockCols * sizeof(T)) * (RES ? 3 : 2) > kStreamBytes;
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
