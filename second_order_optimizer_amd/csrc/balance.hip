// Router balance loss (include/kfac_objectives.h): softmax of each token's
// logits over E experts, per-expert counts and mean probabilities, the
// balance and z losses and the gradient of every logit.
//
// The gradient needs the counts of all tokens, so there are two passes over
// the logits (the second finds them in the caches: at most some tens of MB)
// with a small reduction between them:
//   balance_count_kernel   column sums of p, histogram of the chosen experts
//                          and sum of log-sum-exp^2 per workgroup;
//   balance_reduce_kernel  their sums in a fixed order;
//   balance_grad_kernel    with f[e] = coef E counts[e] / (top_k n^2),
//                          g = p (f - sum p f) + p 2 z_coef / n lse.
//
// A token's E logits sit in LPT neighbouring lanes, one 16-byte vector a lane
// (NV vectors for E beyond 64 lanes), 64 / LPT tokens in a wavefront.  Where E
// is not a multiple of a vector, the row's last lane takes the last whole
// vector of the row instead and leaves the columns its neighbour already has
// out of the sums; both compute the same gradient there.  E below a vector:
// one element a lane.
#include "objectives.h"

#include <algorithm>

namespace kfac {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

struct BalArgs {
  const char* x;
  char* g;
  const void* chosen;
  const uint8_t* mask;
  int64_t tokens;
  int64_t ldx, ldg;      // bytes
  int32_t E, k, index_type;
  int32_t blocks;        // workgroups of the counting pass
  float coef, z, grad_scale;
  int32_t* counts;
  float* prob;
  float* stats;
  uint32_t* flags;
  float* part_p;         // [blocks][E]
  int32_t* part_c;       // [blocks][E]
  double* part_z;        // [blocks]
  int32_t* part_n;       // [blocks]
  double* prob64;        // [E]
  double* total;         // [2]: n, sum of lse^2
};

// Maximum / sum over the LPT lanes of a token; every lane gets it.
template <int LPT, bool MAX>
__device__ inline float group_reduce(float v) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  if constexpr (LPT >= 2) v = op(v, dpp<kXor1>(v));
  if constexpr (LPT >= 4) v = op(v, dpp<kXor2>(v));
  if constexpr (LPT >= 8) v = op(v, dpp<kHalfMirror>(v));
  if constexpr (LPT >= 16) v = op(v, dpp<kMirror>(v));
  if constexpr (LPT >= 32) v = op(v, __shfl_xor(v, 16, kWave));
  if constexpr (LPT >= 64) v = op(v, __shfl_xor(v, 32, kWave));
  return v;
}

// Where a lane's vectors lie in a row, and how many of their first columns
// belong to the lane before (VEC: the lane has nothing there).
template <int VEC, int LPT, int NV>
struct Columns {
  int col[NV], skip[NV];
  __device__ Columns(int lane, int E) {
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int b = (q * LPT + lane) * VEC;
      col[q] = b;
      skip[q] = 0;
      if (b >= E) {
        col[q] = 0;
        skip[q] = VEC;
      } else if (b + VEC > E) {
        col[q] = E - VEC;
        skip[q] = b - col[q];
      }
    }
  }
};

template <typename T, int VEC, int LPT, int NV>
struct Token {
  float p[NV][VEC];      // softmax of the lane's columns
  float lse;

  // p and log-sum-exp of one token; lanes past the row hold p = 0.
  __device__ void softmax(const float (&x)[NV][VEC], const Columns<VEC, LPT, NV>& cols) {
    constexpr float kLog2e = 1.4426950408889634f;
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) m = fmaxf(m, x[q][i]);
    m = group_reduce<LPT, true>(m);
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        p[q][i] = __builtin_amdgcn_exp2f((x[q][i] - m) * kLog2e);
        s += i >= cols.skip[q] ? p[q][i] : 0.f;
      }
    s = group_reduce<LPT, false>(s);
    const float inv = 1.f / s;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[q][i] *= inv;
    lse = m + logf(s);
  }
};

template <typename T, int VEC, int LPT, int NV>
__device__ inline void load_token(float (&x)[NV][VEC], const BalArgs& a, int64_t t, const Columns<VEC, LPT, NV>& cols) {
  const char* row = a.x + t * a.ldx;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    if (cols.skip[q] < VEC) {
      if constexpr (VEC == 1) {
        x[q][0] = Elem<T>::load(row, cols.col[q]);
      } else {
        const u32x4 v = load16(row + static_cast<int64_t>(cols.col[q]) * sizeof(T));
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[q][i] = Elem<T>::get(v, i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[q][i] = -INFINITY;
    }
  }
}

__device__ inline bool token_live(const BalArgs& a, int64_t t) {
  return t < a.tokens && (!a.mask || a.mask[t] != 0);
}

template <typename T, int VEC, int LPT, int NV>
__global__ void __launch_bounds__(kThreads) balance_count_kernel(BalArgs a) {
  constexpr int SLOTS = kWave / LPT, W = LPT * NV * VEC;   // tokens a wavefront, columns a row at most
  __shared__ int hist[kBalanceMaxExperts];
  __shared__ float psum[kWaves][W];
  __shared__ double zred[kWaves];
  __shared__ int nred[kWaves];
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const int slot = lane / LPT, sub = lane % LPT;
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  __syncthreads();
  const Columns<VEC, LPT, NV> cols(sub, a.E);

  float acc[NV][VEC] = {};
  double z = 0.0;
  int n = 0;
  const int64_t per = static_cast<int64_t>(kWaves) * SLOTS;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  for (int64_t t0 = blockIdx.x * per; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + wid * SLOTS + slot;
    const bool live = token_live(a, t);
    float x[NV][VEC];
    if (live) {
      load_token<T, VEC, LPT, NV>(x, a, t, cols);
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[q][i] = 0.f;
    }
    Token<T, VEC, LPT, NV> k;
    k.softmax(x, cols);
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[q][i] += live && i >= cols.skip[q] ? k.p[q][i] : 0.f;
    if (live && sub == 0) {
      z += static_cast<double>(k.lse) * static_cast<double>(k.lse);
      ++n;
    }
  }
  // the chosen experts: integer counts, in any order
  const int64_t slots = a.tokens * a.k;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < slots;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t t = slots <= INT32_MAX ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.k))
                                         : i / a.k;
    if (!token_live(a, t)) continue;
    const int64_t e = load_index(a.chosen, i, a.index_type);
    if (e >= a.E) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    else if (e >= 0) atomicAdd(&hist[e], 1);
  }
  // column sums of the wavefront (over its slots), then of the workgroup
#pragma unroll
  for (int q = 0; q < NV; ++q)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = acc[q][i];
#pragma unroll
      for (int off = LPT; off < kWave; off *= 2) s += __shfl_xor(s, off, kWave);
      // columns that the lane before has are its to write
      if (slot == 0 && i >= cols.skip[q]) psum[wid][cols.col[q] + i] = s;
    }
  z = wave_sum(z);
  for (int off = 1; off < kWave; off *= 2) n += __shfl_xor(n, off, kWave);
  if (lane == 0) {
    zred[wid] = z;
    nred[wid] = n;
  }
  __syncthreads();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float s = 0.f;
    for (int w = 0; w < kWaves; ++w) s += psum[w][e];
    a.part_p[at + e] = s;
    a.part_c[at + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
    int c = 0;
    for (int w = 0; w < kWaves; ++w) {
      s += zred[w];
      c += nred[w];
    }
    a.part_z[blockIdx.x] = s;
    a.part_n[blockIdx.x] = c;
  }
}

// 16 experts a workgroup, 16 threads an expert.
__global__ void __launch_bounds__(256) balance_reduce_kernel(BalArgs a) {
  __shared__ double ps[16][16];
  __shared__ int cs[16][16];
  __shared__ double zr[4], nr[4];
  double z = 0.0, n = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += 256) {
    z += a.part_z[i];
    n += a.part_n[i];
  }
  z = wave_sum(z);
  n = wave_sum(n);
  const int wid = threadIdx.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == 0) {
    zr[wid] = z;
    nr[wid] = n;
  }
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, e = blockIdx.x * 16 + col;
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
    for (int b = grp; b < a.blocks; b += 16) {
      p += a.part_p[static_cast<int64_t>(b) * a.E + e];
      c += a.part_c[static_cast<int64_t>(b) * a.E + e];
    }
  }
  ps[grp][col] = p;
  cs[grp][col] = c;
  __syncthreads();
  n = (nr[0] + nr[1]) + (nr[2] + nr[3]);
  if (threadIdx.x < 16 && e < a.E) {
    double s = 0.0;
    int t = 0;
    for (int g = 0; g < 16; ++g) {
      s += ps[g][col];
      t += cs[g][col];
    }
    s /= fmax(n, 1.0);
    a.prob[e] = static_cast<float>(s);
    a.prob64[e] = s;
    a.counts[e] = t;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.total[0] = n;
    a.total[1] = (zr[0] + zr[1]) + (zr[2] + zr[3]);
  }
}

template <typename T, int VEC, int LPT, int NV>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(BalArgs a) {
  constexpr int SLOTS = kWave / LPT;
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const int slot = lane / LPT, sub = lane % LPT;
  const Columns<VEC, LPT, NV> cols(sub, a.E);
  const double live_n = a.total[0], n = fmax(live_n, 1.0);
  const double per_count = static_cast<double>(a.coef) * a.E / (static_cast<double>(a.k) * n);
  if (blockIdx.x == 0 && wid == 0) {
    double s = 0.0;
    for (int e = lane; e < a.E; e += kWave) s += a.counts[e] * a.prob64[e];
    s = wave_sum(s) * per_count;
    if (lane == 0) {
      const double z = static_cast<double>(a.z) * a.total[1] / n;
      a.stats[0] = static_cast<float>(s + z);
      a.stats[1] = static_cast<float>(s);
      a.stats[2] = static_cast<float>(z);
      a.stats[3] = static_cast<float>(live_n);
      if (!(fabs(s + z) < INFINITY)) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
    }
  }
  const double unit = per_count / n * a.grad_scale;
  const float zs = static_cast<float>(2.0 * a.z / n * a.grad_scale);
  float f[NV][VEC];
#pragma unroll
  for (int q = 0; q < NV; ++q)
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      f[q][i] = cols.skip[q] < VEC ? static_cast<float>(unit * a.counts[cols.col[q] + i]) : 0.f;

  const int64_t per = static_cast<int64_t>(kWaves) * SLOTS;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * per;
  for (int64_t t0 = blockIdx.x * per; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + wid * SLOTS + slot;
    const bool live = token_live(a, t);
    float x[NV][VEC];
    if (live) {
      load_token<T, VEC, LPT, NV>(x, a, t, cols);
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[q][i] = 0.f;
    }
    Token<T, VEC, LPT, NV> k;
    k.softmax(x, cols);
    float pf = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) pf += i >= cols.skip[q] ? k.p[q][i] * f[q][i] : 0.f;
    pf = group_reduce<LPT, false>(pf);
    const float zt = zs != 0.f ? zs * k.lse : 0.f;
    if (t < a.tokens) {
      char* row = a.g + t * a.ldg;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        if (cols.skip[q] < VEC) {
          float g[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] = live ? k.p[q][i] * (f[q][i] - pf) + k.p[q][i] * zt : 0.f;
          if constexpr (VEC == 1) Elem<T>::store(row, cols.col[q], g[0]);
          else store16(row + static_cast<int64_t>(cols.col[q]) * sizeof(T), pack16<T>(g));
        }
      }
    }
  }
}

template <typename T, int VEC, int LPT, int NV>
kfac_status_t run(BalArgs a, hipStream_t st) {
  const int64_t per = static_cast<int64_t>(kWaves) * (kWave / LPT);
  const int64_t need = std::max<int64_t>(1, (a.tokens + per - 1) / per);
  a.blocks = static_cast<int32_t>(std::min<int64_t>(need, kBalanceBlocks));
  hipLaunchKernelGGL((balance_count_kernel<T, VEC, LPT, NV>), dim3(a.blocks), dim3(kThreads), 0, st, a);
  KFAC_HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL(balance_reduce_kernel, dim3((a.E + 15) / 16), dim3(256), 0, st, a);
  KFAC_HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL((balance_grad_kernel<T, VEC, LPT, NV>), dim3(static_cast<int>(std::min<int64_t>(need, 1024))),
                     dim3(kThreads), 0, st, a);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

// Lanes a token by its number of vectors.
template <typename T>
kfac_status_t pick(const BalArgs& a, hipStream_t st) {
  constexpr int VE = Elem<T>::VE;
  if (a.E < VE) return run<T, 1, VE, 1>(a, st);
  const int nvec = (a.E + VE - 1) / VE;
  if (nvec <= 1) return run<T, VE, 1, 1>(a, st);
  if (nvec <= 2) return run<T, VE, 2, 1>(a, st);
  if (nvec <= 4) return run<T, VE, 4, 1>(a, st);
  if (nvec <= 8) return run<T, VE, 8, 1>(a, st);
  if (nvec <= 16) return run<T, VE, 16, 1>(a, st);
  if (nvec <= 32) return run<T, VE, 32, 1>(a, st);
  if (nvec <= 64) return run<T, VE, 64, 1>(a, st);
  if (nvec <= 128) return run<T, VE, 64, 2>(a, st);
  if constexpr (VE == 4) return run<T, VE, 64, 4>(a, st);
  return KFAC_ERR_UNSUPPORTED;
}

struct Regions {
  size_t p, c, z, n, prob, total, end;
};
Regions regions(int32_t E) {
  Regions r;
  r.p = kFlagBytes;
  r.c = r.p + align_up(sizeof(float) * kBalanceBlocks * static_cast<size_t>(E), 256);
  r.z = r.c + align_up(sizeof(int32_t) * kBalanceBlocks * static_cast<size_t>(E), 256);
  r.n = r.z + align_up(sizeof(double) * kBalanceBlocks, 256);
  r.prob = r.n + align_up(sizeof(int32_t) * kBalanceBlocks, 256);
  r.total = r.prob + align_up(sizeof(double) * static_cast<size_t>(E), 256);
  r.end = r.total + 256;
  return r;
}

}  // namespace

size_t balance_workspace_bytes(int32_t experts) { return regions(experts).end; }

kfac_status_t launch_balance(const kfac_balance_t& b, char* ws, hipStream_t st) {
  const Regions r = regions(b.experts);
  const int64_t el = b.dtype == KFAC_BF16 ? 2 : 4;
  BalArgs a{};
  a.x = static_cast<const char*>(b.logits);
  a.g = static_cast<char*>(b.grad);
  a.chosen = b.chosen;
  a.mask = b.mask;
  a.tokens = b.tokens;
  a.ldx = b.ld * el;
  a.ldg = b.grad_ld * el;
  a.E = b.experts;
  a.k = b.top_k;
  a.index_type = b.index_type;
  a.coef = b.coef;
  a.z = b.z_coef;
  a.grad_scale = b.grad_scale;
  a.counts = b.counts;
  a.prob = b.prob;
  a.stats = b.stats;
  a.flags = reinterpret_cast<uint32_t*>(ws);
  a.part_p = reinterpret_cast<float*>(ws + r.p);
  a.part_c = reinterpret_cast<int32_t*>(ws + r.c);
  a.part_z = reinterpret_cast<double*>(ws + r.z);
  a.part_n = reinterpret_cast<int32_t*>(ws + r.n);
  a.prob64 = reinterpret_cast<double*>(ws + r.prob);
  a.total = reinterpret_cast<double*>(ws + r.total);
  return b.dtype == KFAC_BF16 ? pick<__bf16>(a, st) : pick<float>(a, st);
}

}  // namespace kfac
