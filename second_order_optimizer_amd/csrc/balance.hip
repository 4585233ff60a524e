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
//                          g = p (f + 2 z_coef / n lse - sum p f).
// A few tokens (kSmallRounds rounds of one workgroup) take all of it in one
// launch, balance_small_kernel.
//
// A token's E logits sit in LPT neighbouring lanes, one 16-byte vector a lane
// (NV vectors for E beyond 64 lanes), 64 / LPT tokens in a wavefront.  Where E
// is not a multiple of a vector (!EVEN), the row's last lane takes the last
// whole vector of the row instead and leaves the columns its neighbour already
// has out of the sums; both compute the same gradient there.  E below a vector:
// one element a lane.
//
// Bound by vector arithmetic and the lane reductions, not by memory: some 14
// operations an element and pass, the exponential counting four.
#include "objectives.h"

#include <algorithm>

namespace kfac {

namespace {

constexpr int kThreads = 512;
constexpr int kSmallThreads = 1024;
constexpr int kSmallRounds = 8;
constexpr float kLog2e = 1.4426950408889634f;

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

// Sum (maximum) over the LPT lanes of a token; every lane gets it.
template <int LPT, bool MAX>
__device__ inline float group_reduce(float v) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  if constexpr (LPT >= 2) v = op(v, dpp<kXor1>(v));
  if constexpr (LPT >= 4) v = op(v, dpp<kXor2>(v));
  if constexpr (LPT >= 8) v = op(v, dpp<kHalfMirror>(v));
  if constexpr (LPT >= 16) v = op(v, dpp<kMirror>(v));
  if constexpr (LPT >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LPT >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

// Lanes LPT apart, summed.
template <int LPT, typename V>
__device__ inline V slot_sum(V v) {
#pragma unroll
  for (int off = LPT; off < kWave; off *= 2) v += __shfl_xor(v, off, kWave);
  return v;
}

// One shape of the operator: element type, elements a vector, lanes a token,
// vectors a lane, whether E is a whole number of vectors.
template <typename T_, int VEC_, int LPT_, int NV_, bool EVEN_>
struct Shape {
  using T = T_;
  static constexpr int VEC = VEC_, LPT = LPT_, NV = NV_;
  static constexpr bool EVEN = EVEN_;
  static constexpr int SLOTS = kWave / LPT;      // tokens a wavefront
  static constexpr int W = LPT * NV * VEC;       // columns at most
  static constexpr int U = NV == 1 ? 2 : 1;      // tokens a lane works on at once
};

// Where a lane's vectors lie in a row, and how many of their first columns
// belong to the lane before (VEC: the lane has nothing there).
template <typename S>
struct Columns {
  int col[S::NV], skip[S::NV];
  __device__ Columns(int sub, int E) {
#pragma unroll
    for (int q = 0; q < S::NV; ++q) {
      const int b = (q * S::LPT + sub) * S::VEC;
      col[q] = b;
      skip[q] = 0;
      if (b >= E) {
        col[q] = 0;
        skip[q] = S::VEC;
      } else if (b + S::VEC > E) {
        col[q] = E - S::VEC;
        skip[q] = b - col[q];
      }
    }
  }
};

__device__ inline bool token_live(const BalArgs& a, int64_t t) {
  return t < a.tokens && (!a.mask || a.mask[t] != 0);
}

// A token's logits (zeros for one that does not count: it is not looked at),
// minus infinity past the row.
template <typename S>
__device__ inline void load_token(float (&x)[S::NV][S::VEC], const BalArgs& a, int64_t t, bool live,
                                  const Columns<S>& cols) {
  using T = typename S::T;
  const char* row = a.x + t * a.ldx;
#pragma unroll
  for (int q = 0; q < S::NV; ++q) {
#pragma unroll
    for (int i = 0; i < S::VEC; ++i) x[q][i] = live ? -INFINITY : 0.f;
    if (live && cols.skip[q] < S::VEC) {
      if constexpr (S::VEC == 1) {
        x[q][0] = Elem<T>::load(row, cols.col[q]);
      } else {
        const u32x4 v = load16(row + static_cast<int64_t>(cols.col[q]) * sizeof(T));
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) x[q][i] = Elem<T>::get(v, i);
      }
    }
  }
}

template <typename S>
__device__ inline float row_maximum(const float (&x)[S::NV][S::VEC]) {
  float m = x[0][0];
#pragma unroll
  for (int q = 0; q < S::NV; ++q)
#pragma unroll
    for (int i = q == 0 ? 1 : 0; i < S::VEC; i += 2)
      m = max3(m, x[q][i], x[q][i + 1 < S::VEC ? i + 1 : i]);
  return group_reduce<S::LPT, true>(m);
}

// First pass over a wavefront's tokens t0 + slot, t0 + stride + slot, ...:
// adds p to the lane's columns, lse^2 and the tokens that count (in a token's
// first lane).
template <typename S>
__device__ inline void count_tokens(const BalArgs& a, const Columns<S>& cols, int64_t t0, int64_t stride,
                                    float (&acc)[S::NV][S::VEC], double& z, int& n) {
  constexpr int U = S::U;
  const int lane = threadIdx.x & (kWave - 1), slot = lane / S::LPT, sub = lane % S::LPT;
  for (; t0 < a.tokens; t0 += stride * U) {
    float x[U][S::NV][S::VEC];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * stride + slot;
      live[u] = token_live(a, t);
      load_token<S>(x[u], a, t, live[u], cols);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!S::EVEN) {
#pragma unroll
        for (int q = 0; q < S::NV; ++q)
#pragma unroll
          for (int i = 0; i < S::VEC; ++i) x[u][q][i] = i < cols.skip[q] ? -INFINITY : x[u][q][i];
      }
      const float m = row_maximum<S>(x[u]);
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < S::NV; ++q)
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) {
          x[u][q][i] = __builtin_amdgcn_exp2f((x[u][q][i] - m) * kLog2e);
          s += x[u][q][i];
        }
      s = group_reduce<S::LPT, false>(s);
      const float inv = live[u] ? 1.f / s : 0.f;
#pragma unroll
      for (int q = 0; q < S::NV; ++q)
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) acc[q][i] = fmaf(x[u][q][i], inv, acc[q][i]);
      const bool first = live[u] && sub == 0;
      const float lse = first ? m + logf(s) : 0.f;
      z += static_cast<double>(lse) * static_cast<double>(lse);
      n += first;
    }
  }
}

// Histogram of the chosen experts, from thread `first` of `threads`: integer
// counts, in any order.
__device__ inline void count_chosen(const BalArgs& a, int* hist, int64_t first, int64_t threads) {
  const int64_t slots = a.tokens * a.k;
  for (int64_t i = first; i < slots; i += threads) {
    const int64_t t = slots <= INT32_MAX ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.k))
                                         : i / a.k;
    if (!token_live(a, t)) continue;
    const int64_t e = load_index(a.chosen, i, a.index_type);
    if (e >= a.E) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    else if (e >= 0) atomicAdd(&hist[e], 1);
  }
}

// A wavefront's column sums, over its slots, into psum[0 .. E): each column
// from the lane it belongs to.
template <typename S>
__device__ inline void column_sums(const Columns<S>& cols, const float (&acc)[S::NV][S::VEC], float* psum) {
  const int slot = (threadIdx.x & (kWave - 1)) / S::LPT;
#pragma unroll
  for (int q = 0; q < S::NV; ++q)
#pragma unroll
    for (int i = 0; i < S::VEC; ++i) {
      const float s = slot_sum<S::LPT>(acc[q][i]);
      if (slot == 0 && i >= cols.skip[q]) psum[cols.col[q] + i] = s;
    }
}

// Second pass: the gradients, from f of the lane's columns and zs = 2 z_coef /
// n (both times grad_scale).
template <typename S>
__device__ inline void grad_tokens(const BalArgs& a, const Columns<S>& cols, int64_t t0, int64_t stride,
                                   const float (&f)[S::NV][S::VEC], float zs) {
  using T = typename S::T;
  constexpr int U = S::U;
  const int slot = (threadIdx.x & (kWave - 1)) / S::LPT;
  for (; t0 < a.tokens; t0 += stride * U) {
    float x[U][S::NV][S::VEC];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * stride + slot;
      live[u] = token_live(a, t);
      load_token<S>(x[u], a, t, live[u], cols);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * stride + slot;
      const float m = row_maximum<S>(x[u]);
      float s = 0.f, pf = 0.f;
#pragma unroll
      for (int q = 0; q < S::NV; ++q)
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) {
          x[u][q][i] = __builtin_amdgcn_exp2f((x[u][q][i] - m) * kLog2e);
          const float e = S::EVEN || i >= cols.skip[q] ? x[u][q][i] : 0.f;
          s += e;
          pf = fmaf(e, f[q][i], pf);
        }
      s = group_reduce<S::LPT, false>(s);
      pf = group_reduce<S::LPT, false>(pf);
      const float inv = live[u] ? 1.f / s : 0.f;
      const float shift = (zs != 0.f ? zs * (m + logf(s)) : 0.f) - pf * inv;
      if (t < a.tokens) {
        char* row = a.g + t * a.ldg;
#pragma unroll
        for (int q = 0; q < S::NV; ++q) {
          if (cols.skip[q] < S::VEC) {
            float g[S::VEC];
#pragma unroll
            for (int i = 0; i < S::VEC; ++i) g[i] = x[u][q][i] * inv * (f[q][i] + shift);
            if constexpr (S::VEC == 1) Elem<T>::store(row, cols.col[q], g[0]);
            else store16(row + static_cast<int64_t>(cols.col[q]) * sizeof(T), pack16<T>(g));
          }
        }
      }
    }
  }
}

// Factors of a count in f and of lse in the gradient, and the statistics.
struct Scales {
  double n, per_count;
  __device__ Scales(const BalArgs& a, double live) {
    n = fmax(live, 1.0);
    per_count = static_cast<double>(a.coef) * a.E / (static_cast<double>(a.k) * n);
  }
  __device__ double unit(const BalArgs& a) const { return per_count / n * a.grad_scale; }
  __device__ float zs(const BalArgs& a) const { return static_cast<float>(2.0 * a.z / n * a.grad_scale); }
  // dot = sum_e counts[e] prob[e], sq = sum of lse^2
  __device__ void write(const BalArgs& a, double dot, double sq, double live) const {
    const double balance = dot * per_count, z = a.z != 0.f ? static_cast<double>(a.z) * sq / n : 0.0;
    a.stats[0] = static_cast<float>(balance + z);
    a.stats[1] = static_cast<float>(balance);
    a.stats[2] = static_cast<float>(z);
    a.stats[3] = static_cast<float>(live);
    if (!(fabs(balance + z) < INFINITY)) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
  }
};

template <typename S, int THREADS>
struct CountShared {
  static constexpr int WAVES = THREADS / kWave;
  int hist[S::W];
  float psum[WAVES][S::W];
  double z[WAVES];
  int n[WAVES];

  // Everything of the first pass for this workgroup: hist, psum, z and n.
  __device__ void count(const BalArgs& a, const Columns<S>& cols, int block, int blocks) {
    const int wid = threadIdx.x / kWave;
    for (int e = threadIdx.x; e < a.E; e += THREADS) hist[e] = 0;
    __syncthreads();
    float acc[S::NV][S::VEC] = {};
    double zs = 0.0;
    int ns = 0;
    const int64_t per = static_cast<int64_t>(WAVES) * S::SLOTS;
    count_tokens<S>(a, cols, block * per + wid * S::SLOTS, blocks * per, acc, zs, ns);
    count_chosen(a, hist, static_cast<int64_t>(block) * THREADS + threadIdx.x, static_cast<int64_t>(blocks) * THREADS);
    column_sums<S>(cols, acc, psum[wid]);
    zs = wave_sum(zs);
    ns = slot_sum<1>(ns);
    if ((threadIdx.x & (kWave - 1)) == 0) {
      z[wid] = zs;
      n[wid] = ns;
    }
    __syncthreads();
  }
  __device__ float column(int e) const {
    float s = 0.f;
    for (int w = 0; w < WAVES; ++w) s += psum[w][e];
    return s;
  }
  __device__ double z_sum() const {
    double s = 0.0;
    for (int w = 0; w < WAVES; ++w) s += z[w];
    return s;
  }
  __device__ int n_sum() const {
    int s = 0;
    for (int w = 0; w < WAVES; ++w) s += n[w];
    return s;
  }
};

template <typename S>
__global__ void __launch_bounds__(kThreads) balance_count_kernel(BalArgs a) {
  __shared__ CountShared<S, kThreads> sh;
  const Columns<S> cols(threadIdx.x % S::LPT, a.E);
  sh.count(a, cols, blockIdx.x, gridDim.x);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    a.part_p[at + e] = sh.column(e);
    a.part_c[at + e] = sh.hist[e];
  }
  if (threadIdx.x == 0) {
    a.part_z[blockIdx.x] = sh.z_sum();
    a.part_n[blockIdx.x] = sh.n_sum();
  }
}

// 16 experts a workgroup, 64 threads an expert.
__global__ void __launch_bounds__(1024) balance_reduce_kernel(BalArgs a) {
  constexpr int ROWS = 64;
  __shared__ double ps[ROWS][16];
  __shared__ int cs[ROWS][16];
  __shared__ double zr[16], nr[16];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, e = blockIdx.x * 16 + col;
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int b = grp; b < a.blocks; b += ROWS) {
      p += a.part_p[static_cast<int64_t>(b) * a.E + e];
      c += a.part_c[static_cast<int64_t>(b) * a.E + e];
    }
  }
  double z = 0.0, n = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += 1024) {
    z += a.part_z[i];
    n += a.part_n[i];
  }
  z = wave_sum(z);
  n = wave_sum(n);
  if ((threadIdx.x & (kWave - 1)) == 0) {
    zr[threadIdx.x / kWave] = z;
    nr[threadIdx.x / kWave] = n;
  }
  ps[grp][col] = p;
  cs[grp][col] = c;
  __syncthreads();
  if (threadIdx.x < 16) {
    z = n = 0.0;
    for (int w = 0; w < 16; ++w) {
      z += zr[w];
      n += nr[w];
    }
    if (e < a.E) {
      double s = 0.0;
      int t = 0;
      for (int g = 0; g < ROWS; ++g) {
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
      a.total[1] = z;
    }
  }
}

template <typename S>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(BalArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const Columns<S> cols(lane % S::LPT, a.E);
  const double live = a.total[0];
  const Scales sc(a, live);
  if (blockIdx.x == 0 && wid == 0) {
    double dot = 0.0;
    for (int e = lane; e < a.E; e += kWave) dot += a.counts[e] * a.prob64[e];
    dot = wave_sum(dot);
    if (lane == 0) sc.write(a, dot, a.total[1], live);
  }
  const double unit = sc.unit(a);
  float f[S::NV][S::VEC];
#pragma unroll
  for (int q = 0; q < S::NV; ++q)
#pragma unroll
    for (int i = 0; i < S::VEC; ++i)
      f[q][i] = cols.skip[q] < S::VEC ? static_cast<float>(unit * a.counts[cols.col[q] + i]) : 0.f;
  const int64_t per = static_cast<int64_t>(kThreads / kWave) * S::SLOTS;
  grad_tokens<S>(a, cols, blockIdx.x * per + wid * S::SLOTS, gridDim.x * per, f, sc.zs(a));
}

// All of it in one workgroup, for a few tokens.
template <typename S>
__global__ void __launch_bounds__(kSmallThreads) balance_small_kernel(BalArgs a) {
  using Shared = CountShared<S, kSmallThreads>;
  __shared__ Shared sh;
  __shared__ double dots[Shared::WAVES];
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const Columns<S> cols(lane % S::LPT, a.E);
  sh.count(a, cols, 0, 1);
  const double live = sh.n_sum();
  const Scales sc(a, live);
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kSmallThreads) {
    const double p = sh.column(e) / sc.n;
    a.prob[e] = static_cast<float>(p);
    a.counts[e] = sh.hist[e];
    dot += p * sh.hist[e];
  }
  dot = wave_sum(dot);
  if (lane == 0) dots[wid] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    dot = 0.0;
    for (int w = 0; w < Shared::WAVES; ++w) dot += dots[w];
    sc.write(a, dot, sh.z_sum(), live);
  }
  const double unit = sc.unit(a);
  float f[S::NV][S::VEC];
#pragma unroll
  for (int q = 0; q < S::NV; ++q)
#pragma unroll
    for (int i = 0; i < S::VEC; ++i)
      f[q][i] = cols.skip[q] < S::VEC ? static_cast<float>(unit * sh.hist[cols.col[q] + i]) : 0.f;
  const int64_t per = static_cast<int64_t>(Shared::WAVES) * S::SLOTS;
  grad_tokens<S>(a, cols, wid * S::SLOTS, per, f, sc.zs(a));
}

template <typename S>
kfac_status_t run(BalArgs a, hipStream_t st) {
  if (a.tokens <= static_cast<int64_t>(kSmallRounds) * (kSmallThreads / S::LPT)) {
    hipLaunchKernelGGL((balance_small_kernel<S>), dim3(1), dim3(kSmallThreads), 0, st, a);
    KFAC_HIP_TRY(hipGetLastError());
    return KFAC_OK;
  }
  const int64_t per = static_cast<int64_t>(kThreads / kWave) * S::SLOTS;
  const int64_t need = (a.tokens + per - 1) / per;
  a.blocks = static_cast<int32_t>(std::min<int64_t>(need, kBalanceBlocks));
  hipLaunchKernelGGL((balance_count_kernel<S>), dim3(a.blocks), dim3(kThreads), 0, st, a);
  KFAC_HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL(balance_reduce_kernel, dim3((a.E + 15) / 16), dim3(1024), 0, st, a);
  KFAC_HIP_TRY(hipGetLastError());
  hipLaunchKernelGGL((balance_grad_kernel<S>), dim3(static_cast<int>(std::min<int64_t>(need, 1024))), dim3(kThreads), 0,
                     st, a);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

template <typename T, int LPT, int NV>
kfac_status_t run_even(const BalArgs& a, hipStream_t st) {
  constexpr int VE = Elem<T>::VE;
  return a.E % VE == 0 ? run<Shape<T, VE, LPT, NV, true>>(a, st) : run<Shape<T, VE, LPT, NV, false>>(a, st);
}

// Lanes a token by its number of vectors.
template <typename T>
kfac_status_t pick(const BalArgs& a, hipStream_t st) {
  constexpr int VE = Elem<T>::VE;
  if (a.E < VE) return run<Shape<T, 1, VE, 1, true>>(a, st);
  const int nvec = (a.E + VE - 1) / VE;
  if (nvec <= 1) return run_even<T, 1, 1>(a, st);
  if (nvec <= 2) return run_even<T, 2, 1>(a, st);
  if (nvec <= 4) return run_even<T, 4, 1>(a, st);
  if (nvec <= 8) return run_even<T, 8, 1>(a, st);
  if (nvec <= 16) return run_even<T, 16, 1>(a, st);
  if (nvec <= 32) return run_even<T, 32, 1>(a, st);
  if (nvec <= 64) return run_even<T, 64, 1>(a, st);
  if (nvec <= 128) return run_even<T, 64, 2>(a, st);
  if constexpr (VE == 4) return run_even<T, 64, 4>(a, st);
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
