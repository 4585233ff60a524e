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
// 65536 tokens of 256 bf16 logits: first pass 14.0 us, sums 4.5 us (latency),
// second pass 12.3 us, where a copy of the same 34 MB takes 10.3 us.  The first
// pass issues some 115 vector operations for a lane's eight logits (6.7 us in
// all; only 1 us of it the exponentials' own rate), the rest is the launch, the
// first loads and the sums at the end.  The next token's logits are loaded while
// one is worked on, tokens are numbered in 32 bits with rows stepped to, and 8
// wavefronts fit a SIMD.  With workgroups of 512, the mask waited for before the
// logits, addresses multiplied out, every lane dividing for the scales and the
// softmax found twice it was 15.5, 4.6 and 22 us; two vectors a lane and half
// the lanes: 17.1, 4.8 and 11.3 us.
#include "objectives.h"

#include <algorithm>

namespace kfac {

namespace {

constexpr int kThreads = 1024;
constexpr int kGradThreads = 256, kGradBlocks = 2048;
constexpr int kSmallRounds = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
  float* f;              // [E]: a count's weight in the gradient
  float2* stat;          // [tokens]: (maximum, 1 / sum), the latter 0 for a token that does not count
  double* total;         // [2]: n, sum of lse^2
  float* zs;             // [1]: lse's weight in the gradient
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
  static constexpr int WAVES = NV == 1 ? 8 : 4;  // wavefronts a SIMD that the registers have to leave room for
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

// A lane's part of a token's logits, minus infinity past the row.
template <typename S>
__device__ inline void load_row(u32x4 (&v)[S::NV], const char* row, const Columns<S>& cols) {
  using T = typename S::T;
#pragma unroll
  for (int q = 0; q < S::NV; ++q) {
    v[q] = u32x4{Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf};
    if (cols.skip[q] < S::VEC) {
      if constexpr (S::VEC > 1) v[q] = load16(row + static_cast<int64_t>(cols.col[q]) * sizeof(T));
      else if constexpr (sizeof(T) == 2) v[q][0] = reinterpret_cast<const unsigned short*>(row)[cols.col[q]];
      else v[q][0] = reinterpret_cast<const uint32_t*>(row)[cols.col[q]];
    }
  }
}

// A token's logits as they are loaded.  A token that is masked out is loaded
// too, so that its mask and its logits are waited for together, and counts as
// zeros from there on.
template <typename S>
struct TokenIn {
  u32x4 v[S::NV];
  uint8_t live;

  __device__ void load(const BalArgs& a, uint32_t t, const char* row, const Columns<S>& cols) {
#pragma unroll
    for (int q = 0; q < S::NV; ++q) v[q] = u32x4{0u, 0u, 0u, 0u};
    live = 0;
    if (t >= static_cast<uint32_t>(a.tokens)) return;
    load_row<S>(v, row, cols);
    live = a.mask ? a.mask[t] : 1;
  }
  // The logits, minus infinity past the row; zeros for a token that does not count.
  __device__ void expand(float (&x)[S::NV][S::VEC]) const {
#pragma unroll
    for (int q = 0; q < S::NV; ++q) {
      const u32x4 w = live ? v[q] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < S::VEC; ++i) x[q][i] = Elem<typename S::T>::get(w, i);
    }
  }
};

// 1 / s of a sum of exponentials (1 .. 1024), to float32's width.
__device__ inline float inverse(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return fmaf(fmaf(-s, r, 1.f), r, r);
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

// A lane's tokens in either pass: every `stride`th from t, with its row in a
// matrix of `ld` bytes a row.  Tokens are numbered in 32 bits, with room for one
// stride past the last.
struct Tokens {
  uint32_t t, stride;
  int64_t step;
  __device__ Tokens(int64_t first, int64_t every, int64_t ld)
      : t(static_cast<uint32_t>(first)), stride(static_cast<uint32_t>(every)), step(every * ld) {}
};

// First pass over a lane's tokens, the first of which is loaded: adds p to the lane's columns, lse^2 and the tokens
// that count (in a token's first lane); keeps each token's maximum and 1 / sum.
template <typename S>
__device__ inline void count_tokens(const BalArgs& a, const Columns<S>& cols, Tokens at, const char* row,
                                    TokenIn<S> in, float (&acc)[S::NV][S::VEC], double& z, int& n) {
  const int lane = threadIdx.x & (kWave - 1), slot = lane / S::LPT, sub = lane % S::LPT;
  const uint32_t tokens = static_cast<uint32_t>(a.tokens);
  for (; at.t - slot < tokens; at.t += at.stride) {       // as long as the wavefront's first token is one
    const uint32_t t = at.t;
    float x[S::NV][S::VEC];
    const bool live = in.live != 0;
    in.expand(x);
    row += at.step;
    in.load(a, t + at.stride, row, cols);
    if constexpr (!S::EVEN) {
#pragma unroll
      for (int q = 0; q < S::NV; ++q)
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) x[q][i] = i < cols.skip[q] ? -INFINITY : x[q][i];
    }
    const float m = row_maximum<S>(x);
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < S::NV; ++q)
#pragma unroll
      for (int i = 0; i < S::VEC; ++i) {
        x[q][i] = __builtin_amdgcn_exp2f((x[q][i] - m) * kLog2e);
        s += x[q][i];
      }
    s = group_reduce<S::LPT, false>(s);
    const float inv = live ? inverse(s) : 0.f;
    if (sub == 0 && t < tokens) a.stat[t] = make_float2(m, inv);
#pragma unroll
    for (int q = 0; q < S::NV; ++q)
#pragma unroll
      for (int i = 0; i < S::VEC; ++i) acc[q][i] = fmaf(x[q][i], inv, acc[q][i]);
    const bool first = live && sub == 0;
    if (a.z != 0.f) {
      const float lse = first ? fmaf(__builtin_amdgcn_logf(s), kLn2, m) : 0.f;
      z += static_cast<double>(lse) * static_cast<double>(lse);
    }
    n += first;
  }
}

// Histogram of the chosen experts, from thread `first` of `threads`: integer
// counts, in any order.  The first kAhead slots of a thread are loaded before
// the histogram is cleared.
constexpr int kAhead = 2;
struct Chosen {
  int64_t e[kAhead];
  uint8_t live[kAhead];

  static __device__ int64_t token(const BalArgs& a, int64_t i) {
    return a.tokens * a.k <= INT32_MAX
               ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.k)) : i / a.k;
  }
  static __device__ void add(const BalArgs& a, int* hist, int64_t e) {
    if (e >= a.E) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    else if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __device__ void load(const BalArgs& a, int64_t first, int64_t threads) {
    const int64_t slots = a.tokens * a.k;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = first + j * threads;
      live[j] = 0;
      e[j] = -1;
      if (i < slots) {
        e[j] = load_index(a.chosen, i, a.index_type);
        live[j] = a.mask ? a.mask[token(a, i)] : 1;
      }
    }
  }
  __device__ void count(const BalArgs& a, int* hist, int64_t first, int64_t threads) const {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (live[j]) add(a, hist, e[j]);
    const int64_t slots = a.tokens * a.k;
    for (int64_t i = first + kAhead * threads; i < slots; i += threads) {
      const int64_t c = load_index(a.chosen, i, a.index_type);
      if (!a.mask || a.mask[token(a, i)] != 0) add(a, hist, c);
    }
  }
};

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

// The lane's columns of an array [E].
template <typename S>
__device__ inline void own_columns(float (&f)[S::NV][S::VEC], const float* from, const Columns<S>& cols) {
#pragma unroll
  for (int q = 0; q < S::NV; ++q) {
#pragma unroll
    for (int i = 0; i < S::VEC; ++i) f[q][i] = 0.f;
    if (cols.skip[q] < S::VEC) {
      if constexpr (S::VEC == 1) {
        f[q][0] = from[cols.col[q]];
      } else {
#pragma unroll
        for (int k = 0; k < S::VEC / 4; ++k) {
          const u32x4 v = load16(from + cols.col[q] + 4 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[q][4 * k + i] = __uint_as_float(v[i]);
        }
      }
    }
  }
}

// Second pass: the gradients, from each token's maximum and inverse sum as the
// first pass found them (a third less arithmetic than to find them again), from
// f of the lane's columns and zs = 2 z_coef / n (both times grad_scale).
template <typename S>
struct TokenBack {
  u32x4 v[S::NV];
  float2 stat;

  __device__ void load(const BalArgs& a, uint32_t t, const char* row, const Columns<S>& cols) {
#pragma unroll
    for (int q = 0; q < S::NV; ++q) v[q] = u32x4{0u, 0u, 0u, 0u};
    stat = make_float2(0.f, 0.f);
    if (t >= static_cast<uint32_t>(a.tokens)) return;
    load_row<S>(v, row, cols);
    stat = a.stat[t];
  }
};

template <typename S>
__device__ inline void grad_tokens(const BalArgs& a, const Columns<S>& cols, Tokens at, const char* row,
                                   TokenBack<S> in, const float (&f)[S::NV][S::VEC], float zs) {
  using T = typename S::T;
  const int slot = (threadIdx.x & (kWave - 1)) / S::LPT;
  const uint32_t tokens = static_cast<uint32_t>(a.tokens);
  const int64_t grad_step = static_cast<int64_t>(at.stride) * a.ldg;
  char* grad = a.g + static_cast<int64_t>(at.t) * a.ldg;
  bool bad = false;
  for (; at.t - slot < tokens; at.t += at.stride, grad += grad_step) {
    const uint32_t t = at.t;
    const TokenBack<S> cur = in;
    row += at.step;
    in.load(a, t + at.stride, row, cols);
    const float m = cur.stat.x, inv = cur.stat.y;
    float p[S::NV][S::VEC], pf = 0.f;
#pragma unroll
    for (int q = 0; q < S::NV; ++q)
#pragma unroll
      for (int i = 0; i < S::VEC; ++i) {
        p[q][i] = __builtin_amdgcn_exp2f((Elem<T>::get(cur.v[q], i) - m) * kLog2e) * inv;
        pf = fmaf(S::EVEN || i >= cols.skip[q] ? p[q][i] : 0.f, f[q][i], pf);
      }
    pf = group_reduce<S::LPT, false>(pf);
    const bool live = inv != 0.f;
    const float shift = (zs != 0.f ? zs * fmaf(__builtin_amdgcn_logf(inv), -kLn2, m) : 0.f) - pf;
    bad |= live && !finite(shift);      // also where an f is not: its column is in pf
    if (t >= tokens) continue;
#pragma unroll
    for (int q = 0; q < S::NV; ++q) {
      if (cols.skip[q] < S::VEC) {
        float g[S::VEC];
#pragma unroll
        for (int i = 0; i < S::VEC; ++i) g[i] = p[q][i] * (f[q][i] + shift);
        if constexpr (S::VEC == 1) Elem<T>::store(grad, cols.col[q], live ? g[0] : 0.f);
        else store16(grad + static_cast<int64_t>(cols.col[q]) * sizeof(T), live ? pack16<T>(g) : u32x4{0u, 0u, 0u, 0u});
      }
    }
  }
  if (bad && (threadIdx.x & (S::LPT - 1)) == 0) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
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
    if (!(finite(a.stats[0]) && finite(a.stats[1]) && finite(a.stats[2]))) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
  }
};

template <typename S>
struct CountShared {
  static constexpr int WAVES = kThreads / kWave;
  int hist[S::W];
  float psum[WAVES][S::W];
  double z[WAVES];
  int n[WAVES];

  // Everything of the first pass for this workgroup: hist, psum, z and n.
  __device__ void count(const BalArgs& a, const Columns<S>& cols, int block, int blocks) {
    const int wid = threadIdx.x / kWave;
    const int64_t per = static_cast<int64_t>(WAVES) * S::SLOTS, t0 = block * per + wid * S::SLOTS, stride = blocks * per;
    const int64_t first = static_cast<int64_t>(block) * kThreads + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(blocks) * kThreads;
    const Tokens at(t0 + (threadIdx.x & (kWave - 1)) / S::LPT, stride, a.ldx);
    const char* row = a.x + static_cast<int64_t>(at.t) * a.ldx;
    TokenIn<S> in;
    in.load(a, at.t, row, cols);
    Chosen chosen;
    chosen.load(a, first, threads);
    for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    float acc[S::NV][S::VEC] = {};
    double zs = 0.0;
    int ns = 0;
    count_tokens<S>(a, cols, at, row, in, acc, zs, ns);
    chosen.count(a, hist, first, threads);
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
__global__ void __launch_bounds__(kThreads, S::WAVES) balance_count_kernel(BalArgs a) {
  __shared__ CountShared<S> sh;
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
      a.f[e] = static_cast<float>(Scales(a, n).unit(a) * t);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.total[0] = n;
      a.total[1] = z;
      *a.zs = Scales(a, n).zs(a);
    }
  }
}

template <typename S>
__global__ void __launch_bounds__(kGradThreads, S::WAVES) balance_grad_kernel(BalArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const Columns<S> cols(lane % S::LPT, a.E);
  const int64_t per = static_cast<int64_t>(kGradThreads / kWave) * S::SLOTS;
  const Tokens at(blockIdx.x * per + wid * S::SLOTS + lane / S::LPT, gridDim.x * per, a.ldx);
  const char* row = a.x + static_cast<int64_t>(at.t) * a.ldx;
  TokenBack<S> in;
  in.load(a, at.t, row, cols);
  float f[S::NV][S::VEC];
  own_columns<S>(f, a.f, cols);
  const float zs = *a.zs;
  if (blockIdx.x == 0 && wid == 0) {
    const double live = a.total[0];
    double dot = 0.0;
    for (int e = lane; e < a.E; e += kWave) dot += a.counts[e] * a.prob64[e];
    dot = wave_sum(dot);
    if (lane == 0) Scales(a, live).write(a, dot, a.total[1], live);
  }
  grad_tokens<S>(a, cols, at, row, in, f, zs);
}

// All of it in one workgroup, for a few tokens.
template <typename S>
__global__ void __launch_bounds__(kThreads) balance_small_kernel(BalArgs a) {
  using Shared = CountShared<S>;
  __shared__ Shared sh;
  __shared__ double dots[Shared::WAVES];
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const Columns<S> cols(lane % S::LPT, a.E);
  sh.count(a, cols, 0, 1);
  const double live = sh.n_sum();
  const Scales sc(a, live);
  double dot = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
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
  const Tokens at(wid * S::SLOTS + lane / S::LPT, per, a.ldx);
  const char* row = a.x + static_cast<int64_t>(at.t) * a.ldx;
  TokenBack<S> in;
  in.load(a, at.t, row, cols);
  grad_tokens<S>(a, cols, at, row, in, f, sc.zs(a));
}

template <typename S>
kfac_status_t run(BalArgs a, hipStream_t st) {
  if (a.tokens <= static_cast<int64_t>(kSmallRounds) * (kThreads / S::LPT)) {
    hipLaunchKernelGGL((balance_small_kernel<S>), dim3(1), dim3(kThreads), 0, st, a);
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
  const int64_t grad_need = need * (kThreads / kGradThreads);
  hipLaunchKernelGGL((balance_grad_kernel<S>), dim3(static_cast<int>(std::min<int64_t>(grad_need, kGradBlocks))),
                     dim3(kGradThreads), 0, st, a);
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
  size_t p, c, z, n, prob, f, stat, total, end;
};
Regions regions(int64_t tokens, int32_t E) {
  Regions r;
  r.p = kRegions;
  r.c = r.p + align_up(sizeof(float) * kBalanceBlocks * static_cast<size_t>(E), 256);
  r.z = r.c + align_up(sizeof(int32_t) * kBalanceBlocks * static_cast<size_t>(E), 256);
  r.n = r.z + align_up(sizeof(double) * kBalanceBlocks, 256);
  r.prob = r.n + align_up(sizeof(int32_t) * kBalanceBlocks, 256);
  r.f = r.prob + align_up(sizeof(double) * static_cast<size_t>(E), 256);
  r.stat = r.f + align_up(sizeof(float) * static_cast<size_t>(E), 256);
  r.total = r.stat + align_up(sizeof(float2) * static_cast<size_t>(tokens), 256);
  r.end = r.total + 256;
  return r;
}

}  // namespace

size_t balance_workspace_bytes(int64_t tokens, int32_t experts) { return regions(tokens, experts).end; }

kfac_status_t launch_balance(const kfac_balance_t& b, char* ws, hipStream_t st) {
  const Regions r = regions(b.tokens, b.experts);
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
  a.f = reinterpret_cast<float*>(ws + r.f);
  a.stat = reinterpret_cast<float2*>(ws + r.stat);
  a.total = reinterpret_cast<double*>(ws + r.total);
  a.zs = reinterpret_cast<float*>(a.total + 2);
  return b.dtype == KFAC_BF16 ? pick<__bf16>(a, st) : pick<float>(a, st);
}

}  // namespace kfac
