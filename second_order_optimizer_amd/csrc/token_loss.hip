// Objectives over rows of logits (include/kfac_objectives.h): label
// log-probabilities, the clipped policy loss and the preference loss, the two
// losses with the gradient of every logit.
//
// With s the logit scale, M = max_j x_j and S = sum_j exp(s (x_j - M)), a row
// with label l has logp = s (x_l - M) - log S, and the gradient of
// coef * logp is coef s (onehot(l) - exp(s (x - M)) / S).  All three are
// bound by HBM: the logits in, the gradients out.
//
// Arithmetic: differences x - M are formed before scaling, so rows whose
// logits are all huge, or all the type's lowest value, stay exact; exp is the
// hardware's 2^x on a float32 argument; a vector's terms are added as a tree
// in float32 and the vectors of a thread, the threads and the wavefronts in
// 64 bits, in a fixed order; the gradient is rounded once, when it is stored.
#include "objectives.h"
#include "objectives_grid.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace kfac {

namespace {

struct TokArgs {
  const char* x;
  char* g;
  const void* labels;
  float* logp;
  int64_t rows;
  int64_t ldx, ldg;    // bytes
  int32_t vocab;
  int32_t label_type;
  float scale;         // s
  float c, clo;        // s log2(e): exp(s d) = 2^(c d + clo d)
  float near;          // the same to the nearest float32
  float grad_scale;    // s grad_scale
  uint32_t* flags;
};

struct PolArgs {
  const float *adv, *weight, *old_logp, *ref;
  uint64_t* part;      // [gridDim.x][3] doubles
  uint32_t* arrived;   // counters of workgroups that are done, 0 between calls
  float* stats;
  float lo, hi, kl;
  float w0;            // weight where none is given
};

// Running maximum and sum of exp(s (x - max)) of some of a row's logits.
struct Softmax {
  float m;
  double s;
};

// Adds the vectors v[0 .. N) to a thread's running maximum and sum.  Absent
// values are minus infinity; `mu` replaces a maximum of minus infinity so
// that those add exp(-inf) = 0.
// FINE multiplies by s log2(e) to twice float32's width: c alone is off by up
// to 3e-8 of itself, which biases log S by that times the mean exponent, the
// same way in every row; sums of log-probabilities over a sequence would show
// it.  bf16 gradients, and the policy loss's bf16 rows, do without: their c is
// the nearest float32, so that log S is off by at most 6e-8 times the mean
// exponent (the float below the product, which the pair needs, may be twice as
// far: 1.25 and 0.85 are such scales).
template <typename T>
constexpr bool kFine = sizeof(T) == 4;
template <typename T>
__device__ inline float scale_of(const TokArgs& a) { return kFine<T> ? a.c : a.near; }
template <bool FINE>
__device__ inline float exp_of(float d, float c, float clo) {
  return __builtin_amdgcn_exp2f(FINE ? fmaf(d, c, d * clo) : d * c);
}
template <typename T, int N, bool FINE = false>
__device__ inline void absorb(Softmax& a, const u32x4* v, float c, float clo = 0.f) {
  constexpr int VE = Elem<T>::VE;
  float m = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < VE; i += 2) m = max3(m, Elem<T>::get(v[j], i), Elem<T>::get(v[j], i + 1));
  const float mu = m == -INFINITY ? 0.f : m;
  a.s *= static_cast<double>(exp_of<FINE>(a.m - mu, c, clo));
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = exp_of<FINE>(Elem<T>::get(v[j], i) - mu, c, clo);
#pragma unroll
    for (int w = VE / 2; w > 0; w >>= 1)
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] += e[i + w];
    a.s += static_cast<double>(e[0]);
  }
  a.m = m;
}
template <bool FINE = false>
__device__ inline void absorb_one(Softmax& a, float x, float c, float clo = 0.f) {
  const float m = fmaxf(a.m, x);
  const float mu = m == -INFINITY ? 0.f : m;
  a.s = a.s * static_cast<double>(exp_of<FINE>(a.m - mu, c, clo)) + static_cast<double>(exp_of<FINE>(x - mu, c, clo));
  a.m = m;
}

__device__ inline float first_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// A wavefront's maximum and sum from its lanes', and a team's from its
// wavefronts', in the lanes of one.
template <bool FINE>
__device__ inline Softmax wave_softmax(Softmax a, float c, float clo) {
  const float m = wave_max(a.m);
  const float mu = m == -INFINITY ? 0.f : m;
  return {m, wave_sum(a.s * static_cast<double>(exp_of<FINE>(a.m - mu, c, clo)))};
}
template <int NW, bool FINE>
__device__ inline Softmax across(Softmax b, float c, float clo) {
  static_assert(NW <= 16, "one row of lanes");
  const float m = lane_of(row_max(b.m), 0);
  const float mu = m == -INFINITY ? 0.f : m;
  return {m, lane_of(row_sum(b.s * static_cast<double>(exp_of<FINE>(b.m - mu, c, clo))), 0)};
}

// A team's maximum and sum from its threads'.  Several wavefronts meet in
// `red`, whose two halves alternate from use to use (`parity`), so that one
// barrier a row is enough.
template <int TEAM, bool FINE>
__device__ inline Softmax team_softmax(Softmax a, float c, float clo, Softmax* red, int parity) {
  Softmax r = wave_softmax<FINE>(a, c, clo);
  if constexpr (TEAM > kWave) {
    constexpr int NW = TEAM / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    red += parity * NW;
    if (lane == 0) red[threadIdx.x / kWave] = r;
    __syncthreads();
    r = across<NW, FINE>(lane < NW ? red[lane] : Softmax{-INFINITY, 0.0}, c, clo);
  }
  return r;
}

__device__ inline float log_prob(float xl, Softmax r, float scale) {
  const float s = static_cast<float>(r.s);
  return (xl - r.m) * scale - (logf(s) + static_cast<float>(r.s - static_cast<double>(s)) / s);
}

// The label of a row, -1 for one to leave out (a label beyond the vocabulary
// is reported and left out).
__device__ inline int32_t row_label(const TokArgs& a, int64_t row) {
  const int64_t l = load_index(a.labels, row, a.label_type);
  if (l >= a.vocab) {
    if ((threadIdx.x & (kWave - 1)) == 0) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    return -1;
  }
  return l < 0 ? -1 : static_cast<int32_t>(l);
}

// coef / S times exp(s (x - M)), negated and rounded: a vector of the gradient.
template <typename T>
__device__ inline u32x4 grad_vec(u32x4 v, float m, float c, float clo, float neg) {
  float o[Elem<T>::VE];
#pragma unroll
  for (int i = 0; i < Elem<T>::VE; ++i) o[i] = exp_of<kFine<T>>(Elem<T>::get(v, i) - m, c, clo) * neg;
  return pack16<T>(o);
}
template <typename T>
__device__ inline float grad_one(float x, float m, float c, float clo, float neg) {
  return exp_of<kFine<T>>(x - m, c, clo) * neg;
}

// ---------------------------------------------------------------------------
// Clipped policy loss: one team of wavefronts a row, the row held in
// registers between its sum and its gradient, so each logit is read once and
// each gradient written once.  A team walks rows a grid apart and asks for
// the next row's vector in the place of each one it has finished, so loads
// and stores stay mixed and no phase waits for an empty pipe.  LONG: rows
// beyond the registers (TEAM * NV vectors) read the rest twice (512 x 140003 bf16
// 85 us, 1024 x 131072 f32 266: 53 and 75% of a row is read again).
//
// Bound by HBM with reads and writes mixed: 4096 x 131072 bf16 421 us for 2.07 GB
// (the 7% of rows without a label are written, not read), 4.9 TB/s (a copy as
// large: 6.2); without the exponentials it is 2% less.  2047 x 50001 bf16 92 us
// for 0.39 GB, 4.3 TB/s: eight rows a compute unit, so the first loads and the
// last stores, with nothing to pair them with, are a ninth each, which is some 8
// of the 28 us over a copy's time; what the others are was not found.
//
// A row's scalars (logp, ratio, KL term, coefficient, coef / S) are float32,
// formed from the 64-bit sum: logp is off by a few 2^-24 of its two terms, and the
// ratio and the gradient by as much relatively (256 x 1000 f32: 2e-7 against 64
// bits).  Their 64-bit functions are some hundred instructions each for a lane
// that the row waits for.  For the same reason logp here and in logp_kernel,
// which has them, differ in their last bits.

struct RowScalars {
  int32_t label;
  float xl, w, adv, old_logp, ref;
};

// What a row's gradient and log-probability need of its sum.
struct RowTerms {
  float m, coef, neg, logp;      // neg = -coef / S
};

template <typename T>
__device__ inline RowScalars row_scalars(const TokArgs& a, const PolArgs& p, int64_t row, int32_t label) {
  RowScalars r;
  r.label = label;
  r.xl = label >= 0 ? Elem<T>::load(a.x + row * a.ldx, label) : 0.f;
  r.w = p.weight ? p.weight[row] : p.w0;
  r.adv = p.adv[row];
  r.old_logp = p.old_logp ? p.old_logp[row] : 0.f;
  r.ref = p.ref ? p.ref[row] : 0.f;
  return r;
}

// stats from the workgroups' sums: the workgroup that counts itself last adds
// them up, in a fixed order, and leaves the counters at 0 for the next call.
// Workgroups count in groups of kArriveGroup, the last of a group counts it: on
// one counter 1536 workgroups took 18 us.  The sums are stored and loaded at
// device scope, past the XCDs' own caches, and counted once the stores have
// arrived, so no cache has to be written back (a release fence in every
// workgroup does that: 2047 x 50001 bf16 92 -> 103 us).  A kernel of its own
// for these sums took 4 us and a launch.

__device__ inline bool counted_last(uint32_t* counter, uint32_t of) {
  if (__hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != of - 1) return false;
  __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return true;
}

template <int TEAMS>
__device__ inline void policy_stats(const PolArgs& p, uint32_t* flags, const double (*sums)[3], int* last) {
  if (threadIdx.x == 0) {
    uint64_t* q = p.part + static_cast<int64_t>(blockIdx.x) * 3;
    for (int k = 0; k < 3; ++k) {
      double t = 0.0;
      for (int i = 0; i < TEAMS; ++i) t += sums[i][k];
      __hip_atomic_store(q + k, __builtin_bit_cast(uint64_t, t), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t group = blockIdx.x / kArriveGroup, groups = (gridDim.x + kArriveGroup - 1) / kArriveGroup;
    const uint32_t size = min(static_cast<uint32_t>(kArriveGroup), gridDim.x - group * kArriveGroup);
    *last = counted_last(p.arrived + (1 + group) * kArriveStride, size) && counted_last(p.arrived, groups);
  }
  __syncthreads();
  if (!*last) return;
  constexpr int WAVES = 4;                      // of 4 or more
  __shared__ double red[WAVES][3];
  if (threadIdx.x < WAVES * kWave) {
    double t[3] = {0.0, 0.0, 0.0};
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += WAVES * kWave)
      for (int k = 0; k < 3; ++k)
        t[k] += __builtin_bit_cast(double, __hip_atomic_load(p.part + static_cast<int64_t>(i) * 3 + k, __ATOMIC_RELAXED,
                                                             __HIP_MEMORY_SCOPE_AGENT));
    for (int k = 0; k < 3; ++k) {
      t[k] = wave_sum(t[k]);
      if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave][k] = t[k];
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t[3];
    for (int k = 0; k < 3; ++k) t[k] = (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
    const float loss = static_cast<float>(p.kl != 0.f ? t[0] + static_cast<double>(p.kl) * t[1] : t[0]);
    p.stats[0] = loss;
    p.stats[1] = static_cast<float>(t[0]);
    p.stats[2] = static_cast<float>(t[1]);
    p.stats[3] = static_cast<float>(t[2]);
    if (!finite(loss)) raise_flag(flags, KFAC_FLAG_NONFINITE);      // a sum of finite rows may pass float32
  }
}

template <typename T, int TEAM, int NV, bool LONG, bool NT>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) policy_kernel(TokArgs a, PolArgs p) {
  constexpr int VE = Elem<T>::VE;
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM, NW = TEAM / kWave;
  constexpr int CH = NV < 4 ? NV : 4;
  __shared__ Softmax red[NW];
  __shared__ RowTerms shared;
  __shared__ double sums[TEAMS][3];
  __shared__ int last;
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM), tid = threadIdx.x % TEAM;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  const int nfull = a.vocab / VE, ntail = a.vocab % VE;
  const float c = scale_of<T>(a), clo = a.clo;
  constexpr bool FINE = kFine<T>;

  u32x4 v[NV];
  float tail = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = u32x4{Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf};
  double acc_a = 0.0, acc_k = 0.0, acc_c = 0.0;
  bool bad = false;

  int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
  RowScalars cur{};
  if (row < a.rows) {
    const char* x = a.x + row * a.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * TEAM + tid < nfull) v[j] = load16<NT>(x + static_cast<int64_t>(j * TEAM + tid) * 16);
    if (tid < ntail) tail = Elem<T>::load(x, static_cast<int64_t>(nfull) * VE + tid);
    cur = row_scalars<T>(a, p, row, row_label(a, row));
  }
  while (row < a.rows) {
    const int64_t next = row + stride;
    const bool has = next < a.rows;
    const int32_t nlabel = has ? row_label(a, next) : -1;
    const char* xr = a.x + row * a.ldx;
    const char* xn = a.x + next * a.ldx;
    char* gr = a.g + row * a.ldg;

    RowTerms o{0.f, 0.f, 0.f, 0.f};
    if (cur.label >= 0) {
      Softmax t{-INFINITY, 0.0};
#pragma unroll
      for (int j = 0; j < NV; j += CH) absorb<T, CH, FINE>(t, v + j, c, clo);
      if (ntail) absorb_one<FINE>(t, tail, c, clo);
      if constexpr (LONG) {
        constexpr int CL = 4;
        for (int j0 = NV; j0 * TEAM < nfull; j0 += CL) {
          u32x4 u[CL];
#pragma unroll
          for (int j = 0; j < CL; ++j) {
            const int idx = (j0 + j) * TEAM + tid;
            u[j] = u32x4{Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf};
            if (idx < nfull) u[j] = load16<NT>(xr + static_cast<int64_t>(idx) * 16);
          }
          absorb<T, CL, FINE>(t, u, c, clo);
        }
      }
      // what follows from the row's sum is the same for all of it: one wavefront
      // works it out and the others wait (4096 x 12000 bf16 44.6 -> 43.1 us; 2047 x 50001
      // 90.5 -> 92.1)
      auto terms = [&](Softmax r) {
        RowTerms o{r.m, 0.f, 0.f, log_prob(cur.xl, r, a.scale)};
        if (cur.w == 0.f) return o;
        const float ratio = p.old_logp ? expf(o.logp - cur.old_logp) : 1.f;
        const float held = fminf(fmaxf(ratio, p.lo), p.hi);
        // an advantage of 0 is a term of 0, also where the ratio passes float32
        const float first = cur.adv != 0.f ? ratio * cur.adv : 0.f, second = held * cur.adv;
        const bool clipped = second < first;
        const float gain = clipped ? second : first;
        float slope = clipped ? 0.f : -first, kl = 0.f;
        if (p.ref) {
          const float d = cur.ref - o.logp, ed = expm1f(d);
          kl = ed - d;
          if (p.kl != 0.f) slope -= p.kl * ed;
        }
        o.coef = cur.w * slope * a.grad_scale;
        o.neg = -o.coef / static_cast<float>(r.s);
        acc_a -= static_cast<double>(cur.w) * gain;
        acc_k += static_cast<double>(cur.w) * kl;
        acc_c += clipped ? cur.w : 0.f;
        bad |= !(finite(gain) && finite(kl) && finite(o.neg));
        return o;
      };
      Softmax r = wave_softmax<FINE>(t, c, clo);
      if constexpr (TEAM == kWave) {
        o = terms(r);
      } else {
        if ((tid & (kWave - 1)) == 0) red[tid / kWave] = r;
        __syncthreads();
        if (tid < kWave) {
          r = across<NW, FINE>(tid < NW ? red[tid] : Softmax{-INFINITY, 0.0}, c, clo);
          o = terms(r);
          if (tid == 0) shared = o;
        }
        __syncthreads();
        o = shared;
        o.m = first_lane(o.m);
        o.coef = first_lane(o.coef);
        o.neg = first_lane(o.neg);
        o.logp = first_lane(o.logp);
      }
    }
    if (tid == 0) a.logp[row] = o.logp;

    const RowScalars nxt = has ? row_scalars<T>(a, p, next, nlabel) : RowScalars{};
    const bool fetch = nlabel >= 0, zero = o.coef == 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int idx = j * TEAM + tid;
      if (idx < nfull) {
        const int64_t at = static_cast<int64_t>(idx) * 16;
        store16<NT>(gr + at, zero ? u32x4{0u, 0u, 0u, 0u} : grad_vec<T>(v[j], o.m, c, clo, o.neg));
        if (fetch) v[j] = load16<NT>(xn + at);
      }
    }
    if constexpr (LONG) {
      for (int idx = NV * TEAM + tid; idx < nfull; idx += TEAM) {
        const int64_t at = static_cast<int64_t>(idx) * 16;
        u32x4 g = {0u, 0u, 0u, 0u};
        if (!zero) g = grad_vec<T>(load16<NT>(xr + at), o.m, c, clo, o.neg);
        store16<NT>(gr + at, g);
      }
    }
    if (tid < ntail) {
      const int64_t e = static_cast<int64_t>(nfull) * VE + tid;
      Elem<T>::store(gr, e, zero ? 0.f : grad_one<T>(tail, o.m, c, clo, o.neg));
      if (fetch) tail = Elem<T>::load(xn, e);
    }
    // the label's entry, over what its owner has just stored there:
    // coef (1 - p) with 1 - p = -expm1(logp), which does not cancel
    if (!zero) {
      const int lv = cur.label / VE;
      const int owner = lv < nfull ? lv % TEAM : cur.label - nfull * VE;
      if (tid == owner) Elem<T>::store(gr, cur.label, -o.coef * expm1f(o.logp));
    }
    row = next;
    cur = nxt;
  }
  if (tid == 0) {
    sums[team][0] = acc_a;
    sums[team][1] = acc_k;
    sums[team][2] = acc_c;
    if (bad) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
  }
  __syncthreads();
  policy_stats<TEAMS>(p, a.flags, sums, &last);
}

// ---------------------------------------------------------------------------
// Label log-probabilities: a team streams its row, UN vectors a thread at a
// time.  logp is formed in 64 bits, since the preference loss adds up small
// differences of it; with `stat` each row's (M, 1 / S) and with `wide` its logp
// in 64 bits are kept for the kernels below.  Rows before `past` are read past
// the cache.  Bound by HBM reads: 8192 x 32768 bf16 86 us, 6.2 TB/s; 1024 x
// 131072 f32 82 us, 6.5 TB/s (reads alone: 7.2).  64 rows of 32768: 5 us, of which
// the launch is half.  Wavefronts a row by the rows there are: 1024 threads where 256 would
// leave compute units idle.

struct RowStats {
  float2* stat;        // 1 / S to float32: the gradient is off by 2^-24 of itself for it
  double* wide;
  float* coef;         // set to 0 for preference_pair_kernel
  int64_t past;
};

template <typename T, int TEAM, int UN, bool NT>
__device__ inline Softmax stream_row(const TokArgs& a, const char* x, int tid) {
  constexpr int VE = Elem<T>::VE;
  const int nfull = a.vocab / VE, ntail = a.vocab % VE;
  Softmax t{-INFINITY, 0.0};
  for (int j0 = 0; j0 * TEAM < nfull; j0 += UN) {
    u32x4 u[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int idx = (j0 + j) * TEAM + tid;
      u[j] = u32x4{Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf};
      if (idx < nfull) u[j] = load16<NT>(x + static_cast<int64_t>(idx) * 16);
    }
    absorb<T, UN, true>(t, u, a.c, a.clo);
  }
  if (ntail)
    absorb_one<true>(t, tid < ntail ? Elem<T>::load(x, static_cast<int64_t>(nfull) * VE + tid) : -INFINITY, a.c, a.clo);
  return t;
}

// The logarithm in 64 bits is some hundred instructions, whether for one lane or
// for all: over the shortest rows (UN = 1) a team keeps one row a lane and takes
// it for up to 64 rows at once (32768 rows of 500 bf16: 20.0 -> 16.3 us; for
// longer rows the registers cost more, 8192 x 4000 13.5 -> 15.3 us).
template <typename T, int TEAM, int UN>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) logp_kernel(TokArgs a, RowStats out) {
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM, NW = TEAM / kWave;
  __shared__ Softmax red[2 * NW];
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM), tid = threadIdx.x % TEAM;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  constexpr int KEEP = UN == 1 ? kWave : 1;
  int parity = 0, kept = 0;
  double num = 0.0, den = 1.0;       // of the lane's row: s (x_l - M), S
  float top = 0.f;                   // M
  int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team, base = row;
  int32_t next = row < a.rows ? row_label(a, row) : -1;
  for (; row < a.rows; row += stride) {
    const int32_t label = next;
    next = row + stride < a.rows ? row_label(a, row + stride) : -1;      // known when its row comes
    float xl = 0.f;
    Softmax r{0.f, 1.0};
    if (label >= 0) {
      const char* x = a.x + row * a.ldx;
      xl = Elem<T>::load(x, label);
      Softmax t = row < out.past ? stream_row<T, TEAM, UN, true>(a, x, tid) : stream_row<T, TEAM, UN, false>(a, x, tid);
      r = team_softmax<TEAM, true>(t, a.c, a.clo, red, parity);
      parity ^= 1;
    }
    if (tid == kept) {
      num = (static_cast<double>(xl) - static_cast<double>(r.m)) * static_cast<double>(a.scale);
      den = r.s;
      top = r.m;
    }
    if (++kept == KEEP || row + stride >= a.rows) {
      if (tid < kept) {
        const int64_t at = KEEP == 1 ? row : base + tid * stride;
        const double logp = num - log(den);
        a.logp[at] = static_cast<float>(logp);
        if (out.stat) {
          out.stat[at] = make_float2(top, static_cast<float>(1.0 / den));
          out.wide[at] = logp;
          out.coef[at] = 0.f;
        }
      }
      base = row + stride;
      kept = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Preference loss, between its two passes over the logits: workgroup i adds
// up pair i's log ratios and writes d loss / d logp of its rows.

struct PrefArgs {
  const int32_t* offsets;
  const float *ref, *weight;
  float* seq;
  float* stats;
  double* part;        // [pairs][4]
  const double* wide;  // [rows]: logp
  float* coef;         // [rows], zero before preference_pair_kernel
  int32_t pairs, kind, average;
  float beta, eps, w0;
};

__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(TokArgs a, PrefArgs p) {
  constexpr int WAVES = kPairThreads / kWave;
  static_assert(WAVES == 16, "row_sum adds 16 lanes");
  __shared__ double red[WAVES][4];
  __shared__ float coef[2];
  const int i = blockIdx.x, tid = threadIdx.x;
  int lo[2], hi[2];
  for (int k = 0; k < 2; ++k) {
    lo[k] = p.offsets[k * p.pairs + i];
    hi[k] = p.offsets[k * p.pairs + i + 1];
  }
  for (int k = 0; k < 2; ++k)
    if (lo[k] < 0 || hi[k] < lo[k] || hi[k] > a.rows) {
      if (tid == 0) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
      lo[k] = hi[k] = 0;
    }
  // sums of the log ratios and, where they are averaged, numbers of labelled rows
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  auto labelled = [&](int64_t label) { return label >= 0 && label < a.vocab; };
  auto take = [&](int k, double wide, float ref) {
    sum[2 * k] += wide - static_cast<double>(ref);
    sum[2 * k + 1] += 1.0;
  };
  bool first[2] = {false, false};       // the thread's first row of either sequence has a label
  if (a.rows > 0) {
    // both are asked for at once (row 0 for a thread that has none)
    int64_t label[2];
    double wide[2];
    float ref[2];
    for (int k = 0; k < 2; ++k) {
      const int64_t r = tid < hi[k] - lo[k] ? lo[k] + tid : 0;
      label[k] = load_index(a.labels, r, a.label_type);
      wide[k] = p.wide[r];
      ref[k] = p.ref ? p.ref[r] : 0.f;
    }
    for (int k = 0; k < 2; ++k) {
      first[k] = tid < hi[k] - lo[k] && labelled(label[k]);
      if (first[k]) take(k, wide[k], ref[k]);
    }
    for (int k = 0; k < 2; ++k)
      for (int64_t r = static_cast<int64_t>(lo[k]) + kPairThreads + tid; r < hi[k]; r += kPairThreads)
        if (labelled(load_index(a.labels, r, a.label_type))) take(k, p.wide[r], p.ref ? p.ref[r] : 0.f);
  }
  for (int q = 0; q < 4; ++q) {
    if ((q & 1) && !p.average) continue;
    sum[q] = wave_sum(sum[q]);
    if ((tid & (kWave - 1)) == 0) red[tid / kWave][q] = sum[q];
  }
  __syncthreads();
  // one wavefront forms the loss (in all of them its 64-bit functions took 1.6 us more)
  if (tid < kWave) {
    double R[2], share[2];
    for (int k = 0; k < 2; ++k) {
      const double s = lane_of(row_sum(red[tid % WAVES][2 * k]), 0);
      const double n = p.average ? lane_of(row_sum(red[tid % WAVES][2 * k + 1]), 0) : 0.0;
      share[k] = p.average ? (n > 0.0 ? 1.0 / n : 0.0) : 1.0;
      R[k] = s * share[k];
    }
    const double h = R[0] - R[1], beta = p.beta, eps = p.eps;
    const double w = p.weight ? static_cast<double>(p.weight[i]) : static_cast<double>(p.w0);
    double loss, slope;
    if (p.kind == KFAC_PREF_SIGMOID) {
      const double x = beta * h, e = exp(-fabs(x)), l = log1p(e);
      loss = (1.0 - eps) * (fmax(-x, 0.0) + l);                 // log(1 + exp(-x)), and of x below
      if (eps != 0.0) loss += eps * (fmax(x, 0.0) + l);         // no 0 times infinity where x is infinite
      // sigma(x) - (1 - e), with sigma of the side that does not cancel
      const double sig = e / (1.0 + e);                         // sigma(-|x|)
      slope = beta * (x >= 0.0 ? eps - sig : sig - (1.0 - eps));
    } else {
      const double x = h - 0.5 / beta;
      loss = x * x;
      slope = 2.0 * x;
    }
    if (tid == 0) {
      p.seq[i] = static_cast<float>(R[0]);
      p.seq[p.pairs + i] = static_cast<float>(R[1]);
      double* q = p.part + static_cast<int64_t>(i) * 4;
      q[0] = w != 0.0 ? w * loss : 0.0;
      q[1] = h > 0.0 ? w : 0.0;
      q[2] = w != 0.0 ? w * beta * h : 0.0;
      q[3] = w;
      bool bad = !finite(static_cast<float>(q[0]));
      for (int k = 0; k < 2; ++k) {
        coef[k] = w != 0.0 ? static_cast<float>((k ? -w : w) * slope * share[k] * static_cast<double>(a.grad_scale)) : 0.f;
        bad |= !finite(coef[k]);
      }
      if (bad) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
    }
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    const float f = coef[k];
    if (tid < hi[k] - lo[k]) p.coef[lo[k] + tid] = first[k] ? f : 0.f;
    for (int64_t r = static_cast<int64_t>(lo[k]) + kPairThreads + tid; r < hi[k]; r += kPairThreads)
      p.coef[r] = labelled(load_index(a.labels, r, a.label_type)) ? f : 0.f;
  }
}

// Second pass over the logits: the gradient, from each row's (M, 1 / S) and
// coefficient.  The rows are taken last to first: where logits and gradients
// do not fit the cache, the first pass reads all but its last rows past it
// and the gradients are stored past it, so that those last rows are still
// there (the whole loss 287 -> 250 us on 7155 rows of 32768 bf16 logits, 243 now).  The
// extra workgroup adds up the pairs' statistics.  Bound by memory: 161 us for
// the 0.89 GB of gradients and of logits of rows with a label (5.5 TB/s), after 78
// us of first pass and 5 us between; the second read is the price of a coefficient that needs
// the whole pair.
template <typename T, int TEAM, int UN, bool NTL, bool NTS>
__device__ inline void grad_row(const TokArgs& a, const char* x, char* g, int tid, float m, float neg, bool zero) {
  const int nfull = a.vocab / Elem<T>::VE;
  for (int j0 = 0; j0 * TEAM < nfull; j0 += UN) {
    u32x4 u[UN];
    if (!zero) {
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        const int idx = (j0 + j) * TEAM + tid;
        if (idx < nfull) u[j] = load16<NTL>(x + static_cast<int64_t>(idx) * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int idx = (j0 + j) * TEAM + tid;
      if (idx < nfull)
        store16<NTS>(g + static_cast<int64_t>(idx) * 16,
                     zero ? u32x4{0u, 0u, 0u, 0u} : grad_vec<T>(u[j], m, scale_of<T>(a), a.clo, neg));
    }
  }
}

template <typename T, int TEAM, int UN, bool NT>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) preference_grad_kernel(TokArgs a, PrefArgs p,
                                                                                  RowStats rs) {
  constexpr int VE = Elem<T>::VE;
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
  if (blockIdx.x == 0) {
    if (threadIdx.x < kWave) {
      for (int q = 0; q < 4; ++q) {
        double t = 0.0;
        for (int i = threadIdx.x; i < p.pairs; i += kWave) t += p.part[static_cast<int64_t>(i) * 4 + q];
        t = wave_sum(t);
        if (threadIdx.x == 0) {
          p.stats[q] = static_cast<float>(t);
          if (q == 0 && !finite(p.stats[0])) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
        }
      }
    }
    return;
  }
  const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM), tid = threadIdx.x % TEAM;
  const int64_t stride = static_cast<int64_t>(gridDim.x - 1) * TEAMS;
  const int nfull = a.vocab / VE, ntail = a.vocab % VE;
  for (int64_t back = static_cast<int64_t>(blockIdx.x - 1) * TEAMS + team; back < a.rows; back += stride) {
    const int64_t row = a.rows - 1 - back;
    const char* x = a.x + row * a.ldx;
    char* g = a.g + row * a.ldg;
    const float coef = p.coef[row];
    const float2 ms = rs.stat[row];
    const bool zero = coef == 0.f;
    const float neg = -coef * ms.y;
    const int32_t label = zero ? -1 : row_label(a, row);
    if (NT && row < rs.past) grad_row<T, TEAM, UN, true, NT>(a, x, g, tid, ms.x, neg, zero);
    else grad_row<T, TEAM, UN, false, NT>(a, x, g, tid, ms.x, neg, zero);
    if (tid < ntail) {
      const int64_t e = static_cast<int64_t>(nfull) * VE + tid;
      Elem<T>::store(g, e, zero ? 0.f : grad_one<T>(Elem<T>::load(x, e), ms.x, scale_of<T>(a), a.clo, neg));
    }
    if (!zero) {
      const int lv = label / VE;
      const int owner = lv < nfull ? lv % TEAM : label - nfull * VE;
      if (tid == owner) Elem<T>::store(g, label, -coef * expm1f(a.logp[row]));
    }
  }
}

__global__ void zero_stats_kernel(float* stats) {
  if (threadIdx.x < 4) stats[threadIdx.x] = 0.f;
}

TokArgs tok_args(const kfac_token_rows_t& t, char* ws) {
  const int64_t el = t.dtype == KFAC_BF16 ? 2 : 4;
  TokArgs a{};
  a.x = static_cast<const char*>(t.logits);
  a.g = static_cast<char*>(t.grad);
  a.labels = t.labels;
  a.logp = t.logp;
  a.rows = t.rows;
  a.ldx = t.ld * el;
  a.ldg = t.grad_ld * el;
  a.vocab = t.vocab;
  a.label_type = t.label_type;
  a.scale = t.logit_scale;
  const double c = static_cast<double>(t.logit_scale) * 1.4426950408889634;
  a.c = a.near = static_cast<float>(c);
  // c below the exact product and clo above 0, so that a difference of minus
  // infinity stays one in d c + d clo
  if (static_cast<double>(a.c) >= c) a.c = std::nextafter(a.c, 0.f);
  a.clo = std::max(static_cast<float>(c - static_cast<double>(a.c)), FLT_MIN);
  a.grad_scale = t.logit_scale * t.grad_scale;
  a.flags = reinterpret_cast<uint32_t*>(ws);
  return a;
}

template <typename T, int TEAM, int NV, bool LONG>
void run_policy(const TokArgs& a, const PolArgs& p, int per_cu, hipStream_t st) {
  constexpr int THREADS = TEAM < 256 ? 256 : TEAM;
  const int grid = grid_of(a.rows, THREADS / TEAM, per_cu);
  // the part of a LONG row that is read again is best left in the cache
  if (!LONG && 2 * a.rows * a.vocab * static_cast<int64_t>(sizeof(T)) > kCacheBytes)
    hipLaunchKernelGGL((policy_kernel<T, TEAM, NV, LONG, !LONG>), dim3(grid), dim3(THREADS), 0, st, a, p);
  else
    hipLaunchKernelGGL((policy_kernel<T, TEAM, NV, LONG, false>), dim3(grid), dim3(THREADS), 0, st, a, p);
}

// The team and its registers by the row's length alone: the smallest that hold
// the row, a wavefront a row as far as 512 vectors (no barriers; 16384 x 500
// bf16 with registers for 256 vectors instead of 64: 21.6 us against 17.3 us).
// From 4096 vectors one row a workgroup and compute unit: two of half the size
// would count 512 workgroups' sums in and load no faster (2047 x 50001 bf16 with
// a label in every row 98 us, 103 with two).  Past 16384 vectors half of the registers hold the row's
// start and the other half its stream: with more for the start they spill
// (1024 x 131072 f32 272 us with 12 vectors, 262 with 8).
template <typename T>
void pick_policy(const TokArgs& a, const PolArgs& p, hipStream_t st) {
  const int nvec = a.vocab / Elem<T>::VE;
  if (nvec <= 64) return run_policy<T, 64, 1, false>(a, p, 6, st);
  if (nvec <= 64 * 2) return run_policy<T, 64, 2, false>(a, p, 6, st);
  if (nvec <= 64 * 4) return run_policy<T, 64, 4, false>(a, p, 6, st);
  if (nvec <= 64 * 8) return run_policy<T, 64, 8, false>(a, p, 4, st);
  if (nvec <= 256 * 4) return run_policy<T, 256, 4, false>(a, p, 6, st);
  if (nvec <= 256 * 8) return run_policy<T, 256, 8, false>(a, p, 5, st);
  if (nvec <= 512 * 8) return run_policy<T, 512, 8, false>(a, p, 2, st);
  if (nvec <= 1024 * 8) return run_policy<T, 1024, 8, false>(a, p, 1, st);
  if (nvec <= 1024 * 16) return run_policy<T, 1024, 16, false>(a, p, 1, st);
  return run_policy<T, 1024, 8, true>(a, p, 1, st);
}

template <typename T>
void run_logp(const TokArgs& a, const RowStats& rs, hipStream_t st) {
  const int nvec = a.vocab / Elem<T>::VE;
  if (nvec <= 64)
    hipLaunchKernelGGL((logp_kernel<T, 64, 1>), dim3(grid_of(a.rows, 4, 8)), dim3(256), 0, st, a, rs);
  else if (nvec <= 64 * 8)
    hipLaunchKernelGGL((logp_kernel<T, 64, 4>), dim3(grid_of(a.rows, 4, 8)), dim3(256), 0, st, a, rs);
  else if (a.rows >= 2 * kCus)
    hipLaunchKernelGGL((logp_kernel<T, 256, 8>), dim3(grid_of(a.rows, 1, 8)), dim3(256), 0, st, a, rs);
  else
    hipLaunchKernelGGL((logp_kernel<T, 1024, 4>), dim3(grid_of(a.rows, 1, 2)), dim3(1024), 0, st, a, rs);
}

template <typename T, bool NT>
void run_pref_grad(const TokArgs& a, const PrefArgs& p, const RowStats& rs, hipStream_t st) {
  const int nvec = a.vocab / Elem<T>::VE;
  if (nvec <= 64 * 8)
    hipLaunchKernelGGL((preference_grad_kernel<T, 64, 4, NT>), dim3(1 + grid_of(a.rows, 4, 8)), dim3(256), 0, st, a,
                       p, rs);
  else if (NT || a.rows >= 2 * kCus)
    hipLaunchKernelGGL((preference_grad_kernel<T, 256, 4, NT>), dim3(1 + grid_of(a.rows, 1, 8)), dim3(256), 0, st, a,
                       p, rs);
  else      // few rows: 1024 threads each (160 rows of 16384 f32: 11 us with 256)
    hipLaunchKernelGGL((preference_grad_kernel<T, 1024, 4, false>), dim3(1 + grid_of(a.rows, 1, 2)), dim3(1024), 0, st,
                       a, p, rs);
}

template <typename T>
kfac_status_t run_preference(const TokArgs& a, const PrefArgs& q, RowStats rs, hipStream_t st) {
  const int64_t row_bytes = static_cast<int64_t>(a.vocab) * sizeof(T);
  const bool nt = 2 * a.rows * row_bytes > kCacheBytes;
  rs.past = nt ? std::max<int64_t>(0, a.rows - kCacheBytes * 3 / 4 / row_bytes) : 0;
  if (a.rows > 0) {
    run_logp<T>(a, rs, st);
    KFAC_HIP_TRY(hipGetLastError());
  }
  hipLaunchKernelGGL(preference_pair_kernel, dim3(q.pairs), dim3(kPairThreads), 0, st, a, q);
  KFAC_HIP_TRY(hipGetLastError());
  if (nt) run_pref_grad<T, true>(a, q, rs, st);
  else run_pref_grad<T, false>(a, q, rs, st);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

// Regions.  policy: part [kMaxPartials][3] double.  preference: part [pairs][4]
// double, stat [rows] float2, wide [rows] double, coef [rows] float.
struct PrefRegions {
  size_t part, stat, wide, coef, end;
};
PrefRegions pref_regions(int64_t rows, int32_t pairs) {
  PrefRegions r;
  r.part = kRegions;
  r.stat = r.part + align_up(static_cast<size_t>(pairs) * 4 * sizeof(double), 256);
  r.wide = r.stat + align_up(static_cast<size_t>(rows) * sizeof(float2), 256);
  r.coef = r.wide + align_up(static_cast<size_t>(rows) * sizeof(double), 256);
  r.end = r.coef + align_up(static_cast<size_t>(rows) * sizeof(float), 256);
  return r;
}

}  // namespace

size_t token_workspace_bytes(int objective, int64_t rows, int32_t groups) {
  if (objective == KFAC_OBJ_POLICY) return kRegions + sizeof(double) * 3 * kMaxPartials;
  if (objective == KFAC_OBJ_PREFERENCE) return pref_regions(rows, groups).end;
  return kFlagBytes;
}

kfac_status_t launch_token_logp(const kfac_token_rows_t& t, char* ws, hipStream_t st) {
  if (t.rows == 0) return KFAC_OK;
  const TokArgs a = tok_args(t, ws);
  // each logit is read once: past the cache, which serves reads as fast at any size
  const RowStats rs{nullptr, nullptr, nullptr, t.rows};
  if (t.dtype == KFAC_BF16) run_logp<__bf16>(a, rs, st);
  else run_logp<float>(a, rs, st);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

kfac_status_t launch_policy(const kfac_token_rows_t& t, const kfac_policy_t& p, char* ws, hipStream_t st) {
  if (t.rows == 0) {
    hipLaunchKernelGGL(zero_stats_kernel, dim3(1), dim3(64), 0, st, p.stats);
    KFAC_HIP_TRY(hipGetLastError());
    return KFAC_OK;
  }
  const TokArgs a = tok_args(t, ws);
  PolArgs q{};
  q.adv = p.advantage;
  q.weight = p.weight;
  q.old_logp = p.old_logp;
  q.ref = p.ref_logp;
  q.part = reinterpret_cast<uint64_t*>(ws + kRegions);
  q.lo = static_cast<float>(1.0 - static_cast<double>(p.clip_low));
  q.hi = static_cast<float>(1.0 + static_cast<double>(p.clip_high));
  q.kl = p.kl_coef;
  q.stats = p.stats;
  q.arrived = reinterpret_cast<uint32_t*>(ws + kFlagBytes);
  q.w0 = static_cast<float>(1.0 / static_cast<double>(t.rows));
  if (t.dtype == KFAC_BF16) pick_policy<__bf16>(a, q, st);
  else pick_policy<float>(a, q, st);
  KFAC_HIP_TRY(hipGetLastError());
  return KFAC_OK;
}

kfac_status_t launch_preference(const kfac_token_rows_t& t, const kfac_preference_t& p, char* ws, hipStream_t st) {
  // with no rows every sequence is empty, and the losses at h = 0 still count
  const TokArgs a = tok_args(t, ws);
  const PrefRegions r = pref_regions(t.rows, p.pairs);
  PrefArgs q{};
  q.offsets = p.offsets;
  q.ref = p.ref_logp;
  q.weight = p.pair_weight;
  q.seq = p.seq;
  q.stats = p.stats;
  q.part = reinterpret_cast<double*>(ws + r.part);
  q.coef = reinterpret_cast<float*>(ws + r.coef);
  q.pairs = p.pairs;
  q.kind = p.kind;
  q.average = p.average;
  q.beta = p.beta;
  q.eps = p.kind == KFAC_PREF_SIGMOID ? p.label_smoothing : 0.f;
  q.w0 = static_cast<float>(1.0 / p.pairs);
  RowStats rs{};
  rs.stat = reinterpret_cast<float2*>(ws + r.stat);
  rs.wide = reinterpret_cast<double*>(ws + r.wide);
  rs.coef = q.coef;
  q.wide = rs.wide;
  return t.dtype == KFAC_BF16 ? run_preference<__bf16>(a, q, rs, st) : run_preference<float>(a, q, rs, st);
}

}  // namespace kfac
