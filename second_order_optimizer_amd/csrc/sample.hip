// Sampling of a token from each row of logits (include/kfac_tokens.h).
//
// With M the row's maximum, w[i] = exp((x[i] - M) / T), and columns ordered by
// falling x, equal ones by rising number, the kept columns are a prefix of that
// order: all columns above one border (x, number), which is what is looked for.
// No row is sorted.  One workgroup a row (few long rows of which top_k keeps few:
// sixteen, which list the k largest of a part each, and one that joins the lists):
//
//   top_k  The k-th largest of the threads' own maxima is at most the row's k-th
//          largest: the columns from there on, hardly more than k, are put in a
//          list, where each finds its place by comparison with the others.  The
//          draw is made in the list.
//   top_p  Two histograms of float32 masses, over 32 bins of (M - x) / T and over 32
//          parts of the bin in which the border lies, say in which part it is; one
//          pass then takes the exact masses: of all columns, of those above the part
//          by blocks of columns, and a list of the part's.  Exact sums say whether
//          the border is in the list, where each column finds its place by
//          comparison.  The draw goes through the blocks' sums to a block, and
//          through the block to a column.
//   neither  the exact masses by blocks, and the draw.
//
// Rows that these do not settle (long runs of equal logits, a k beyond half the
// threads, a border among the unlikeliest columns) take histograms of exact masses
// and counts, narrowed by digits of (x, number) until a list holds what is left.
//
// w is held as a whole multiple of 2^-44: sums of integers have no rounding and
// no order, so that LDS atomics add them, and a border or a draw is decided as
// in 64-bit arithmetic.  It is formed in 64 bits (20 instructions a column);
// only the log-probability's sum over columns that are not kept takes the
// hardware's exp, 2^-22 off, and the first histograms, which decide nothing.  Those
// are each thread's own, 32 words of LDS 4 NT bytes apart: an LDS atomic on float32
// took 190 cycles of a compute unit a wavefront (1023 rows of 100257 columns: 126 us),
// a read, an addition and a write take 18.
#include "tokens.h"

#include <cmath>

namespace kfac {

namespace {

constexpr int kBins = 1024;
constexpr double kLog2e = 1.4426950408889634;
constexpr float kGreedy = 1e-6f;          // temperatures below this keep the maximum alone
constexpr float kBinsPerOctave = 16.f;    // 1024 bins reach 2^-64 of the maximum's weight

// What a workgroup finds in its part of a row that several take.
constexpr int kSplitRows = 16, kSplitVocab = 65536, kSplitTopK = 64, kParts = 16;
constexpr uint32_t kNoList = 0xFFFFFFFFu;
struct Head {
  double rest;             // sum of its columns' weights against its own maximum
  float top;
  uint32_t n;              // listed columns, or kNoList
  uint64_t place[kSplitTopK];      // by rank
};

struct SampleArgs {
  const char* x;
  const float *u, *row_t, *row_p, *row_m;
  const int32_t* row_k;
  int64_t* token;
  float* logp;
  int32_t* kept;
  int64_t ldx;       // bytes
  double t, p, m;
  int32_t k, vocab;
  uint32_t* flags;
  Head* heads;       // [rows][parts], or none
  int32_t parts;
};

// Columns above this one, and itself, in the order.
struct Border {
  float x;
  int32_t i;
  __device__ bool keeps(float v, int32_t at) const { return v > x || (v == x && at <= i); }
};

// (x, column) as one number that rises with the order's rank from the end.
__device__ inline uint64_t place_of(float x, int32_t i) {
  const uint32_t b = __float_as_uint(x + 0.f);       // -0 is equal to 0
  const uint32_t key = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ inline Border border_of(uint64_t place) {
  const uint32_t key = static_cast<uint32_t>(place >> 32);
  return {__uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key),
          static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(place))};
}

// 2^z in multiples of 2^-44, z <= 0: z's nearest integer is left in the low bits by
// adding 1.5 2^52; e^(r ln 2) is its series to the 11th power (|r| <= 1/2: 7e-15 of
// it is left out); and 2^52 is added so that the significand's low bits are the
// integer.
__device__ inline uint64_t mass_of(double z) {
  constexpr double shift = 6755399441055744.0;
  z = fmax(z, -60.0);
  const double t = z + shift, r = z - (t - shift);
  double e = 4.44553827187081e-10;                 // ln2^k / k!, k = 11 .. 1
  e = fma(e, r, 7.054911620801121e-09);
  e = fma(e, r, 1.0178086009239696e-07);
  e = fma(e, r, 1.3215486790144305e-06);
  e = fma(e, r, 1.5252733804059838e-05);
  e = fma(e, r, 0.00015403530393381606);
  e = fma(e, r, 0.0013333558146428441);
  e = fma(e, r, 0.009618129107628477);
  e = fma(e, r, 0.055504108664821576);
  e = fma(e, r, 0.2402265069591007);
  e = fma(e, r, 0.6931471805599453);
  e = fma(e, r, 1.0);
  // times 2^n in its exponent
  const uint64_t bits = __builtin_bit_cast(uint64_t, e) + (__builtin_bit_cast(uint64_t, t) << 52);
  const double scaled = fma(__builtin_bit_cast(double, bits), 17592186044416.0, 4503599627370496.0);
  return __builtin_bit_cast(uint64_t, scaled) - 0x4330000000000000ull;
}

// The row: vectors of 16 bytes.  Held in registers where a thread has one (HELD);
// longer rows are read again by each pass, from the caches, two vectors a thread
// ahead.  (Rows of up to 16 vectors a thread in registers left the passes too few:
// 1023 x 100257 with top_p 961 us, of which most were moves and spills.)
template <typename T, int NT, bool HELD>
struct Row {
  static constexpr int VE = Elem<T>::VE;
  const char* x;
  int nfull, ntail, nvec;
  u32x4 v;

  __device__ __forceinline__ u32x4 load(int idx) const {
    u32x4 r{Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf};
    if (idx < nfull) r = load16(x + static_cast<int64_t>(idx) * 16);
    else if (idx == nfull && ntail) {
      float f[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i)
        f[i] = i < ntail ? Elem<T>::load(x, static_cast<int64_t>(nfull) * VE + i) : -INFINITY;
      r = pack16<T>(f);
    }
    return r;
  }
  __device__ __forceinline__ void fill(const char* row, int vocab) {
    x = row;
    nfull = vocab / VE;
    ntail = vocab % VE;
    nvec = nfull + (ntail != 0);
    if constexpr (HELD) v = load(static_cast<int>(threadIdx.x));
  }
  __device__ int blocks() const { return (nvec + NT - 1) / NT; }
  // f(vector, block) over the thread's vectors in the columns' order; every lane of a
  // wavefront is there (absent columns are minus infinity).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (HELD) {
      f(v, 0);
    } else {
      const int tid = static_cast<int>(threadIdx.x), n = blocks();
      u32x4 a = load(tid), b = load(NT + tid);
#pragma unroll 1
      for (int j = 0; j < n; j += 2) {
        const u32x4 c = load((j + 2) * NT + tid), d = load((j + 3) * NT + tid);
        f(a, j);
        if (j + 1 < n) f(b, j + 1);
        a = c;
        b = d;
      }
    }
  }
  __device__ int column(int j, int i) const { return (j * NT + static_cast<int>(threadIdx.x)) * VE + i; }
};

constexpr int kOwn = 32;                  // bins of a thread's own histogram

// A listed column and its mass: sixteen bytes, one read.  A list has a column a thread
// at most, and lies in the histograms' LDS.
struct alignas(16) Listed {
  uint64_t place, mass;
};

template <int NT>
struct Shared {
  static constexpr int NW = NT / kWave;
  uint64_t mass[kBins];
  uint32_t count[kBins];
  uint64_t wave_mass[NW], sums[3][NW];
  uint32_t wave_count[NW];
  uint64_t before_mass, place_min, total_mass;
  uint32_t before_count, bin, inside, listed, total_count;
  float fmax[NW], hist[kOwn];
  int fbad[NW];
  double rest[NW];
  uint64_t chosen_base;
  int32_t chosen_block;
  uint64_t border, above_mass, list_mass;
  uint32_t above_count, chosen;
};

// What a row's columns are compared and weighed by.
struct Scale {
  float m, bins;       // maximum; bins of 1 / bins wide
  double c;            // log2(e) / T
  __device__ uint64_t mass(float x) const { return mass_of((static_cast<double>(x) - static_cast<double>(m)) * c); }
  __device__ int bin(float x) const {
    return static_cast<int>(fminf((m - x) * bins, static_cast<float>(kBins - 1)));
  }
};

// Where the border lies among n <= kBins counted bins: the first at which the
// running count reaches k, or the running mass reaches `goal` of all (by_mass).
// Returns false where all columns together do not pass it.
template <int NT>
__device__ __forceinline__ bool find_bin(Shared<NT>& s, int n, bool by_mass, uint32_t k, double goal, bool first) {
  constexpr int PER = kBins / NT;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  uint32_t c[PER], csum = 0;
  uint64_t m[PER], msum = 0;
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int b = tid * PER + q;
    c[q] = b < n ? s.count[b] : 0;
    m[q] = b < n && by_mass ? s.mass[b] : 0;
    csum += c[q];
    msum += m[q];
  }
  const uint32_t cs = wave_scan(csum);
  const uint64_t ms = by_mass ? wave_scan(msum) : 0;
  if (lane == kWave - 1) {
    s.wave_count[wave] = cs;
    s.wave_mass[wave] = ms;
  }
  __syncthreads();
  uint32_t cb = first ? 0 : s.before_count, ct = cb;
  uint64_t mb = first ? 0 : s.before_mass, mt = mb;
  for (int w = 0; w < NT / kWave; ++w) {
    if (w == wave) cb = ct, mb = mt;
    ct += s.wave_count[w];
    mt += s.wave_mass[w];
  }
  cb += cs - csum;
  mb += ms - msum;
  if (first) {
    if (by_mass) goal = fmax(goal * static_cast<double>(mt), 0.5);
    else if (ct < k) return false;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const bool here = by_mass ? static_cast<double>(mb) < goal && static_cast<double>(mb + m[q]) >= goal
                              : cb < k && cb + c[q] >= k;
    if (here && c[q]) {
      s.bin = tid * PER + q;
      s.before_count = cb;
      s.before_mass = mb;
      s.inside = c[q];
      if (first) s.total_mass = mt;
    }
    cb += c[q];
    mb += m[q];
  }
  __syncthreads();
  return true;
}

template <int NT>
__device__ __forceinline__ void clear_bins(Shared<NT>& s) {
#pragma unroll
  for (int b = threadIdx.x; b < kBins; b += NT) {
    s.count[b] = 0;
    s.mass[b] = 0;
  }
  __syncthreads();
}

// Sums over the workgroup; every thread gets them.
template <int NT, int N>
__device__ __forceinline__ void all_sums(Shared<NT>& s, uint64_t (&v)[N]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum_u64(v[i]);
  __syncthreads();
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s.sums[i][wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // a wavefront's lanes read the wavefronts' sums at once
    v[i] = wave_sum_u64(lane < NT / kWave ? s.sums[i][lane] : 0);
  }
}
template <int NT>
__device__ __forceinline__ uint64_t all_sum(Shared<NT>& s, uint64_t v) {
  uint64_t one[1] = {v};
  all_sums<NT, 1>(s, one);
  return one[0];
}

// Of a list of n columns: how many come before `mine` in the order, and their mass.
__device__ __forceinline__ void before_in_list(const Listed* list, uint32_t n, uint64_t mine, uint32_t* rank, uint64_t* mass) {
  uint32_t r = 0;
  uint64_t m = 0;
  uint32_t f = 0;
  for (; f + 8 <= n; f += 8) {
    Listed e[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) e[q] = list[f + q];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool first = e[q].place > mine;
      r += first;
      m += first ? e[q].mass : 0;
    }
  }
  for (; f < n; ++f) {
    const bool first = list[f].place > mine;
    r += first;
    m += first ? list[f].mass : 0;
  }
  *rank += r;
  *mass += m;
}

// The border of top_k (by_mass false) or top_p among the columns within `in`.
template <typename T, int NT, bool HELD>
__device__ __forceinline__ Border select(Shared<NT>& s, Listed* list, Row<T, NT, HELD>& row, const Scale& sc, Border in, bool by_mass, uint32_t k,
                         double p) {
  constexpr int VE = Elem<T>::VE;
  clear_bins<NT>(s);
  auto count = [&](u32x4 v, int j) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float x = Elem<T>::get(v, i);
      if (x > -INFINITY && in.keeps(x, row.column(j, i))) {
        const int b = sc.bin(x);
        atomicAdd(&s.count[b], 1u);
        if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), static_cast<unsigned long long>(sc.mass(x)));
      }
    }
  };
  row.each(count);
  __syncthreads();
  if (!find_bin<NT>(s, kBins, by_mass, k, p, true)) return in;
  const double goal = by_mass ? fmax(p * static_cast<double>(s.total_mass), 0.5) : 0.0;
  const int bin = s.bin;
  uint64_t digits = 0;
  int shift = 64;
  // a full bin: narrowed by eight bits of the place at a time
  while (s.inside > NT) {
    __syncthreads();
    clear_bins<NT>(s);
    shift -= 8;
    row.each([&](u32x4 v, int j) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float x = Elem<T>::get(v, i);
        if (!(x > -INFINITY) || !in.keeps(x, row.column(j, i)) || sc.bin(x) != bin) continue;
        const uint64_t place = place_of(x, row.column(j, i));
        if (shift < 56 && (place >> (shift + 8)) != digits) continue;
        const int b = 255 - static_cast<int>((place >> shift) & 255);
        atomicAdd(&s.count[b], 1u);
        if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), static_cast<unsigned long long>(sc.mass(x)));
      }
    });
    __syncthreads();
    find_bin<NT>(s, 256, by_mass, k, goal, false);
    digits = (digits << 8) | (255 - s.bin);
  }
  // the columns left, in a list, each with its place in the order
  if (threadIdx.x == 0) {
    s.listed = 0;
    s.place_min = ~0ull;
  }
  __syncthreads();
  row.each([&](u32x4 v, int j) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float x = Elem<T>::get(v, i);
      if (!(x > -INFINITY) || sc.bin(x) != bin || !in.keeps(x, row.column(j, i))) continue;
      const uint64_t place = place_of(x, row.column(j, i));
      if (shift < 64 && (place >> shift) != digits) continue;
      const uint32_t at = atomicAdd(&s.listed, 1u);
      list[at].place = place;
    }
  });
  __syncthreads();
  const uint32_t n = s.inside;
  uint64_t mine = 0;
  if (threadIdx.x < n) {
    mine = list[threadIdx.x].place;
    list[threadIdx.x].mass = by_mass ? sc.mass(border_of(mine).x) : 0;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    uint32_t rank = s.before_count;
    uint64_t mass = s.before_mass;
    before_in_list(list, n, mine, &rank, &mass);
    if (by_mass ? static_cast<double>(mass) < goal : rank < k)
      atomicMin(reinterpret_cast<unsigned long long*>(&s.place_min), static_cast<unsigned long long>(mine));
  }
  __syncthreads();
  return border_of(s.place_min);
}

// What a row's draw gives.
struct Drawn {
  int32_t token, kept;
  float x;
  double sum;            // of all w
};

// top_k, with top_p and min_p on what it keeps, and the draw, in a list of n <= NT
// columns that holds the k largest (their places are in it); the whole row's sum is
// in s.rest.
template <int NT>
__device__ __forceinline__ void draw_in_list(Shared<NT>& s, Listed* list, const Scale& sc, uint32_t n, uint32_t k, double p, float low, float u,
                                             Drawn* out) {
  const int tid = threadIdx.x;
  uint64_t mine = 0, weight = 0;
  float x = 0.f;
  int32_t column = 0;
  if (tid < n) {
    mine = list[tid].place;
    const Border b = border_of(mine);
    x = b.x;
    column = b.i;
    weight = sc.mass(x);
    list[tid].mass = weight;
  }
  __syncthreads();
  uint32_t rank = 0;
  uint64_t before = 0;
  if (tid < n) before_in_list(list, n, mine, &rank, &before);
  bool keep = tid < n && rank < k;
  if (p < 1.0) {
    const double goal = fmax(p * static_cast<double>(all_sum<NT>(s, keep ? weight : 0)), 0.5);
    keep = keep && static_cast<double>(before) < goal;
  }
  keep = keep && x >= low;
  uint64_t sums[2] = {keep ? weight : 0, keep ? 1u : 0u};
  all_sums<NT, 2>(s, sums);
  const uint64_t total = sums[0], count = sums[1];
  if (tid < n) list[tid] = {static_cast<uint32_t>(mine), keep ? weight : 0};      // in the columns' order from here on
  if (tid == 0) s.chosen = ~0u;
  __syncthreads();
  const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
  if (keep) {
    // the kept columns before this one: their places' low halves fall as the number rises
    uint64_t run = 0;
    uint32_t rank_by_number = 0;
    before_in_list(list, n, static_cast<uint32_t>(mine), &rank_by_number, &run);
    if (run <= at && at < run + weight) s.chosen = tid;
  }
  __syncthreads();
  if (tid == s.chosen) {
    double sum = 0.0;
    for (int w = 0; w < NT / kWave; ++w) sum += s.rest[w];
    *out = {column, static_cast<int32_t>(count), x, sum};
  }
}

// How far from the maximum, in bins, the k-th largest of the threads' `own` lies;
// `all` where that is no bound (fewer than k have one, or it is in the last bin).
template <int NT>
__device__ __forceinline__ float reach_of(Shared<NT>& s, const Scale& sc, float own, uint32_t k, bool* all) {
  for (int b = threadIdx.x; b < kBins; b += NT) s.count[b] = 0;
  if (threadIdx.x == 0) s.listed = 0;
  __syncthreads();
  if (own > -INFINITY) atomicAdd(&s.count[sc.bin(own)], 1u);
  __syncthreads();
  *all = !find_bin<NT>(s, kBins, false, k, 0.0, true) || s.bin == kBins - 1;
  return *all ? 0.f : static_cast<float>(s.bin + 1);
}

// The draw of a row of which top_k keeps few, in a list of the columns from the k-th
// largest of the threads' maxima (`own`) on.  False where the list does not hold them.
template <typename T, int NT, bool HELD>
__device__ __forceinline__ bool draw_of_few(Shared<NT>& s, Listed* list, Row<T, NT, HELD>& row, const Scale& sc, float own, uint32_t k, double p, float low,
                            float u, Drawn* out) {
  constexpr int VE = Elem<T>::VE;
  const int tid = threadIdx.x;
  bool all;
  const float reach = reach_of<NT>(s, sc, own, k, &all);
  const float cf = static_cast<float>(sc.c);
  double rest = 0.0;
  row.each([&](u32x4 v, int j) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float x = Elem<T>::get(v, i);
      sum += __builtin_amdgcn_exp2f((x - sc.m) * cf);
      if (((sc.m - x) * sc.bins < reach || all) && x > -INFINITY) {
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < NT) list[at].place = place_of(x, row.column(j, i));
      }
    }
    rest += static_cast<double>(sum);
  });
  rest = wave_sum(rest);
  if ((tid & (kWave - 1)) == 0) s.rest[tid / kWave] = rest;
  __syncthreads();
  if (s.listed > NT) return false;
  draw_in_list<NT>(s, list, sc, s.listed, k, p, low, u, out);
  return true;
}

// The border of top_p over the whole row, with the kept masses of the blocks of
// columns in block_mass, their number in s.above_count and the whole row's mass in
// s.total_mass.  False where the first histogram's bin does not hold it.
template <typename T, int NT, bool HELD>
__device__ __forceinline__ bool border_of_mass(Shared<NT>& s, float* own, uint64_t* block_mass, Row<T, NT, HELD>& row, const Scale& sc,
                                               double p, int vocab, Border* out) {
  constexpr int VE = Elem<T>::VE;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const float cf = static_cast<float>(sc.c);
  // columns of less than (1 - p) / vocab of the maximum's weight together weigh less
  // than 1 - p: the border is above them, and the last bin is theirs
  const float octaves = fminf(fmaxf(1.f + log2f(static_cast<float>(vocab)) - log2f(fmaxf(static_cast<float>(1.0 - p), 1e-9f)), 2.f), 60.f);
  float width = cf * (static_cast<float>(kOwn - 1) / octaves), above = 0.f, mass_above = 0.f, goal = 0.f;
  // twice: bins of (m - x) width, then parts of the bin [above, above + 1)
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    for (int i = 0; i < kOwn; ++i) own[i * NT + tid] = 0.f;
    if (tid == 0) s.bin = kOwn;
    __syncthreads();
    const float coarse = width;
    row.each([&](u32x4 v, int) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float d = sc.m - Elem<T>::get(v, i);
        const float at = d * coarse;
        if (level == 0 || (at >= above && at < above + 1.f)) {
          const int b = static_cast<int>(fminf(level == 0 ? at : (at - above) * static_cast<float>(kOwn), static_cast<float>(kOwn - 1)));
          own[b * NT + tid] += __builtin_amdgcn_exp2f(-d * cf);
        }
      }
    });
    __syncthreads();
    // the bins' sums: NT / kOwn threads each
    constexpr int PER = NT / kOwn;
    float sum = 0.f;
    for (int i = 0; i < NT / PER; ++i) sum += own[(tid / PER) * NT + i * PER + tid % PER];
#pragma unroll
    for (int d = 1; d < PER; d <<= 1) sum += __shfl_xor(sum, d);
    if (tid % PER == 0) s.hist[tid / PER] = sum;
    __syncthreads();
    if (tid < kWave) {
      const float mass = lane < kOwn ? s.hist[lane] : 0.f;
      const float upto = wave_scan(mass) + mass_above;
      if (level == 0) goal = static_cast<float>(p) * __shfl(upto, kWave - 1);
      if (mass > 0.f && upto >= goal) atomicMin(&s.bin, static_cast<uint32_t>(lane));
      if (lane < kOwn) s.hist[lane] = upto - mass;
    }
    __syncthreads();
    const int bin = s.bin;
    if (bin >= kOwn || (level == 0 && bin == kOwn - 1)) return false;
    mass_above = s.hist[bin];
    if (level == 0) above = static_cast<float>(bin);
    else s.bin = bin;
    __syncthreads();
  }
  const float part = static_cast<float>(s.bin);
  if (tid == 0) s.listed = 0;
  __syncthreads();
  Listed* list = reinterpret_cast<Listed*>(own);
  uint64_t all = 0;
  uint32_t kept = 0;
  uint64_t above_own = 0;
  row.each([&](u32x4 v, int j) {
    uint64_t mass = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float x = Elem<T>::get(v, i), at = (sc.m - x) * width;
      const float in = fminf((at - above) * static_cast<float>(kOwn), static_cast<float>(kOwn - 1));
      const uint64_t w = sc.mass(x);
      all += w;
      if (at < above || (at < above + 1.f && in < part)) {
        mass += w;
        ++kept;
      } else if (at < above + 1.f && in < part + 1.f) {
        const uint32_t to = atomicAdd(&s.listed, 1u);
        if (to < NT) list[to].place = place_of(x, row.column(j, i));
      }
    }
    above_own += mass;
    const uint64_t sum = wave_sum_u64(mass);
    if (lane == 0 && sum) atomicAdd(reinterpret_cast<unsigned long long*>(&block_mass[j]), static_cast<unsigned long long>(sum));
  });
  uint64_t sums[3] = {all, kept, above_own};
  all_sums<NT, 3>(s, sums);
  const uint64_t total = sums[0], count = sums[1], above_mass = sums[2];
  const uint32_t n = s.listed;
  const double want = fmax(p * static_cast<double>(total), 0.5);
  if (n > NT || !(static_cast<double>(above_mass) < want)) return false;
  uint64_t mine = 0, own_mass = 0;
  if (tid < n) {
    mine = list[tid].place;
    list[tid].mass = own_mass = sc.mass(border_of(mine).x);
  }
  const uint64_t list_mass = all_sum<NT>(s, own_mass);
  if (!(static_cast<double>(above_mass + list_mass) >= want)) return false;
  if (tid == 0) s.place_min = ~0ull;
  __syncthreads();
  bool keep = false;
  if (tid < n) {
    uint64_t before = above_mass;
    uint32_t rank = 0;
    before_in_list(list, n, mine, &rank, &before);
    keep = static_cast<double>(before) < want;
    if (keep) {
      atomicMin(reinterpret_cast<unsigned long long*>(&s.place_min), static_cast<unsigned long long>(mine));
      atomicAdd(reinterpret_cast<unsigned long long*>(&block_mass[border_of(mine).i / (VE * NT)]), static_cast<unsigned long long>(own_mass));
    }
  }
  const uint64_t listed = all_sum<NT>(s, keep ? 1 : 0);
  if (tid == 0) {
    s.above_count = static_cast<uint32_t>(count + listed);
    s.total_mass = total;
  }
  __syncthreads();
  *out = border_of(s.place_min);
  return true;
}

// The least float whose weight is at least m (0 < m <= 1): the comparison in 64 bits
// rises with the float, so that its first float lies between one that fails (minus
// infinity does) and one that holds (the maximum does).  These are the floats on either
// side of the border's rounding, two or three apart, but where it cancels to about 0:
// there all floats below 2^-53 of the maximum compare alike, 10^9 of them, and are
// halved 32 times at most.
__device__ inline Border min_p_border(const Scale& sc, double m) {
  const double z = log(m) * kLog2e, top = static_cast<double>(sc.m), below = z / sc.c, at = top + below;
  const double off = 0x1p-50 * (fabs(top) + fabs(below));
  auto holds = [&](float x) { return (static_cast<double>(x) - top) * sc.c >= z; };
  // floats as whole numbers in their order
  auto order = [](float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return (b >> 31) ? ~b : b | 0x80000000u;
  };
  auto float_of = [](uint32_t o) { return __builtin_bit_cast(float, (o >> 31) ? o & 0x7FFFFFFFu : ~o); };
  const uint32_t least = order(-INFINITY), most = order(sc.m);
  auto clamped = [&](uint32_t o) { return o < least ? least : o > most ? most : o; };
  uint32_t lo = clamped(order(static_cast<float>(at - off)) - 1), hi = clamped(order(static_cast<float>(at + off)) + 1);
  if (holds(float_of(lo))) lo = least;
  if (!holds(float_of(hi))) hi = most;
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (holds(float_of(mid))) hi = mid;
    else lo = mid;
  }
  return {float_of(hi), INT32_MAX};
}

// A row's settings.
struct Settings {
  float u;
  double p, m, inv_t;
  int32_t k;
  bool valid;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t r) {
  Settings s;
  s.u = a.u[r];
  const float t = a.row_t ? a.row_t[r] : static_cast<float>(a.t);
  s.p = a.row_p ? static_cast<double>(a.row_p[r]) : a.p;
  s.m = a.row_m ? static_cast<double>(a.row_m[r]) : a.m;
  s.k = a.row_k ? a.row_k[r] : a.k;
  s.valid = s.u >= 0.f && s.u < 1.f && t >= 0.f && s.p == s.p && s.m == s.m;
  s.inv_t = t < kGreedy ? 1.0 : 1.0 / fmin(a.row_t ? static_cast<double>(t) : a.t, 1e30);
  if (t < kGreedy) s.k = 1;
  return s;
}
__device__ __forceinline__ Scale scale_of(float top, double inv_t) {
  Scale sc;
  sc.m = top;
  sc.c = kLog2e * inv_t;
  sc.bins = static_cast<float>(sc.c) * kBinsPerOctave;
  return sc;
}

// A part of a row of which top_k keeps few: its maximum, its sum, and its k largest.
template <typename T>
__global__ void __launch_bounds__(256) sample_head_kernel(SampleArgs a) {
  constexpr int NT = 256, VE = Elem<T>::VE, NW = NT / kWave;
  __shared__ Shared<NT> s;
  __shared__ Listed list[NT];
  const int64_t r = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts, tid = threadIdx.x;
  Head& head = a.heads[blockIdx.x];
  Row<T, NT, false> row;
  row.fill(a.x + r * a.ldx, a.vocab);
  const int per = (row.nvec + a.parts - 1) / a.parts, v0 = part * per, v1 = min(v0 + per, row.nvec);
  const Settings set = settings_of(a, r);
  float own = -INFINITY;
  bool bad = false;
#pragma unroll 4
  for (int i = v0 + tid; i < v1; i += NT) {
    const u32x4 v = row.load(i);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float x = Elem<T>::get(v, e);
      bad |= !(x < INFINITY);
      own = fmaxf(own, x);
    }
  }
  float top = wave_max(own);
  const bool any = __any(bad);
  if (tid % kWave == 0) {
    s.fmax[tid / kWave] = top;
    s.fbad[tid / kWave] = any;
  }
  __syncthreads();
  int nan = 0;
  for (int w = 0; w < NW; ++w) {
    top = fmaxf(top, s.fmax[w]);
    nan |= s.fbad[w];
  }
  const bool few = set.valid && set.k > 0 && set.k <= kSplitTopK && !nan;
  if (!few || top == -INFINITY) {
    if (tid == 0) {
      head.rest = 0.0;
      head.top = top;
      head.n = few ? 0 : kNoList;
    }
    return;
  }
  const Scale sc = scale_of(top, set.inv_t);
  const float cf = static_cast<float>(sc.c);
  bool all;
  const float reach = reach_of<NT>(s, sc, own, static_cast<uint32_t>(set.k), &all);
  double rest = 0.0;
#pragma unroll 4
  for (int i = v0 + tid; i < v1; i += NT) {
    const u32x4 v = row.load(i);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float x = Elem<T>::get(v, e);
      sum += __builtin_amdgcn_exp2f((x - top) * cf);
      if (((top - x) * sc.bins < reach || all) && x > -INFINITY) {
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < NT) list[at] = {place_of(x, i * VE + e), 0};
      }
    }
    rest += static_cast<double>(sum);
  }
  rest = wave_sum(rest);
  if (tid % kWave == 0) s.rest[tid / kWave] = rest;
  __syncthreads();
  const uint32_t n = s.listed;
  if (n <= NT && tid < n) {
    const uint64_t mine = list[tid].place;
    uint32_t rank = 0;
    uint64_t mass = 0;
    before_in_list(list, n, mine, &rank, &mass);
    if (rank < set.k) head.place[rank] = mine;
  }
  if (tid == 0) {
    head.rest = (s.rest[0] + s.rest[1]) + (s.rest[2] + s.rest[3]);
    head.top = top;
    head.n = n <= NT ? min(n, static_cast<uint32_t>(set.k)) : kNoList;
  }
}

// The lists of a row's parts, one column a thread: the row's maximum and sum in *top
// and s.rest, the columns from the k-th largest on in `list`.  False where a part has
// no list, or they are more than the threads.
template <int NT>
__device__ __forceinline__ bool join_heads(Shared<NT>& s, Listed* list, const Head* heads, int parts, const Settings& set, Scale* sc, uint32_t* n) {
  // a lane a part: one read of memory in place of one after the other
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const uint32_t own_n = lane < parts ? heads[lane].n : 0;
  const float top = wave_max(lane < parts ? heads[lane].top : -INFINITY);
  if (__any(own_n == kNoList)) return false;
  const uint32_t upto = wave_scan(own_n), count = __shfl(upto, kWave - 1);
  if (count == 0 || count > NT) return false;
  int from = 0;
  uint32_t at = tid;
  for (int g = 0; g + 1 < parts; ++g) {
    const uint32_t end = __shfl(upto, g);
    if (static_cast<uint32_t>(tid) >= end) {
      from = g + 1;
      at = tid - end;
    }
  }
  *sc = scale_of(top, set.inv_t);
  uint64_t place = 0;
  float own = -INFINITY;
  if (static_cast<uint32_t>(tid) < count) {
    place = heads[from].place[at];
    own = border_of(place).x;
  }
  bool all;
  const float reach = reach_of<NT>(s, *sc, own, static_cast<uint32_t>(set.k), &all);
  if (own > -INFINITY && ((top - own) * sc->bins < reach || all)) list[atomicAdd(&s.listed, 1u)].place = place;
  if (tid < kWave) {
    double rest = tid < parts ? heads[tid].rest : 0.0;
    if (rest > 0.0) rest *= exp2((static_cast<double>(heads[tid].top) - static_cast<double>(top)) * sc->c);
    rest = wave_sum(rest);
    if (tid == 0) s.rest[0] = rest;
  } else if (tid % kWave == 0) {
    s.rest[tid / kWave] = 0.0;
  }
  __syncthreads();
  *n = s.listed;
  return true;
}

// The one thread that has the draw writes it.
__device__ __forceinline__ void give(const SampleArgs& a, int64_t r, const Drawn& d, const Scale& sc, double inv_t) {
  a.token[r] = d.token;
  a.logp[r] = static_cast<float>((static_cast<double>(d.x) - static_cast<double>(sc.m)) * inv_t - log(d.sum));
  a.kept[r] = d.kept;
}

template <typename T, int NT, bool HELD, bool CUT, bool SPLIT>
__global__ void __launch_bounds__(NT) sample_kernel(SampleArgs a) {
  constexpr int VE = Elem<T>::VE, NW = NT / kWave;
  __shared__ Shared<NT> s;
  extern __shared__ uint64_t block_mass[];         // kept mass of each block of NT vectors
  __shared__ Listed lists[CUT ? kOwn * NT / 4 : 1];        // or the threads' histograms
  float* histograms = reinterpret_cast<float*>(lists);
  static_assert(kOwn * NT * sizeof(float) >= NT * sizeof(Listed));
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  Row<T, NT, HELD> row;
  row.fill(a.x + r * a.ldx, a.vocab);
  const int blocks = row.blocks();
  for (int j = tid; j < blocks; j += NT) block_mass[j] = 0;

  const Settings set = settings_of(a, r);
  const float u = set.u;
  const double p = set.p, m = set.m, inv_t = set.inv_t;
  const int32_t k = set.k;
  const bool valid = set.valid;
  if constexpr (SPLIT) {
    Scale sc;
    uint32_t n;
    if (join_heads<NT>(s, lists, a.heads + r * a.parts, a.parts, set, &sc, &n)) {
      Border low{-INFINITY, -1};
      if (m > 0.0) low = min_p_border(sc, fmin(m, 1.0));
      Drawn d;
      d.token = -1;
      draw_in_list<NT>(s, lists, sc, n, static_cast<uint32_t>(k), k == 1 ? 1.0 : p, low.x, u, &d);
      if (d.token >= 0) give(a, r, d, sc, inv_t);
      return;
    }
    __syncthreads();
  }

  // maximum, and whether every value is a number below infinity
  float top = -INFINITY;
  bool bad = false;
  row.each([&](u32x4 v, int) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float x = Elem<T>::get(v, i);
      bad |= !(x < INFINITY);
      top = fmaxf(top, x);
    }
  });
  const float own = top;
  top = wave_max(top);
  const bool any_bad = __any(bad);
  if (lane == 0) {
    s.fmax[wave] = top;
    s.fbad[wave] = any_bad;
  }
  __syncthreads();
  top = s.fmax[0];
  int nan = s.fbad[0];
  for (int w = 1; w < NW; ++w) {
    top = fmaxf(top, s.fmax[w]);
    nan |= s.fbad[w];
  }
  if (!valid || nan || top == -INFINITY) {
    if (tid == 0) {
      a.token[r] = -1;
      a.logp[r] = 0.f;
      a.kept[r] = 0;
      if (nan) raise_flag(a.flags, KFAC_FLAG_NONFINITE);
      if (!valid) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    }
    return;
  }

  const Scale sc = scale_of(top, inv_t);
  Border border{-INFINITY, -1};
  bool summed = false;                       // block_mass and the count are there
  if constexpr (CUT) {
    Border low{-INFINITY, -1};
    if (m > 0.0) low = min_p_border(sc, fmin(m, 1.0));
    if (k > 0 && k <= NT / 2) {
      Drawn d;
      d.token = -1;
      if (draw_of_few<T, NT, HELD>(s, lists, row, sc, own, static_cast<uint32_t>(k), k == 1 ? 1.0 : p, low.x, u, &d)) {
        if (d.token >= 0) give(a, r, d, sc, inv_t);
        return;
      }
      __syncthreads();
    }
    if (k > 0) border = select<T, NT, HELD>(s, lists, row, sc, border, false, static_cast<uint32_t>(k), 0.0);
    if (p < 1.0 && k != 1) {
      summed = k <= 0 && border_of_mass<T, NT, HELD>(s, histograms, block_mass, row, sc, p, a.vocab, &border);
      if (!summed) border = select<T, NT, HELD>(s, lists, row, sc, border, true, 0, p);
    }
    if (low.x > border.x) {
      border = low;
      summed = false;
    }
    if (!summed) {
      __syncthreads();
      for (int j = tid; j < blocks; j += NT) block_mass[j] = 0;
      __syncthreads();
    }
  }

  // the kept mass of each block of columns, the other columns' in 32-bit terms
  if (!summed) {
    const float cf = static_cast<float>(sc.c);
    double rest = 0.0;
    uint32_t kept = 0;
    row.each([&](u32x4 v, int j) {
      uint64_t mass = 0;
      float others = 0.f;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float x = Elem<T>::get(v, i);
        if (x > -INFINITY && (!CUT || border.keeps(x, row.column(j, i)))) {
          mass += sc.mass(x);
          ++kept;
        } else if (CUT) {
          others += __builtin_amdgcn_exp2f((x - top) * cf);
        }
      }
      if (CUT) rest += static_cast<double>(others);
      if (__any(mass != 0)) {
        const uint64_t sum = wave_sum_u64(mass);
        if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&block_mass[j]), static_cast<unsigned long long>(sum));
      }
    });
    rest = wave_sum(rest);
    const uint32_t count = wave_scan(kept);
    if (lane == kWave - 1) s.wave_count[wave] = count;
    if (lane == 0) s.rest[wave] = rest;
  }
  __syncthreads();

  // the block where u falls
  if (wave == 0) {
    uint64_t total = 0;
    for (int j0 = 0; j0 < blocks; j0 += kWave) total += wave_sum_u64(j0 + lane < blocks ? block_mass[j0 + lane] : 0);
    const uint64_t at = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
    uint64_t before = 0;
    for (int j0 = 0; j0 < blocks; j0 += kWave) {
      const uint64_t own = j0 + lane < blocks ? block_mass[j0 + lane] : 0;
      const uint64_t upto = wave_scan(own) + before;
      if (upto > at && upto - own <= at) {
        s.chosen_block = j0 + lane;
        s.chosen_base = at - (upto - own);        // what is left within the block
      }
      before = lane_of(upto, kWave - 1);
    }
    if (lane == 0) s.list_mass = total;          // of the kept
  }
  __syncthreads();
  const int block = s.chosen_block;
  u32x4 v = row.load(block * NT + tid);
  uint64_t each[VE], mass = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    const float x = Elem<T>::get(v, i);
    each[i] = x > -INFINITY && (!CUT || border.keeps(x, row.column(block, i))) ? sc.mass(x) : 0;
    mass += each[i];
  }
  uint64_t upto = wave_scan(mass);
  if (lane == kWave - 1) s.wave_mass[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += s.wave_mass[w];
  const uint64_t at = s.chosen_base;
  if (upto > at && upto - mass <= at) {
    uint64_t run = upto - mass;
    int found = 0;
    float xt = 0.f;
#pragma unroll
    for (int i = VE - 1; i >= 0; --i) {
      // the last i with run + each[0 .. i) <= at and a mass of its own
      uint64_t below = run;
#pragma unroll
      for (int f = 0; f < VE; ++f)
        if (f < i) below += each[f];
      if (below <= at && at < below + each[i]) {
        found = i;
        xt = Elem<T>::get(v, i);
      }
    }
    uint32_t n = 0;
    double sum = 0.0;
    if (summed) {
      n = s.above_count;
      sum = static_cast<double>(s.total_mass) * 0x1p-44;
    } else {
      for (int w = 0; w < NW; ++w) {
        n += s.wave_count[w];
        sum += s.rest[w];
      }
      sum += static_cast<double>(s.list_mass) * 0x1p-44;
    }
    a.token[r] = row.column(block, found);
    a.logp[r] = static_cast<float>((static_cast<double>(xt) - static_cast<double>(top)) * inv_t - log(sum));
    a.kept[r] = static_cast<int32_t>(n);
  }
}

template <typename T, bool CUT>
kfac_status_t launch_typed(const SampleArgs& a, int64_t rows, hipStream_t st) {
  constexpr int VE = Elem<T>::VE;
  const int nvec = (a.vocab + VE - 1) / VE;
  auto go = [&](auto kernel, int nt) -> kfac_status_t {
    const size_t lds = sizeof(uint64_t) * ((nvec + nt - 1) / nt);
    // a launch has at most 2^31 - 1 workgroups and 2^32 - 1 threads
    const int64_t most = INT64_C(0xFFFFFFFF) / nt;
    for (int64_t r0 = 0; r0 < rows; r0 += most) {
      SampleArgs b = a;
      const int64_t n = rows - r0 < most ? rows - r0 : most;
      b.x += r0 * a.ldx;
      b.u += r0;
      if (b.row_t) b.row_t += r0;
      if (b.row_k) b.row_k += r0;
      if (b.row_p) b.row_p += r0;
      if (b.row_m) b.row_m += r0;
      b.token += r0;
      b.logp += r0;
      b.kept += r0;
      hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(n)), dim3(nt), lds, st, b);
      if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
    }
    return KFAC_OK;
  };
  // Wavefronts enough to fill the compute units with the rows that there are: a
  // workgroup of 1024 threads a unit, or two of 512, or (short rows) many of 256.
  if (nvec <= 256) return go(sample_kernel<T, 256, true, CUT, false>, 256);
  if (nvec <= 1024) return go(sample_kernel<T, 256, false, CUT, false>, 256);
  if (rows > 256) return go(sample_kernel<T, 512, false, CUT, false>, 512);
  if constexpr (CUT) {
    // few rows of which top_k keeps few: several workgroups a row find the largest
    // columns of a part each
    if (a.heads) {
      hipLaunchKernelGGL(sample_head_kernel<T>, dim3(static_cast<uint32_t>(rows * a.parts)), dim3(256), 0, st, a);
      return go(sample_kernel<T, 1024, false, CUT, true>, 1024);
    }
  }
  return go(sample_kernel<T, 1024, false, CUT, false>, 1024);
}

}  // namespace

// Workgroups of a row, where few long rows leave most compute units idle; 0: one alone.
// (Two launches, a row as far as 131072 columns: 20 us against 30 alone; 8 rows of
// 50000 21 against 22, one of 16384 13 against 11.)
int sample_parts(int64_t rows, int32_t vocab) {
  if (rows > kSplitRows || vocab < kSplitVocab) return 0;
  return kParts;
}
size_t sample_workspace_bytes(int64_t rows, int32_t vocab) {
  return kRegions + align_up(sizeof(Head) * static_cast<size_t>(rows) * sample_parts(rows, vocab), 256);
}

kfac_status_t launch_sample(const kfac_sample_t& s, char* ws, hipStream_t st) {
  if (s.rows == 0) return KFAC_OK;
  SampleArgs a{};
  a.x = static_cast<const char*>(s.logits);
  a.u = s.u;
  a.row_t = s.row_temperature;
  a.row_k = s.row_top_k;
  a.row_p = s.row_top_p;
  a.row_m = s.row_min_p;
  a.token = s.token;
  a.logp = s.logp;
  a.kept = s.kept;
  a.ldx = s.ld * (s.dtype == KFAC_BF16 ? 2 : 4);
  a.t = s.temperature;
  a.p = s.top_p;
  a.m = s.min_p;
  a.k = s.top_k;
  a.vocab = s.vocab;
  a.flags = reinterpret_cast<uint32_t*>(ws);
  a.parts = sample_parts(s.rows, s.vocab);
  // (with top_k by row the rows without it take the longest, and the parts' launch is lost)
  if (a.parts && !s.row_top_k && ((s.top_k > 0 && s.top_k <= kSplitTopK) || (!s.row_temperature && s.temperature < kGreedy)))
    a.heads = reinterpret_cast<Head*>(ws + kRegions);
  const bool cut = s.row_temperature || s.row_top_k || s.row_top_p || s.row_min_p || s.top_k > 0 || s.top_p < 1.0 ||
                   s.min_p > 0.0 || s.temperature < kGreedy;
  if (s.dtype == KFAC_BF16) return cut ? launch_typed<__bf16, true>(a, s.rows, st) : launch_typed<__bf16, false>(a, s.rows, st);
  return cut ? launch_typed<float, true>(a, s.rows, st) : launch_typed<float, false>(a, s.rows, st);
}

}  // namespace kfac
