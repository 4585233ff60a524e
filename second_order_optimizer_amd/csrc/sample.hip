// Sampling of a token from each row of logits (include/kfac_tokens.h).
//
// With M the row's maximum, w[i] = exp((x[i] - M) / T), and columns ordered by
// falling x, equal ones by rising number, the kept columns are a prefix of that
// order: all columns above one border (x, number), which is what is looked for.
// No row is sorted.  One workgroup a row:
//
//   1. the row is read once, into registers, with its maximum;
//   2. for top_k a histogram of counts, for top_p one of masses, over 1024 bins
//      of (M - x) / T: the bin in which the border lies;
//   3. that bin's columns, a few hundred at most in practice, are put in a list
//      and each finds its place in the order by comparison with the others (a
//      bin with more is narrowed by digits of (x, number) first);
//   4. sums of the kept w, a column block at a time, in the columns' order, and
//      the token in the block where u falls.
//
// w is held as a whole multiple of 2^-44: sums of integers have no rounding and
// no order, so that LDS atomics add them, and a border or a draw is decided as
// in 64-bit arithmetic.  It is formed in 64 bits (20 instructions a column);
// only the log-probability's sum over columns that are not kept takes the
// hardware's exp, 2^-22 off.
#include "tokens.h"

#include <cmath>

namespace kfac {

namespace {

constexpr int kBins = 1024;
constexpr double kLog2e = 1.4426950408889634;
constexpr float kGreedy = 1e-6f;          // temperatures below this keep the maximum alone
constexpr float kBinsPerOctave = 16.f;    // 1024 bins reach 2^-64 of the maximum's weight
constexpr int kMassBits = 44;

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

// 2^z in multiples of 2^-44, z <= 0: e^(r ln 2) as its series to the 11th power
// (|r| <= 1/2: 7e-15 of it is left out), and 2^52 added so that the significand's
// low bits are the integer.
__device__ inline uint64_t mass_of(double z) {
  z = fmax(z, -60.0);
  const double n = rint(z), r = z - n;
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
  const double scaled = ldexp(e, static_cast<int>(n) + kMassBits) + 4503599627370496.0;
  return __builtin_bit_cast(uint64_t, scaled) - 0x4330000000000000ull;
}

// The row: vectors of 16 bytes, NV a thread in registers, the others read again.
template <typename T, int NT, int NV>
struct Row {
  static constexpr int VE = Elem<T>::VE;
  const char* x;
  int nfull, ntail, nvec;
  u32x4 v[NV];

  __device__ u32x4 load(int idx) const {
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
  __device__ void fill(const char* row, int vocab) {
    x = row;
    nfull = vocab / VE;
    ntail = vocab % VE;
    nvec = nfull + (ntail != 0);
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = load(j * NT + static_cast<int>(threadIdx.x));
  }
  __device__ int blocks() const { return (nvec + NT - 1) / NT; }
  // f(vector, block) over the thread's vectors in the columns' order.
  template <typename F>
  __device__ void each(F f) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * NT < nvec) f(v[j], j);
    for (int j = NV; j * NT < nvec; ++j) f(load(j * NT + static_cast<int>(threadIdx.x)), j);
  }
  // The same for long bodies, which are laid out CH times and not NV times: the
  // registers move round.
  template <typename F>
  __device__ void each_long(F f) {
    constexpr int CH = NV < 4 ? NV : 4;
#pragma unroll 1
    for (int j0 = 0; j0 < NV; j0 += CH) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if ((j0 + j) * NT < nvec) f(v[j], j0 + j);
      if constexpr (NV > CH) {
        u32x4 t[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) t[j] = v[j];
#pragma unroll
        for (int j = 0; j + CH < NV; ++j) v[j] = v[j + CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) v[NV - CH + j] = t[j];
      }
    }
    for (int j = NV; j * NT < nvec; ++j) f(load(j * NT + static_cast<int>(threadIdx.x)), j);
  }
  __device__ int column(int j, int i) const { return (j * NT + static_cast<int>(threadIdx.x)) * VE + i; }
};

template <int NT>
struct Shared {
  static constexpr int NW = NT / kWave;
  uint64_t mass[kBins];
  uint64_t place[NT], weight[NT];         // a bin's columns
  uint32_t count[kBins];
  uint64_t wave_mass[NW];
  uint32_t wave_count[NW];
  uint64_t before_mass, place_min, total_mass;
  uint32_t before_count, bin, inside, listed, total_count;
  float fmax[NW];
  int fbad[NW];
  double rest[NW];
  uint64_t chosen_base;
  int32_t chosen_block;
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
__device__ bool find_bin(Shared<NT>& s, int n, bool by_mass, uint32_t k, double goal, bool first) {
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
    else if (ct <= k) return false;
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
__device__ void clear_bins(Shared<NT>& s) {
#pragma unroll
  for (int b = threadIdx.x; b < kBins; b += NT) {
    s.count[b] = 0;
    s.mass[b] = 0;
  }
  __syncthreads();
}

// The border of top_k (by_mass false) or top_p among the columns within `in`.
template <typename T, int NT, int NV>
__device__ Border select(Shared<NT>& s, Row<T, NT, NV>& row, const Scale& sc, Border in, bool by_mass, uint32_t k,
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
  row.each_long(count);
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
    row.each_long([&](u32x4 v, int j) {
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
      s.place[at] = place;
    }
  });
  __syncthreads();
  const uint32_t n = s.inside;
  uint64_t mine = 0;
  if (threadIdx.x < n) {
    mine = s.place[threadIdx.x];
    if (by_mass) s.weight[threadIdx.x] = sc.mass(border_of(mine).x);
  }
  __syncthreads();
  if (threadIdx.x < n) {
    uint32_t rank = s.before_count;
    uint64_t mass = s.before_mass;
    for (uint32_t f = 0; f < n; ++f) {
      if (s.place[f] > mine) {
        ++rank;
        if (by_mass) mass += s.weight[f];
      }
    }
    if (by_mass ? static_cast<double>(mass) < goal : rank < k)
      atomicMin(reinterpret_cast<unsigned long long*>(&s.place_min), static_cast<unsigned long long>(mine));
  }
  __syncthreads();
  return border_of(s.place_min);
}

// The least float whose weight is at least m (0 < m <= 1).
__device__ inline Border min_p_border(const Scale& sc, double m) {
  const double z = log(m) * kLog2e;
  auto holds = [&](float x) { return (static_cast<double>(x) - static_cast<double>(sc.m)) * sc.c >= z; };
  float x = fminf(static_cast<float>(static_cast<double>(sc.m) + z / sc.c), sc.m);
  while (!holds(x) && x < sc.m) x = nextafterf(x, INFINITY);
  for (float y = nextafterf(x, -INFINITY); y > -INFINITY && holds(y); y = nextafterf(x, -INFINITY)) x = y;
  return {x, INT32_MAX};
}

template <typename T, int NT, int NV, bool CUT>
__global__ void __launch_bounds__(NT) sample_kernel(SampleArgs a) {
  constexpr int VE = Elem<T>::VE, NW = NT / kWave;
  __shared__ Shared<NT> s;
  extern __shared__ uint64_t block_mass[];        // kept mass of each block of NT vectors
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  Row<T, NT, NV> row;
  row.fill(a.x + r * a.ldx, a.vocab);
  const int blocks = row.blocks();
  for (int j = tid; j < blocks; j += NT) block_mass[j] = 0;

  // the row's settings
  const float u = a.u[r];
  float t = a.row_t ? a.row_t[r] : static_cast<float>(a.t);
  double p = a.row_p ? static_cast<double>(a.row_p[r]) : a.p, m = a.row_m ? static_cast<double>(a.row_m[r]) : a.m;
  int32_t k = a.row_k ? a.row_k[r] : a.k;
  const bool valid = u >= 0.f && u < 1.f && t >= 0.f && p == p && m == m;
  const double inv_t = t < kGreedy ? 1.0 : 1.0 / (a.row_t ? static_cast<double>(t) : a.t);
  if (t < kGreedy) k = 1;

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

  Scale sc;
  sc.m = top;
  sc.c = kLog2e * inv_t;
  sc.bins = static_cast<float>(sc.c) * kBinsPerOctave;
  Border border{-INFINITY, -1};
  if constexpr (CUT) {
    if (k > 0) border = select<T, NT, NV>(s, row, sc, border, false, static_cast<uint32_t>(k), 0.0);
    if (p < 1.0 && k != 1) border = select<T, NT, NV>(s, row, sc, border, true, 0, p);
    if (m > 0.0) {
      const Border low = min_p_border(sc, fmin(m, 1.0));
      if (low.x > border.x) border = low;
    }
  }

  // the kept mass of each block of columns, the other columns' in 32-bit terms
  const float cf = static_cast<float>(sc.c);
  double rest = 0.0;
  uint32_t kept = 0;
  row.each_long([&](u32x4 v, int j) {
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
  uint32_t count = wave_scan(kept);
  if (lane == kWave - 1) s.wave_count[wave] = count;
  if (lane == 0) s.rest[wave] = rest;
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
    if (lane == 0) s.total_mass = total;
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
    double others = 0.0;
    for (int w = 0; w < NW; ++w) {
      n += s.wave_count[w];
      others += s.rest[w];
    }
    const double sum = static_cast<double>(s.total_mass) * 0x1p-44 + others;
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
  if (nvec <= 256) return go(sample_kernel<T, 256, 1, CUT>, 256);
  if (nvec <= 1024) return go(sample_kernel<T, 256, 4, CUT>, 256);
  if (nvec <= 4096) return go(sample_kernel<T, 1024, 4, CUT>, 1024);
  if (nvec <= 8192) return go(sample_kernel<T, 1024, 8, CUT>, 1024);
  return go(sample_kernel<T, 1024, 16, CUT>, 1024);
}

}  // namespace

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
  const bool cut = s.row_temperature || s.row_top_k || s.row_top_p || s.row_min_p || s.top_k > 0 || s.top_p < 1.0 ||
                   s.min_p > 0.0 || s.temperature < kGreedy;
  if (s.dtype == KFAC_BF16) return cut ? launch_typed<__bf16, true>(a, s.rows, st) : launch_typed<__bf16, false>(a, s.rows, st);
  return cut ? launch_typed<float, true>(a, s.rows, st) : launch_typed<float, false>(a, s.rows, st);
}

}  // namespace kfac
