// Embedding lookup and its gradient (include/kfac_tokens.h).
//
// Both are bound by HBM: the lookup reads T rows and writes T, the gradient
// reads the T rows of dy and writes the table's V rows whole.
//
// The gradient adds a token's rows in the order of their positions, so that it
// does not depend on scheduling: positions are sorted by token with a stable
// radix sort (tiles of positions, a histogram and a scatter a pass), a token's
// rows are then a run of the sorted positions.  These are cut into tiles of equal
// length, whatever the tokens: a wavefront adds a tile's rows one after the other
// and writes each token's sum as its run ends.  A run that crosses a tile's border
// leaves a part in each tile, and the tile in which it begins has them joined, in
// order.  So a token that fills a tenth of the batch is many wavefronts' work, and
// one of which the batch has a single row no wavefront's of its own.
#include "tokens.h"

#include <algorithm>
#include <type_traits>

namespace kfac {

namespace {

constexpr int kThreads = 256;
constexpr int kSortWaves = 8, kSortThreads = kSortWaves * kWave;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kMostTiles = 256;           // tiles of a sort: every workgroup of a scatter reads all their histograms
constexpr int kLeastTile = 1024;
constexpr int kAhead = 8;                 // rows asked for before they are added
constexpr int kTile = 32;                 // sorted positions of a tile: fewer where there are few, so that
constexpr int kSumTiles = 1024;           // enough workgroups run, more where there are many, so that few
constexpr int kMostSumTiles = 4096;       // parts are joined

struct SortPlan {
  int64_t tile;       // positions a workgroup sorts, a multiple of kSortThreads
  int tiles, passes, bits;
};
SortPlan sort_plan(int64_t tokens, int32_t vocab) {
  SortPlan p;
  p.tile = kLeastTile;
  if (tokens > p.tile * kMostTiles) p.tile = ((tokens + kMostTiles - 1) / kMostTiles + kSortThreads - 1) / kSortThreads * kSortThreads;
  p.tiles = static_cast<int>((tokens + p.tile - 1) / p.tile);
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;      // vocab itself stands for ids that are none
  p.passes = (bits + kDigitBits - 1) / kDigitBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  return p;
}

// Floats of a part: a row's columns, in whole vectors of a lane.
size_t part_ld(int32_t width) { return align_up(static_cast<size_t>(width), 8); }

// Sorted positions of a tile of the sums.
int sum_tile(int64_t tokens) {
  auto share = [&](int tiles, int of) { return ((tokens + tiles - 1) / tiles + of - 1) / of * of; };
  return static_cast<int>(std::max(std::min<int64_t>(kTile, std::max<int64_t>(kAhead, share(kSumTiles, kAhead))), share(kMostSumTiles, kTile) <= kTile ? 0 : share(kMostSumTiles, kTile)));
}

struct Regions {
  size_t keys[2], perm[2], hist, partial, bytes;
};
Regions regions(int64_t tokens, int32_t vocab, int32_t width) {
  const SortPlan p = sort_plan(tokens, vocab);
  Regions r;
  size_t at = kRegions;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = align_up(at + n, 256);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    r.keys[i] = take(4 * static_cast<size_t>(tokens));
    r.perm[i] = take(4 * static_cast<size_t>(tokens));
  }
  r.hist = take(4 * static_cast<size_t>(p.tiles) * kDigits);
  const int64_t tile = sum_tile(tokens);
  r.partial = take(8 * part_ld(width) * static_cast<size_t>((tokens + tile - 1) / tile));
  r.bytes = at;
  return r;
}

// -- vectors ----------------------------------------------------------------

// N values of a row from column c on, of `width` columns; those past it read as 0.
template <typename T, int N, bool NT = false>
__device__ inline void load_cols(float (&f)[N], const char* row, int c, int width) {
  constexpr int VE = Elem<T>::VE;
  if (c + N <= width) {
    if constexpr (N >= VE) {
#pragma unroll
      for (int q = 0; q < N / VE; ++q) {
        const u32x4 v = load16<NT>(row + static_cast<int64_t>(c + q * VE) * sizeof(T));
#pragma unroll
        for (int i = 0; i < VE; ++i) f[q * VE + i] = Elem<T>::get(v, i);
      }
    } else {
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(row + static_cast<int64_t>(c) * sizeof(T));
      const u32x4 w{v[0], v[1], 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = Elem<T>::get(w, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = c + i < width ? Elem<T>::load(row, c + i) : 0.f;
  }
}
template <typename T, int N, bool NT = false>
__device__ inline void store_cols(char* row, int c, int width, const float (&f)[N]) {
  constexpr int VE = Elem<T>::VE;
  if (c + N <= width) {
    if constexpr (N >= VE) {
#pragma unroll
      for (int q = 0; q < N / VE; ++q) store16<NT>(row + static_cast<int64_t>(c + q * VE) * sizeof(T), pack16<T>(f + q * VE));
    } else {
      float g[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) g[i] = i < N ? f[i] : 0.f;
      const u32x4 w = pack16<T>(g);
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<u32x2_any*>(row + static_cast<int64_t>(c) * sizeof(T)) = u32x2_any{w[0], w[1]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < width) Elem<T>::store(row, c + i, f[i]);
  }
}
// Columns a lane takes at a time: 16 bytes of the wider type, so that the lanes of
// a store lie side by side (two stores of 16 bytes a lane, 32 bytes apart between
// lanes, past the cache: 65536 x 4096 f32 422 instead of 178 us).
template <typename TT, typename TY>
constexpr int kCols = Elem<TT>::VE < Elem<TY>::VE ? Elem<TT>::VE : Elem<TY>::VE;

// -- lookup -----------------------------------------------------------------

struct LookupArgs {
  const char* table;
  char* y;
  const void* ids;
  int64_t tokens, table_ld, y_ld;      // strides in bytes
  int32_t vocab, width, id_type;
  float scale;
  uint32_t* flags;
};

template <typename TT, typename TY, int TEAM, bool NT>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs a) {
  constexpr int N = Elem<TY>::VE, TEAMS = kThreads / TEAM;
  const int lane = threadIdx.x % TEAM;
  const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM; t < a.tokens; t += step) {
    const int64_t id = load_index(a.ids, t, a.id_type);
    const bool there = id >= 0 && id < a.vocab;
    if (id >= a.vocab && lane == 0) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    const char* from = a.table + (there ? id : 0) * a.table_ld;
    char* to = a.y + t * a.y_ld;
    for (int c = lane * N; c < a.width; c += TEAM * N) {
      float f[N];
      if (there) {
        load_cols<TT, N>(f, from, c, a.width);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] *= a.scale;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = 0.f;
      }
      store_cols<TY, N, NT>(to, c, a.width, f);
    }
  }
}

// -- positions sorted by token ------------------------------------------------

struct SortArgs {
  const void* ids;              // the first pass reads these
  const uint32_t *keys, *perm;  // later ones these
  uint32_t *keys_out, *perm_out, *hist;
  int64_t tokens, tile;
  int32_t vocab, id_type, shift, bits, tiles;
  uint32_t* flags;
};

template <bool FIRST>
__device__ inline uint32_t key_at(const SortArgs& a, int64_t t) {
  if constexpr (!FIRST) return a.keys[t];
  const int64_t id = load_index(a.ids, t, a.id_type);
  return id >= 0 && id < a.vocab ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.vocab);
}

// How often each digit occurs in each tile.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) digits_kernel(SortArgs a) {
  __shared__ uint32_t count[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) count[d] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.tokens);
  const uint32_t mask = (1u << a.bits) - 1;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads) {
    if (FIRST && load_index(a.ids, t, a.id_type) >= a.vocab) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    atomicAdd(&count[(key_at<FIRST>(a, t) >> a.shift) & mask], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) a.hist[static_cast<int64_t>(blockIdx.x) * kDigits + d] = count[d];
}

// Moves a tile's positions to their places: those of all smaller digits, of the
// same digit in earlier tiles, in earlier wavefronts of this one (each has a run
// of the tile) and in earlier rounds and lanes.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) scatter_kernel(SortArgs a) {
  static_assert(kDigits == kSortThreads, "a thread for each digit");
  __shared__ uint32_t base[kSortWaves][kDigits];
  __shared__ uint32_t wave_total[kSortWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int w = 0; w < kSortWaves; ++w) base[w][tid] = 0;
  // this digit in earlier tiles, and in all
  uint32_t before = 0, total = 0;
#pragma unroll 8
  for (int b = 0; b < a.tiles; ++b) {
    const uint32_t n = a.hist[static_cast<int64_t>(b) * kDigits + tid];
    before += b < static_cast<int>(blockIdx.x) ? n : 0;
    total += n;
  }
  const uint32_t upto = wave_scan(total);
  if (lane == kWave - 1) wave_total[wave] = upto;
  __syncthreads();
  uint32_t place = upto - total + before;
  for (int w = 0; w < wave; ++w) place += wave_total[w];

  const int64_t t0 = blockIdx.x * a.tile, t1 = min(t0 + a.tile, a.tokens);
  const int64_t run = a.tile / kSortWaves;
  const int64_t r0 = t0 + wave * run, r1 = min(r0 + run, t1);
  for (int64_t t = r0 + lane; t < r1; t += kWave) atomicAdd(&base[wave][(key_at<FIRST>(a, t) >> a.shift) & mask], 1u);
  __syncthreads();
  for (int w = 0; w < kSortWaves; ++w) {
    const uint32_t n = base[w][tid];
    base[w][tid] = place;
    place += n;
  }
  __syncthreads();
  for (int64_t t = r0; t < r1; t += kWave) {
    const bool in = t + lane < r1;
    const uint32_t key = in ? key_at<FIRST>(a, t + lane) : 0;
    const uint32_t digit = (key >> a.shift) & mask;
    uint64_t same = __ballot(in);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t set = __ballot((digit >> b) & 1);
      same &= (digit >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    uint32_t to = 0;
    if (in) to = base[wave][digit] + rank;
    __builtin_amdgcn_wave_barrier();
    if (in && rank == 0) base[wave][digit] = to + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      a.keys_out[to] = key;
      a.perm_out[to] = FIRST ? static_cast<uint32_t>(t + lane) : a.perm[t + lane];
    }
  }
}

// The whole sort of up to kSmall positions in one workgroup, in LDS.
constexpr int kSmall = 8192;
constexpr int kSmallWaves = 16, kSmallThreads = kSmallWaves * kWave;

__global__ void __launch_bounds__(kSmallThreads) sort_small_kernel(SortArgs a, int passes) {
  __shared__ uint32_t keys[2][kSmall];
  __shared__ uint16_t perm[2][kSmall];
  __shared__ uint32_t base[kSmallWaves][kDigits];
  __shared__ uint32_t wave_total[kDigits / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int n = static_cast<int>(a.tokens);
  const uint32_t mask = (1u << a.bits) - 1;
  for (int t = tid; t < n; t += kSmallThreads) {
    if (load_index(a.ids, t, a.id_type) >= a.vocab) raise_flag(a.flags, KFAC_FLAG_BAD_INDEX);
    keys[0][t] = key_at<true>(a, t);
    perm[0][t] = static_cast<uint16_t>(t);
  }
  const int run = ((n + kSmallWaves - 1) / kSmallWaves + kWave - 1) / kWave * kWave;
  const int r0 = wave * run, r1 = min(r0 + run, n);
  for (int pass = 0; pass < passes; ++pass) {
    const int from = pass & 1, shift = pass * a.bits;
    for (int i = tid; i < kSmallWaves * kDigits; i += kSmallThreads) base[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    for (int t = r0 + lane; t < r1; t += kWave) atomicAdd(&base[wave][(keys[from][t] >> shift) & mask], 1u);
    __syncthreads();
    uint32_t total = 0, upto = 0;
    if (tid < kDigits) {
      for (int w = 0; w < kSmallWaves; ++w) total += base[w][tid];
      upto = wave_scan(total);
      if (lane == kWave - 1) wave_total[wave] = upto;
    }
    __syncthreads();
    if (tid < kDigits) {
      uint32_t place = upto - total;
      for (int w = 0; w < wave; ++w) place += wave_total[w];
      for (int w = 0; w < kSmallWaves; ++w) {
        const uint32_t c = base[w][tid];
        base[w][tid] = place;
        place += c;
      }
    }
    __syncthreads();
    for (int t = r0; t < r1; t += kWave) {
      const bool in = t + lane < r1;
      const uint32_t key = in ? keys[from][t + lane] : 0;
      const uint32_t digit = (key >> shift) & mask;
      uint64_t same = __ballot(in);
      for (int b = 0; b < a.bits; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1);
        same &= (digit >> b) & 1 ? set : ~set;
      }
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      uint32_t to = 0;
      if (in) to = base[wave][digit] + rank;
      __builtin_amdgcn_wave_barrier();
      if (in && rank == 0) base[wave][digit] = to + __popcll(same);
      __builtin_amdgcn_wave_barrier();
      if (in) {
        const uint32_t position = perm[from][t + lane];
        if (pass + 1 == passes) {
          a.keys_out[to] = key;
          a.perm_out[to] = position;
        } else {
          keys[from ^ 1][to] = key;
          perm[from ^ 1][to] = static_cast<uint16_t>(position);
        }
      }
    }
    __syncthreads();
  }
}

// -- sums -------------------------------------------------------------------

struct SumArgs {
  const char* dy;
  char* grad;
  int32_t* counts;
  const uint32_t *keys, *perm;
  float* partial;                      // [tiles][2][part_ld]
  int64_t tokens, dy_ld, grad_ld, part_ld;      // strides of dy and grad in bytes
  int32_t vocab, width, accumulate, tile;
  int32_t tiles, fill_first;           // the first group of tokens that the join's launch fills
  float scale;
};

// The first sorted position whose token is at least v.
__device__ inline int64_t first_at(const uint32_t* keys, int64_t n, uint32_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <typename TT, int N, bool NT>
__device__ inline void write_sum(const SumArgs& a, int64_t v, int c, const float (&s)[N]) {
  char* row = a.grad + v * a.grad_ld;
  float f[N];
  if (a.accumulate) {
    load_cols<TT, N>(f, row, c, a.width);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fmaf(s[i], a.scale, f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = s[i] * a.scale;
  }
  store_cols<TT, N, NT>(row, c, a.width, f);
}
template <int N>
__device__ inline void write_part(const SumArgs& a, int64_t tile, int which, int c, const float (&s)[N]) {
  float* to = a.partial + (tile * 2 + which) * a.part_ld + c;
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4*>(to + i) = f32x4{s[i], s[i + 1], s[i + 2], s[i + 3]};
}

// Counts, and zeros for the tokens that do not occur, of 64 tokens.
template <typename TT, typename TY, bool NT>
__device__ inline void fill(const SumArgs& a, int group) {
  constexpr int N = kCols<TT, TY>;
  __shared__ int64_t start[kWave + 1];
  const int64_t v0 = static_cast<int64_t>(group) * kWave;
  for (int i = threadIdx.x; i <= kWave; i += blockDim.x)
    start[i] = first_at(a.keys, a.tokens, static_cast<uint32_t>(min(v0 + i, static_cast<int64_t>(a.vocab))));
  __syncthreads();
  if (a.counts && blockIdx.y == 0 && threadIdx.x < kWave && v0 + threadIdx.x < a.vocab)
    a.counts[v0 + threadIdx.x] = static_cast<int32_t>(start[threadIdx.x + 1] - start[threadIdx.x]);
  if (a.accumulate) return;
  const float zero[N] = {};
  for (int i = blockIdx.y; i < kWave && v0 + i < a.vocab; i += gridDim.y)        // whole rows, one after the other
    if (start[i] == start[i + 1])
      for (int c = threadIdx.x * N; c < a.width; c += blockDim.x * N) store_cols<TT, N, NT>(a.grad + (v0 + i) * a.grad_ld, c, a.width, zero);
}

// A tile of sorted positions a workgroup (further ones fill), kAhead rows asked for before they are
// added.  Part 0 of a tile is the run that began before it, part 1 the one that
// goes on after it (a run that does both is part 0).
template <typename TT, typename TY, bool NT>
__global__ void __launch_bounds__(kThreads) sums_kernel(SumArgs a) {
  constexpr int N = kCols<TT, TY>;
  if (static_cast<int>(blockIdx.x) >= a.tiles) return fill<TT, TY, NT>(a, blockIdx.x - a.tiles);
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile, t1 = min(t0 + a.tile, a.tokens);
  if (c >= a.width) return;
  const uint32_t none = static_cast<uint32_t>(a.vocab);
  float s[N] = {};
  uint32_t run = a.keys[t0];
  bool head = t0 > 0 && a.keys[t0 - 1] == run;        // the run began before the tile
  for (int64_t p0 = t0; p0 < t1 && run != none; p0 += kAhead) {
    float f[kAhead][N];
    uint32_t key[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t p = min(p0 + j, t1 - 1);
      key[j] = a.keys[p];
      load_cols<TY, N, NT>(f[j], a.dy + a.perm[p] * a.dy_ld, c, a.width);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (p0 + j >= t1) break;
      if (key[j] != run) {
        if (head) write_part<N>(a, blockIdx.x, 0, c, s);
        else write_sum<TT, N, NT>(a, run, c, s);
        head = false;
        run = key[j];
        if (run == none) break;                       // what is left are positions without a token
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = f[j][i];
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += f[j][i];
      }
    }
  }
  if (run == none) return;
  if (head) write_part<N>(a, blockIdx.x, 0, c, s);
  else if (t1 < a.tokens && a.keys[t1] == run) write_part<N>(a, blockIdx.x, 1, c, s);
  else write_sum<TT, N, NT>(a, run, c, s);
}

// The sum of the run that begins in a tile and goes on after it; further workgroups fill.
template <typename TT, typename TY, bool NT>
__global__ void __launch_bounds__(kThreads) join_kernel(SumArgs a) {
  constexpr int N = kCols<TT, TY>;
  if (static_cast<int>(blockIdx.x) >= a.tiles) return fill<TT, TY, NT>(a, blockIdx.x - a.tiles + a.fill_first);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile, t1 = t0 + a.tile;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  if (t1 >= a.tokens || c >= a.width) return;
  const uint32_t v = a.keys[t1 - 1];
  if (v == static_cast<uint32_t>(a.vocab) || a.keys[t1] != v || (a.keys[t0] == v && t0 > 0 && a.keys[t0 - 1] == v)) return;
  const int64_t last = (first_at(a.keys, a.tokens, v + 1) - 1) / a.tile;
  float s[N];
  const float* from = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * a.part_ld + c;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = from[i];
  int64_t tile = blockIdx.x + 1;
  for (; tile + kAhead <= last + 1; tile += kAhead) {
    f32x4 f[kAhead][N / 4];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int q = 0; q < N / 4; ++q)
        f[j][q] = *reinterpret_cast<const f32x4*>(a.partial + (tile + j) * 2 * a.part_ld + c + 4 * q);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += f[j][i / 4][i % 4];
  }
  for (; tile <= last; ++tile) {
    const float* f = a.partial + tile * 2 * a.part_ld + c;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += f[i];
  }
  write_sum<TT, N, NT>(a, v, c, s);
}

template <typename F>
kfac_status_t by_types(const kfac_embedding_t& e, F f) {
  const bool tb = e.table_dtype == KFAC_BF16, yb = e.dtype == KFAC_BF16;
  if (tb) return yb ? f(__bf16{}, __bf16{}) : f(__bf16{}, float{});
  return yb ? f(float{}, __bf16{}) : f(float{}, float{});
}
int64_t stride_bytes(int64_t ld, int32_t dtype) { return ld * (dtype == KFAC_BF16 ? 2 : 4); }

}  // namespace

size_t embedding_workspace_bytes(int64_t tokens, int32_t vocab, int32_t width) {
  return regions(tokens, vocab, width).bytes;
}

kfac_status_t launch_embedding_lookup(const kfac_embedding_t& e, char* ws, hipStream_t st) {
  if (e.tokens == 0) return KFAC_OK;
  LookupArgs a{};
  a.table = static_cast<const char*>(e.table);
  a.y = static_cast<char*>(e.y);
  a.ids = e.ids;
  a.tokens = e.tokens;
  a.table_ld = stride_bytes(e.table_ld, e.table_dtype);
  a.y_ld = stride_bytes(e.y_ld, e.dtype);
  a.vocab = e.vocab;
  a.width = e.width;
  a.id_type = e.id_type;
  a.scale = e.scale;
  a.flags = reinterpret_cast<uint32_t*>(ws);
  return by_types(e, [&](auto tt, auto ty) -> kfac_status_t {
    using TT = decltype(tt);
    using TY = decltype(ty);
    const int64_t most = 1 << 16;
    if (e.width <= kWave * Elem<TY>::VE) {
      const int64_t n = std::min<int64_t>((e.tokens + 3) / 4, most);
      hipLaunchKernelGGL((lookup_kernel<TT, TY, kWave, false>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, st, a);
    } else {
      const int64_t n = std::min<int64_t>(e.tokens, most);
      // rows that do not fit the memory-side cache go past it: what is read again are the table's
      if (e.tokens * e.width > kCacheBytes / 2 / static_cast<int64_t>(sizeof(TY)))
        hipLaunchKernelGGL((lookup_kernel<TT, TY, kThreads, true>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, st, a);
      else
        hipLaunchKernelGGL((lookup_kernel<TT, TY, kThreads, false>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? KFAC_OK : KFAC_ERR_HIP;
  });
}

kfac_status_t launch_embedding_grad(const kfac_embedding_t& e, char* ws, hipStream_t st) {
  const Regions r = regions(e.tokens, e.vocab, e.width);
  const SortPlan plan = sort_plan(e.tokens, e.vocab);
  SumArgs a{};
  a.dy = static_cast<const char*>(e.y);
  a.grad = static_cast<char*>(e.table);
  a.counts = e.counts;
  a.tokens = e.tokens;
  a.dy_ld = stride_bytes(e.y_ld, e.dtype);
  a.grad_ld = stride_bytes(e.table_ld, e.table_dtype);
  a.vocab = e.vocab;
  a.width = e.width;
  a.accumulate = e.accumulate;
  a.scale = e.scale;
  a.partial = reinterpret_cast<float*>(ws + r.partial);
  a.part_ld = static_cast<int64_t>(part_ld(e.width));
  a.tile = sum_tile(e.tokens);
  a.tiles = static_cast<int32_t>((e.tokens + a.tile - 1) / a.tile);

  SortArgs s{};
  s.ids = e.ids;
  s.hist = reinterpret_cast<uint32_t*>(ws + r.hist);
  s.tokens = e.tokens;
  s.tile = plan.tile;
  s.vocab = e.vocab;
  s.id_type = e.id_type;
  s.bits = plan.bits;
  s.tiles = plan.tiles;
  s.flags = reinterpret_cast<uint32_t*>(ws);
  // positions that fit one workgroup's LDS: one launch in place of two a pass (5003 positions: 22 -> 16 us)
  const bool small = e.tokens <= kSmall;
  if (small && e.tokens > 0) {
    s.keys_out = reinterpret_cast<uint32_t*>(ws + r.keys[0]);
    s.perm_out = reinterpret_cast<uint32_t*>(ws + r.perm[0]);
    hipLaunchKernelGGL(sort_small_kernel, dim3(1), dim3(kSmallThreads), 0, st, s, plan.passes);
    if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
    a.keys = s.keys_out;
    a.perm = s.perm_out;
  }
  for (int pass = 0; pass < plan.passes && !small; ++pass) {
    const int to = pass & 1;
    s.shift = pass * plan.bits;
    s.keys = reinterpret_cast<const uint32_t*>(ws + r.keys[to ^ 1]);
    s.perm = reinterpret_cast<const uint32_t*>(ws + r.perm[to ^ 1]);
    s.keys_out = reinterpret_cast<uint32_t*>(ws + r.keys[to]);
    s.perm_out = reinterpret_cast<uint32_t*>(ws + r.perm[to]);
    const dim3 grid(plan.tiles), block(kSortThreads);
    if (pass == 0) {
      hipLaunchKernelGGL(digits_kernel<true>, grid, block, 0, st, s);
      hipLaunchKernelGGL(scatter_kernel<true>, grid, block, 0, st, s);
    } else {
      hipLaunchKernelGGL(digits_kernel<false>, grid, block, 0, st, s);
      hipLaunchKernelGGL(scatter_kernel<false>, grid, block, 0, st, s);
    }
    if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
    a.keys = s.keys_out;
    a.perm = s.perm_out;
  }
  return by_types(e, [&](auto tt, auto ty) -> kfac_status_t {
    using TT = decltype(tt);
    using TY = decltype(ty);
    const int64_t vectors = (static_cast<int64_t>(e.width) + kCols<TT, TY> - 1) / kCols<TT, TY>;
    const uint32_t slabs = static_cast<uint32_t>((vectors + kThreads - 1) / kThreads);
    const uint32_t threads = static_cast<uint32_t>(((vectors + slabs - 1) / slabs + kWave - 1) / kWave * kWave);
    const uint32_t groups = static_cast<uint32_t>((static_cast<int64_t>(e.vocab) + kWave - 1) / kWave);
    // The sums wait for rows and the joins for parts, the fills only write: half of
    // them beside each.
    const uint32_t beside = a.tiles ? groups / 2 : 0;
    a.fill_first = static_cast<int32_t>(beside);
    // dy and the gradient past the memory-side cache where they do not fit it
    const bool past = (e.tokens * static_cast<int64_t>(sizeof(TY)) + e.vocab * static_cast<int64_t>(sizeof(TT))) * e.width > kCacheBytes;
    auto go = [&](auto nt) {
      constexpr bool NT = decltype(nt)::value;
      if (a.tiles) hipLaunchKernelGGL((sums_kernel<TT, TY, NT>), dim3(a.tiles + beside, slabs), dim3(threads), 0, st, a);
      hipLaunchKernelGGL((join_kernel<TT, TY, NT>), dim3(a.tiles + groups - beside, slabs), dim3(threads), 0, st, a);
    };
    if (past) go(std::true_type{});
    else go(std::false_type{});
    return hipGetLastError() == hipSuccess ? KFAC_OK : KFAC_ERR_HIP;
  });
}

}  // namespace kfac
