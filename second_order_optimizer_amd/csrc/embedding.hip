// Embedding lookup and its gradient (include/kfac_tokens.h).
//
// Both are bound by HBM: the lookup reads T rows and writes T, the gradient
// reads the T rows of dy and writes the table's V rows whole.
//
// The gradient adds a token's rows in the order of their positions, so that it
// does not depend on scheduling: positions are sorted by token with a stable
// radix sort (tiles of positions, a histogram and a scatter a pass), a token's
// rows are then a run of the sorted positions.  Wavefronts walk the tokens, 64
// of them each; a token with more than kLong rows is left to the tiles of kLong
// sorted positions, whose partial sums are joined in order, so that a token that
// fills a tenth of the batch does not wait for one wavefront.
#include "tokens.h"

#include <algorithm>

namespace kfac {

namespace {

constexpr int kThreads = 256;
constexpr int kSortWaves = 8, kSortThreads = kSortWaves * kWave;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kMostTiles = 256;           // tiles of a sort: every workgroup of a scatter reads all their histograms
constexpr int kLeastTile = 1024;
constexpr int kLong = 128;

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
  r.partial = take(8 * static_cast<size_t>(width) * static_cast<size_t>((tokens + kLong - 1) / kLong));
  r.bytes = at;
  return r;
}

// -- vectors ----------------------------------------------------------------

// N values of a row from column c on, of `width` columns; those past it read as 0.
template <typename T, int N>
__device__ inline void load_cols(float (&f)[N], const char* row, int c, int width) {
  constexpr int VE = Elem<T>::VE;
  if (c + N <= width) {
    if constexpr (N >= VE) {
#pragma unroll
      for (int q = 0; q < N / VE; ++q) {
        const u32x4 v = load16(row + static_cast<int64_t>(c + q * VE) * sizeof(T));
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
template <typename T, int N>
__device__ inline void store_cols(char* row, int c, int width, const float (&f)[N]) {
  constexpr int VE = Elem<T>::VE;
  if (c + N <= width) {
    if constexpr (N >= VE) {
#pragma unroll
      for (int q = 0; q < N / VE; ++q) store16(row + static_cast<int64_t>(c + q * VE) * sizeof(T), pack16<T>(f + q * VE));
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
// Columns a lane takes at a time: 16 bytes of the rows of dtype.
template <typename TY>
constexpr int kCols = Elem<TY>::VE;

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

template <typename TT, typename TY, int TEAM>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs a) {
  constexpr int N = kCols<TY>, TEAMS = kThreads / TEAM;
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
      store_cols<TY, N>(to, c, a.width, f);
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
  for (int b = 0; b < a.tiles; ++b) {
    const uint32_t n = a.hist[static_cast<int64_t>(b) * kDigits + tid];
    if (b < static_cast<int>(blockIdx.x)) before += n;
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

// -- sums -------------------------------------------------------------------

struct SumArgs {
  const char* dy;
  char* grad;
  int32_t* counts;
  const uint32_t *keys, *perm;
  float* partial;                      // [tiles of kLong sorted positions][2][width]
  int64_t tokens, dy_ld, grad_ld;      // strides in bytes
  int32_t vocab, width, accumulate;
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

template <typename TY, int N>
__device__ inline void add_row(float (&s)[N], const char* row, int c, int width) {
  float f[N];
  load_cols<TY, N>(f, row, c, width);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] += f[i];
}
template <typename TT, int N>
__device__ inline void write_sum(const SumArgs& a, int64_t v, int c, float (&s)[N]) {
  char* row = a.grad + v * a.grad_ld;
  if (a.accumulate) {
    float old[N];
    load_cols<TT, N>(old, row, c, a.width);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = fmaf(s[i], a.scale, old[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= a.scale;
  }
  store_cols<TT, N>(row, c, a.width, s);
}

// Tokens of at most kLong rows: 64 of them a workgroup, a wavefront for kWave * N columns.
template <typename TT, typename TY>
__global__ void __launch_bounds__(kThreads) sums_kernel(SumArgs a) {
  constexpr int N = kCols<TY>;
  __shared__ int64_t start[kWave + 1];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kWave;
  if (wave == 0) {
    start[lane] = first_at(a.keys, a.tokens, static_cast<uint32_t>(min(v0 + lane, static_cast<int64_t>(a.vocab))));
    if (lane == 0) start[kWave] = first_at(a.keys, a.tokens, static_cast<uint32_t>(min(v0 + kWave, static_cast<int64_t>(a.vocab))));
  }
  __syncthreads();
  if (a.counts && blockIdx.y == 0 && wave == 0 && v0 + lane < a.vocab)
    a.counts[v0 + lane] = static_cast<int32_t>(start[lane + 1] - start[lane]);
  const int c = ((blockIdx.y * (kThreads / kWave) + wave) * kWave + lane) * N;
  if (c >= a.width) return;
  for (int i = 0; i < kWave && v0 + i < a.vocab; ++i) {
    const int64_t p0 = start[i], p1 = start[i + 1];
    if (p1 - p0 > kLong || (p1 == p0 && a.accumulate)) continue;
    float s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = 0.f;
    for (int64_t p = p0; p < p1; ++p) add_row<TY, N>(s, a.dy + a.perm[p] * a.dy_ld, c, a.width);
    write_sum<TT, N>(a, v0 + i, c, s);
  }
}

// Where a token's rows lie, and whether they are left to the tiles.
struct Run {
  int64_t p0, p1;
  __device__ Run(const SumArgs& a, uint32_t v) : p0(first_at(a.keys, a.tokens, v)), p1(first_at(a.keys, a.tokens, v + 1)) {}
  __device__ bool by_tiles() const { return p1 - p0 > kLong; }
};

// A tile holds rows of at most two tokens of more than kLong: of its first
// position's, whose sum goes to place 0, and of its last one's, to place 1.
template <typename TY>
__global__ void __launch_bounds__(kThreads) tiles_kernel(SumArgs a) {
  constexpr int N = kCols<TY>;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kLong, t1 = min(t0 + kLong, a.tokens);
  const int c = (blockIdx.y * kThreads + threadIdx.x) * N;
  const uint32_t tokens[2] = {a.keys[t0], a.keys[t1 - 1]};
  for (int which = 0; which < 2; ++which) {
    const uint32_t v = tokens[which];
    if (v >= static_cast<uint32_t>(a.vocab) || (which == 1 && v == tokens[0])) continue;
    const Run r(a, v);
    if (!r.by_tiles() || c >= a.width) continue;
    float s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = 0.f;
    const int64_t p1 = min(r.p1, t1);
#pragma unroll 4
    for (int64_t p = max(r.p0, t0); p < p1; ++p) add_row<TY, N>(s, a.dy + a.perm[p] * a.dy_ld, c, a.width);
    float* to = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.width;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < a.width) to[c + e] = s[e];
  }
}

// The sums of the tokens of more than kLong rows that begin in this tile.
template <typename TT, typename TY>
__global__ void __launch_bounds__(kThreads) join_kernel(SumArgs a) {
  constexpr int N = kCols<TY>;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kLong, t1 = min(t0 + kLong, a.tokens);
  const int c = (blockIdx.y * kThreads + threadIdx.x) * N;
  const uint32_t v = a.keys[t1 - 1];         // one that begins here has rows to the tile's end, or is no long one
  if (v >= static_cast<uint32_t>(a.vocab)) return;
  const Run r(a, v);
  if (!r.by_tiles() || r.p0 < t0 || c >= a.width) return;
  float s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = 0.f;
  const int64_t last = (r.p1 - 1) / kLong;
  for (int64_t tile = blockIdx.x; tile <= last; ++tile) {
    const int which = tile == static_cast<int64_t>(blockIdx.x) && a.keys[t0] != v ? 1 : 0;
    const float* from = a.partial + (tile * 2 + which) * a.width;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < a.width) s[e] += from[c + e];
  }
  write_sum<TT, N>(a, v, c, s);
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
    if (e.width <= kWave * kCols<TY>) {
      const int64_t n = std::min<int64_t>((e.tokens + 3) / 4, most);
      hipLaunchKernelGGL((lookup_kernel<TT, TY, kWave>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, st, a);
    } else {
      const int64_t n = std::min<int64_t>(e.tokens, most);
      hipLaunchKernelGGL((lookup_kernel<TT, TY, kThreads>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, st, a);
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
  for (int pass = 0; pass < plan.passes && e.tokens > 0; ++pass) {
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
    constexpr int per = kThreads * kCols<TY>;
    const uint32_t slabs = static_cast<uint32_t>((static_cast<int64_t>(e.width) + per - 1) / per);
    const uint32_t groups = static_cast<uint32_t>((static_cast<int64_t>(e.vocab) + kWave - 1) / kWave);
    hipLaunchKernelGGL((sums_kernel<TT, TY>), dim3(groups, slabs), dim3(kThreads), 0, st, a);
    if (e.tokens > kLong) {
      const uint32_t tiles = static_cast<uint32_t>((e.tokens + kLong - 1) / kLong);
      hipLaunchKernelGGL(tiles_kernel<TY>, dim3(tiles, slabs), dim3(kThreads), 0, st, a);
      hipLaunchKernelGGL((join_kernel<TT, TY>), dim3(tiles, slabs), dim3(kThreads), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? KFAC_OK : KFAC_ERR_HIP;
  });
}

}  // namespace kfac
