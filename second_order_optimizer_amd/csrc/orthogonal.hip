// Orthogonalised updates (include/kfac_orthogonal.h) on CDNA4 half-precision
// matrix cores, for any number of matrices of any shapes in the same launches.
//
// With X the matrix, d <= n its sides, a step is three products:
//     A = X X^T (symmetric),  B = b A + c A A (symmetric),  X <- a X + B X
// of 2 d^2 n / 2, 2 d^3 / 2 and 2 d^2 n operations.  All are products P Q^T of
// two matrices whose rows run along the contraction: A of X with itself, A A of
// A with itself, B X of B and X^T.  So X is kept both ways round, and each
// product's epilogue writes its tile and the tile's transpose: for A and B the
// mirror image (tiles below the diagonal are not computed), for X its X^T.
//
// Numbers.  Sums are float32 (MFMA).  Between products a matrix is held in IEEE
// half: with `products` HALF in one plane, rounded to 11 bits, with FULL in two,
// the value's rounding to half and the half of what that left, 22 bits together;
// a product is then high x high + high x low + low x high.  A value's own bits
// beyond those are left out; low x low is 2^-22 of a term.  With HALF, B's
// diagonal is kept apart in float32 and meets X in the last product's epilogue
// (where the singular values have come near 1 it is most of B), and so are X's
// low halves, for the term a X: where a few strong directions make up most of X,
// its rounding to 11 bits is large against all the others, which that term
// carries; as operands of the products, where B hardly has them yet, 11 bits do.
// (Both together: 1.5e-3 -> 5e-4 of the result.  Where x has a few directions and
// nothing else the diagonal apart costs, as the operand's roundings then reach the
// others through it: 6e-4 -> 1.6e-3 for eight of 128 x 128.)  bfloat16 outputs take
// HALF, float32 ones FULL.  Each matrix carries a power of two that keeps |value| <= 2^15:
// the norm bounds every element, and the polynomial's maximum bounds the norm after
// each step.
//
// Pairs.  Of a long X two of three products grow with n.  With FULL, where those
// weigh enough, two steps meet X in one: with P = a I + B of the first step, X's
// next X X^T is P A P, B' comes of that, and
//     X <- (a' I + B') P X = a a' X + (a' P + B' P - a a' I) X,
// one product with X, one X X^T and five d x d ones (symmetric all, as the factors
// are polynomials of A) in place of two, two and two; an odd step stays by itself.
// In 22 bits that is as exact (2e-6 of the result where a step at a time is 1e-6,
// both 2e-5 to 5e-5 where eight directions make up nearly all of X); in 11 bits it would
// double the error, so HALF takes a step at a time.  Eight layers of 1024 x 4096:
// 2.51 -> 2.01 ms.
//
// Layout.  Planes are row-major, both sides padded with zeros to whole tiles,
// which every product keeps at zero: no bounds checks outside the first and last
// pass.
#include "orthogonal_load.h"

#include <algorithm>
#include <cmath>

namespace kfac {

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kNormBlocks = 1024;     // most partial sums of a matrix's squares
constexpr int kMaxProbs = 14;         // problems a launch
constexpr int kBand = 4;              // tile rows whose tiles of a column run together

__device__ inline void split(float v, f16& hi, f16& lo) {
  hi = static_cast<f16>(v);
  lo = static_cast<f16>(v - static_cast<float>(hi));
}

// -- first pass: momentum, sums of squares ------------------------------------

struct PrepProb {
  const void* x;
  float* mom;
  int64_t ld, stride;
  int32_t rows, cols, batch, bf16, blk_begin, blocks;      // blocks a matrix
  double* part;                                            // [batch][kNormBlocks]
  float *bias, *bias_mom;
  const float* bias_grad;
  // second pass
  f16* same;            // planes laid out as x, [rows_p, cols_p]
  f16* turned;          // [cols_p, rows_p]
  int64_t plane, same_stride, turned_stride;
  int32_t rows_p, cols_p, tiles_c, blk2_begin;
  float scale;          // power of two
};
struct PrepBatch {
  PrepProb p[kMaxProbs];
  int32_t n, nesterov;
  float mu, lr, wd;
  double eps;
  uint32_t* flags;
};
static_assert(sizeof(PrepBatch) <= 4096, "kernel arguments");

template <int WHICH>
__device__ inline int find(const PrepBatch& b, int blk) {
  int i = 0;
  while (i + 1 < b.n && (WHICH ? b.p[i + 1].blk2_begin : b.p[i + 1].blk_begin) <= blk) ++i;
  return i;
}

__device__ inline const void* row_at(const PrepProb& P, int64_t at) {
  return P.bf16 ? static_cast<const void*>(static_cast<const unsigned short*>(P.x) + at)
                : static_cast<const void*>(static_cast<const float*>(P.x) + at);
}
// The matrix that is orthogonalised, from a gradient and its momentum after the update.
__device__ inline float direction(const PrepBatch& b, float g, float m) { return b.nesterov ? fmaf(b.mu, m, g) : m; }

__global__ void __launch_bounds__(256) orth_norm_kernel(PrepBatch b) {
  __shared__ double red[4];
  const PrepProb& P = b.p[find<0>(b, blockIdx.x)];
  const int t = blockIdx.x - P.blk_begin;
  const int mat = t / P.blocks, blk = t % P.blocks;
  double sum = 0.0;
  const int per_row = (P.cols + 7) / 8;
  const int64_t vectors = static_cast<int64_t>(P.rows) * per_row;
  for (int64_t i = static_cast<int64_t>(blk) * 256 + threadIdx.x; i < vectors; i += static_cast<int64_t>(P.blocks) * 256) {
    const int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<int64_t>(r) * per_row) * 8;
    float u[8];
    load8(u, row_at(P, mat * P.stride + r * P.ld), c, P.cols, P.bf16);
    if (P.mom) {
      float* at = P.mom + static_cast<int64_t>(r) * P.cols;
      float m[8];
      load8(m, at, c, P.cols, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = fmaf(b.mu, m[e], u[e]);
        u[e] = direction(b, u[e], m[e]);
      }
      if (c + 8 <= P.cols) {
        store16(at + c, pack16<float>(m));
        store16(at + c + 4, pack16<float>(m + 4));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < P.cols) at[c + e] = m[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(u[e]), static_cast<double>(u[e]), sum);
  }
  if (P.bias) {
    for (int r = blk * 256 + threadIdx.x; r < P.rows; r += P.blocks * 256) {
      const float v = fmaf(b.mu, P.bias_mom[r], fmaf(b.wd, P.bias[r], P.bias_grad[r]));
      P.bias_mom[r] = v;
      P.bias[r] = fmaf(-b.lr, v, P.bias[r]);
    }
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x == 0) P.part[static_cast<int64_t>(mat) * kNormBlocks + blk] = (red[0] + red[1]) + (red[2] + red[3]);
}

// -- second pass: the normalised matrix in planes, both ways round ---------------

// With HALF the low halves are stored of the matrix as x lies, not of the turned one.
template <int PLANES>
__global__ void __launch_bounds__(256) orth_load_kernel(PrepBatch b) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const PrepProb& P = b.p[find<1>(b, blockIdx.x)];
  int t = blockIdx.x - P.blk2_begin;
  const int tiles = (P.rows_p / 64) * P.tiles_c;
  const int mat = t / tiles;
  t -= mat * tiles;
  const int r0 = t / P.tiles_c * 64, c0 = t % P.tiles_c * 64;
  const int tid = threadIdx.x;
  double sum = 0.0;
  for (int i = tid; i < P.blocks; i += 256) sum += P.part[static_cast<int64_t>(mat) * kNormBlocks + i];
  sum = wave_sum(sum);
  if ((tid & 63) == 0) red[tid / 64] = sum;
  __syncthreads();
  sum = (red[0] + red[1]) + (red[2] + red[3]);
  if (!(sum < INFINITY) && t == 0 && tid == 0) raise_flag(b.flags, KFAC_FLAG_NONFINITE);
  const double norm = sqrt(sum) + b.eps;
  const double inv = norm > 0.0 ? static_cast<double>(P.scale) / norm : 0.0;
  f16* same = P.same + mat * P.same_stride;
  f16* turned = P.turned + mat * P.turned_stride;
  const int tr = tid / 8, tc = tid % 8 * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + tr + 32 * h, c = c0 + tc;
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < P.rows && c < P.cols) {
      load8(u, row_at(P, mat * P.stride + r * P.ld), c, P.cols, P.bf16);
      if (P.mom) {
        float m[8];
        load8(m, P.mom + static_cast<int64_t>(r) * P.cols, c, P.cols, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = direction(b, u[e], m[e]);
      }
    }
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u[e] = static_cast<float>(static_cast<double>(u[e]) * inv);
      f16 x, y;
      split(u[e], x, y);
      hi[e] = x;
      lo[e] = y;
      tile[tr + 32 * h][tc + e] = u[e];
    }
    const int64_t at = static_cast<int64_t>(r) * P.cols_p + c;
    *reinterpret_cast<f16x8*>(same + at) = hi;
    *reinterpret_cast<f16x8*>(same + P.plane + at) = lo;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f16 x, y;
      split(tile[tc + e][tr + 32 * h], x, y);
      hi[e] = x;
      lo[e] = y;
    }
    const int64_t at = static_cast<int64_t>(c0 + tr + 32 * h) * P.rows_p + r0 + tc;
    *reinterpret_cast<f16x8*>(turned + at) = hi;
    if constexpr (PLANES == 2) *reinterpret_cast<f16x8*>(turned + P.plane + at) = lo;
  }
}

// -- the products --------------------------------------------------------------

struct GemmProb {
  const f16 *a, *b, *c;       // P, Q and the matrix that is added; second planes `*_plane` elements on
  f16 *o, *ot;                // result and its transpose (one matrix where it is symmetric)
  int64_t a_plane, b_plane, c_plane, o_plane, ot_plane;
  int64_t a_batch, b_batch, c_batch, o_batch, ot_batch;
  int32_t lda, ldb, ldo, ldot;      // c is laid out as o
  int32_t k, tm, tn, tiles, blk_begin;      // tiles of a matrix; the first of all
  int64_t unit_begin;                       // the first stage of all
  float s_acc, s_c, s_diag;   // result = s_acc P Q^T + s_c C + s_diag I (s_diag: FULL, kPoly)
  float *d_out, *d_in;        // HALF: the diagonal that the result leaves out, and the one that B left out,
  int32_t d_batch, d_cols;    // a value a row of C, or a column
  // last product: the update goes to y, or into w
  void* y;
  float* w;
  int64_t y_ld, y_batch;
  int32_t rows, cols, y_bf16;
  float decay, factor;
};
// Workgroups take whole tiles (units 0), or equal shares of all tiles' stages one
// after the other: `units` stages over the grid's workgroups.  A share that is not
// a whole tile goes to `partial`, place 2 w for the tile it begins in and 2 w + 1 for
// the one it ends in, and the join kernel adds a tile's shares in order.
struct GemmBatch {
  GemmProb p[kMaxProbs];
  int32_t n;
  int32_t workgroups;       // of the shares
  int64_t units;
  float* partial;
};
static_assert(sizeof(GemmBatch) <= 4096, "kernel arguments");

// s_waitcnt with only the vector-memory counter limited to n (n < 64)
#define KFAC_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | (0x7 << 4) | (0xF << 8))

// instruction classes of __builtin_amdgcn_sched_group_barrier
constexpr int kSchedMfma = 0x008;
constexpr int kSchedDsRead = 0x100;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ inline f16x8 turned_rows(const f16* a, const f16* b) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)b);
  return __builtin_bit_cast(f16x8, s16x8(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
}

// What a product is for, and with it what its epilogue does.
enum Kind { kGram, kPoly, kNext, kLast, kWeight };      // A; B; X; O; the weight that takes O

// A kernel's tile: BM x BN, the contraction BK a stage, SLOTS stages in LDS, wavefronts
// of 32 MI x 32 NJ each.
template <int PLANES_, int BM_, int BN_, int MI_, int NJ_, int BK_, int SLOTS_>
struct Tile {
  static constexpr int PLANES = PLANES_, BM = BM_, BN = BN_, MI = MI_, NJ = NJ_, BK = BK_, SLOTS = SLOTS_;
  static constexpr int WN = BN / (32 * NJ), WAVES = BM / (32 * MI) * WN, THREADS = WAVES * 64;
};

// A problem entry read once from the kernel arguments and kept in scalar
// registers (see arg_reg).
__device__ inline GemmProb prob_regs(const GemmProb& p) {
  GemmProb q;
  q.a = arg_reg(p.a), q.b = arg_reg(p.b), q.c = arg_reg(p.c), q.o = arg_reg(p.o), q.ot = arg_reg(p.ot);
  q.a_plane = arg_reg(p.a_plane), q.b_plane = arg_reg(p.b_plane), q.c_plane = arg_reg(p.c_plane);
  q.o_plane = arg_reg(p.o_plane), q.ot_plane = arg_reg(p.ot_plane);
  q.a_batch = arg_reg(p.a_batch), q.b_batch = arg_reg(p.b_batch), q.c_batch = arg_reg(p.c_batch);
  q.o_batch = arg_reg(p.o_batch), q.ot_batch = arg_reg(p.ot_batch);
  q.lda = arg_reg(p.lda), q.ldb = arg_reg(p.ldb), q.ldo = arg_reg(p.ldo), q.ldot = arg_reg(p.ldot);
  q.k = arg_reg(p.k), q.tm = arg_reg(p.tm), q.tn = arg_reg(p.tn), q.tiles = arg_reg(p.tiles);
  q.blk_begin = arg_reg(p.blk_begin), q.unit_begin = arg_reg(p.unit_begin);
  q.s_acc = arg_reg(p.s_acc), q.s_c = arg_reg(p.s_c), q.s_diag = arg_reg(p.s_diag), q.d_out = arg_reg(p.d_out), q.d_in = arg_reg(p.d_in);
  q.d_batch = arg_reg(p.d_batch), q.d_cols = arg_reg(p.d_cols);
  q.y = arg_reg(p.y), q.w = arg_reg(p.w), q.y_ld = arg_reg(p.y_ld), q.y_batch = arg_reg(p.y_batch);
  q.rows = arg_reg(p.rows), q.cols = arg_reg(p.cols), q.y_bf16 = arg_reg(p.y_bf16);
  q.decay = arg_reg(p.decay), q.factor = arg_reg(p.factor);
  return q;
}

// Where tile t of a problem lies.
struct Place {
  int mat, ti, tj;
};
template <bool SYM>
__device__ inline Place place_of_tile(const GemmProb& P, int t) {
  Place at;
  at.mat = t / P.tiles;
  t -= at.mat * P.tiles;
  if (SYM) {                       // upper tiles, in bands of kBand rows, column after column
    int r0 = 0;
    for (;;) {
      const int h = min(kBand, P.tn - r0), n = h * (h + 1) / 2 + (P.tn - r0 - h) * h;
      if (t < n) {
        int c = 0;
        while (t >= min(c + 1, h)) t -= min(++c, h);
        at.ti = r0 + t;
        at.tj = r0 + c;
        return at;
      }
      t -= n;
      r0 += h;
    }
  }
  // bands of kBand tile rows, column after column
  const int band = t / (kBand * P.tn), h = min(kBand, P.tm - band * kBand);
  t -= band * kBand * P.tn;
  at.ti = band * kBand + t % h;
  at.tj = t / h;
  return at;
}

template <typename C>
using Ring = f16[C::SLOTS][C::PLANES][(C::BM + C::BN) * C::BK];

// acc = the product over the stages s0 .. s1 - 1 of a tile.
template <typename C>
__device__ inline void sum_stages(const GemmProb& P, const Place& at, int s0, int s1, Ring<C>& ring, f32x16 (&acc)[C::MI][C::NJ]) {
  constexpr int PLANES = C::PLANES, BM = C::BM, BN = C::BN, MI = C::MI, NJ = C::NJ, BK = C::BK, SLOTS = C::SLOTS;
  constexpr int THREADS = C::THREADS;
  constexpr int CHUNKS = BK / 8;                      // 16-byte chunks of a row
  constexpr int PL = (BM + BN) * BK;                  // elements of a plane of a stage, P's rows first
  constexpr int LOADS = PL / 8 / THREADS;             // loads a thread and plane
  constexpr int LOADS_P = BM * BK / 8 / THREADS;      // of these, of P
  static_assert(BM * BK % (8 * THREADS) == 0 && BN * BK % (8 * THREADS) == 0);
  const int mat = at.mat, i0 = at.ti * BM, j0 = at.tj * BN;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int wm = wid / C::WN * (32 * MI), wn = wid % C::WN * (32 * NJ);

  // operands: a buffer resource of the tile's rows each
  i32x4 rsrc[2][PLANES];
  uint32_t off[LOADS];
  auto swizzle = [](int row) { return CHUNKS == 8 ? (row >> 1) & 7 : (row >> 2) & 3; };
#pragma unroll
  for (int op = 0; op < 2; ++op) {
    const int ld = op ? P.ldb : P.lda;
    const f16* base = op ? P.b + mat * P.b_batch + static_cast<int64_t>(j0) * ld : P.a + mat * P.a_batch + static_cast<int64_t>(i0) * ld;
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl) {
      const uint64_t at = reinterpret_cast<uint64_t>(base + (pl ? (op ? P.b_plane : P.a_plane) : 0));
      rsrc[op][pl] = i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(at & 0xffffffffu)),
                           __builtin_amdgcn_readfirstlane(static_cast<int>((at >> 32) & 0xffffu)), (op ? BN : BM) * ld * 2, 0x00020000};
    }
  }
#pragma unroll
  for (int u = 0; u < LOADS; ++u) {
    const int p = u * THREADS + tid, row = p / CHUNKS, r = row < BM ? row : row - BM;
    off[u] = static_cast<uint32_t>(r * (u < LOADS_P ? P.lda : P.ldb) + ((p % CHUNKS) ^ swizzle(row)) * 8) * 2;
  }
  auto issue = [&](int s, int slot) {
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
            (__attribute__((address_space(3))) void*)(&ring[slot][pl][(u * THREADS + wid * 64) * 8])));
        asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off[u]), "s"(rsrc[u >= LOADS_P][pl]),
                       "s"(__builtin_amdgcn_readfirstlane(s * BK * 2))
                     : "memory");
      }
  };

#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // a lane's fragment of rows r0 .. r0 + 31: row r0 + lane % 32, 8 of the contraction from ks + 8 (lane / 32)
  auto frag = [&](const f16* stage, int r0, int ks) {
    const int row = r0 + (lane & 31), c = ks / 8 + (lane >> 5);
    return *reinterpret_cast<const f16x8*>(stage + row * BK + (c ^ swizzle(row)) * 8);
  };

#pragma unroll
  for (int s = 0; s < SLOTS - 1; ++s) issue(min(s0 + s, s1 - 1), s);       // (a short contraction asks for its last stage again)
  for (int s = s0, slot = 0; s < s1; ++s, slot = slot + 1 == SLOTS ? 0 : slot + 1) {
    // this stage has arrived: all but the newest SLOTS - 2 stages' loads
    KFAC_WAIT_VM((SLOTS - 2) * LOADS * PLANES);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");           // the loads above wrote what is read below
    // into the slot that every wavefront has left; past the end the last stage again, so that counts stay the same
    issue(min(s + SLOTS - 1, s1 - 1), slot == 0 ? SLOTS - 1 : slot - 1);
    // the fragments of a step of 16 are read while the products of the one before run
    f16x8 fa[2][PLANES][MI], fb[2][PLANES][NJ];
    auto read = [&](int ks, int to) {
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[to][pl][i] = frag(ring[slot][pl], wm + 32 * i, ks);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[to][pl][j] = frag(ring[slot][pl], BM + wn + 32 * j, ks);
      }
    };
    constexpr int READS = PLANES * (MI + NJ), MFMAS = (PLANES == 2 ? 3 : 1) * MI * NJ;
    read(0, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedDsRead, READS, 0);
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      const int cur = (ks / 16) & 1;
      if (ks + 16 < BK) read(ks + 16, cur ^ 1);
#pragma unroll
      for (int x = 0; x < (PLANES == 2 ? 3 : 1); ++x)      // high x high, high x low, low x high
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[cur][PLANES == 2 && x == 2][i], fb[cur][PLANES == 2 && x == 1][j],
                                                               acc[i][j], 0, 0, 0);
      if (ks + 16 < BK && MFMAS >= READS) {
#pragma unroll
        for (int u = 0; u < READS; ++u) {
          __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kSchedMfma, MFMAS >= READS ? MFMAS - READS : 0, 0);
      } else if (ks + 16 >= BK) {
        __builtin_amdgcn_sched_group_barrier(kSchedMfma, MFMAS, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0): this wavefront has read the slot before the next barrier
  }

  KFAC_WAIT_VM(0);                           // the stages asked for past the end
  __syncthreads();
}

// What becomes of a wavefront's sums, 32 rows at a time, through LDS of its own
// (`mine`): the sums (accumulator r of block (i, j): row 8 (r / 4) + 4 (lane / 32) +
// r % 4, column lane % 32) are turned into 8 columns a lane, so that C is read and
// the result written in 16-byte pieces; the result's halves go back to LDS, from
// where transposing reads give 8 rows a lane for the transpose.  C's next rows are asked
// for before a row is stored: a load waits for the stores before it.
constexpr int LS = 68;                       // row length in LDS, of floats and of halves
constexpr int kMine = 32 * LS;               // floats of a wavefront

template <typename C, Kind KIND>
__device__ inline void finish(const GemmProb& P, const Place& at, int wid, f32x16 (&acc)[C::MI][C::NJ], float* mine) {
  constexpr int PLANES = C::PLANES, MI = C::MI, NJ = C::NJ;
  constexpr bool SYM = KIND == kGram || KIND == kPoly;
  static_assert(NJ == 2, "64 columns a wavefront");
  const int mat = at.mat, i0 = at.ti * C::BM, j0 = at.tj * C::BN;
  const int lane = threadIdx.x & 63;
  const int wm = wid / C::WN * (32 * MI), wn = wid % C::WN * (32 * NJ);
  f16* halves = reinterpret_cast<f16*>(mine);
  const int lr = lane >> 3, lc = (lane & 7) * 8;
  const int col = j0 + wn + lc;
  // a symmetric result: 64 x 64 blocks below the diagonal are not written, those on it whole, those above it both ways
  auto below = [&](int i) { return SYM ? (i0 + wm + 32 * i) / 64 - (j0 + wn) / 64 : -1; };
  constexpr bool HAS_C = KIND != kGram, C_LOW = PLANES == 2 || KIND >= kNext, LAST = KIND >= kLast;
  constexpr bool DIAG_IN = PLANES == 1 && KIND >= kNext;
  const int64_t row_step = static_cast<int64_t>(8) * P.ldo;
  const f16* c_at = P.c + mat * P.c_batch + static_cast<int64_t>(i0 + wm + lr) * P.ldo + col;
  f16x8 ch[2][4], cl[2][4];
  float d_row[2][4] = {};
  const bool whole = j0 + wn + 64 <= P.cols; // no columns past the matrix (LAST)
  auto read_c = [&](int i) {
    if constexpr (!HAS_C) return;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f16* c = c_at + (4 * i + t) * row_step;
      ch[i & 1][t] = *reinterpret_cast<const f16x8*>(c);
      if constexpr (C_LOW) cl[i & 1][t] = *reinterpret_cast<const f16x8*>(c + P.c_plane);
    }
    if (DIAG_IN && !P.d_cols) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        d_row[i & 1][t] = P.d_in[static_cast<int64_t>(mat) * P.d_batch + i0 + wm + 32 * i + 8 * t + lr];
    }
  };
  // what multiplies C: s_c, and with it the diagonal that B left out, of the lane's columns or of a row
  float fc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) fc[e] = P.s_c;
  if (DIAG_IN && P.d_cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) fc[e] = fmaf(P.s_acc, P.d_in[static_cast<int64_t>(mat) * P.d_batch + col + e], P.s_c);
  }
  read_c(0);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if (i + 1 < MI) read_c(i + 1);
    const int row0 = i0 + wm + 32 * i;
    if (below(i) > 0) continue;
    u32x4 keep[8];                           // the result: 4 rows' halves and what they leave
    u32x4 wv[8];                             // kWeight: the weight's rows
    if (KIND == kWeight && whole) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float* from = P.w + static_cast<int64_t>(min(row0 + 8 * t + lr, P.rows - 1)) * P.y_ld + col;
        wv[2 * t] = load16(from);
        wv[2 * t + 1] = load16(from + 4);
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) mine[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * LS + 32 * j + (lane & 31)] = acc[i][j][r];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = row0 + 8 * t + lr;
      f32x4* at = reinterpret_cast<f32x4*>(mine + (8 * t + lr) * LS + lc);
      const f32x4 x0 = at[0], x1 = at[1];
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = P.s_acc * (e < 4 ? x0[e & 3] : x1[e & 3]);
        if constexpr (HAS_C) {
          float c = static_cast<float>(ch[i & 1][t][e]);
          if constexpr (C_LOW) c += static_cast<float>(cl[i & 1][t][e]);
          v[e] = fmaf(DIAG_IN ? fmaf(P.s_acc, d_row[i & 1][t], fc[e]) : fc[e], c, v[e]);
        }
      }
      if constexpr (LAST) {
        if (!whole) {
          at[0] = f32x4{v[0], v[1], v[2], v[3]};
          at[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else if (row < P.rows) {
          const int64_t to = mat * P.y_batch + static_cast<int64_t>(row) * P.y_ld + col;
          if (KIND == kLast && P.y_bf16) {
            store16(static_cast<unsigned short*>(P.y) + to, pack16<__bf16>(v));
          } else {
            float* y = (KIND == kWeight ? P.w : static_cast<float*>(P.y)) + to;
            if constexpr (KIND == kWeight) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaf(-P.factor, v[e], P.decay * __uint_as_float(wv[2 * t + (e >> 2)][e & 3]));
            }
            store16(y, pack16<float>(v));
            store16(y + 4, pack16<float>(v + 4));
          }
        }
      } else {
        if (KIND == kPoly && PLANES == 1 && below(i) == 0) {
          float d = 0.f;
          const int at_e = row - col;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (at_e == e) d = v[e], v[e] = 0.f;
          if (at_e >= 0 && at_e < 8) P.d_out[static_cast<int64_t>(mat) * P.d_batch + row] = d;
        }
        if (KIND == kPoly && PLANES == 2 && below(i) == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row - col == e) v[e] += P.s_diag;
        }
        f16x8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f16 h, l;
          split(v[e], h, l);
          hi[e] = h;
          lo[e] = l;
        }
        keep[t] = __builtin_bit_cast(u32x4, hi);
        if constexpr (PLANES == 2 || KIND == kNext) keep[4 + t] = __builtin_bit_cast(u32x4, lo);
      }
    }
    if constexpr (LAST) {
      if (!whole && j0 + wn + lane < P.cols) {         // a lane a column
        const int64_t at = mat * P.y_batch + static_cast<int64_t>(row0) * P.y_ld + j0 + wn + lane;
#pragma unroll 1
        for (int r = 0; r < min(32, P.rows - row0); ++r) {
          const float v = mine[r * LS + lane];
          const int64_t to = at + r * P.y_ld;
          if (KIND == kWeight) P.w[to] = fmaf(-P.factor, v, P.decay * P.w[to]);
          else if (P.y_bf16) Elem<__bf16>::store(P.y, to, v);
          else static_cast<float*>(P.y)[to] = v;
        }
      }
    }
    if constexpr (!LAST) {
      f16* o = P.o + mat * P.o_batch + static_cast<int64_t>(row0 + lr) * P.ldo + col;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        *reinterpret_cast<u32x4*>(o + t * row_step) = keep[t];
        if constexpr (PLANES == 2 || KIND == kNext) *reinterpret_cast<u32x4*>(o + t * row_step + P.o_plane) = keep[4 + t];
      }
      if (below(i) == 0) {
        __builtin_amdgcn_sched_barrier(0);
        continue;
      }
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          u32x2* to = reinterpret_cast<u32x2*>(halves + pl * 32 * LS + (8 * t + lr) * LS + lc);
          const u32x4 x = keep[4 * pl + t];
          to[0] = u32x2{x[0], x[1]};
          to[1] = u32x2{x[2], x[3]};
        }
      // 16 lanes: 4 rows of 16 columns in, a column of 4 rows each out
      const int g = lane >> 4, s = lane & 15;
      f16* ot = P.ot + mat * P.ot_batch + static_cast<int64_t>(j0 + wn + s) * P.ldot + row0 + 8 * g;
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f16* from = halves + pl * 32 * LS + (8 * g + (s >> 2)) * LS + 16 * q + 4 * (s & 3);
          *reinterpret_cast<f16x8*>(ot + static_cast<int64_t>(16 * q) * P.ldot + (pl ? P.ot_plane : 0)) =
              turned_rows(from, from + 4 * LS);
        }
    }
    __builtin_amdgcn_sched_barrier(0);       // (rows taken ahead of each other would not fit the registers)
  }
}

// The shares of a launch that workgroup w takes, and the first that reaches unit u.
__device__ inline int64_t share_begin(const GemmBatch& b, int64_t w) { return w * b.units / b.workgroups; }
__device__ inline int share_of(const GemmBatch& b, int64_t u) {
  int64_t w = u * b.workgroups / b.units;
  while (share_begin(b, w + 1) <= u) ++w;
  while (share_begin(b, w) > u) --w;
  return static_cast<int>(w);
}

template <typename C, Kind KIND>
__global__ void __launch_bounds__(C::THREADS) orth_gemm_kernel(GemmBatch batch) {
  constexpr bool SYM = KIND == kGram || KIND == kPoly;
  static_assert(C::BM == C::BN, "symmetric tiles");
  __shared__ __attribute__((aligned(16))) Ring<C> ring;
  static_assert(sizeof(ring) >= C::WAVES * kMine * sizeof(float));
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float* mine = reinterpret_cast<float*>(&ring[0][0][0]) + wid * kMine;
  // workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles, so that the
  // panels that its tiles share are read into its L2 once
  const int per = gridDim.x / 8, w0 = blockIdx.x;
  const int w = w0 < 8 * per ? (w0 % 8) * per + w0 / 8 : w0;
  f32x16 acc[C::MI][C::NJ];
  if (batch.units == 0) {
    int pi = 0;
    while (pi + 1 < batch.n && batch.p[pi + 1].blk_begin <= w) ++pi;
    const GemmProb P = prob_regs(batch.p[pi]);
    const Place at = place_of_tile<SYM>(P, w - P.blk_begin);
    sum_stages<C>(P, at, 0, P.k / C::BK, ring, acc);
    finish<C, KIND>(P, at, wid, acc, mine);
    return;
  }
  const int64_t end = share_begin(batch, w + 1);
  bool first = true;
  for (int64_t u = share_begin(batch, w); u < end; first = false) {
    int pi = 0;
    while (pi + 1 < batch.n && batch.p[pi + 1].unit_begin <= u) ++pi;
    const GemmProb P = prob_regs(batch.p[pi]);
    const int stages = P.k / C::BK;
    const int64_t in = u - P.unit_begin;
    const int tile = static_cast<int>(in / stages), s0 = static_cast<int>(in - static_cast<int64_t>(tile) * stages);
    const int s1 = static_cast<int>(min(static_cast<int64_t>(stages), s0 + end - u));
    const Place at = place_of_tile<SYM>(P, tile);
    sum_stages<C>(P, at, s0, s1, ring, acc);
    if (s0 == 0 && s1 == stages) {
      finish<C, KIND>(P, at, wid, acc, mine);
      __syncthreads();                       // the ring is the next tile's
    } else {
      f32x4* to = reinterpret_cast<f32x4*>(batch.partial + (2 * static_cast<int64_t>(w) + !first) * (C::BM * C::BN)) +
                  wid * (C::MI * C::NJ * 4 * 64) + lane;
#pragma unroll
      for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int j = 0; j < C::NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            to[((i * C::NJ + j) * 4 + q) * 64] = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    u += s1 - s0;
  }
}

// 32 rows of a wavefront's part of a tile whose stages were shared: the shares in
// order.  (A whole part a wavefront, 64 rows or 128, took twice as long: 21 tiles
// of 20 shares 27 us, here 11.)
template <typename C, Kind KIND>
__global__ void __launch_bounds__(64) orth_join_kernel(GemmBatch batch) {
  constexpr bool SYM = KIND == kGram || KIND == kPoly;
  using J = Tile<C::PLANES, C::BM, C::BN, 1, C::NJ, C::BK, C::SLOTS>;
  static_assert(J::WN == C::WN);
  __shared__ __attribute__((aligned(16))) float mine[kMine];
  const int lane = threadIdx.x, part = blockIdx.x % J::WAVES, tile = blockIdx.x / J::WAVES;
  const int i = part / C::WN % C::MI, wid = part / C::WN / C::MI * C::WN + part % C::WN;
  int pi = 0;
  while (pi + 1 < batch.n && batch.p[pi + 1].blk_begin <= tile) ++pi;
  const GemmProb P = prob_regs(batch.p[pi]);
  const int stages = P.k / C::BK;
  const int64_t begin = P.unit_begin + static_cast<int64_t>(tile - P.blk_begin) * stages;
  const int w0 = share_of(batch, begin), w1 = share_of(batch, begin + stages - 1);
  if (w0 == w1) return;                      // one workgroup had all of it
  f32x16 acc[1][C::NJ];
#pragma unroll
  for (int j = 0; j < C::NJ; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[0][j][r] = 0.f;
  const int begun = share_begin(batch, w0) < begin;        // the first share's workgroup had begun with another tile
#pragma unroll 4
  for (int w = w0; w <= w1; ++w) {
    const int second = w == w0 && begun;
    const f32x4* from = reinterpret_cast<const f32x4*>(batch.partial + (2 * static_cast<int64_t>(w) + second) * (C::BM * C::BN)) +
                        (wid * C::MI + i) * (C::NJ * 4 * 64) + lane;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 x = from[(j * 4 + q) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][j][4 * q + e] += x[e];
      }
  }
  finish<J, KIND>(P, place_of_tile<SYM>(P, tile - P.blk_begin), part, acc, mine);
}

// -- plan ----------------------------------------------------------------------

int round_up(int v, int to) { return (v + to - 1) / to * to; }

struct Shape {
  int d, n, dp, np, tile;
  bool tall;
  int64_t x_plane, a_plane;          // elements of a plane of X and of A
};
Shape shape_of(const OrthTask& t) {
  Shape s;
  s.d = std::min(t.rows, t.cols);
  s.n = std::max(t.rows, t.cols);
  s.tall = t.rows > t.cols;
  // whole tiles of 256 where that adds less than an eighth to a side
  s.tile = round_up(s.d, 256) * 8 <= round_up(s.d, 128) * 9 && round_up(s.n, 256) * 8 <= round_up(s.n, 128) * 9 ? 256 : 128;
  s.dp = round_up(s.d, s.tile);
  s.np = round_up(s.n, s.tile);
  s.x_plane = static_cast<int64_t>(s.dp) * s.np;
  s.a_plane = static_cast<int64_t>(s.dp) * s.dp;
  return s;
}

struct Region {
  size_t part, same[2], turned[2], a, b, s, diag;      // X as x lies and turned; what B X reads is not what it writes
};
size_t plan(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how, std::vector<Region>* out) {
  const int planes = how.products == KFAC_PRODUCTS_FULL ? 2 : 1;
  size_t at = kRegions;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = align_up(at + n, 256);
    return here;
  };
  for (const OrthTask& t : tasks) {
    const Shape s = shape_of(t);
    Region r{};
    const size_t batch = static_cast<size_t>(t.batch);
    r.part = take(sizeof(double) * kNormBlocks * batch);
    const size_t both = 2 * 2 * batch * s.x_plane, some = 2 * planes * batch * s.x_plane;
    r.same[0] = take(both);
    r.same[1] = s.tall ? take(both) : r.same[0];
    r.turned[0] = take(some);
    r.turned[1] = s.tall ? r.turned[0] : take(some);
    r.a = take(2 * planes * batch * s.a_plane);
    r.b = take(2 * planes * batch * s.a_plane);
    if (planes == 2) r.s = take(2 * planes * batch * s.a_plane);
    r.diag = take(sizeof(float) * batch * s.dp);
    if (out) out->push_back(r);
  }
  return at;
}

// Bits to scale a matrix whose norm is at most `bound` by, so that no element passes 2^15.
int bits_for(double bound) { return 15 - static_cast<int>(std::ceil(std::log2(std::max(bound, 1e-30)))); }

// Norm bounds after each step, over all singular values that the last one allows.
struct StepScale {
  int x, a, b;           // powers of two of X, A, B in this step
  double rho, pb;        // bounds of |X| and |B|
};
std::vector<StepScale> step_scales(const kfac_orthogonal_t& how, int* last) {
  std::vector<StepScale> out;
  double rho = 1.0;
  for (int s = 0; s < how.steps; ++s) {
    const PolyBound p = poly_of(how.coefs + 3 * s, rho);
    out.push_back({bits_for(rho), bits_for(rho * rho), bits_for(p.b), rho, p.b});
    rho = p.next;
  }
  *last = bits_for(rho);
  return out;
}

using Half256 = Tile<1, 256, 256, 4, 2, 64, 2>;
using Half128 = Tile<1, 128, 128, 2, 2, 64, 2>;
using Half128Wide = Tile<1, 128, 128, 1, 2, 64, 3>;
using Full256 = Tile<2, 256, 256, 4, 2, 32, 2>;
using Full128 = Tile<2, 128, 128, 2, 2, 32, 2>;
using Full128Wide = Tile<2, 128, 128, 1, 2, 32, 3>;

// How a launch's tiles are cut: their size, and the workgroups that share their
// stages (0: each takes a tile).
struct Cut {
  int tile, shares;
  bool wide;             // eight wavefronts a tile of 128, for at most a workgroup a compute unit
  double time;           // what it should take, us
};
struct Product {
  int64_t tiles[2], units[2];      // of 128 and of 256
};
// The cut that takes least time, by what the kernels measured: a stage of one
// workgroup a compute unit (two, for tiles of 128, where there are that many), an
// epilogue, and shares written and read again at 4 TB/s with a launch of their own.
Cut cut_of(const Product& p, int planes, bool may256) {
  Cut best{128, 0, false, 0.0};
  double least = 1e30;
  for (int big = may256 ? 1 : 0; big >= 0; --big) {
    const double tiles = static_cast<double>(p.tiles[big]), units = static_cast<double>(p.units[big]), stages = units / tiles;
    const int slots = big ? 256 : 512;
    auto stage = [&](double running) {
      if (big) return planes == 2 ? 2.1 : 1.4;
      return running > 256 ? (planes == 2 ? 1.45 : 0.8) : (planes == 2 ? 1.0 : 0.55);
    };
    const double rounds = std::ceil(tiles / slots), end = big ? 30.0 : 12.0;
    const double whole = rounds * (stages * stage(std::min(tiles, static_cast<double>(slots))) + end);
    if (whole < least) least = whole, best = {big ? 256 : 128, 0, !big && tiles <= 256.0, whole};
    const double bytes = big ? 524288.0 : 131072.0;          // a share's sums, written and read
    if (big && tiles > 0.5 * slots && tiles < slots) {
      // Whole tiles would leave up to half of the compute units idle: thirds, of which
      // two rounds run, at the same places of the contraction (X X^T of 4096 x 16384, 136
      // tiles: 342 us whole, 282 and a join of 30 in thirds).
      const double t = std::ceil(3.0 * tiles / slots) * stages / 3.0 * stage(0) + 4.0 * tiles * bytes / 4e6 + 10.0 + end;
      if (t < 0.95 * least) least = t, best = {256, static_cast<int>(3 * p.tiles[big]), false, t};
    }
    for (int g = 32; g <= slots; g += 32) {
      if (units < 2.0 * g || g < tiles * 0.5) continue;
      // (workgroups at different places of the contraction read no panels together)
      const double t = units / g * stage(0) * (1.0 + g / (big ? 256.0 : 350.0)) + (g + tiles) * bytes / 4e6 + 10.0 + end;
      if (t < 0.95 * least) least = t, best = {big ? 256 : 128, g, !big && g <= 256, t};
    }
  }
  return best;
}

template <typename C, Kind KIND>
kfac_status_t launch_tiles(std::vector<GemmProb>& probs, const std::vector<int>& batch, int shares, float* partial, hipStream_t st) {
  GemmBatch b{};
  int64_t tiles = 0, units = 0;
  for (size_t i = 0; i < probs.size(); ++i) {
    GemmProb& p = probs[i];
    p.tm /= C::BM;                  // rows and columns so far
    p.tn /= C::BN;
    p.tiles = KIND == kGram || KIND == kPoly ? p.tn * (p.tn + 1) / 2 : p.tm * p.tn;
    p.blk_begin = static_cast<int>(tiles);
    p.unit_begin = units;
    tiles += static_cast<int64_t>(p.tiles) * batch[i];
    units += static_cast<int64_t>(p.tiles) * batch[i] * (p.k / C::BK);
    b.p[b.n++] = p;
  }
  b.workgroups = shares;
  b.units = shares ? units : 0;
  b.partial = partial;
  hipLaunchKernelGGL((orth_gemm_kernel<C, KIND>), dim3(static_cast<uint32_t>(shares ? shares : tiles)), dim3(C::THREADS), 0, st, b);
  if (shares)
    hipLaunchKernelGGL((orth_join_kernel<C, KIND>), dim3(static_cast<uint32_t>(tiles * (C::WAVES * C::MI))), dim3(64), 0, st, b);
  return hipGetLastError() == hipSuccess ? KFAC_OK : KFAC_ERR_HIP;
}

template <Kind KIND>
kfac_status_t launch_products(std::vector<GemmProb>& probs, const std::vector<int>& batch, int planes, Cut cut, float* partial, hipStream_t st) {
  if (planes == 2)
    return cut.tile == 256 ? launch_tiles<Full256, KIND>(probs, batch, cut.shares, partial, st)
           : cut.wide      ? launch_tiles<Full128Wide, KIND>(probs, batch, cut.shares, partial, st)
                           : launch_tiles<Full128, KIND>(probs, batch, cut.shares, partial, st);
  return cut.tile == 256 ? launch_tiles<Half256, KIND>(probs, batch, cut.shares, partial, st)
         : cut.wide      ? launch_tiles<Half128Wide, KIND>(probs, batch, cut.shares, partial, st)
                         : launch_tiles<Half128, KIND>(probs, batch, cut.shares, partial, st);
}

// Matrices whose products go into the same launches.
struct Group {
  std::vector<size_t> tasks;
  Cut gram, poly, next;
  bool pairs;            // two steps a product with X
};
std::vector<Group> groups_of(const std::vector<OrthTask>& tasks, int planes) {
  std::vector<Group> out;
  for (int tile : {256, 128}) {
    Group g;
    auto close = [&] {
      if (g.tasks.empty()) return;
      Product a{}, b{}, x{};
      for (size_t i : g.tasks) {
        const Shape s = shape_of(tasks[i]);
        for (int big = 0; big < 2; ++big) {
          const int bt = big ? 256 : 128, bk = planes == 2 ? 32 : 64;
          const int64_t nd = s.dp / bt, nn = s.np / bt, batch = tasks[i].batch;
          const int64_t upper = nd * (nd + 1) / 2 * batch, all = nd * nn * batch;
          a.tiles[big] += upper, a.units[big] += upper * (s.np / bk);
          b.tiles[big] += upper, b.units[big] += upper * (s.dp / bk);
          x.tiles[big] += all, x.units[big] += all * (s.dp / bk);
        }
      }
      g.gram = cut_of(a, planes, tile == 256);
      g.poly = cut_of(b, planes, tile == 256);
      g.next = cut_of(x, planes, tile == 256);
      // three more d x d products against an X X^T and a product with X
      g.pairs = planes == 2 && g.gram.time + g.next.time > 3.3 * g.poly.time;
      out.push_back(g);
      g = Group{};
    };
    for (size_t i = 0; i < tasks.size(); ++i) {
      if (shape_of(tasks[i]).tile != tile) continue;
      g.tasks.push_back(i);
      if (g.tasks.size() == kMaxProbs) close();
    }
    close();
  }
  return out;
}
size_t partial_bytes(const Cut& c) { return static_cast<size_t>(c.shares) * 2 * c.tile * c.tile * sizeof(float); }

}  // namespace

size_t orth_workspace_bytes(const std::vector<OrthTask>& all, const kfac_orthogonal_t& how) {
  std::vector<OrthTask> small, tasks;
  for (const OrthTask& t : all) (orth_is_small(t) ? small : tasks).push_back(t);
  size_t partial = orth_small_bytes(small);
  for (const Group& g : groups_of(tasks, how.products == KFAC_PRODUCTS_FULL ? 2 : 1))
    for (const Cut& c : {g.gram, g.poly, g.next}) partial = std::max(partial, partial_bytes(c));      // one after the other
  return plan(tasks, how, nullptr) + partial;
}

kfac_status_t launch_orthogonal(const std::vector<OrthTask>& all, const kfac_orthogonal_t& how, const OrthStep& step,
                                char* ws, hipStream_t st) {
  std::vector<OrthTask> small, tasks;
  for (const OrthTask& t : all) (orth_is_small(t) ? small : tasks).push_back(t);
  const int planes = how.products == KFAC_PRODUCTS_FULL ? 2 : 1;
  std::vector<Region> regions;
  char* rest = ws + plan(tasks, how, &regions);
  float* partial = reinterpret_cast<float*>(rest);
  if (!small.empty()) {
    const kfac_status_t r = launch_orth_small(small, how, step, rest, reinterpret_cast<uint32_t*>(ws), st);
    if (r != KFAC_OK || tasks.empty()) return r;
  }
  int last_bits = 0;
  const std::vector<StepScale> scales = step_scales(how, &last_bits);

  // both first passes
  for (size_t i0 = 0; i0 < tasks.size(); i0 += kMaxProbs) {
    PrepBatch b{};
    b.nesterov = how.nesterov;
    b.mu = step.momentum;
    b.lr = step.lr;
    b.wd = step.weight_decay;
    b.eps = how.eps;
    b.flags = reinterpret_cast<uint32_t*>(ws);
    int64_t blocks = 0, blocks2 = 0;
    for (size_t i = i0; i < tasks.size() && i < i0 + kMaxProbs; ++i) {
      const OrthTask& t = tasks[i];
      const Shape s = shape_of(t);
      const Region& r = regions[i];
      PrepProb& p = b.p[b.n++];
      p.x = t.x;
      p.mom = t.mom;
      p.ld = t.ld;
      p.stride = t.stride;
      p.rows = t.rows;
      p.cols = t.cols;
      p.batch = t.batch;
      p.bf16 = t.dtype == KFAC_BF16;
      p.blocks = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(t.rows) * ((t.cols + 7) / 8) + 1023) / 1024, kNormBlocks));
      p.blk_begin = static_cast<int>(blocks);
      blocks += static_cast<int64_t>(p.blocks) * t.batch;
      p.part = reinterpret_cast<double*>(ws + r.part);
      p.bias = t.bias;
      p.bias_mom = t.bias_mom;
      p.bias_grad = t.bias_grad;
      p.same = reinterpret_cast<f16*>(ws + r.same[0]);
      p.turned = reinterpret_cast<f16*>(ws + r.turned[0]);
      p.plane = s.x_plane;
      p.same_stride = s.x_plane * 2;
      p.turned_stride = s.x_plane * planes;
      p.rows_p = s.tall ? s.np : s.dp;
      p.cols_p = s.tall ? s.dp : s.np;
      p.tiles_c = p.cols_p / 64;
      p.blk2_begin = static_cast<int>(blocks2);
      blocks2 += static_cast<int64_t>(p.rows_p / 64) * p.tiles_c * t.batch;
      p.scale = std::ldexp(1.f, scales[0].x);
    }
    if (b.n == 0) return KFAC_OK;
    hipLaunchKernelGGL(orth_norm_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, st, b);
    if (planes == 2) hipLaunchKernelGGL(orth_load_kernel<2>, dim3(static_cast<uint32_t>(blocks2)), dim3(256), 0, st, b);
    else hipLaunchKernelGGL(orth_load_kernel<1>, dim3(static_cast<uint32_t>(blocks2)), dim3(256), 0, st, b);
    if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
  }

  auto two = [](int e) { return std::ldexp(1.f, e); };
  for (const Group& g : groups_of(tasks, planes)) {
    int from = 0;                        // where X is: of the two, for products with X so far
    for (int k = 0, n; k < how.steps; k += n, from ^= 1) {
      n = g.pairs && k + 1 < how.steps ? 2 : 1;
      const float *c1 = how.coefs + 3 * k, *c2 = c1 + 3;
      const StepScale& sc = scales[k];
      const bool last = k + n == how.steps;
      const int xb = last ? 0 : scales[k + n].x;         // the last X is written as it is
      std::vector<GemmProb> pa, px;
      std::vector<std::vector<GemmProb>> polys(n == 2 ? 5 : 1);
      std::vector<int> batch;
      for (size_t i : g.tasks) {
        const OrthTask& t = tasks[i];
        batch.push_back(t.batch);
        const Shape s = shape_of(t);
        const Region& r = regions[i];
        // X as x lies, [rows_p, cols_p], and turned; the one with d rows and n columns
        f16* same = reinterpret_cast<f16*>(ws + r.same[from]);
        f16* turned = reinterpret_cast<f16*>(ws + r.turned[from]);
        f16 *A = reinterpret_cast<f16*>(ws + r.a), *B = reinterpret_cast<f16*>(ws + r.b), *S = reinterpret_cast<f16*>(ws + r.s);
        const int64_t a_plane2 = planes == 2 ? s.a_plane : 0;
        GemmProb p{};
        p.a = p.b = s.tall ? turned : same;
        p.a_plane = p.b_plane = s.x_plane;
        p.a_batch = p.b_batch = s.x_plane * (s.tall ? planes : 2);
        p.lda = p.ldb = s.np;
        p.o = p.ot = A;
        p.o_plane = p.ot_plane = a_plane2;
        p.o_batch = p.ot_batch = s.a_plane * planes;
        p.ldo = p.ldot = s.dp;
        p.k = s.np;
        p.tm = p.tn = s.dp;
        p.s_acc = two(sc.a - 2 * sc.x);
        pa.push_back(p);
        // among d x d matrices: out = by s_acc, s_c and s_diag from left right and c
        p.a_plane = p.b_plane = s.a_plane;
        p.a_batch = p.b_batch = s.a_plane * planes;
        p.lda = p.ldb = s.dp;
        p.c_plane = a_plane2;
        p.c_batch = s.a_plane * planes;
        p.d_out = reinterpret_cast<float*>(ws + r.diag);
        p.d_batch = s.dp;
        p.k = s.dp;
        auto poly = [&](int which, f16* out, const f16* left, const f16* right, const f16* c, float s_acc, float s_c, float s_diag) {
          p.o = p.ot = out;
          p.a = left;
          p.b = right;
          p.c = c;
          p.s_acc = s_acc;
          p.s_c = s_c;
          p.s_diag = s_diag;
          polys[which].push_back(p);
        };
        float a = c1[0];                   // X <- a X + M X
        f16* M = B;
        int m_bits = sc.b;
        if (n == 1) {
          poly(0, B, A, A, A, c1[2] * two(sc.b - 2 * sc.a), c1[1] * two(sc.b - sc.a), 0.f);
        } else {
          const StepScale& next = scales[k + 1];
          const int pbits = bits_for(std::fabs(c1[0]) + sc.pb), sbits = bits_for(sc.rho * next.rho);
          // (the last term: what P's rounding leaves of a I - a I)
          m_bits = bits_for(std::fabs(c1[0]) * next.pb + std::fabs(c2[0]) * sc.pb + sc.pb * next.pb +
                            std::ldexp(std::fabs(c2[0]) * (std::fabs(c1[0]) + sc.pb), -18));
          a = c1[0] * c2[0];
          M = A;
          poly(0, B, A, A, A, c1[2] * two(pbits - 2 * sc.a), c1[1] * two(pbits - sc.a), c1[0] * two(pbits));          // P
          poly(1, S, B, A, A, two(sbits - pbits - sc.a), 0.f, 0.f);                                                   // P A
          poly(2, A, S, B, B, two(next.a - sbits - pbits), 0.f, 0.f);                                                 // P A P
          poly(3, S, A, A, A, c2[2] * two(next.b - 2 * next.a), c2[1] * two(next.b - next.a), 0.f);                   // B of it
          poly(4, A, S, B, B, two(m_bits - next.b - pbits), c2[0] * two(m_bits - pbits), -a * two(m_bits));
        }
        // M X, or X^T M where x is taller than wide
        const f16* xt = s.tall ? same : turned;
        const int64_t xt_batch = s.x_plane * (s.tall ? 2 : planes);
        p.a = s.tall ? xt : M;
        p.b = s.tall ? M : xt;
        p.a_plane = s.tall ? s.x_plane : s.a_plane;
        p.b_plane = s.tall ? s.a_plane : s.x_plane;
        p.a_batch = s.tall ? xt_batch : s.a_plane * planes;
        p.b_batch = s.tall ? s.a_plane * planes : xt_batch;
        p.d_in = p.d_out;
        p.d_cols = s.tall;
        p.d_out = nullptr;
        p.c = same;
        p.o = reinterpret_cast<f16*>(ws + r.same[from ^ 1]);
        p.c_plane = p.o_plane = s.x_plane;
        p.c_batch = p.o_batch = s.x_plane * 2;
        p.ldo = s.tall ? s.dp : s.np;
        p.ot = reinterpret_cast<f16*>(ws + r.turned[from ^ 1]);
        p.ot_plane = s.x_plane;
        p.ot_batch = s.x_plane * planes;
        p.ldot = s.tall ? s.np : s.dp;
        p.tm = s.tall ? s.np : s.dp;
        p.tn = s.tall ? s.dp : s.np;
        p.s_acc = two(xb - m_bits - sc.x);
        p.s_c = a * two(xb - sc.x);
        p.y = t.y;
        p.w = t.w;
        p.y_ld = t.w ? t.cols : t.y_ld;
        p.y_batch = t.w ? 0 : t.y_stride;
        p.rows = t.rows;
        p.cols = t.cols;
        p.y_bf16 = t.dtype == KFAC_BF16;
        p.decay = 1.f - step.lr * step.weight_decay;
        p.factor = t.factor;
        px.push_back(p);
      }
      kfac_status_t r = launch_products<kGram>(pa, batch, planes, g.gram, partial, st);
      for (std::vector<GemmProb>& q : polys)
        if (r == KFAC_OK) r = launch_products<kPoly>(q, batch, planes, g.poly, partial, st);
      if (r == KFAC_OK)
        r = !last ? launch_products<kNext>(px, batch, planes, g.next, partial, st)
            : px[0].w ? launch_products<kWeight>(px, batch, planes, g.next, partial, st)
                      : launch_products<kLast>(px, batch, planes, g.next, partial, st);
      if (r != KFAC_OK) return r;
    }
  }
  return KFAC_OK;
}

}  // namespace kfac
