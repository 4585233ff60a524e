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
// carries; as operands of the products, where B hardly has them yet, 11 bits do.  bfloat16 outputs take HALF, float32 ones FULL.  Each
// matrix carries a power of two that keeps |value| <= 2^15: the norm bounds
// every element, and the polynomial's maximum bounds the norm after each step.
//
// Layout.  Planes are row-major, both sides padded with zeros to whole tiles,
// which every product keeps at zero: no bounds checks outside the first and last
// pass.
#include "orthogonal.h"
#include "objectives.h"

#include <algorithm>
#include <cmath>

namespace kfac {

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kNormBlocks = 256;      // partial sums of a matrix's squares
constexpr int kMaxProbs = 16;         // problems a launch

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
  int32_t rows_p, cols_p, tiles_c, blk2_begin, tall;
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

__device__ inline float load_any(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_bits_to_float(static_cast<const unsigned short*>(p)[i]) : static_cast<const float*>(p)[i];
}
// The matrix that is orthogonalised, from a gradient and its momentum after the update.
__device__ inline float direction(const PrepBatch& b, float g, float m) { return b.nesterov ? fmaf(b.mu, m, g) : m; }

__global__ void __launch_bounds__(256) orth_norm_kernel(PrepBatch b) {
  __shared__ double red[4];
  const PrepProb& P = b.p[find<0>(b, blockIdx.x)];
  const int t = blockIdx.x - P.blk_begin;
  const int mat = t / P.blocks, blk = t % P.blocks;
  const int64_t base = mat * P.stride;
  double sum = 0.0;
  for (int r = blk; r < P.rows; r += P.blocks) {
    for (int c = threadIdx.x; c < P.cols; c += 256) {
      float u = load_any(P.x, base + r * P.ld + c, P.bf16);
      if (P.mom) {
        float* m = P.mom + static_cast<int64_t>(r) * P.cols + c;
        const float v = fmaf(b.mu, *m, u);
        *m = v;
        u = direction(b, u, v);
      }
      sum += static_cast<double>(u) * static_cast<double>(u);
    }
    if (P.bias && threadIdx.x == 0) {
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

// With HALF the low halves are stored with X alone.
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
  double sum = tid < P.blocks ? P.part[static_cast<int64_t>(mat) * kNormBlocks + tid] : 0.0;
  sum = wave_sum(sum);
  if ((tid & 63) == 0) red[tid / 64] = sum;
  __syncthreads();
  sum = (red[0] + red[1]) + (red[2] + red[3]);
  if (!(sum < INFINITY) && t == 0 && tid == 0) raise_flag(b.flags, KFAC_FLAG_NONFINITE);
  const double norm = sqrt(sum) + b.eps;
  const double inv = norm > 0.0 ? static_cast<double>(P.scale) / norm : 0.0;
  const int64_t base = mat * P.stride;
  f16* same = P.same + mat * P.same_stride;
  f16* turned = P.turned + mat * P.turned_stride;
  for (int i = tid; i < 64 * 64; i += 256) {
    const int r = r0 + i / 64, c = c0 + i % 64;
    float u = 0.f;
    if (r < P.rows && c < P.cols) {
      u = load_any(P.x, base + r * P.ld + c, P.bf16);
      if (P.mom) u = direction(b, u, P.mom[static_cast<int64_t>(r) * P.cols + c]);
      u = static_cast<float>(static_cast<double>(u) * inv);
    }
    tile[i / 64][i % 64] = u;
    f16 hi, lo;
    split(u, hi, lo);
    const int64_t at = static_cast<int64_t>(r) * P.cols_p + c;
    same[at] = hi;
    if (PLANES == 2 || !P.tall) same[P.plane + at] = lo;
  }
  __syncthreads();
  for (int i = tid; i < 64 * 64; i += 256) {
    f16 hi, lo;
    split(tile[i % 64][i / 64], hi, lo);
    const int64_t at = static_cast<int64_t>(c0 + i / 64) * P.rows_p + r0 + i % 64;
    turned[at] = hi;
    if (PLANES == 2 || P.tall) turned[P.plane + at] = lo;
  }
}

// -- the products --------------------------------------------------------------

struct GemmProb {
  const f16 *a, *b, *c;       // P, Q and the matrix that is added; second planes `*_plane` elements on
  f16 *o, *ot;                // result and its transpose (one matrix where it is symmetric)
  int64_t a_plane, b_plane, c_plane, o_plane, ot_plane;
  int64_t a_batch, b_batch, c_batch, o_batch, ot_batch;
  int32_t lda, ldb, ldo, ldot;      // c is laid out as o
  int32_t k, tn, tiles, sym, blk_begin;
  float s_acc, s_c;           // result = s_acc P Q^T + s_c C
  float *d_out, *d_in;        // HALF: the diagonal that the result leaves out, and the one that P left out
  int64_t d_batch;
  // last product: the update goes to y, or into w
  void* y;
  float* w;
  int64_t y_ld, y_batch;
  int32_t rows, cols, tall, y_bf16;
  float decay, factor;
};
struct GemmBatch {
  GemmProb p[kMaxProbs];
  int32_t n;
};
static_assert(sizeof(GemmBatch) <= 4096, "kernel arguments");

#define KFAC_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (0x7 << 4) | (0xF << 8))

template <int PLANES, int BT, bool LAST>
__global__ void __launch_bounds__(BT == 256 ? 512 : 256) orth_gemm_kernel(GemmBatch batch) {
  constexpr int THREADS = BT == 256 ? 512 : 256;
  constexpr int BK = PLANES == 2 ? 32 : 64;           // contraction a stage
  constexpr int CHUNKS = BK / 8;                      // 16-byte chunks of a row
  constexpr int OP = BT * BK;                         // elements of an operand's plane of a stage
  constexpr int LOADS = OP / 8 / THREADS;             // loads a thread and plane
  constexpr int MI = BT == 256 ? 4 : 2, NJ = 2;       // 32 x 32 blocks of a wavefront
  __shared__ __attribute__((aligned(16))) f16 ring[2][2][PLANES][OP];
  int pi = 0;
  while (pi + 1 < batch.n && batch.p[pi + 1].blk_begin <= static_cast<int>(blockIdx.x)) ++pi;
  const GemmProb& P = batch.p[pi];
  int t = blockIdx.x - P.blk_begin;
  const int mat = t / P.tiles;
  t -= mat * P.tiles;
  int ti, tj;
  if (P.sym) {                       // upper tiles, row by row
    ti = 0;
    int width = P.tn;
    while (t >= width) { t -= width; --width; ++ti; }
    tj = ti + t;
  } else {
    ti = t / P.tn;
    tj = t % P.tn;
  }
  const int i0 = ti * BT, j0 = tj * BT;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int wm = BT == 256 ? (wid >> 2) * 128 : (wid >> 1) * 64;
  const int wn = BT == 256 ? (wid & 3) * 64 : (wid & 1) * 64;

  // operands: a buffer resource of the tile's rows each
  i32x4 rsrc[2][PLANES];
  uint32_t off[2][LOADS];
#pragma unroll
  for (int op = 0; op < 2; ++op) {
    const int ld = op ? P.ldb : P.lda;
    const f16* base = op ? P.b + mat * P.b_batch + static_cast<int64_t>(j0) * ld : P.a + mat * P.a_batch + static_cast<int64_t>(i0) * ld;
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl) {
      const uint64_t at = reinterpret_cast<uint64_t>(base + (pl ? (op ? P.b_plane : P.a_plane) : 0));
      rsrc[op][pl] = i32x4{static_cast<int>(at & 0xffffffffu), static_cast<int>((at >> 32) & 0xffffu), BT * ld * 2, 0x00020000};
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int p = u * THREADS + tid, row = p / CHUNKS;
      const int c = (p % CHUNKS) ^ (CHUNKS == 8 ? (row >> 1) & 7 : (row >> 2) & 3);
      off[op][u] = static_cast<uint32_t>(row * ld + c * 8) * 2;
    }
  }
  auto issue = [&](int s, int slot) {
#pragma unroll
    for (int op = 0; op < 2; ++op)
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
          const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
              (__attribute__((address_space(3))) void*)(&ring[slot][op][pl][(u * THREADS + wid * 64) * 8])));
          asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                       :
                       : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(static_cast<uint32_t>(s * BK * 2) + off[op][u]),
                         "s"(rsrc[op][pl])
                       : "memory", "m0");
        }
  };

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // a lane's fragment of rows r0 .. r0 + 31 of an operand: row r0 + lane % 32, 8 of the contraction from ks + 8 (lane / 32)
  auto frag = [&](const f16* op, int r0, int ks) {
    const int row = r0 + (lane & 31), c = ks / 8 + (lane >> 5);
    return *reinterpret_cast<const f16x8*>(op + row * BK + (c ^ (CHUNKS == 8 ? (row >> 1) & 7 : (row >> 2) & 3)) * 8);
  };

  const int stages = P.k / BK;
  issue(0, 0);
  for (int s = 0; s < stages; ++s) {
    KFAC_WAIT_VM(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");           // the loads above wrote what is read below
    if (s + 1 < stages) issue(s + 1, (s + 1) & 1);
    const int slot = s & 1;
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      f16x8 fa[PLANES][MI], fb[PLANES][NJ];
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[pl][i] = frag(ring[slot][0][pl], wm + 32 * i, ks);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[pl][j] = frag(ring[slot][1][pl], wn + 32 * j, ks);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[0][j], acc[i][j], 0, 0, 0);
          if constexpr (PLANES == 2) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[1][j], acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[1][i], fb[0][j], acc[i][j], 0, 0, 0);
          }
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0): this wavefront has read the slot before the next barrier
  }

  // accumulator r of block (i, j): row 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
  const bool diag = P.sym && ti == tj;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col = j0 + wn + 32 * j + (lane & 31);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row0 = i0 + wm + 32 * i + 8 * q + 4 * (lane >> 5);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = row0 + e;
          float v = P.s_acc * acc[i][j][4 * q + e];
          const int64_t at = static_cast<int64_t>(row) * P.ldo + col;
          if (P.c) {
            const f16* c = P.c + mat * P.c_batch + at;
            float x = static_cast<float>(c[0]);
            if (PLANES == 2 || P.c_plane) x += static_cast<float>(c[P.c_plane]);
            if (PLANES == 1 && P.d_in) v = fmaf(P.s_acc * P.d_in[mat * P.d_batch + row], x, v);
            v = fmaf(P.s_c, x, v);
          }
          if constexpr (LAST) {
            if (row >= P.rows || col >= P.cols) continue;       // rows, cols of X
            const int64_t to = P.tall ? static_cast<int64_t>(col) * P.y_ld + row : static_cast<int64_t>(row) * P.y_ld + col;
            if (P.w) {
              P.w[to] = fmaf(-P.factor, v, P.decay * P.w[to]);
            } else if (P.y_bf16) {
              static_cast<unsigned short*>(P.y)[mat * P.y_batch + to] = static_cast<unsigned short>(Elem<__bf16>::bits(v));
            } else {
              static_cast<float*>(P.y)[mat * P.y_batch + to] = v;
            }
          } else {
            if (diag && row > col) continue;
            if (PLANES == 1 && P.d_out && row == col) {
              P.d_out[mat * P.d_batch + row] = v;
              v = 0.f;
            }
            f16 hi, lo;
            split(v, hi, lo);
            f16* o = P.o + mat * P.o_batch + at;
            o[0] = hi;
            if (PLANES == 2 || P.o_plane) o[P.o_plane] = lo;
            f16* ot = P.ot + mat * P.ot_batch + static_cast<int64_t>(col) * P.ldot + row;
            ot[0] = hi;
            if constexpr (PLANES == 2) ot[P.ot_plane] = lo;
          }
        }
      }
    }
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
  s.tile = s.d >= 2048 ? 256 : 128;
  s.dp = round_up(s.d, s.tile);
  s.np = round_up(s.n, s.tile);
  s.x_plane = static_cast<int64_t>(s.dp) * s.np;
  s.a_plane = static_cast<int64_t>(s.dp) * s.dp;
  return s;
}

struct Region {
  size_t part, x, xt[2], a, b, diag;
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
    Region r;
    const size_t batch = static_cast<size_t>(t.batch);
    r.part = take(sizeof(double) * kNormBlocks * batch);
    r.x = take(2 * 2 * batch * s.x_plane);
    r.xt[0] = take(2 * planes * batch * s.x_plane);
    r.xt[1] = take(2 * planes * batch * s.x_plane);
    r.a = take(2 * planes * batch * s.a_plane);
    r.b = take(2 * planes * batch * s.a_plane);
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
};
std::vector<StepScale> step_scales(const kfac_orthogonal_t& how, int* last) {
  std::vector<StepScale> out;
  double rho = 1.0;
  for (int s = 0; s < how.steps; ++s) {
    const PolyBound p = poly_of(how.coefs + 3 * s, rho);
    out.push_back({bits_for(rho), bits_for(rho * rho), bits_for(p.b)});
    rho = p.next;
  }
  *last = bits_for(rho);
  return out;
}

template <bool LAST>
kfac_status_t launch_products(const std::vector<GemmProb>& probs, const std::vector<int>& tile, const std::vector<int>& batch,
                              int planes, hipStream_t st) {
  for (int bt : {256, 128}) {
    size_t i = 0;
    while (i < probs.size()) {
      GemmBatch b{};
      int64_t blocks = 0;
      for (; i < probs.size() && b.n < kMaxProbs; ++i) {
        if (tile[i] != bt) continue;
        GemmProb p = probs[i];
        if (blocks + static_cast<int64_t>(p.tiles) * batch[i] > (1 << 22)) {
          if (b.n) break;                 // the rest in a launch of their own
        }
        p.blk_begin = static_cast<int>(blocks);
        blocks += static_cast<int64_t>(p.tiles) * batch[i];
        b.p[b.n++] = p;
      }
      if (b.n == 0) continue;
      const dim3 grid(static_cast<uint32_t>(blocks)), block(bt == 256 ? 512 : 256);
      if (planes == 2) {
        if (bt == 256) hipLaunchKernelGGL((orth_gemm_kernel<2, 256, LAST>), grid, block, 0, st, b);
        else hipLaunchKernelGGL((orth_gemm_kernel<2, 128, LAST>), grid, block, 0, st, b);
      } else {
        if (bt == 256) hipLaunchKernelGGL((orth_gemm_kernel<1, 256, LAST>), grid, block, 0, st, b);
        else hipLaunchKernelGGL((orth_gemm_kernel<1, 128, LAST>), grid, block, 0, st, b);
      }
      if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
    }
  }
  return KFAC_OK;
}

}  // namespace

size_t orth_workspace_bytes(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how) {
  return plan(tasks, how, nullptr);
}

kfac_status_t launch_orthogonal(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how, const OrthStep& step,
                                char* ws, hipStream_t st) {
  const int planes = how.products == KFAC_PRODUCTS_FULL ? 2 : 1;
  std::vector<Region> regions;
  plan(tasks, how, &regions);
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
      p.blocks = std::min(t.rows, kNormBlocks);
      p.blk_begin = static_cast<int>(blocks);
      blocks += static_cast<int64_t>(p.blocks) * t.batch;
      p.part = reinterpret_cast<double*>(ws + r.part);
      p.bias = t.bias;
      p.bias_mom = t.bias_mom;
      p.bias_grad = t.bias_grad;
      f16* x = reinterpret_cast<f16*>(ws + r.x);
      f16* xt = reinterpret_cast<f16*>(ws + r.xt[0]);
      p.same = s.tall ? xt : x;
      p.turned = s.tall ? x : xt;
      p.plane = s.x_plane;
      p.same_stride = s.x_plane * (s.tall ? planes : 2);
      p.turned_stride = s.x_plane * (s.tall ? 2 : planes);
      p.tall = s.tall;
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

  std::vector<int> tile, batch;
  for (const OrthTask& t : tasks) {
    tile.push_back(shape_of(t).tile);
    batch.push_back(t.batch);
  }
  auto two = [](int e) { return std::ldexp(1.f, e); };
  for (int k = 0; k < how.steps; ++k) {
    const float a = how.coefs[3 * k], b = how.coefs[3 * k + 1], c = how.coefs[3 * k + 2];
    const StepScale& sc = scales[k];
    const bool last = k + 1 == how.steps;
    const int xb = last ? 0 : scales[k + 1].x;         // the last X is written as it is
    std::vector<GemmProb> pa, pb, px;
    for (size_t i = 0; i < tasks.size(); ++i) {
      const OrthTask& t = tasks[i];
      const Shape s = shape_of(t);
      const Region& r = regions[i];
      f16* x = reinterpret_cast<f16*>(ws + r.x);
      f16* xt = reinterpret_cast<f16*>(ws + r.xt[k & 1]);
      f16* xt_next = reinterpret_cast<f16*>(ws + r.xt[(k + 1) & 1]);
      f16* A = reinterpret_cast<f16*>(ws + r.a);
      f16* B = reinterpret_cast<f16*>(ws + r.b);
      const int nd = s.dp / s.tile;
      GemmProb p{};
      p.a = p.b = x;
      p.a_plane = p.b_plane = s.x_plane;
      p.a_batch = p.b_batch = s.x_plane * 2;
      p.lda = p.ldb = s.np;
      p.o = p.ot = A;
      p.o_plane = p.ot_plane = planes == 2 ? s.a_plane : 0;
      p.o_batch = p.ot_batch = s.a_plane * planes;
      p.ldo = p.ldot = s.dp;
      p.k = s.np;
      p.tn = nd;
      p.tiles = nd * (nd + 1) / 2;
      p.sym = 1;
      p.s_acc = two(sc.a - 2 * sc.x);
      pa.push_back(p);
      p.a = p.b = A;
      p.a_plane = p.b_plane = s.a_plane;
      p.a_batch = p.b_batch = s.a_plane * planes;
      p.lda = p.ldb = s.dp;
      p.c = A;
      p.c_plane = planes == 2 ? s.a_plane : 0;
      p.c_batch = s.a_plane * planes;
      p.o = p.ot = B;
      p.d_out = reinterpret_cast<float*>(ws + r.diag);
      p.d_batch = s.dp;
      p.k = s.dp;
      p.s_acc = c * two(sc.b - 2 * sc.a);
      p.s_c = b * two(sc.b - sc.a);
      pb.push_back(p);
      p.a = B;
      p.d_in = p.d_out;
      p.d_out = nullptr;
      p.b = xt;
      p.b_plane = s.x_plane;
      p.b_batch = s.x_plane * planes;
      p.c = x;
      p.c_plane = s.x_plane;
      p.c_batch = s.x_plane * 2;
      p.o = x;
      p.o_plane = s.x_plane;
      p.o_batch = s.x_plane * 2;
      p.ldo = s.np;
      p.ot = xt_next;
      p.ot_plane = s.x_plane;
      p.ot_batch = s.x_plane * planes;
      p.ldot = s.dp;
      p.tn = s.np / s.tile;
      p.tiles = nd * p.tn;
      p.sym = 0;
      p.s_acc = two(xb - sc.b - sc.x);
      p.s_c = a * two(xb - sc.x);
      p.y = t.y;
      p.w = t.w;
      p.y_ld = t.w ? t.cols : t.y_ld;
      p.y_batch = t.y_stride;
      p.rows = s.d;
      p.cols = s.n;
      p.tall = s.tall;
      p.y_bf16 = t.dtype == KFAC_BF16;
      p.decay = 1.f - step.lr * step.weight_decay;
      p.factor = t.factor;
      px.push_back(p);
    }
    kfac_status_t r = launch_products<false>(pa, tile, batch, planes, st);
    if (r == KFAC_OK) r = launch_products<false>(pb, tile, batch, planes, st);
    if (r == KFAC_OK) r = last ? launch_products<true>(px, tile, batch, planes, st) : launch_products<false>(px, tile, batch, planes, st);
    if (r != KFAC_OK) return r;
  }
  return KFAC_OK;
}

}  // namespace kfac
