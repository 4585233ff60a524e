// Orthogonalised updates of matrices with a side of at most 64 (include/
// kfac_orthogonal.h), in three launches for all of them.
//
// With d the shorter side, every X of the iteration is Q X0 with Q a polynomial in
// R0 = X0 X0^T, so the iteration runs on d x d matrices alone:
//     P = a I + b R + c R R,   Q <- P Q,   R <- P R P      for each step,
// and the update is Q X0 at the end.  Here that is not only less work (n does not
// enter) but the whole of it fits one workgroup's LDS.  A small singular value's
// square is what R holds of it, and R's errors grow by a^2 a step against it: all
// of this is done in 64 bits, by 64-bit matrix instructions.  The norm is R0's
// trace.  Only the last product, Q X0, is in float32.
//
// Three launches: R0 by slices of n (and the momentum on the way), the iteration,
// the product.  Of the path for larger matrices every product is a launch: 16
// matrices of 64 x 1024 165 us, here 65 (R0 10, the iteration 43, the product 13);
// one of 32 x 64 140, here 27 (6, 14 and 7).  The iteration is a chain of up to
// four products a step; its matrix instructions alone take 22 of the 43 us (ten
// tiles on four matrix cores, 64 cycles an instruction), the rest are its reads
// from LDS, and a barrier after each.
#include "orthogonal_load.h"

namespace kfac {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kD = kOrthSmall;           // largest d
constexpr int kTiles = 10;               // upper 16 x 16 tiles of d x d
constexpr int kChunk = 128;              // columns of X at a time
constexpr int kLeastSlice = 128;         // columns of a slice
constexpr int kMostSlices = 16;
constexpr int kProbs = 16;

struct SmallProb {
  const void* x;
  float* mom;
  int64_t ld, stride;
  int32_t rows, cols, d, n, nt, tall, bf16;
  int32_t slices, slice, slice_begin, mat_begin, chunks, chunk_begin;
  double* part;             // [batch][slices][kTiles][256]: R0's parts
  float* q;                 // [batch][kD][kD]
  double* inv;              // [batch]: 1 / norm
  float *bias, *bias_mom;
  const float* bias_grad;
  void* y;
  float* w;
  int64_t y_ld, y_stride;
  float factor;
};
struct SmallBatch {
  SmallProb p[kProbs];
  float coefs[3 * KFAC_ORTHOGONAL_MAX_STEPS];
  int32_t n, steps, nesterov;
  float mu, lr, wd;
  double eps;
  uint32_t* flags;
};
static_assert(sizeof(SmallBatch) <= 4096, "kernel arguments");

// X's columns c0 .. c0 + kChunk - 1 of matrix `mat` into LDS, rows past d and columns
// past n as 0.  MOVE: the momentum is brought up to date on the way.
constexpr int kXs = kChunk + 4;
template <bool MOVE>
__device__ inline void load_chunk(const SmallBatch& b, const SmallProb& P, int mat, int c0, float (*xs)[kXs], double scale) {
  const int rows = 16 * P.nt, per = P.tall ? rows / 8 : kChunk / 8;       // vectors of 8 neighbours in memory
  const int vectors = rows * kChunk / 8;
#pragma unroll 2
  for (int e = threadIdx.x; e < vectors; e += 256) {
    const int line = e / per, at = e % per * 8;
    const int64_t r = P.tall ? c0 + line : line;
    const int c = P.tall ? at : c0 + at;
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < P.rows && c < P.cols) {
      const int64_t from = mat * P.stride + r * P.ld;
      load8(u, P.bf16 ? static_cast<const void*>(static_cast<const unsigned short*>(P.x) + from)
                      : static_cast<const void*>(static_cast<const float*>(P.x) + from), c, P.cols, P.bf16);
      if (P.mom) {
        float* m = P.mom + r * P.cols;
        float v[8];
        load8(v, m, c, P.cols, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (MOVE) {
            v[i] = fmaf(b.mu, v[i], u[i]);
            if (c + i < P.cols) m[c + i] = v[i];
          }
          u[i] = b.nesterov ? fmaf(b.mu, v[i], u[i]) : v[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = MOVE ? u[i] : static_cast<float>(static_cast<double>(u[i]) * scale);
      if (P.tall) xs[at + i][line] = f;
      else xs[line][at + i] = f;
    }
  }
}

// A problem entry read once from the kernel arguments and kept in scalar
// registers (see arg_reg).
__device__ inline SmallProb small_regs(const SmallProb& p) {
  SmallProb q;
  q.x = arg_reg(p.x), q.mom = arg_reg(p.mom), q.ld = arg_reg(p.ld), q.stride = arg_reg(p.stride);
  q.rows = arg_reg(p.rows), q.cols = arg_reg(p.cols), q.d = arg_reg(p.d), q.n = arg_reg(p.n), q.nt = arg_reg(p.nt);
  q.tall = arg_reg(p.tall), q.bf16 = arg_reg(p.bf16), q.slices = arg_reg(p.slices), q.slice = arg_reg(p.slice);
  q.slice_begin = arg_reg(p.slice_begin), q.mat_begin = arg_reg(p.mat_begin), q.chunks = arg_reg(p.chunks);
  q.chunk_begin = arg_reg(p.chunk_begin), q.part = arg_reg(p.part), q.q = arg_reg(p.q), q.inv = arg_reg(p.inv);
  q.bias = arg_reg(p.bias), q.bias_mom = arg_reg(p.bias_mom), q.bias_grad = arg_reg(p.bias_grad);
  q.y = arg_reg(p.y), q.w = arg_reg(p.w), q.y_ld = arg_reg(p.y_ld), q.y_stride = arg_reg(p.y_stride);
  q.factor = arg_reg(p.factor);
  return q;
}

__device__ inline void upper_tile(int t, int nt, int* ti, int* tj) {
  int i = 0;
  while (t >= nt - i) t -= nt - i++;
  *ti = i;
  *tj = i + t;
}

// R0's part of a slice: tile (ti, tj) of 16 x 16, accumulator r of a lane at row
// lane / 16 + 4 r, column lane % 16.
__global__ void __launch_bounds__(256) small_gram_kernel(SmallBatch b) {
  __shared__ float xs[kD][kXs];
  int pi = 0;
  while (pi + 1 < b.n && b.p[pi + 1].slice_begin <= static_cast<int>(blockIdx.x)) ++pi;
  const SmallProb P = small_regs(b.p[pi]);
  const int t = blockIdx.x - P.slice_begin, mat = t / P.slices, slice = t % P.slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nt = P.nt, tiles = nt * (nt + 1) / 2;
  f64x4 acc[3] = {};
  const int c1 = min(P.n, (slice + 1) * P.slice);
  for (int c0 = slice * P.slice; c0 < c1; c0 += kChunk) {
    __syncthreads();
    load_chunk<true>(b, P, mat, c0, xs, 1.0);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int tile = wave + 4 * q;
      if (tile >= tiles) continue;
      int ti, tj;
      upper_tile(tile, nt, &ti, &tj);
#pragma unroll 8
      for (int k = 0; k < kChunk; k += 4) {
        const double a = xs[16 * ti + (lane & 15)][k + (lane >> 4)], c = xs[16 * tj + (lane & 15)][k + (lane >> 4)];
        acc[q] = __builtin_amdgcn_mfma_f64_16x16x4f64(a, c, acc[q], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int tile = wave + 4 * q;
    if (tile >= tiles) continue;
    f64x4* to = reinterpret_cast<f64x4*>(P.part + ((static_cast<int64_t>(mat) * P.slices + slice) * kTiles + tile) * 256);
    to[lane] = acc[q];
  }
  if (P.bias && slice == 0) {
    for (int r = threadIdx.x; r < P.rows; r += 256) {
      const float v = fmaf(b.mu, P.bias_mom[r], fmaf(b.wd, P.bias[r], P.bias_grad[r]));
      P.bias_mom[r] = v;
      P.bias[r] = fmaf(-b.lr, v, P.bias[r]);
    }
  }
}

// The iteration, a wavefront for each upper tile; a matrix's lower half mirrors the
// upper.  Rows of 68 values: a 16 x 4 operand lies in all banks alike.
constexpr int kLd = 68;
__global__ void __launch_bounds__(kTiles * 64) small_iterate_kernel(SmallBatch b) {
  __shared__ double R[kD * kLd], P_[kD * kLd], Q[kD * kLd], W[kD * kLd];
  int pi = 0;
  while (pi + 1 < b.n && b.p[pi + 1].mat_begin <= static_cast<int>(blockIdx.x)) ++pi;
  const SmallProb P = small_regs(b.p[pi]);
  const int mat = blockIdx.x - P.mat_begin;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nt = P.nt;
  const bool works = wave < nt * (nt + 1) / 2;
  int ti = 0, tj = 0;
  if (works) upper_tile(wave, nt, &ti, &tj);
  const int row = 16 * ti + (lane >> 4), col = 16 * tj + (lane & 15);     // of accumulator 0; the others 4 rows on each
  auto put = [&](double* m, const f64x4& v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (row + 4 * r <= col) {
        m[(row + 4 * r) * kLd + col] = v[r];
        m[col * kLd + row + 4 * r] = v[r];
      }
    }
  };
  auto times = [&](const double* x, const double* y) {
    const double* a = x + (16 * ti + (lane & 15)) * kLd + (lane >> 4);
    const double* c = y + (16 * tj + (lane & 15)) * kLd + (lane >> 4);
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
    double u = a[0], v = c[0];
    for (int k = 4; k < 16 * nt; k += 4) {
      const double un = a[k], vn = c[k];
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(u, v, acc, 0, 0, 0);
      u = un;
      v = vn;
    }
    acc = __builtin_amdgcn_mfma_f64_16x16x4f64(u, v, acc, 0, 0, 0);
    return acc;
  };
  if (works) {
    f64x4 sum = {0.0, 0.0, 0.0, 0.0};
    for (int s = 0; s < P.slices; ++s)
      sum += reinterpret_cast<const f64x4*>(P.part + ((static_cast<int64_t>(mat) * P.slices + s) * kTiles + wave) * 256)[lane];
    put(R, sum);
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < P.d; ++i) trace += R[i * kLd + i];
  if (!(trace < INFINITY) && threadIdx.x == 0) raise_flag(b.flags, KFAC_FLAG_NONFINITE);
  const double norm = sqrt(trace) + b.eps;
  const double inv = norm > 0.0 || norm != norm ? 1.0 / norm : 0.0;
  if (threadIdx.x == 0) P.inv[mat] = inv;
  __syncthreads();
  for (int e = threadIdx.x; e < 256 * nt * nt; e += kTiles * 64) {
    double* at = R + e / (16 * nt) * kLd + e % (16 * nt);
    *at = *at * inv * inv;
  }
  __syncthreads();
  for (int s = 0; s < b.steps; ++s) {
    const double ca = b.coefs[3 * s], cb = b.coefs[3 * s + 1], cc = b.coefs[3 * s + 2];
    const bool last = s + 1 == b.steps;
    if (works) {
      f64x4 p = times(R, R);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p[r] = fma(cc, p[r], fma(cb, R[(row + 4 * r) * kLd + col], row + 4 * r == col ? ca : 0.0));
      put(P_, p);
      if (s == 0) put(Q, p);
    }
    __syncthreads();
    f64x4 q, w;
    if (works && s > 0) q = times(P_, Q);
    if (works && !last) w = times(P_, R);
    __syncthreads();
    if (works && s > 0) put(Q, q);
    if (works && !last) put(W, w);
    __syncthreads();
    if (works && !last) put(R, times(W, P_));
    __syncthreads();
  }
  float* to = P.q + static_cast<int64_t>(mat) * kD * kD;
  for (int e = threadIdx.x; e < 256 * nt * nt; e += kTiles * 64) {
    const int i = e / (16 * nt), j = e % (16 * nt);
    to[i * kD + j] = static_cast<float>(Q[i * kLd + j]);
  }
}

// The update Q X0 of a chunk of columns, or the weight that takes it.
__global__ void __launch_bounds__(256) small_apply_kernel(SmallBatch b) {
  __shared__ float xs[kD][kXs];
  __shared__ float q[kD][kLd];
  int pi = 0;
  while (pi + 1 < b.n && b.p[pi + 1].chunk_begin <= static_cast<int>(blockIdx.x)) ++pi;
  const SmallProb P = small_regs(b.p[pi]);
  const int t = blockIdx.x - P.chunk_begin, mat = t / P.chunks, c0 = t % P.chunks * kChunk;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nt = P.nt;
  load_chunk<false>(b, P, mat, c0, xs, P.inv[mat]);
  const float* from = P.q + static_cast<int64_t>(mat) * kD * kD;
#pragma unroll
  for (int h = 0; h < kD * kD / 1024; ++h) {             // (what the iteration did not write is not used)
    const int e = (h * 256 + threadIdx.x) * 4;
    *reinterpret_cast<f32x4*>(&q[e / kD][e % kD]) = *reinterpret_cast<const f32x4*>(from + e);
  }
  __syncthreads();
  f32x4 acc[2][kD / 16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = 16 * (2 * wave + h) + (lane & 15);
#pragma unroll
    for (int ti = 0; ti < kD / 16; ++ti) acc[h][ti] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < 16 * nt; k += 4) {
      const float x = xs[k + (lane >> 4)][j];
#pragma unroll
      for (int ti = 0; ti < kD / 16; ++ti)
        if (ti < nt) acc[h][ti] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[16 * ti + (lane & 15)][k + (lane >> 4)], x, acc[h][ti], 0, 0, 0);
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int ti = 0; ti < kD / 16; ++ti)
#pragma unroll
      for (int r = 0; r < 4; ++r) xs[16 * ti + 4 * (lane >> 4) + r][16 * (2 * wave + h) + (lane & 15)] = acc[h][ti][r];
  __syncthreads();
  const int rows = 16 * nt, per = P.tall ? rows / 8 : kChunk / 8;
  const float decay = 1.f - b.lr * b.wd;
#pragma unroll 2
  for (int e = threadIdx.x; e < rows * kChunk / 8; e += 256) {
    const int line = e / per, at = e % per * 8;
    const int64_t r = P.tall ? c0 + line : line;
    const int c = P.tall ? at : c0 + at;
    if (r >= P.rows || c >= P.cols) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = P.tall ? xs[at + i][line] : xs[line][at + i];
    const int64_t to = mat * P.y_stride + r * P.y_ld + c;
    const bool whole = c + 8 <= P.cols;
    if (P.w) {
      float w[8];
      load8(w, P.w + r * P.y_ld, c, P.cols, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(-P.factor, v[i], decay * w[i]);
    }
    if (!P.w && P.bf16) {
      unsigned short* y = static_cast<unsigned short*>(P.y) + to;
      if (whole) store16(y, pack16<__bf16>(v));
      else
        for (int i = 0; i < 8; ++i)
          if (c + i < P.cols) Elem<__bf16>::store(y, i, v[i]);
    } else {
      float* y = (P.w ? P.w : static_cast<float*>(P.y)) + to;
      if (whole) {
        store16(y, pack16<float>(v));
        store16(y + 4, pack16<float>(v + 4));
      } else {
        for (int i = 0; i < 8; ++i)
          if (c + i < P.cols) y[i] = v[i];
      }
    }
  }
}

struct SmallShape {
  int d, n, slices, slice;
};
SmallShape small_shape(const OrthTask& t) {
  SmallShape s;
  s.d = std::min(t.rows, t.cols);
  s.n = std::max(t.rows, t.cols);
  const int least = std::max(kLeastSlice, (s.n + kMostSlices - 1) / kMostSlices);
  s.slice = (least + kChunk - 1) / kChunk * kChunk;
  s.slices = (s.n + s.slice - 1) / s.slice;
  return s;
}
size_t small_bytes(const OrthTask& t) {
  const SmallShape s = small_shape(t);
  return static_cast<size_t>(t.batch) * (static_cast<size_t>(s.slices) * kTiles * 256 * sizeof(double) + kD * kD * sizeof(float) + 256);
}

}  // namespace

size_t orth_small_bytes(const std::vector<OrthTask>& tasks) {
  size_t n = 0;
  for (const OrthTask& t : tasks) n += align_up(small_bytes(t), 256);
  return n;
}

kfac_status_t launch_orth_small(const std::vector<OrthTask>& tasks, const kfac_orthogonal_t& how, const OrthStep& step,
                                char* regions, uint32_t* flags, hipStream_t st) {
  for (size_t i0 = 0; i0 < tasks.size(); i0 += kProbs) {
    SmallBatch b{};
    std::copy(how.coefs, how.coefs + 3 * how.steps, b.coefs);
    b.steps = how.steps;
    b.nesterov = how.nesterov;
    b.mu = step.momentum;
    b.lr = step.lr;
    b.wd = step.weight_decay;
    b.eps = how.eps;
    b.flags = flags;
    int64_t slices = 0, mats = 0, chunks = 0;
    for (size_t i = i0; i < tasks.size() && i < i0 + kProbs; ++i) {
      const OrthTask& t = tasks[i];
      const SmallShape s = small_shape(t);
      SmallProb& p = b.p[b.n++];
      p.x = t.x;
      p.mom = t.mom;
      p.ld = t.ld;
      p.stride = t.stride;
      p.rows = t.rows;
      p.cols = t.cols;
      p.d = s.d;
      p.n = s.n;
      p.nt = (s.d + 15) / 16;
      p.tall = t.rows > t.cols;
      p.bf16 = t.dtype == KFAC_BF16;
      p.slices = s.slices;
      p.slice = s.slice;
      p.slice_begin = static_cast<int>(slices);
      slices += static_cast<int64_t>(s.slices) * t.batch;
      p.mat_begin = static_cast<int>(mats);
      mats += t.batch;
      p.chunks = (s.n + kChunk - 1) / kChunk;
      p.chunk_begin = static_cast<int>(chunks);
      chunks += static_cast<int64_t>(p.chunks) * t.batch;
      p.part = reinterpret_cast<double*>(regions);
      p.q = reinterpret_cast<float*>(p.part + static_cast<int64_t>(t.batch) * s.slices * kTiles * 256);
      p.inv = reinterpret_cast<double*>(p.q + static_cast<int64_t>(t.batch) * kD * kD);
      regions += align_up(small_bytes(t), 256);
      p.bias = t.bias;
      p.bias_mom = t.bias_mom;
      p.bias_grad = t.bias_grad;
      p.y = t.y;
      p.w = t.w;
      p.y_ld = t.w ? t.cols : t.y_ld;
      p.y_stride = t.w ? 0 : t.y_stride;
      p.factor = t.factor;
    }
    if (mats == 0) continue;
    hipLaunchKernelGGL(small_gram_kernel, dim3(static_cast<uint32_t>(slices)), dim3(256), 0, st, b);
    hipLaunchKernelGGL(small_iterate_kernel, dim3(static_cast<uint32_t>(mats)), dim3(kTiles * 64), 0, st, b);
    hipLaunchKernelGGL(small_apply_kernel, dim3(static_cast<uint32_t>(chunks)), dim3(256), 0, st, b);
    if (hipGetLastError() != hipSuccess) return KFAC_ERR_HIP;
  }
  return KFAC_OK;
}

}  // namespace kfac
