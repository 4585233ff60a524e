// Declarations shared by the token kernels and their C entry points
// (include/kfac_tokens.h).
#pragma once

#include "objectives.h"
#include "../../include/kfac_tokens.h"

namespace kfac {

constexpr int32_t kSampleMaxVocab = (1 << 20) - 1;      // weights of up to 2^44 are added in 64 bits
// one launch covers 2^32 - 1 threads: 256 for 64 tokens of the table, and for 128 positions
constexpr int32_t kEmbeddingMaxVocab = 1 << 29;
constexpr int64_t kEmbeddingMaxTokens = 1 << 30;
constexpr int32_t kEmbeddingMaxWidth = 1 << 24;

size_t sample_workspace_bytes(int64_t rows, int32_t vocab);
size_t embedding_workspace_bytes(int64_t tokens, int32_t vocab, int32_t width);

kfac_status_t launch_sample(const kfac_sample_t& s, char* ws, hipStream_t st);
kfac_status_t launch_embedding_lookup(const kfac_embedding_t& e, char* ws, hipStream_t st);
kfac_status_t launch_embedding_grad(const kfac_embedding_t& e, char* ws, hipStream_t st);

// -- device helpers ---------------------------------------------------------

// 64-bit integers through the lane operations of objectives.h.
template <int CTRL>
__device__ inline uint64_t dpp(uint64_t u) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ inline uint64_t lane_of(uint64_t u, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), l);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ inline uint64_t row_sum_u64(uint64_t v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return v;
}
__device__ inline uint64_t wave_sum_u64(uint64_t v) {
  v = row_sum_u64(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
// Sum of the lanes up to and with this one.
template <typename V>
__device__ inline V wave_scan(V v) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const V below = __shfl_up(v, d);
    if (lane >= d) v += below;
  }
  return v;
}

}  // namespace kfac
