// Declarations shared by the objective and dropout kernels and their C entry
// points (include/kfac_objectives.h).
#pragma once

#include "common.h"
#include "../../include/kfac_objectives.h"

namespace kfac {

// An objective's workspace: the flag word, the counters of the policy loss, then
// the operator's regions, all 256-byte aligned.  The counters are 0 between calls,
// so no objective has a region there and they can take turns on one workspace.
// They are 256 bytes apart: packed into the flag word's 256 bytes, which would
// let a step share the workspace too, they cost 4096 x 90 bf16 8.5 -> 16.2 us and
// 16384 x 500 17.5 -> 23.6 us.
constexpr int kMaxPartials = 2048;        // policy: (A, K, clipped) sums, one triple a workgroup
constexpr int kArriveGroup = 32;          // workgroups that count on one counter
constexpr int kArriveStride = 64;         // words between counters
constexpr size_t kArriveBytes = sizeof(uint32_t) * kArriveStride * (1 + kMaxPartials / kArriveGroup);
constexpr size_t kRegions = kFlagBytes + kArriveBytes;
static_assert(kRegions % 256 == 0 && kMaxPartials % kArriveGroup == 0);
constexpr int kPairThreads = 1024;        // preference: threads of a pair's workgroup
constexpr int kBalanceMaxExperts = 1024;
constexpr int64_t kDropoutMaxBlocks = (int64_t(1) << 32) - 1024;  // generator blocks a call
constexpr int kBalanceBlocks = 512;       // balance: workgroups of the first pass

size_t token_workspace_bytes(int objective, int64_t rows, int32_t groups);
size_t balance_workspace_bytes(int64_t tokens, int32_t experts);

kfac_status_t launch_token_logp(const kfac_token_rows_t& t, char* ws, hipStream_t st);
kfac_status_t launch_policy(const kfac_token_rows_t& t, const kfac_policy_t& p, char* ws, hipStream_t st);
kfac_status_t launch_preference(const kfac_token_rows_t& t, const kfac_preference_t& p, char* ws, hipStream_t st);
kfac_status_t launch_balance(const kfac_balance_t& b, char* ws, hipStream_t st);
kfac_status_t launch_dropout(const kfac_dropout_t& d, hipStream_t st);

// -- device helpers ---------------------------------------------------------

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at any element alignment (gfx950 global accesses need none: one
// 16-byte instruction, whatever the address).  NT: nontemporal, for data that
// is not worth a place in the caches.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool NT = false>
__device__ inline u32x4 load16(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
  else return *static_cast<const u32x4_any*>(p);
}
template <bool NT = false>
__device__ inline void store16(void* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(static_cast<u32x4_any>(v), static_cast<u32x4_any*>(p));
  else *static_cast<u32x4_any*>(p) = v;
}

// The memory-side cache.  Streams that fit it together find what was written
// just before and leave theirs for what comes next; larger ones go past it
// with nontemporal accesses.  Measured on copies and reads of 2 GiB: 5.7 TB/s
// and 6.4 TB/s through the cache, 6.2 and 7.2 past it (128 MiB copied again
// and again: 7.0 through it, 6.2 past it).
constexpr int64_t kCacheBytes = int64_t(256) << 20;

// Element type traits: VE elements per 16-byte vector.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VE = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ float get(u32x4 v, int i) { return __uint_as_float(v[i]); }
  static __device__ float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ void store(void* p, int64_t i, float x) { static_cast<float*>(p)[i] = x; }
};
template <>
struct Elem<__bf16> {
  static constexpr int VE = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ float get(u32x4 v, int i) {
    return __uint_as_float((i & 1) ? (v[i >> 1] & 0xFFFF0000u) : (v[i >> 1] << 16));
  }
  static __device__ uint32_t bits(float x) { return __builtin_bit_cast(unsigned short, static_cast<__bf16>(x)); }
  static __device__ float load(const void* p, int64_t i) {
    return bf16_bits_to_float(static_cast<const unsigned short*>(p)[i]);
  }
  static __device__ void store(void* p, int64_t i, float x) {
    static_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(bits(x));
  }
};

// Eight (bf16) or four (f32) floats rounded to nearest even into one vector
// (bf16: two at a time, one instruction).
template <typename T>
__device__ inline u32x4 pack16(const float* f) {
  u32x4 v;
  if constexpr (Elem<T>::VE == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
  } else {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
  }
  return v;
}

// max of three without the canonicalising moves that fmaxf needs for
// signalling NaNs (a NaN operand is passed over; the sums still carry it).
__device__ inline float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

__device__ inline bool finite(float v) { return fabsf(v) < INFINITY; }

// v from the lane that the DPP control names (all controls used here have a
// source inside the same 16 lanes).
template <int CTRL>
__device__ inline float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ inline double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ inline float lane_of(float v, int l) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}
__device__ inline double lane_of(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), l);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// Sum / maximum over 16 lanes (every lane gets it), and over the wavefront
// (uniform); the order is fixed.
template <typename V>
__device__ inline V row_sum(V v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return v;
}
__device__ inline float row_max(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  v = fmaxf(v, dpp<kMirror>(v));
  return v;
}
template <typename V>
__device__ inline V wave_sum(V v) {
  v = row_sum(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ inline float wave_max(float v) {
  v = row_max(v);
  return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}

__device__ inline int64_t load_index(const void* p, int64_t i, int type) {
  return type == KFAC_I64 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

}  // namespace kfac
