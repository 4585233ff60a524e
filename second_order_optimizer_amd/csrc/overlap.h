// Which tensors of a call share memory, on the host.
#pragma once

#include <algorithm>
#include <cstdint>
#include <vector>

#include "../../include/kfac.h"

namespace kfac {

// Contiguous memory that a call reads or writes.
struct Span {
  uintptr_t begin, end;
  bool written;
};
inline Span span_of(const void* p, int64_t bytes, bool written) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, at + static_cast<uintptr_t>(bytes), written};
}

// Whether one that is written shares memory with any other.
inline bool share_memory(std::vector<Span>& spans) {
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t end = 0, written_end = 0;      // of those that begin no later
  for (const Span& s : spans) {
    if (s.begin == s.end) continue;
    if (s.begin < (s.written ? end : written_end)) return true;
    end = std::max(end, s.end);
    if (s.written) written_end = std::max(written_end, s.end);
  }
  return false;
}

// Whether what a step of these layers writes (weights, momenta, biases) shares memory
// with itself or with a gradient: one that another workgroup of the launch writes would
// be read before or after, by chance.
inline bool step_shares_memory(const kfac_layer_t* layers, int64_t n) {
  std::vector<Span> spans;
  for (int64_t i = 0; i < n; ++i) {
    const kfac_layer_t& L = layers[i];
    const int64_t bias = 4 * static_cast<int64_t>(L.d_out), matrix = bias * L.d_in;
    for (const float* p : {L.w, L.mom_w}) spans.push_back(span_of(p, matrix, true));
    spans.push_back(span_of(L.grad_w, matrix, false));
    if (!L.has_bias) continue;
    for (const float* p : {L.b, L.mom_b}) spans.push_back(span_of(p, bias, true));
    spans.push_back(span_of(L.grad_b, bias, false));
  }
  return share_memory(spans);
}

}  // namespace kfac
