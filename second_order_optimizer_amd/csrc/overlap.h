// Which tensors of a call share memory, on the host.
#pragma once

#include <algorithm>
#include <cstdint>
#include <numeric>
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

// Strided memory: `mats` matrices of `rows` rows of `run` bytes, rows `ld` and matrices
// `stride` bytes apart.
struct Lines {
  uintptr_t begin;
  int64_t run, rows, ld, mats = 1, stride = 0;
};
inline Lines lines_of(const void* p, int64_t run, int64_t rows = 1, int64_t ld = 0, int64_t mats = 1, int64_t stride = 0) {
  return {reinterpret_cast<uintptr_t>(p), run, rows, ld, mats, stride};
}

// Whether the two may share memory.  No where their extents do not meet, and none where
// all distances are multiples of one number (as between column slices of a matrix) and
// the runs lie apart within it; what neither shows apart counts as shared.
inline bool overlap(const Lines& a, const Lines& b) {
  auto extent = [](const Lines& l) { return l.run + (l.rows - 1) * l.ld + (l.mats - 1) * l.stride; };
  if (a.run < 1 || a.rows < 1 || a.mats < 1 || b.run < 1 || b.rows < 1 || b.mats < 1) return false;
  if (a.begin + static_cast<uintptr_t>(extent(a)) <= b.begin || b.begin + static_cast<uintptr_t>(extent(b)) <= a.begin) return false;
  int64_t g = 0;
  for (const Lines* l : {&a, &b}) {
    if (l->rows > 1) g = std::gcd(g, l->ld);
    if (l->mats > 1) g = std::gcd(g, l->stride);
  }
  if (g == 0) return true;
  const int64_t apart = static_cast<int64_t>(b.begin - a.begin) % g, d = apart < 0 ? apart + g : apart;
  return d < a.run || d + b.run > g;
}

}  // namespace kfac
