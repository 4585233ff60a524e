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

// Whether the two share memory.  Not where their extents do not meet, nor where all
// distances between their rows (or matrices) are multiples of one number, as between
// column slices of a matrix (row slices of a batch), and the rows (matrices) lie apart
// within it.  What that leaves is looked at row by row, if there are not too many (then
// it counts as shared).
inline bool overlap(const Lines& a, const Lines& b) {
  if (a.run < 1 || a.rows < 1 || a.mats < 1 || b.run < 1 || b.rows < 1 || b.mats < 1) return false;
  auto matrix = [](const Lines& l) { return l.run + (l.rows - 1) * l.ld; };
  auto extent = [&](const Lines& l) { return matrix(l) + (l.mats - 1) * l.stride; };
  if (a.begin + static_cast<uintptr_t>(extent(a)) <= b.begin || b.begin + static_cast<uintptr_t>(extent(b)) <= a.begin) return false;
  const int64_t between = static_cast<int64_t>(b.begin - a.begin);
  auto apart = [&](int64_t a_run, int64_t b_run, int64_t step) {      // runs `step`, or a multiple of it, apart
    if (step == 0) return false;
    const int64_t d = (between % step + step) % step;
    return d >= a_run && d + b_run <= step;
  };
  int64_t rows = 0, mats = 0;
  for (const Lines* l : {&a, &b}) {
    if (l->rows > 1) rows = std::gcd(rows, l->ld);
    if (l->mats > 1) mats = std::gcd(mats, l->stride);
  }
  if (apart(a.run, b.run, std::gcd(rows, mats)) || apart(matrix(a), matrix(b), mats)) return false;
  constexpr int64_t most = 1 << 18;         // some 2 ms
  if (a.mats > most / b.mats || a.rows > most / (a.mats * b.mats)) return true;
  for (int64_t m = 0; m < a.mats; ++m)
    for (int64_t n = 0; n < b.mats; ++n) {
      const int64_t from = between + n * b.stride - m * a.stride;      // b's matrix, from a's
      for (int64_t r = 0; r < a.rows; ++r) {
        // the last of b's rows that begins before a's row ends: if none meets it, that one does not
        const int64_t end = r * a.ld + a.run - 1 - from;
        if (end < 0) continue;
        const int64_t last = b.rows > 1 ? std::min(b.rows - 1, end / b.ld) : 0;
        if (from + last * b.ld + b.run > r * a.ld) return true;
      }
    }
  return false;
}

}  // namespace kfac
