// Whether the buffers of a call share memory (internal, host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssd {

// A caller's buffer: rows of `row` bytes, `stride` bytes apart.
struct Span {
  uint64_t at, row, rows, stride;
  bool none() const { return at == 0 || row == 0 || rows == 0; }
  bool one() const { return rows == 1 || stride == row; }
  uint64_t end() const { return at + (rows - 1) * stride + row; }
};
inline Span rows_of(const void* p, int64_t rows, int64_t row, int64_t stride, size_t elem) {
  return {(uint64_t)reinterpret_cast<uintptr_t>(p), (uint64_t)row * elem, (uint64_t)rows,
          (uint64_t)stride * elem};
}
inline Span bytes_of(const void* p, uint64_t bytes) {
  return {(uint64_t)reinterpret_cast<uintptr_t>(p), bytes, 1, bytes};
}

// a b, at most 2^62 (more than there is memory; an address and it still fit 64 bits).
inline uint64_t capped(uint64_t a, uint64_t b) {
  const uint64_t most = (uint64_t)1 << 62;
  return b != 0 && a > most / b ? most : a * b;
}

// Whether two buffers share a byte.  Rows of the same stride may lie beside one another
// (columns of one wider tensor); rows of different strides may not.
inline bool overlap(Span a, Span b) {
  if (a.none() || b.none()) return false;
  if (b.at < a.at) {
    const Span t = a;
    a = b;
    b = t;
  }
  if (b.at >= a.end()) return false;
  if (a.one()) return true;                       // b begins inside a
  const uint64_t d = (b.at - a.at) % a.stride;    // behind the start of a's row before it
  if (d < a.row) return true;
  if (b.one()) return b.end() - b.at > a.stride - d;
  return b.stride != a.stride || b.row > a.stride - d;
}

// Whether a buffer that the call writes shares memory with any other: its workgroups run
// in any order, so another may read it before or after.
template <int NW, int NR>
inline bool aliased(const Span (&written)[NW], const Span (&read)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return true;
    for (int j = 0; j < NR; ++j)
      if (overlap(written[i], read[j])) return true;
  }
  return false;
}

}  // namespace ssd
