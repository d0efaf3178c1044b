// Do two arrays of a call overlap? Rows may lie apart, so that columns of one wider buffer do not.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

// `rows` runs of `bytes` bytes, the starts `step` bytes apart (step >= bytes).
struct Runs {
  int64_t at, rows, bytes, step;
  // packed rows, or one of them, are a single run
  Runs(const void* p, int64_t n, int64_t row_bytes, int64_t row_step)
      : at((int64_t)reinterpret_cast<uintptr_t>(p)), rows(n), bytes(row_bytes), step(row_step) {
    if (rows <= 1 || step == bytes) {
      bytes *= rows;
      rows = bytes > 0 ? 1 : 0;
      step = bytes;
    }
  }
  Runs(const void* p, int64_t n) : Runs(p, 1, n, n) {}
  int64_t end() const { return at + (rows - 1) * step + bytes; }
  // does a run overlap the bytes lo .. hi - 1?
  bool meets(int64_t lo, int64_t hi) const {
    const int64_t before = lo - at - bytes;  // the first run that ends beyond lo
    const int64_t j = before < 0 ? 0 : before / step + 1;
    return j < rows && at + j * step < hi;
  }
};

// Exact. Rows of one step: run i of a and run j of b overlap if (i - j) step lies between the bounds below. Of
// different steps (rare: no columns of one buffer): row by row.
inline bool overlap(const Runs& a, const Runs& b) {
  if (a.rows == 0 || b.rows == 0 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows == 1) return b.meets(a.at, a.at + a.bytes);
  if (b.rows == 1) return a.meets(b.at, b.at + b.bytes);
  if (a.step == b.step) {
    const int64_t s = a.step, lo = b.at - a.at - a.bytes, hi = b.at - a.at + b.bytes;
    const int64_t first = (lo >= 0 ? lo / s : -((-lo + s - 1) / s)) + 1;  // the least m with m s > lo
    const int64_t m = std::max(first, 1 - b.rows);
    return m < a.rows && m * s < hi;
  }
  const Runs &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
  for (int64_t i = 0; i < few.rows; ++i)
    if (many.meets(few.at + i * few.step, few.at + i * few.step + few.bytes)) return true;
  return false;
}

}  // namespace moe
