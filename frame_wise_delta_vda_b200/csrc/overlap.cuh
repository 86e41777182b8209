// Do two strided pieces of memory have a byte in common?  Host code, for the
// checks that results lie apart from inputs and from one another.
#pragma once

#include <stdint.h>

namespace vda {

// Runs of `len` bytes at addr + i * s1 + j * s0, i < n1, j < n0 (strides >= 0).
struct Region {
  int64_t addr, len;
  int64_t n1, s1, n0, s0;
};

// The outer axis has the larger stride; an axis that nothing steps over has one
// place; axes that follow one another without a gap are one, and contiguous
// runs are one run.
inline Region make_region(const void* p, int64_t len, int64_t na = 1, int64_t sa = 0, int64_t nb = 1, int64_t sb = 0) {
  Region r{(int64_t)reinterpret_cast<uintptr_t>(p), len, 1, 0, 1, 0};
  if (na < 2 || sa == 0) na = 1, sa = 0;
  if (nb < 2 || sb == 0) nb = 1, sb = 0;
  if (sa >= sb) {
    r.n1 = na; r.s1 = sa; r.n0 = nb; r.s0 = sb;
  } else {
    r.n1 = nb; r.s1 = sb; r.n0 = na; r.s0 = sa;
  }
  if (r.n0 > 1 && r.s1 == r.n0 * r.s0) {
    r.n1 *= r.n0; r.s1 = r.s0;
    r.n0 = 1; r.s0 = 0;
  }
  if (r.n0 > 1 && r.s0 == len) {
    r.len *= r.n0;
    r.n0 = 1; r.s0 = 0;
  }
  if (r.n0 == 1 && r.s1 == r.len) {
    r.len *= r.n1;
    r.n1 = 1; r.s1 = 0;
  }
  return r;
}

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }   // b > 0

// Is there an m in [m0, m1] with lo < m * s < hi?
inline bool multiple_between(int64_t lo, int64_t hi, int64_t s, int64_t m0, int64_t m1) {
  if (s == 0) return m0 <= m1 && lo < 0 && 0 < hi;
  const int64_t first = floor_div(lo, s) + 1, last = -floor_div(-hi, s) - 1;
  return (first > m0 ? first : m0) <= (last < m1 ? last : m1);
}

// True when an overlap is found.  Exact for regions whose outer strides are
// alike, as those of views of one tensor are, or of which one has a single
// axis or none (a contiguous tensor); others count as apart.
inline bool overlap(Region a, Region b) {
  if (a.len <= 0 || b.len <= 0) return false;
  const int64_t enda = a.addr + (a.n1 - 1) * a.s1 + (a.n0 - 1) * a.s0 + a.len;
  const int64_t endb = b.addr + (b.n1 - 1) * b.s1 + (b.n0 - 1) * b.s0 + b.len;
  if (enda <= b.addr || endb <= a.addr) return false;
  // an axis of one place has any stride; a single axis stands outside where its stride is the other's outer one
  const auto adapt = [](Region& x, const Region& y) {
    if (x.n0 == 1 && x.n1 > 1 && x.s1 != y.s1) {
      x.n0 = x.n1; x.s0 = x.s1;
      x.n1 = 1;
    }
    if (x.n1 == 1) x.s1 = y.s1;
  };
  if (b.n1 > 1) adapt(a, b);
  if (a.n1 > 1) adapt(b, a);
  if (a.s1 != b.s1 && a.n1 > 1 && b.n1 > 1) return false;
  // they meet where  lo < m s + j a.s0 - l b.s0 < hi  for some m = i - k, j, l
  const int64_t lo = b.addr - a.addr - a.len, hi = b.addr - a.addr + b.len;
  const int64_t s = a.s1 > b.s1 ? a.s1 : b.s1;
  const int64_t up = (a.n0 - 1) * a.s0, down = (b.n0 - 1) * b.s0;   // the inner axes move by [-down, up]
  int64_t m0 = -(b.n1 - 1), m1 = a.n1 - 1;
  if (s > 0) {
    const int64_t first = floor_div(lo - up, s) + 1, last = -floor_div(-(hi + down), s) - 1;
    if (first > m0) m0 = first;
    if (last < m1) m1 = last;
  }
  // few, as the inner axes of results stay within one step of the outer one;
  // inputs whose rows run over one another a thousandfold are not followed
  for (int64_t m = m0; m <= m1 && m - m0 < 1024; ++m) {
    const int64_t l0 = lo - m * s, h0 = hi - m * s;
    if (a.n0 == 1 || b.n0 == 1 || a.s0 == b.s0) {
      const int64_t t = a.n0 > 1 ? a.s0 : b.s0;
      if (multiple_between(l0, h0, t, -(b.n0 - 1), a.n0 - 1)) return true;
    } else {
      for (int64_t j = 0; j < a.n0; ++j)   // heads
        if (multiple_between(j * a.s0 - h0, j * a.s0 - l0, b.s0, 0, b.n0 - 1)) return true;
    }
  }
  return false;
}

}  // namespace vda
