// Whether strided tensors share memory, exactly. Host only.
//
// A tensor is rows of `width` bytes at lo + sum_k i_k stride_k, 0 <= i_k < n_k. Rows of a and b share
// a byte where sum_k i_k s_k - sum_k j_k t_k lies strictly between b.lo - a.lo - a.width and
// b.lo - a.lo + b.width, so the question is whether a bounded integer combination of strides reaches a
// window. It is answered stride by stride, the largest first: what the smaller ones can add leaves only
// the multiples that come near enough, one or two where tensors nest as they usually do (parts of a
// projection's output, keys and values in one array of pages). Strides that do not nest may leave
// many; after kShareSteps the answer is yes.
#pragma once

#include <cstdint>

namespace engram {

struct Strided {
  uintptr_t lo;
  int64_t width;
  int64_t n[3], stride[3];   // n = 1: the stride is not read; (n - 1) stride < 2^57

  Strided(const void* p, int64_t bytes, int64_t n0 = 1, int64_t s0 = 0, int64_t n1 = 1,
          int64_t s1 = 0, int64_t n2 = 1, int64_t s2 = 0)
      : lo(reinterpret_cast<uintptr_t>(p)), width(bytes), n{n0, n1, n2}, stride{s0, s1, s2} {}

  uintptr_t hi() const {
    uintptr_t h = lo + static_cast<uintptr_t>(width);
    for (int k = 0; k < 3; ++k)
      if (n[k] > 1) h += static_cast<uintptr_t>((n[k] - 1) * stride[k]);
    return h;
  }
};

constexpr int kShareSteps = 1 << 14;

// sum_k x_k stride_k with lo_k <= x_k <= hi_k, strides falling.
struct StrideSums {
  int count = 0;
  int64_t stride[6], lo[6], hi[6];
  int steps = 0;

  void add(int64_t s, int64_t from, int64_t to) {
    if (from == 0 && to == 0) return;
    int at = 0;
    while (at < count && stride[at] > s) ++at;
    if (at < count && stride[at] == s) {
      lo[at] += from;
      hi[at] += to;
      return;
    }
    for (int k = count++; k > at; --k) {
      stride[k] = stride[k - 1];
      lo[k] = lo[k - 1];
      hi[k] = hi[k - 1];
    }
    stride[at] = s;
    lo[at] = from;
    hi[at] = to;
  }

  static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }   // b > 0

  // Whether the sums of the strides from `k` on reach [from, to].
  bool reach(int64_t from, int64_t to, int k = 0) {
    if (++steps > kShareSteps) return true;
    if (k == count) return from <= 0 && to >= 0;
    int64_t least = 0, most = 0;   // of the smaller strides
    for (int i = k + 1; i < count; ++i) {
      least += lo[i] * stride[i];
      most += hi[i] * stride[i];
    }
    int64_t x0 = -floor_div(most - from, stride[k]), x1 = floor_div(to - least, stride[k]);
    if (x0 < lo[k]) x0 = lo[k];
    if (x1 > hi[k]) x1 = hi[k];
    for (int64_t x = x0; x <= x1; ++x)
      if (reach(from - x * stride[k], to - x * stride[k], k + 1)) return true;
    return false;
  }
};

inline bool shares_memory(const Strided& a, const Strided& b) {
  if (a.width <= 0 || b.width <= 0 || a.lo >= b.hi() || b.lo >= a.hi()) return false;
  StrideSums s;
  for (int k = 0; k < 3; ++k) {
    if (a.n[k] > 1) s.add(a.stride[k], 0, a.n[k] - 1);
    if (b.n[k] > 1) s.add(b.stride[k], -(b.n[k] - 1), 0);
  }
  const int64_t d = static_cast<int64_t>(b.lo - a.lo);
  return s.reach(d - a.width + 1, d + b.width - 1);
}

// Whether two different rows of `a` share a byte: they differ first in some place k, and by symmetry
// upwards.
inline bool rows_share_memory(const Strided& a) {
  for (int k = 0; k < 3; ++k) {
    if (a.n[k] <= 1) continue;
    StrideSums s;
    s.add(a.stride[k], 1, a.n[k] - 1);
    for (int i = k + 1; i < 3; ++i)
      if (a.n[i] > 1) s.add(a.stride[i], -(a.n[i] - 1), a.n[i] - 1);
    if (s.reach(-(a.width - 1), a.width - 1)) return true;
  }
  return false;
}

}  // namespace engram
