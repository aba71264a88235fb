// zo_spans.h -- whether two strided arrays share a byte, on the host: by number
// theory, not row by row, so that a call's check costs nanoseconds whatever the arrays'
// lengths.
#pragma once

#include <cstdint>

namespace zo {

// `rows` rows of `width` bytes, each `stride` bytes behind the one before.  No rows or no
// address: nothing.
struct Span {
  __int128 at = 0, stride = 0, width = 0, end = 0;
  int64_t rows = 0;
  Span() = default;
  Span(const void* p, int64_t n, int64_t stride_elems, int64_t width_elems, int elem_bytes)
      : at(static_cast<__int128>(reinterpret_cast<uintptr_t>(p))),
        stride(static_cast<__int128>(stride_elems) * elem_bytes),
        width(static_cast<__int128>(width_elems) * elem_bytes), rows(p != nullptr ? n : 0) {
    if (rows < 1 || width < 1) {
      rows = 0;
      return;
    }
    if (rows > 1 && stride < 0) {              // from the lowest address on
      at += (rows - 1) * stride;
      stride = -stride;
    }
    if (rows > 1 && stride <= width) {         // rows that touch are one
      width += (rows - 1) * stride;
      rows = 1;
    }
    end = at + (rows - 1) * stride + width;
  }
  Span(const void* p, int64_t bytes) : Span(p, 1, 0, bytes, 1) {}
};

// The smallest x >= 0 with low <= a x mod m <= high, -1 if there is none; 0 <= a < m, 0 <= low
// <= high < m.  If no multiple of a lies in the interval before the first wrap, the multiples
// of m that the wraps take off have to, modulo a: Euclid's steps.
inline __int128 first_multiple_in(__int128 a, __int128 m, __int128 low, __int128 high) {
  if (low == 0) return 0;
  if (a == 0) return -1;
  if (2 * a > m) return first_multiple_in(m - a, m, m - high, m - low);
  const __int128 x = (low + a - 1) / a;
  if (a * x <= high) return x;
  const __int128 y = first_multiple_in((a - m % a) % a, a, low % a, high % a);
  return y < 0 ? -1 : (low + m * y + a - 1) / a;
}

// Rows i of a and j of b meet if -a.width < a.at + i a.stride - b.at - j b.stride < b.width.
inline bool overlap(const Span& a, const Span& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  if (a.end <= b.at || b.end <= a.at) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (b.rows == 1) return overlap(b, a);
  constexpr __int128 kReach = __int128(1) << 57;   // no two rows in memory are further apart
  if (a.stride > kReach || b.stride > kReach) return true;
  // the rows of a that lie in b's stretch: from `first` on, `count` of them
  const __int128 d = a.at - b.at, length = b.end - b.at;
  __int128 first = 0, last = a.rows - 1;
  if (a.rows > 1) {
    if (d + a.width <= 0) first = (-a.width - d) / a.stride + 1;
    const __int128 to = (length - 1 - d) / a.stride;
    if (to < last) last = to;
  }
  if (first > last) return false;
  // row i meets one of b's if (c + i a.stride) mod b.stride <= window
  const __int128 m = b.stride, window = a.width + b.width - 2;
  if (window >= m - 1) return true;
  const __int128 c = (d + first * a.stride + a.width - 1) % m;
  if (c <= window) return true;
  const __int128 x = first_multiple_in((a.rows > 1 ? a.stride : 0) % m, m, m - c, m - c + window);
  return x >= 0 && x <= last - first;
}

// A call's arrays: what it writes may meet nothing else that it touches.  (An output that may be one
// of the inputs stands among the outputs alone where it is.)
template <int OUT, int IN>
class Arrays {
 public:
  void writes(const Span& s) { out_[outs_++] = s; }
  void reads(const Span& s) { in_[ins_++] = s; }
  bool apart() const {
    for (int i = 0; i < outs_; ++i) {
      for (int j = 0; j < ins_; ++j)
        if (overlap(out_[i], in_[j])) return false;
      for (int j = 0; j < i; ++j)
        if (overlap(out_[i], out_[j])) return false;
    }
    return true;
  }

 private:
  Span out_[OUT], in_[IN];
  int outs_ = 0, ins_ = 0;
};

}  // namespace zo
