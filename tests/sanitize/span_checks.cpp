// Whether two strided arrays share a byte (zo_spans.h), against every pair of rows.
#include <cstdint>
#include <cstdio>
#include <random>

#include "zo_spans.h"

static const void* at(int64_t x) { return reinterpret_cast<const void*>(static_cast<uintptr_t>(x)); }

struct Case {
  int64_t at, rows, stride, width;
};

static bool pairs(const Case& a, const Case& b) {
  for (int64_t i = 0; i < a.rows; ++i)
    for (int64_t j = 0; j < b.rows; ++j) {
      const int64_t x = a.at + i * a.stride, y = b.at + j * b.stride;
      if (x < y + b.width && y < x + a.width) return true;
    }
  return false;
}

static bool spans(const Case& a, const Case& b, int bytes) {
  return zo::overlap(zo::Span(at(a.at * bytes), a.rows, a.stride, a.width, bytes),
                     zo::Span(at(b.at * bytes), b.rows, b.stride, b.width, bytes));
}

int main() {
  std::mt19937_64 rng(5);
  const auto pick = [&](int64_t lo, int64_t hi) {
    return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1));
  };
  long met = 0, apart = 0, inside = 0;
  for (int n = 0; n < 3000000; ++n) {
    const int64_t most = pick(1, 60);
    const auto any = [&] {
      Case c{pick(2000, 2000 + 3 * most), pick(0, 12), pick(-most, most), pick(0, pick(1, most))};
      if (c.width > 4 && pick(0, 1)) c.width = pick(1, 3);
      return c;
    };
    const Case a = any(), b = any();
    const bool want = a.width > 0 && b.width > 0 && pairs(a, b);
    const int bytes = 1 << pick(0, 2);
    if (spans(a, b, bytes) != want || spans(b, a, bytes) != want) {
      std::printf("%d: at %lld rows %lld stride %lld width %lld; at %lld rows %lld stride %lld width %lld\n", want,
                  (long long)a.at, (long long)a.rows, (long long)a.stride, (long long)a.width, (long long)b.at,
                  (long long)b.rows, (long long)b.stride, (long long)b.width);
      return 1;
    }
    (want ? met : apart) += 1;
    inside += !want && a.rows > 1 && b.rows > 1;
  }
  if (met < 100000 || apart < 100000 || inside < 100000) return 2;
  // long arrays: columns of one buffer beside each other, rows in turn, and one element too many
  const int64_t C = 4096, T = 1 << 21;
  for (int64_t more = 0; more < 2; ++more) {
    if (spans({1 << 20, T, 3 * C, C + more}, {(1 << 20) + C, T, 3 * C, C}, 2) != (more == 1)) return 3;
    if (spans({1 << 20, T, 6 * C, C}, {(1 << 20) + 3 * C, T, 6 * C, 3 * C + more}, 4) != (more == 1))
      return 4;
    // (rows of 7 and of 11 columns' stride meet at some multiple of 77 or never within the shorter one)
    if (spans({1 << 20, T, 7 * C, C}, {(1 << 20) + 3 * C, more ? T : 1, 11 * C, C}, 2) != (more == 1)) return 5;
  }
  // arrays that no memory holds: refused, and no overflow
  if (!spans({16, 3, INT64_MAX / 8, 8}, {64, 3, INT64_MIN / 8, 8}, 4)) return 6;
  if (spans({0, 5, 8, 8}, {64, 0, 8, 8}, 4) || spans({0, 5, 8, 8}, {16, 3, 8, 8}, 4)) return 7;
  std::puts("ok");
  return 0;
}
