// Which bytes the attention kernels' direct loads fetch (zo_tile.h), on the host:
// every load that its descriptor lets through is of a row that is there, by the lane's
// offset alone, and the 256 threads' loads together are the tile, each piece once.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "zo_tile.h"

static int failures = 0;
#define CHECK(ok, ...)                 \
  do {                                 \
    if (!(ok)) {                       \
      std::fprintf(stderr, __VA_ARGS__); \
      if (++failures > 20) return;     \
    }                                  \
  } while (0)

template <int D>
static void check(int64_t stride) {
  using M = zo::TileMap<D>;
  static_assert(M::kLoads * zo::kWaves * 64 * 16 == zo::kTileBytes<D>, "a tile's loads");
  for (int rows = -3; rows <= zo::kTile + 3; ++rows)
    for (int on = 0; on < 2; ++on) {
      const int n = on ? (rows < 0 ? 0 : rows > zo::kTile ? zo::kTile : rows) : 0;
      std::vector<int> got(zo::kTile * D / 8, 0);
      for (int wave = 0; wave < zo::kWaves; ++wave)
        for (int u = 0; u < M::kLoads; ++u) {
          // the load's descriptor: from which row, and how many bytes
          const int from = M::rows_on(u), left = rows - from;
          const int n = !on || left < 0 ? 0 : left > zo::kTile ? zo::kTile : left;
          const uint64_t bytes = M::bytes(left, stride, on != 0);
          CHECK(bytes == (n ? (static_cast<uint64_t>(n - 1) * stride + D) * 2 : 0),
                "D %d stride %lld rows %d on %d: %llu bytes\n", D, (long long)stride, left, on,
                (unsigned long long)bytes);
          for (int lane = 0; lane < 64; ++lane) {
            const int r = M::row(wave, u, lane), c = M::column(wave, u, lane);
            CHECK(r >= from && r < zo::kTile && c >= 0 && c < D / 8, "D %d: row %d column %d\n", D, r, c);
            const uint64_t at = M::first_offset(wave, u % M::kOffs, lane, stride);
            CHECK(at == (static_cast<uint64_t>(r - from) * stride + 8 * c) * 2,
                  "D %d stride %lld wave %d load %d lane %d: offset %llu\n", D, (long long)stride,
                  wave, u, lane, (unsigned long long)at);
            if (stride >= D)
              CHECK((at + 16 <= bytes) == (on && r < rows) && (at >= bytes) == !(on && r < rows),
                    "D %d stride %lld rows %d on %d: row %d at %llu of %llu\n", D,
                    (long long)stride, rows, on, r, (unsigned long long)at,
                    (unsigned long long)bytes);
            // its place in shared memory, and that it holds what the swizzle says
            const int place = (wave * M::kLoads + u) * 64 + lane;
            CHECK(place / (D / 8) == r && (place % (D / 8)) == (c ^ zo::swizzle<D>(r)),
                  "D %d: place %d\n", D, place);
            ++got[r * (D / 8) + c];
          }
        }
      for (int x : got) CHECK(x == 1, "D %d: a piece fetched %d times\n", D, x);
    }
}

template <int D>
static void check_all() {
  for (int64_t stride : {int64_t(0), int64_t(8), int64_t(D), int64_t(D + 8), int64_t(12 * D),
                         int64_t(40 * 128), int64_t(1) << 20, (int64_t(1) << 23) - 8}) {
    CHECK(zo::TileMap<D>::near(stride), "D %d: stride %lld is near\n", D, (long long)stride);
    check<D>(stride);
  }
  CHECK(!zo::TileMap<D>::near(int64_t(1) << 23) && !zo::TileMap<D>::near(-8), "far strides\n");
}

int main() {
  check_all<32>();
  check_all<64>();
  check_all<96>();
  check_all<128>();
  if (failures == 0) std::puts("ok");
  return failures != 0;
}
