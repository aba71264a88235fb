// zo_tile.h -- the tiles that the attention kernels stage in shared memory: their
// layout, and which bytes of memory each lane's direct loads fetch.  Plain arithmetic,
// so that the host can check which bytes those are.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zo {

constexpr int kWaves = 4;
constexpr int kTile = 64;  // rows of a staged tile

// A staged tile is 64 rows of D bf16 without gaps (the direct loads to shared
// memory write 64 lanes' 16 bytes one after another), and the 16-byte pieces of
// row r are stored at piece ^ swizzle(r), which spreads 8 rows that start on the same bank
// over 8 places (256-byte rows; 128-byte rows alternate between two halves of the banks, 64-
// and 192-byte rows repeat after 4).  It does not spread 16: counted, conflicts are 43 to 50 %
// of the active shared-memory cycles at 128 columns and 30 to 36 % at 64, as 64 banks would
// give, where 16 lanes' 16-byte reads find 8 places and the 4 rows of a transposing read 2
// pairs of pieces.
template <int D>
__host__ __device__ __forceinline__ constexpr int swizzle(int r) {
  return D == 128 ? (r & 7) << 1 : D == 64 ? r & 6 : (r >> 2) & 1;
}
template <int D>
constexpr int kTileBytes = kTile * D * 2;

// Load u of a lane of a wave fetches one 16-byte piece of the tile.
template <int D>
struct TileMap {
  static constexpr int kLoads = D / 32;                // of the workgroup's D / 8, 64 pieces each
  // (8 rows further the swizzle is the same: loads that start there share a lane offset)
  static constexpr int kOffs = D == 128 ? 2 : D == 64 ? 1 : kLoads;

  static __host__ __device__ __forceinline__ constexpr int piece(int wave, int u, int lane) {
    return (wave * kLoads + u) * 64 + lane;
  }
  static __host__ __device__ __forceinline__ constexpr int row(int wave, int u, int lane) {
    return piece(wave, u, lane) / (D / 8);
  }
  static __host__ __device__ __forceinline__ constexpr int column(int wave, int u, int lane) {
    return (piece(wave, u, lane) % (D / 8)) ^ swizzle<D>(row(wave, u, lane));
  }
  // Whether rows `stride` elements apart are within 32-bit offsets of a tile's first row.
  static __host__ __device__ __forceinline__ constexpr bool near(int64_t stride) {
    return stride >= 0 && stride < (1 << 23);          // (64 rows of 16 MiB stay below 2^30)
  }
  // Bytes from the tile's first row on to the piece of load u < kOffs; a later load's is
  // that of load u % kOffs, rows_on(u) rows further on.
  static __host__ __device__ __forceinline__ constexpr uint32_t first_offset(int wave, int u, int lane,
                                                                             int64_t stride) {
    return static_cast<uint32_t>(row(wave, u, lane)) * static_cast<uint32_t>(stride) * 2u +
           column(wave, u, lane) * 16u;
  }
  static __host__ __device__ __forceinline__ constexpr int rows_on(int u) { return u / kOffs * 8; }
  // Bytes of a descriptor that begins at a row and ends with the last of the `rows` rows from
  // there on (0: none, or not `on`).
  static __host__ __device__ __forceinline__ constexpr uint32_t bytes(int rows, int64_t stride, bool on) {
    const int n = rows < 0 ? 0 : rows > kTile ? kTile : rows;
    return ((n - 1) * static_cast<uint32_t>(stride) + D) * 2u * static_cast<uint32_t>(on & (n > 0));
  }
};

}  // namespace zo
