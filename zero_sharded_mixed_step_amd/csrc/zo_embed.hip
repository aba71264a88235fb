// zo_embed.hip -- the embedding lookup with a factor, and the table's gradient.
//
// Both move rows and compute next to nothing: bound by memory.  Forward, a wave
// copies a piece of a token's row.
//
// Backward, sum over the tokens of a row in a fixed order: the tokens are sorted by
// id (equal ids by place), the sorted list is cut into chunks of P places, a wave sums
// the rows of a chunk for 512 columns, one run of equal ids after another, and what a
// chunk's first and last run share with its neighbours goes through the workspace and is
// joined chunk by chunk.  The work of a wave does not depend on how often an id occurs.
// Waves beside those write the rows that no id names.
//
// Sorting needs each place's rank, the number of (id, place) pairs below its own.  It is
// counted: within a tile of 1024 places by comparing with all of them (a few instructions a
// comparison, spread over the card), and over the other tiles by searching their sorted lists, 16
// lists at a time.  No pass depends on the ids' distribution, and there are one launch for 1024
// tokens, two for 16384, three for 262144.
// Up to 256 tokens need none of this: see embed_direct_kernel.
//
// Measured, bf16: forward of 16384 x 4096 41 us, 6.6 TB/s (rows met again come from the
// caches; fp32 97 us, 5.6); backward of the same into a table of 50257 rows with an fp32 base 264 us, 5.2 TB/s:
// ranks 7, joining the tiles 5, sums and rows without a token 244, joining the runs 11; a table of
// 50257 x 768 in fp32 for 61 tokens 29 us, 5.4 TB/s of zeros.
#include <algorithm>

#include "zo_device.h"
#include "zo_internal.h"
#include "zo_rows.h"

namespace zo {

// Places that are ranked by comparison.  (16384 tokens: 6.7 us for the ranks and 4.8 for joining the
// tiles, with 2048 10.2 and 4.9.)
constexpr int kRankTile = 1024;
constexpr int kRankWaves = 16;                // waves that share a tile's comparisons
// Sorted lists that are joined at a time.  (262144 tokens of 768 columns: 275 us, two passes of 36 of
// them; with 32 lists 288 in all, with 64 324; all 256 lists in one pass take 235 alone.)
constexpr int kMergeLists = 16;
constexpr int kFillColumns = 4096;            // columns of a wave that writes what no id names
constexpr int kSlice = 512;                   // columns of a wave: 8 a lane
constexpr int kEmbedThreads = 256, kEmbedWaves = kEmbedThreads / 64;
// Waves that join 512 columns of a run's parts.  (262144 tokens of 768 columns, 43000 of them in one
// run: 36 us, with 8 waves 44, with 4 70.)
constexpr int kJoinWaves = 16;

struct EmbedParams {
  int64_t N, V;
  int C, slices, P, chunks;
  float scale;
  const int32_t* ids;
  const void* table;
  void* out;
  const void* dout;
  const void* base;
  void* dtable;
  int64_t table_s, out_s, dout_s, base_s, dtable_s;
  int32_t *key, *place;                       // sorted
  int32_t *tile_key, *tile_place;             // sorted within tiles
  float* part;                                // [chunks][2][C]: a chunk's first and last run
  int64_t sum_units, fill_units;
  int64_t search_step;                        // 64 times it are at least N; 0: see fill_rows
  int fill_parts;                             // parts of a table row that waves take
  int fill_rows;                              // table rows of a wave that writes what no id names; 0: none does
};

// A wave's columns: 8 of a slice to a lane, 4 and 4 of its halves where one of their
// two types is fp32.
template <typename E, typename G>
constexpr bool kSplit = sizeof(E) == 4 || sizeof(G) == 4;
template <bool S>
__device__ __forceinline__ int column(int64_t slice, int lane) {
  return static_cast<int>(slice) * kSlice + (S ? 4 : 8) * lane;
}

// Loads of a row's columns from c on; of lanes behind its end from its first ones, which nobody stores.
// (Without a branch for every row that is under way: 16384 x 4096 with a base 264 us, 268 with it.)
template <bool S>
struct Columns {
  int a, b;
  __device__ __forceinline__ Columns(int c, int C) {
    a = c < C ? c : 0;
    b = S ? (c + kHalf < C ? c + kHalf : 0) : a + 4;
  }
  __device__ __forceinline__ void load(const bf16* p, Vec8<bf16>& v) const {
    if constexpr (S) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(p + a), y = *reinterpret_cast<const u32x2*>(p + b);
      v.r = u32x4{x[0], x[1], y[0], y[1]};
    } else {
      v.load(p, a);
    }
  }
  __device__ __forceinline__ void load(const float* p, Vec8<float>& v) const {
    v.a = *reinterpret_cast<const f32x4*>(p + a);
    v.b = *reinterpret_cast<const f32x4*>(p + b);
  }
};

// ---------------------------------------------------------------- forward ---

template <typename E>
__global__ __launch_bounds__(kEmbedThreads) void embed_fwd_kernel(const EmbedParams p) {
  constexpr int kU = 4;
  constexpr bool S = kSplit<E, E>;
  const int lane = threadIdx.x & 63;
  const int64_t unit =
      static_cast<int64_t>(blockIdx.x) * kEmbedWaves + uniform(threadIdx.x >> 6);
  const int64_t n = unit / p.slices;
  if (n >= p.N) return;
  const int c0 = column<S>(unit % p.slices * kU, lane);
  const int32_t id = p.ids[n];
  const bool on = id >= 0 && id < p.V;
  Vec8<E> raw[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    raw[u] = Vec8<E>{};
    if (on && c0 + u * kSlice < p.C)
      Columns<S>(c0 + u * kSlice, p.C).load(static_cast<const E*>(p.table) + id * p.table_s, raw[u]);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    float x[8];
    raw[u].get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= p.scale;
    if (!on) {                                // (a factor that is not finite, too)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    store8<E, S>(static_cast<E*>(p.out) + n * p.out_s, c0 + u * kSlice, p.C, x);
  }
}

// ------------------------------------------------------------------- sort ---

// The id of place n, those outside the table behind all others.
__device__ __forceinline__ int32_t key_of(const EmbedParams& p, int64_t n) {
  const int32_t id = p.ids[n];
  return id >= 0 && id < p.V ? id : static_cast<int32_t>(p.V);
}

// Ranks 64 places of a tile, one a lane: each of the 16 waves compares them with 64 of it.
__global__ __launch_bounds__(64 * kRankWaves) void embed_rank_kernel(const EmbedParams p,
                                                                    int32_t* key,
                                                                    int32_t* place) {
  __shared__ int below[kRankWaves][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * 64 / kRankTile * kRankTile;
  constexpr int kShare = kRankTile / kRankWaves;
  const int32_t mine = n < p.N ? key_of(p, n) : 0;
  const int32_t own = static_cast<int32_t>(n - tile);
  int rank = 0;
#pragma unroll
  for (int h = 0; h < kShare / 64; ++h) {
    const int first = wave * kShare + h * 64;
    if (tile + first >= p.N) break;            // (uniform)
    const int64_t m = tile + first + lane;
    const int32_t other = m < p.N ? key_of(p, m) : INT32_MAX;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) {
      const int32_t k = __builtin_amdgcn_readlane(other, i);
      rank += k < mine + (first + i < own ? 1 : 0);
    }
  }
  below[wave][lane] = rank;
  __syncthreads();
  if (wave == 0 && n < p.N) {
    rank = 0;
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) rank += below[w][lane];
    key[tile + rank] = mine;
    place[tile + rank] = static_cast<int32_t>(n);
  }
}

// How many keys of the sorted list of n <= `size` (a power of 2) are below `mine` (with `equal`:
// or equal to it).
__device__ __forceinline__ int count_below(const int32_t* list, int n, int size, int32_t mine,
                                           bool equal) {
  const int32_t limit = mine + (equal ? 1 : 0);
  int at = 0;
  for (int step = size; step > 0; step >>= 1) {
    const int next = at + step;
    if (next <= n && list[next - 1] < limit) at = next;
  }
  return at;
}

// Joins every kMergeLists sorted lists of 1 << log2_len places: a place's rank is its rank in its
// list and, of the others, what is below it (of lists before its own also what is equal).
__global__ __launch_bounds__(64 * kRankWaves) void embed_merge_kernel(
    int64_t N, int log2_len, const int32_t* list_key, const int32_t* list_place, int32_t* key,
    int32_t* place) {
  __shared__ int below[kRankWaves][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int own = static_cast<int>(static_cast<int64_t>(blockIdx.x) * 64 >> log2_len);
  const int group = own / kMergeLists * kMergeLists;
  const int lists = static_cast<int>((N + (int64_t(1) << log2_len) - 1) >> log2_len);
  const int32_t mine = at < N ? list_key[at] : 0;
  int rank = 0;
  for (int t = group + wave; t < min(lists, group + kMergeLists); t += kRankWaves) {
    if (t == own) continue;
    const int64_t first = static_cast<int64_t>(t) << log2_len;
    const int n = static_cast<int>(min(N - first, int64_t(1) << log2_len));
    rank += count_below(list_key + first, n, 1 << log2_len, mine, t < own);
  }
  below[wave][lane] = rank;
  __syncthreads();
  if (wave == 0 && at < N) {
    int64_t to = at - (static_cast<int64_t>(own - group) << log2_len);
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) to += below[w][lane];
    key[to] = mine;
    place[to] = list_place[at];
  }
}

// --------------------------------------------------------------- backward ---

// dtable[v] = base[v] + scale * sum, a piece of 8 columns, past the caches.  (16384 x 4096 into bf16:
// 102 us, through them some 18 more.)
template <typename G, typename B, bool S>
__device__ __forceinline__ void store_row(const EmbedParams& p, int64_t v, int c,
                                          const float sum[8]) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = sum[j] * p.scale;
  if (p.base != nullptr) {
    Vec8<B> r;
    Columns<S>(c, p.C).load(static_cast<const B*>(p.base) + v * p.base_s, r);
    float b[8];
    r.get(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(sum[j], p.scale, b[j]);
  }
  store8<G, S, true>(static_cast<G*>(p.dtable) + v * p.dtable_s, c, p.C, y);
}

template <bool S>
__device__ __forceinline__ void store_part(const EmbedParams& p, int64_t chunk, int which, int c,
                                           const float sum[8]) {
  store8<float, S>(p.part + (chunk * 2 + which) * p.C, c, p.C, sum);
}

// A wave's chunk of sorted places, for 512 columns.
template <typename E, typename G, typename B>
__device__ __forceinline__ void sum_chunk(const EmbedParams& p, int64_t unit, int lane) {
  constexpr int kAtOnce = 8;                  // rows under way
  constexpr bool S = kSplit<E, G>;
  const int64_t chunk = unit / p.slices, first = chunk * p.P;
  const int c = column<S>(unit % p.slices, lane);
  const bool on = c < p.C;
  const Columns<S> columns(c, p.C);
  const int32_t none = static_cast<int32_t>(p.V);
  const bool in = lane < p.P && first + lane < p.N;
  const int32_t key = in ? p.key[first + lane] : none;
  const int32_t place = in ? p.place[first + lane] : 0;
  const int32_t before = first > 0 ? p.key[first - 1] : -1;
  const int32_t after = first + p.P < p.N ? p.key[first + p.P] : none;
  const int count = __popcll(__ballot(key < none));        // (sorted: the first lanes)
  if (count == 0) return;
  float sum[8] = {};
  int32_t run = __builtin_amdgcn_readlane(key, 0);
  bool shared = run == before;                // the run began in an earlier chunk
  for (int i0 = 0; i0 < count; i0 += kAtOnce) {
    Vec8<E> raw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      raw[u] = Vec8<E>{};
      if (i0 + u < count) {
        const int64_t n = __builtin_amdgcn_readlane(place, i0 + u);
        columns.load(static_cast<const E*>(p.dout) + n * p.dout_s, raw[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (i0 + u >= count) break;
      const int32_t k = __builtin_amdgcn_readlane(key, i0 + u);
      float x[8];
      raw[u].get(x);
      if (k != run) {
        if (on) {
          if (shared) store_part<S>(p, chunk, 0, c, sum);
          else store_row<G, B, S>(p, run, c, sum);
        }
        run = k;
        shared = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = x[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += x[j];
      }
    }
  }
  if (!on) return;
  if (shared) store_part<S>(p, chunk, 0, c, sum);
  else if (run == after) store_part<S>(p, chunk, 1, c, sum);
  else store_row<G, B, S>(p, run, c, sum);
}

// N columns as they are in memory, past the caches: one access of 16 bytes or fewer, so that a
// wave's accesses leave no gaps.  (13357 rows of 7896, base and gradient in fp32: 174 us; two
// accesses of 16 bytes with gaps 286.)
template <typename T, int N>
using Piece = T __attribute__((ext_vector_type(N)));
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const Piece<T, N>*>(p));
}
template <typename T, typename From>
__device__ __forceinline__ void store_piece(T* p, From x) {
  constexpr int kN = sizeof(From) / sizeof(x[0]);
  __builtin_nontemporal_store(__builtin_convertvector(x, Piece<T, kN>),
                              reinterpret_cast<Piece<T, kN>*>(p));
}

// A wave's share of the table: rows v0 + i, i < count, for the bits i of `rows`, and of long rows a
// part: base, or zeros.  The lanes take the rows' pieces one after another over
// all the rows, four to a lane under way.
template <typename G, typename B>
__device__ __forceinline__ void write_base(const EmbedParams& p, int64_t unit, int count,
                                           uint64_t rows, int lane) {
  constexpr int kU = 4;
  const int64_t v0 = unit / p.fill_parts * p.fill_rows;
  const int c0 = static_cast<int>(unit % p.fill_parts) * kFillColumns;
  const int columns = min(p.C - c0, kFillColumns);
  const bool zeros = p.base == nullptr;
  constexpr int kWide = sizeof(G) == 2 && sizeof(B) == 2 ? 8 : 4;                  // columns of a piece
  const int pieces = zeros ? columns * static_cast<int>(sizeof(G)) / 16 : columns / kWide;   // of a row
  for (int i0 = lane; i0 < count * pieces; i0 += 64 * kU) {
    Piece<B, kWide> raw[kU];
    int row[kU], piece[kU];
    bool on[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + 64 * u;
      row[u] = count == 1 ? 0 : i / pieces;
      piece[u] = i - row[u] * pieces;
      on[u] = i < count * pieces && ((rows >> row[u]) & 1) != 0;
      raw[u] = {};
      if (on[u] && !zeros)
        raw[u] = load_piece<B, kWide>(static_cast<const B*>(p.base) + (v0 + row[u]) * p.base_s + c0 +
                                      kWide * piece[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!on[u]) continue;
      G* to = static_cast<G*>(p.dtable) + (v0 + row[u]) * p.dtable_s + c0;
      if (zeros) {
        __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4*>(to) + piece[u]);
      } else {
        store_piece<G>(to + kWide * piece[u], raw[u]);
      }
    }
  }
}

// Rows of the table that no id names.  The lanes look together for the keys below the first row, 64
// times fewer places a step; the 64 keys from there on say which rows are named, but where runs fill
// them.  Then, and for long rows, whose writes hide the steps of a search that asks for less, every lane
// looks for its own row.  (16384 tokens, 50257 rows in bf16: of 2048 columns 54 us, each lane for itself
// 65; of 4096 105, 102.)
template <typename G, typename B>
__device__ __forceinline__ void fill_rows(const EmbedParams& p, int64_t unit, int lane) {
  const int64_t v0 = unit / p.fill_parts * p.fill_rows;
  const int here = static_cast<int>(min(p.V - v0, static_cast<int64_t>(p.fill_rows)));
  int64_t at = 0;                             // how many keys are below v0, or the lane's row
  uint64_t absent = 0;
  bool found = p.search_step > 0;
  if (found) {
    for (int64_t step = p.search_step; step > 0; step >>= 6) {
      const int64_t i = at + (lane + 1) * step - 1;
      at += step * __popcll(__ballot(i < p.N && p.key[i] < v0));
    }
    const int64_t key = at + lane < p.N ? p.key[at + lane] : p.V;
    for (int r = 0; r < here; ++r)
      if (!__any(key == v0 + r)) absent |= 1ull << r;
    found = __any(key >= v0 + here);
  }
  if (!found) {
    bool none = lane < here;
    if (none) {
      const int64_t v = v0 + lane;
      for (int64_t step = int64_t(1) << 21; step > 0; step >>= 1)
        if (at + step <= p.N && p.key[at + step - 1] < v) at += step;
      none = at >= p.N || p.key[at] != v;
    }
    absent = __ballot(none);
  }
  write_base<G, B>(p, unit, here, absent, lane);
}

template <typename E, typename G, typename B>
__global__ __launch_bounds__(kEmbedThreads) void embed_sum_kernel(const EmbedParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit =
      static_cast<int64_t>(blockIdx.x) * kEmbedWaves + uniform(threadIdx.x >> 6);
  if (unit < p.sum_units) sum_chunk<E, G, B>(p, unit, lane);
  else if (unit - p.sum_units < p.fill_units)
    fill_rows<G, B>(p, unit - p.sum_units, lane);
}

// Up to 256 tokens: every wave has all of them in its lanes and finds an id's places by itself.
// The wave of an id's first place sums its rows in order, and no sort, parts or join are needed:
// one launch.  (200 tokens of 768 columns, added in place: 5 us, sorted 12; where they are all one
// token 22, sorted 13.)
constexpr int kDirectTokens = 256;

template <typename E, typename G, typename B>
__global__ __launch_bounds__(kEmbedThreads) void embed_direct_kernel(const EmbedParams p) {
  constexpr int kK = kDirectTokens / 64, kAtOnce = 4;
  constexpr bool S = kSplit<E, G>;
  const int lane = threadIdx.x & 63;
  const int64_t unit =
      static_cast<int64_t>(blockIdx.x) * kEmbedWaves + uniform(threadIdx.x >> 6);
  int32_t key[kK];
#pragma unroll
  for (int k = 0; k < kK; ++k)
    key[k] = 64 * k + lane < p.N ? key_of(p, 64 * k + lane) : static_cast<int32_t>(p.V);
  if (unit >= p.sum_units) {
    if (unit - p.sum_units >= p.fill_units) return;
    const int64_t v0 = (unit - p.sum_units) / p.fill_parts * p.fill_rows;
    const int here = static_cast<int>(min(p.V - v0, static_cast<int64_t>(p.fill_rows)));
    uint64_t rows = 0;
    for (int r = 0; r < here; ++r) {
      bool named = false;
#pragma unroll
      for (int k = 0; k < kK; ++k) named |= key[k] == v0 + r;
      if (!__any(named)) rows |= 1ull << r;
    }
    write_base<G, B>(p, unit - p.sum_units, here, rows, lane);
    return;
  }
  const int n = static_cast<int>(unit / p.slices);
  const int c = column<S>(unit % p.slices, lane);
  const bool on = c < p.C;
  int32_t run = 0;
#pragma unroll
  for (int k = 0; k < kK; ++k)
    if (n / 64 == k) run = __builtin_amdgcn_readlane(key[k], n % 64);
  if (run >= p.V) return;
  uint64_t places[kK];
  bool first = true;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    places[k] = __ballot(key[k] == run);
    const int before = n - 64 * k;             // places of these 64 that are before n
    first &= before <= 0 || (places[k] & (before >= 64 ? ~0ull : (1ull << before) - 1)) == 0;
  }
  if (!first) return;
  float sum[8] = {};
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    while (places[k] != 0) {
      Vec8<E> raw[kAtOnce];
      int count = 0;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        raw[u] = Vec8<E>{};
        if (places[k] == 0) continue;
        const int64_t at = 64 * k + __builtin_ctzll(places[k]);
        places[k] &= places[k] - 1;
        ++count;
        Columns<S>(c, p.C).load(static_cast<const E*>(p.dout) + at * p.dout_s, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (u >= count) break;
        float x[8];
        raw[u].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += x[j];
      }
    }
  }
  if (on) store_row<G, B, S>(p, run, c, sum);
}

// The runs that go over a chunk's end, by the chunk that they begin in: its last part
// and the first parts of the chunks after it.  A workgroup has a slice of a run, and a wave every
// 16th of its parts.
template <typename G, typename B>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(const EmbedParams p) {
  __shared__ float fold[kJoinWaves][kSlice];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t chunk = blockIdx.x, first = chunk * p.P;
  if (first + p.P >= p.N) return;
  const int32_t run = p.key[first + p.P - 1];
  if (run >= p.V || p.key[first + p.P] != run || (first > 0 && p.key[first - 1] == run)) return;
  int64_t more = 0;                           // chunks after this one that begin with the run
  const auto count = [&](int64_t step) {      // adds every step-th, until one does not
    const int64_t at = (chunk + more + (lane + 1) * step) * p.P;
    const uint64_t same = __ballot(at < p.N && p.key[at] == run);
    const int n = ~same == 0 ? 64 : __builtin_ctzll(~same);
    more += n * step;
    return n == 64;
  };
  if (count(1))
    for (int64_t step = 4096; step > 0; step >>= 6) count(step);
  constexpr bool S = true;                    // (the parts are fp32)
  const int c = column<S>(blockIdx.y, lane);
  const bool on = c < p.C;
  float sum[8] = {};
  constexpr int kAtOnce = 8;                  // parts under way
  for (int64_t q0 = wave; q0 <= more; q0 += kAtOnce * kJoinWaves) {
    Vec8<float> raw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t q = min(q0 + u * kJoinWaves, more);
      Columns<S>(c, p.C).load(p.part + ((chunk + q) * 2 + (q == 0 ? 1 : 0)) * p.C, raw[u]);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (q0 + u * kJoinWaves > more) break;
      float x[8];
      raw[u].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += x[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) fold[wave][8 * lane + j] = sum[j];
  __syncthreads();
  if (wave > 0 || !on) return;
  for (int w = 1; w < kJoinWaves && w <= more; ++w)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += fold[w][8 * lane + j];
  store_row<G, B, S>(p, run, c, sum);
}

namespace {

// Places of a chunk, no more than a wave's lanes.  Longer chunks leave fewer runs and parts to
// join, and 256 of them, by 8 slices, still fill the card (16384 x 4096, all 50257 rows / added in
// place / one id for all tokens: 274 / 101 / 54 us; with 512 chunks 277 / 101 / 65, with 1024 284 /
// 110 / 91).
int chunk_places(int64_t N) {
  const int64_t p = (N + 255) / 256;
  return static_cast<int>(p < 4 ? 4 : p > 64 ? 64 : p);
}

int64_t chunks_of(int64_t N) { return (N + chunk_places(N) - 1) / chunk_places(N); }

// Rows of a wave that writes what no id names: one, or up to 4096 columns of it, so that the writes'
// front is compact (50257 rows of 4096 with a base: 260 us; two rows 302 and eight 328 where one took
// 293; 2048 columns 269; 13357 rows of 7896 for 20 tokens: 174, whole rows 184).  Of shorter rows as many
// as are 4 KiB of the gradient (16384 tokens, 50257 rows of 768 in fp32: one 42 us, two 45; in bf16
// two 34, one 39; of 1024 in bf16 two 37, one 40), of a small table no more than leave 4096 waves.
int fill_rows_of(int64_t V, int C, int grad_dtype) {
  const int64_t rows = std::min<int64_t>(4096 / (C * (grad_dtype == ZERO_BF16 ? 2 : 4)), V / 4096);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, 64)));
}

size_t rounded(size_t n) { return (n + 15) & ~size_t(15); }

template <typename E, typename G, typename B>
hipError_t run_sums(const EmbedParams& p, hipStream_t s) {
  if (p.N <= kDirectTokens) {
    EmbedParams q = p;
    q.sum_units = p.N * p.slices;
    const int64_t units = q.sum_units + p.fill_units;
    const unsigned grid = static_cast<unsigned>((units + kEmbedWaves - 1) / kEmbedWaves);
    if (grid == 0) return hipSuccess;
    embed_direct_kernel<E, G, B><<<grid, kEmbedThreads, 0, s>>>(q);
    return hipGetLastError();
  }
  const int64_t units = p.sum_units + p.fill_units;
  const unsigned grid = static_cast<unsigned>((units + kEmbedWaves - 1) / kEmbedWaves);
  embed_sum_kernel<E, G, B><<<grid, kEmbedThreads, 0, s>>>(p);
  embed_join_kernel<G, B>
      <<<dim3(p.chunks, p.slices), 64 * kJoinWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <typename E, typename G>
hipError_t pick_base(const EmbedParams& p, int base_dtype, hipStream_t s) {
  return base_dtype == ZERO_BF16 ? run_sums<E, G, bf16>(p, s) : run_sums<E, G, float>(p, s);
}

template <typename E>
hipError_t pick_grad(const EmbedParams& p, const zero_embed_args& a, hipStream_t s) {
  return a.grad_dtype == ZERO_BF16 ? pick_base<E, bf16>(p, a.base_dtype, s)
                                   : pick_base<E, float>(p, a.base_dtype, s);
}

}  // namespace

size_t embed_workspace(int64_t N, int C) {
  if (N <= kDirectTokens) return 0;
  return 4 * rounded(N * sizeof(int32_t)) +
         static_cast<size_t>(chunks_of(N)) * 2 * C * sizeof(float);
}

hipError_t launch_embed_fwd(const zero_embed_args& a, hipStream_t s) {
  EmbedParams p = {};
  p.N = a.N;
  p.V = a.V;
  p.C = a.C;
  p.scale = static_cast<float>(a.scale);
  p.ids = a.ids;
  p.table = a.table;
  p.out = a.out;
  p.table_s = a.table_stride;
  p.out_s = a.out_stride;
  p.slices = (a.C + 4 * kSlice - 1) / (4 * kSlice);
  const unsigned grid =
      static_cast<unsigned>((p.N * p.slices + kEmbedWaves - 1) / kEmbedWaves);
  if (a.dtype == ZERO_BF16) embed_fwd_kernel<bf16><<<grid, kEmbedThreads, 0, s>>>(p);
  else embed_fwd_kernel<float><<<grid, kEmbedThreads, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_embed_bwd(const zero_embed_args& a, hipStream_t s) {
  EmbedParams p = {};
  p.N = a.N;
  p.V = a.V;
  p.C = a.C;
  p.scale = static_cast<float>(a.scale);
  p.ids = a.ids;
  p.dout = a.dout;
  p.base = a.base;
  p.dtable = a.dtable;
  p.dout_s = a.dout_stride;
  p.base_s = a.base_stride;
  p.dtable_s = a.dtable_stride;
  p.slices = (a.C + kSlice - 1) / kSlice;
  p.P = chunk_places(a.N);
  p.chunks = static_cast<int>(chunks_of(a.N));
  p.sum_units = static_cast<int64_t>(p.chunks) * p.slices;
  if (a.base != a.dtable) {
    p.fill_rows = fill_rows_of(a.V, a.C, a.grad_dtype);
    p.fill_parts = (a.C + kFillColumns - 1) / kFillColumns;
    p.fill_units = (a.V + p.fill_rows - 1) / p.fill_rows * p.fill_parts;
    if (a.C < kFillColumns)
      for (p.search_step = 1; p.search_step * 64 < a.N;) p.search_step *= 64;
  }
  char* ws = static_cast<char*>(a.workspace);
  const size_t list = rounded(a.N * sizeof(int32_t));
  p.key = reinterpret_cast<int32_t*>(ws);
  p.place = reinterpret_cast<int32_t*>(ws + list);
  p.tile_key = reinterpret_cast<int32_t*>(ws + 2 * list);
  p.tile_place = reinterpret_cast<int32_t*>(ws + 3 * list);
  p.part = reinterpret_cast<float*>(ws + 4 * list);
  if (a.N > kDirectTokens) {
    const unsigned grid = static_cast<unsigned>((a.N + 63) / 64);
    // the lists go to and fro between two places, the last ones to p.key
    int passes = 0;
    for (int64_t n = kRankTile; n < a.N; n *= kMergeLists) ++passes;
    int32_t* const lists[2][2] = {{p.key, p.place}, {p.tile_key, p.tile_place}};
    embed_rank_kernel<<<grid, 64 * kRankWaves, 0, s>>>(p, lists[passes % 2][0], lists[passes % 2][1]);
    for (int64_t n = kRankTile; n < a.N; n *= kMergeLists, --passes) {
      int32_t* const* from = lists[passes % 2];
      int32_t* const* to = lists[(passes + 1) % 2];
      embed_merge_kernel<<<grid, 64 * kRankWaves, 0, s>>>(a.N, __builtin_ctzll(n), from[0], from[1],
                                                         to[0], to[1]);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return a.dtype == ZERO_BF16 ? pick_grad<bf16>(p, a, s) : pick_grad<float>(p, a, s);
}

}  // namespace zo
