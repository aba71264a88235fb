// zo_attn.h -- what the attention kernels share: parameters, the tile layout
// in shared memory, the matrix-core fragments, masks and the distance bias.
//
// Matrix products use v_mfma_f32_32x32x16_bf16.  A lane l of a wave holds, of
// the 32 x 16 operand A (and, with columns for rows, of B), row l % 32 and the
// 8 contraction indices 8 (l / 32) .. + 7; of the 32 x 32 result it holds
// column l % 32 and the 16 rows 8 (r / 4) + 4 (l / 32) + r % 4, r = 0..15.
//
// Every kernel computes its scores with the rows it owns (queries in the
// forward and dq kernels, keys in the dk/dv kernel) as the result's columns.
// A lane then holds scores of one owned row only, so softmax statistics, the
// rescaling of outputs and the bias need no exchange beyond the two half
// waves, and the result's registers, rounded to bf16, are already an operand of
// the next product: the contraction index may run in any order that both
// operands share, so the 8 rows a lane holds of a 16-row group
// (4h .. 4h + 3 and 8 + 4h .. + 3, h = l / 32) are taken as its 8 indices, and
// the other operand, which has to be read transposed from shared memory, is
// fetched in that order by two transposing reads of 4 rows each.
#pragma once

#include "zo_device.h"
#include "zo_tile.h"
#include "zero_ops.h"

namespace zo {

constexpr int kAttnThreads = 256;
constexpr int kUnits = 256;  // compute units of the card

// Of a tile of 128 keys: the tiles of 64 queries that see any of it, first and one past
// the last, and a bit for each key that is seen.
constexpr int kTileWords = 6;

struct Strides3 {
  int64_t b, t, h;
};

struct AttnParams {
  int B, Tq, Tk, Hq, Hk, group, causal, off;
  float scale, cap;
  const bf16 *q, *k, *v;
  const int32_t* ranges;
  const void* table;
  const int32_t* buckets;
  int table_f32, n_buckets, reach;
  bf16* o;
  float* lse;
  const bf16* d_o;
  bf16 *dq, *dk, *dv;
  void* dtable;
  Strides3 qs, ks, vs, os, dos, dqs, dks, dvs;
  // workspace
  int tq64;         // Tq up to a multiple of 64: the rows below are padded to it
  float* base;      // [B][Hq][tq64]  -lse * log2(e), plus cap * log2(e) if kByU; -inf: no keys
  float* delta;     // [B][Hq][tq64]  do . o
  int *qlo, *qhi;   // [B][tq64]      the keys a query sees; 0, 0 for none
  int* tile;        // [B][key tiles][kTileWords] of what sees a tile of 128 keys
  float* dpart;     // [B][Hq][query tiles][bias_entries]: ds by distance
  float* dsum;      // [Hq][bias_entries]
  float* kvpart;    // [2][parts][B][Hk][Tk][D]: dk and dv of parts of a group's heads
  int parts;        // 1: no parts
  float* osplit;    // split forward: [splits][B * Hq * Tq][D] and, behind it, two statistics
  int splits, tiles_per_split;
};

// The keys [lo, hi) that query i of batch row b sees; {0, 0} for none.
__device__ __forceinline__ int2 key_range(const AttnParams& p, int b, int i) {
  int lo = 0, hi = 0;
  if (i < p.Tq) {
    if (p.ranges) {
      const int2 r = reinterpret_cast<const int2*>(p.ranges)[static_cast<int64_t>(b) * p.Tq + i];
      lo = max(r.x, 0);
      hi = min(r.y, p.Tk);
    } else {
      hi = p.causal ? min(i + 1 + p.off, p.Tk) : p.Tk;
    }
    if (hi <= lo) lo = hi = 0;
  }
  return make_int2(lo, hi);
}

// Hull of the lanes' non-empty ranges over a wave ({INT_MAX, 0}: none).  Uniform,
// and known to be: what decides a wave's loops has to live in scalar registers.
__device__ __forceinline__ int2 wave_hull(int2 r) {
  const int lo = join_lanes<64>(r.y > r.x ? r.x : 0x7FFFFFFF, MinOp());
  const int hi = join_lanes<64>(r.y, MaxOp());
  return make_int2(uniform(lo), uniform(hi));
}

__device__ __forceinline__ bf16x8 load8(const bf16* p) {
  return *reinterpret_cast<const bf16x8*>(p);
}

// Shared memory is addressed by its 32-bit offsets: a fragment's address is one
// exclusive or away from the lane's place in the tile.
#define ZO_LDS __attribute__((address_space(3)))

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((const ZO_LDS char*)static_cast<const char*>(p)));
}

// A lane's place in the fragments of a staged tile.
template <int D>
struct FragAt {
  uint32_t rows, cols;
  __device__ __forceinline__ explicit FragAt(int lane) {
    const int r = lane & 31, half = lane >> 5;
    rows = r * 2 * D + ((half ^ swizzle<D>(r)) << 4);
    const int i = lane & 15, c = 4 * half + (i >> 2), g = (lane >> 4) & 1;
    cols = c * 2 * D + (((2 * g + ((i >> 1) & 1)) ^ swizzle<D>(c)) << 4) + 8 * (i & 1);
  }
  // The same in the tile at `tile` (aligned to 1 KiB, so that or-ing and adding
  // agree).  Opaque to the compiler, which otherwise keeps every fragment's
  // address in a register of its own across the loop, 40 of them.
  __device__ __forceinline__ FragAt in(uint32_t tile) const {
    FragAt f = *this;
    f.rows += tile;
    f.cols += tile;
    asm volatile("" : "+v"(f.rows), "+v"(f.cols));
    return f;
  }
};

// Operand fragment, contraction along the row: rows 32 t + l % 32, elements
// 16 c + 8 (l / 32) .. + 7.  (Swizzles repeat after 8 rows, and piece 2 c + half
// is 2 c ^ half: moving along the row is one exclusive or, or for swizzles of
// one bit a sum.  `beyond`: of a tile that lies so many bytes behind, a constant.)
template <int D>
__device__ __forceinline__ bf16x8 frag_rows(const FragAt<D>& at, int t, int c, int beyond = 0) {
  const uint32_t x = (D == 64 || D == 128 ? at.rows ^ (c << 5) : at.rows + (c << 5));
  return *reinterpret_cast<const ZO_LDS bf16x8*>(x + (t * 64 * D + beyond));
}

// Operand fragment, contraction along the column: columns 32 t + l % 32 and, of
// the 16 rows from 16 u, the 8 in the order in which a score result holds
// them.  A transposing read hands each of 16 lanes a column of the 4 x 16
// block whose rows those lanes address by fours.
template <int D>
__device__ __forceinline__ bf16x8 frag_cols(const FragAt<D>& at, int u, int t, int beyond = 0) {
  const uint32_t x =
      (D == 64 || D == 128 ? at.cols ^ (t << 6) : at.cols + (t << 6)) + (u * 32 * D + beyond);
  using P = ZO_LDS s16x4*;
  union {
    s16x4 s[2];
    bf16x8 v;
  } f;
  f.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<P>(x));
  f.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<P>(x + 16 * D));
  return f.v;
}

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Row of a 32 x 32 result that register r of a lane holds.
__device__ __forceinline__ int result_row(int r, int lane) {
  return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
}

// Eight registers of a score result as an operand fragment: p or dx, rounded to bf16.  A
// binary32 product would take sixteen times as long on the matrix units; with bf16 an output
// is up to 1.4 times as far from the exact one as its own rounding to bf16 leaves it (2.0e-3
// and 1.6e-3 of it, one token on 5003 keys).
__device__ __forceinline__ bf16x8 to_frag(const float* x) {
  bf16x8 f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = static_cast<bf16>(x[j]);
  return f;
}

// Direct loads to shared memory: 64 lanes' 16 (or 4) bytes each, one after the
// other from the uniform address `to`, with no registers on the way.  They are
// written as instructions because the compiler, which cannot tell the buffers
// apart, waits for all of them before the next transposing read and so loses
// what two buffers are for; nothing here returns a value, and wait_tile() holds the
// only wait they need.  (m0, which nothing else here uses, takes the address.  The wait
// states cover its write, and scalar registers that a vector instruction wrote just
// before: inside the text no one else inserts them.)
// The form with a scalar offset is for rows that are all there; the one without is also
// for descriptors that end before the tile does: what is beyond is then told by the lane's
// offset alone.
__device__ __forceinline__ void lds_load16_whole(uint32_t to, u32x4 buffer, uint32_t lane_offset,
                                                 uint32_t offset) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                   uniform(to)),
               "v"(lane_offset), "s"(buffer), "s"(uniform(offset))
               : "memory");
#endif
}
__device__ __forceinline__ void lds_load16(uint32_t to, u32x4 buffer, uint32_t lane_offset) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
                   uniform(to)),
               "v"(lane_offset), "s"(buffer)
               : "memory");
#endif
}
__device__ __forceinline__ void lds_load16(uint32_t to, const void* from) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uniform(to)), "v"(from)
               : "memory");
#endif
}
__device__ __forceinline__ void lds_load4(uint32_t to, u32x4 buffer, uint32_t lane_offset) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                   uniform(to)),
               "v"(lane_offset), "s"(buffer)
               : "memory");
#endif
}
__device__ __forceinline__ void lds_load4(uint32_t to, const void* from) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off" ::"s"(uniform(to)), "v"(from)
               : "memory");
#endif
}

// A descriptor of the memory from `base` on, for 32-bit offsets; beyond `bytes` reads are 0.
__device__ __forceinline__ u32x4 buffer_at(const void* base, uint32_t bytes = 0xFFFFFFFFu) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{uniform(static_cast<uint32_t>(a)), uniform(static_cast<uint32_t>(a >> 32) & 0xFFFFu),
               uniform(bytes), 0x00020000u};
}

// Loads of tiles of 64 rows of D columns.  A lane's offsets from a tile's
// first row are formed once, and a tile inside [first, last) takes a uniform
// base and these 32-bit offsets: forming 64-bit addresses a tile cost as much
// as a quarter of the softmax (integer products run at a quarter of the rate).  At
// the ends, rows outside are replaced by one inside (no owned row sees them),
// and rows too far apart for the offsets go the same way.
template <int D>
struct TileLoad {
  using Map = TileMap<D>;
  static constexpr int kLoads = Map::kLoads;
  const bf16* base;
  int64_t stride;
  int first, last;
  bool near;
  uint32_t off[Map::kOffs];

  __device__ __forceinline__ TileLoad(const bf16* b, int64_t s, int from, int to, int wave, int lane)
      : base(b), stride(s), first(from), last(to) {
    near = Map::near(s);
#pragma unroll
    for (int u = 0; u < Map::kOffs; ++u) off[u] = Map::first_offset(wave, u, lane, s);
  }

  // For near rows, without a branch: rows from `last` on become 0, and all of them do
  // without `on`.  Each run of loads has a descriptor of its own, which ends where the rows do.
  __device__ __forceinline__ void start_near(uint32_t tile, int row0, bool on, int wave) const {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int row = row0 + Map::rows_on(u);
      const u32x4 from = buffer_at(base + row * stride, Map::bytes(last - row, stride, on));
      lds_load16(tile + wave * (kLoads * 1024) + u * 1024, from, off[u % Map::kOffs]);
    }
  }

  __device__ __forceinline__ void start(uint32_t tile, int row0, int wave, int lane) const {
    const uint32_t to = tile + wave * (kLoads * 1024);
    if (near && row0 >= first && row0 + kTile <= last) {
      const u32x4 from = buffer_at(base + row0 * stride);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        lds_load16_whole(to + u * 1024, from, off[u % Map::kOffs],
                         static_cast<uint32_t>(Map::rows_on(u) * 2 * stride));
    } else {
#pragma unroll 1
      for (int u = 0; u < kLoads; ++u) {
        const int r = Map::row(wave, u, lane), c = Map::column(wave, u, lane);
        lds_load16(to + u * 1024, base + min(max(row0 + r, first), last - 1) * stride + c * 8);
      }
    }
  }
};

// Tiles of a pair of tensors under way or in use in the backward kernels.  With three, a
// tile's loads have two turns to arrive: 274 us instead of 279 with two (4096 keys, 16 heads
// of 64, no bias).  Where two workgroups share a compute unit, three of 128 columns do not fit.
// The rule goes by columns alone.  A bias adds its tables: at 96 columns the queries' kernel
// then has room for one workgroup a unit (354 us, where two tiles and two workgroups took 340:
// 4096 keys, 16 heads, causal, reach 128), and so has the joint launch at 64 columns from a
// reach of 256 on (364 us at 512, 209 at 128).
template <int D, bool ALONE>
constexpr int kBuffers = D <= 96 || ALONE ? 3 : 2;

// The calling wave's direct loads are done but for the last `LATER`; the
// workgroup's after the barrier.  (Loads end in the order they were started in.)
template <int LATER = 0>
__device__ __forceinline__ void wait_tile() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER) : "memory");
  __syncthreads();
}

// Has the compiler wait for a value's load here: at its first use, in the loop, the
// wait would be there every turn and for all direct loads under way (a full trip to
// memory a turn, which the buffers are there to hide).
template <typename T>
__device__ __forceinline__ void arrived(T& x) {
  asm volatile("" : "+v"(x));
}

// The larger of a value and the other half wave's at the same lane.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The distance bias in shared memory, times log2(e), at distance d + kSpan(reach):
// it goes on past the reach by kOver at either end, so that in a tile with
// any distance inside the reach no index has to be clipped.
constexpr int kOver = 2 * kTile;
__host__ __device__ constexpr int bias_span(int reach) { return reach + kOver; }
__host__ __device__ constexpr int bias_entries(int reach) { return 2 * bias_span(reach) + 1; }

__device__ __forceinline__ int bias_bucket(const AttnParams& p, int d) {
  return min(max(p.buckets[min(max(d, -p.reach), p.reach) + p.reach], 0), p.n_buckets - 1);
}

// The head's bias into shared memory, in three steps with other work between
// them: every entry is two loads, one after the other, and waiting for both in
// one place took 2.4 us of each workgroup.  Four entries a thread go this way, what a
// longer reach has beyond them (from 1025 entries on) at the end.  A finite bias stays
// finite.
struct BiasStage {
  static constexpr int kAtOnce = 4;
  int bucket[kAtOnce];
  float b[kAtOnce];

  static __device__ __forceinline__ float entry(const AttnParams& p, int h, int bucket) {
    const int64_t at = static_cast<int64_t>(bucket) * p.Hq + h;
    return p.table_f32 ? static_cast<const float*>(p.table)[at]
                       : static_cast<float>(static_cast<const bf16*>(p.table)[at]);
  }
  static __device__ __forceinline__ float in_log2(float b) {
    const float x = b * kLog2e;
    return __builtin_isinf(x) && !__builtin_isinf(b) ? __builtin_copysignf(-kLowest, b) : x;
  }

  __device__ __forceinline__ void buckets(const AttnParams& p, int tid) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      bucket[k] = bias_bucket(p, tid + k * kAttnThreads - bias_span(p.reach));   // (clips)
  }
  __device__ __forceinline__ void values(const AttnParams& p, int h) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) b[k] = entry(p, h, bucket[k]);
  }
  __device__ __forceinline__ void store(const AttnParams& p, int h, float* out, int tid) const {
    const int n = bias_entries(p.reach);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (tid + k * kAttnThreads < n) out[tid + k * kAttnThreads] = in_log2(b[k]);
    for (int e = tid + kAtOnce * kAttnThreads; e < n; e += kAttnThreads)
      out[e] = in_log2(entry(p, h, bias_bucket(p, e - bias_span(p.reach))));
  }
};

// Where a block of distances lies: all at or past one end of the reach (-1, 1),
// where the bias is one number, or not (0).
__device__ __forceinline__ int bias_side(int lowest, int highest, int reach) {
  return highest <= -reach ? -1 : lowest >= reach ? 1 : 0;
}

// How a score is capped.  cap tanh(y) = cap - 2 cap u with u = 1 / (exp(2 y) + 1), which
// is off by two steps (exponential, sum, reciprocal): the score is off by up to cap 2^-22,
// however small it is itself.  Up to kUCap that is 1.5e-5, a 250th of the rounding of p to
// bf16.  A larger cap takes small y by the tanh's series instead, which costs (us, 4096 keys,
// 32 on 8 heads, by u and by the series): forward 141 and 176 at 128 columns, 98 and 119 at
// 64; backward 480 and 759, 276 and 503.
constexpr float kUCap = 64.f;
enum CapForm { kNoCap = 0, kByU = 1, kAnyCap = 2 };
__host__ __device__ constexpr int cap_form(float cap) {
  return cap > 0.f ? (cap <= kUCap ? kByU : kAnyCap) : kNoCap;
}

// Factors of the scores.  Without a cap a score in units of log2 is x * a.
// With one, exp(2 y) is exp2(x * a) and the score c2 - 2 c2 u, or, of kAnyCap for small y,
// x * s times the series.  A negative scale is taken to q, so a > 0:
// the largest score is that of the largest x, and of the smallest u.  (A scale
// of 0 becomes one that vanishes beside any score; the factor of a tiny cap stays finite,
// so that a score of 0 is one.)
struct ScoreFactors {
  float a, c2, s;
  bool flip;
  __device__ __forceinline__ ScoreFactors(const AttnParams& p, int cap) {
    s = fmaxf(fabsf(p.scale), 1e-30f) * kLog2e;
    a = cap ? fminf(fmaxf(2.f * s / p.cap, 1e-30f), 1e30f) : s;
    c2 = cap ? p.cap * kLog2e : 0.f;
    flip = p.scale < 0.f;
  }
  __device__ __forceinline__ float u_of(float x) const { return rcp_hw(exp2_hw(x * a) + 1.f); }
  // The capped score of kAnyCap, in units of log2: tanh(y) / y = 1 - y^2 / 3 + 2 y^4 / 15 -
  // 17 y^6 / 315 + 62 y^8 / 2835 - 1382 y^10 / 155925 + .., whose next term is below 2^-26
  // for y < 0.35; beyond, u's error is below 12 steps of the score.
  __device__ __forceinline__ float any_cap(float x, float u) const {
    const float y = x * a * (0.5f * kLn2), w = y * y;
    float t = __builtin_fmaf(w, -1382.f / 155925.f, 62.f / 2835.f);
    t = __builtin_fmaf(w, t, -17.f / 315.f);
    t = __builtin_fmaf(w, t, 2.f / 15.f);
    t = __builtin_fmaf(w, t, -1.f / 3.f);
    t = __builtin_fmaf(w, t, 1.f);
    return w < 0.35f * 0.35f ? x * s * t : __builtin_fmaf(u, -2.f * c2, c2);
  }
};

// q's fragment times the sign of the scale.
__device__ __forceinline__ bf16x8 signed_frag(bf16x8 f, bool flip) {
  union {
    bf16x8 v;
    uint32_t u[4];
  } x;
  x.v = f;
#pragma unroll
  for (int j = 0; j < 4; ++j) x.u[j] ^= flip ? 0x80008000u : 0u;
  return x.v;
}

// Workgroup index along x to (batch, head): the 8 dies take workgroups in turn, so
// eighths of the heads in a row go to one die, whose cache then serves the query
// heads of a key head together (457 us instead of 459, backward, 4001 keys, 32 on 8 heads).
__device__ __forceinline__ int head_of_group(int x, int n) {
  return n % 8 == 0 ? (x % 8) * (n / 8) + x / 8 : x;
}

// Writes zeros over the rows of two staged tiles whose bit in `rows` is 0, by
// the whole workgroup.
template <int D>
__device__ __forceinline__ void clear_rows(uint32_t tile0, uint32_t tile1, uint64_t rows, int tid) {
  for (int piece = tid; piece < kTile * D / 8; piece += kAttnThreads)
    if (!((rows >> (piece / (D / 8))) & 1)) {
      *reinterpret_cast<ZO_LDS u32x4*>(tile0 + piece * 16) = u32x4{0, 0, 0, 0};
      *reinterpret_cast<ZO_LDS u32x4*>(tile1 + piece * 16) = u32x4{0, 0, 0, 0};
    }
}

// Whether some key between the first and the last that a workgroup's 128
// queries see is seen by none of them (padding between documents).  Such a key may
// hold anything, a NaN too, and is cleared from the staged tile, since a weight of 0 does
// not stop a NaN.  Keys in no gap are seen by a query of the workgroup, so what
// they hold counts; without gaps nothing needs clearing.  A range's end that
// lies in no other range, short of the last end, begins a gap.
// Ranges whose ends do not step back, none empty, as of causal documents and
// prefixes, are compared with their neighbours only.
__device__ __forceinline__ bool has_gaps(const int2* ranges, int last, int tid) {
  const int k = tid & 127;
  const int2 r = ranges[k], next = ranges[k < 127 ? k + 1 : k];
  const bool plain = r.y > r.x && next.x >= r.x && next.y >= r.y;
  if (__syncthreads_and(plain)) return __syncthreads_or(next.x > r.y) != 0;
  bool inside = false;
#pragma unroll 16
  for (int i = 0; i < 128; ++i) {        // (no early end: the reads follow one another)
    const int2 o = ranges[i];
    inside |= (o.x <= r.y) & (o.y > r.y);
  }
  return __syncthreads_or((r.y > r.x) & (r.y < last) & !inside) != 0;
}

// The keys k0 .. + 63 that some of the 128 queries see; `flags`: 2 words.
__device__ __forceinline__ uint64_t seen_keys(const int2* ranges, int k0, uint32_t* flags, int tid) {
  __syncthreads();
  if (tid < 2) flags[tid] = 0;
  __syncthreads();
  const int j = k0 + (tid & 63);
  bool seen = false;
#pragma unroll 8
  for (int k = 0; k < 32; ++k) {
    const int2 o = ranges[32 * (tid >> 6) + k];
    seen |= (j >= o.x) & (j < o.y);
  }
  if (seen) atomicOr(&flags[(tid & 63) >> 5], 1u << (tid & 31));
  __syncthreads();
  return flags[0] | static_cast<uint64_t>(flags[1]) << 32;
}

// A workgroup's place in its kernel's grid, or in its part of a grid that two share.
struct Place {
  int x, y, nx, ny;
};
__device__ __forceinline__ Place place() {
  return {static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y), static_cast<int>(gridDim.x),
          static_cast<int>(gridDim.y)};
}

// Which tile the workgroup at place y of its batch row's launch order takes:
// the one of rank y by decreasing cost (ties by index), so that the longest start first
// and the last to start are short; documents give a tile's cost no order that its index
// would tell.  cost(t) is an estimate; `scratch`: n + 1 words, n <= 256.
template <typename Cost>
__device__ __forceinline__ int tile_of_rank(int y, int n, int* scratch, int tid, Cost cost) {
  if (tid < n) scratch[tid] = cost(tid);
  __syncthreads();
  if (tid < n) {
    const int mine = scratch[tid];
    int rank = 0;
    for (int k = 0; k < n; ++k) rank += scratch[k] > mine || (scratch[k] == mine && k < tid);
    if (rank == y) scratch[n] = tid;
  }
  __syncthreads();
  const int t = scratch[n];
  __syncthreads();
  return t;
}
// (Ranked, 134 us instead of 154 forward and 457 instead of 476 backward: 4096 and 4001 keys
// in two documents.  Eight tiles, 1024 keys: the same.  256 threads rank 255 tiles.)
constexpr int kMinRanked = 16, kMaxRanked = 255;

// The same for a tile of 128 queries: its cost is the span of keys that four of its
// queries see.  Without ranges, or where all workgroups run `at_once` anyway, the last
// tile first: the order of a causal mask.
__device__ __forceinline__ int query_tile(const AttnParams& p, const Place& w, int b, int* scratch,
                                          int tid, int at_once) {
  const int n = w.ny, y = w.y;
  if (!p.ranges || n < kMinRanked || n > kMaxRanked || w.nx * n <= at_once) return n - 1 - y;
  return tile_of_rank(y, n, scratch, tid, [&](int t) {
    int lo = 0x7FFFFFFF, hi = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int2 r = key_range(p, b, min(128 * t + 42 * k, p.Tq - 1));
      if (r.y > r.x) {
        lo = min(lo, r.x);
        hi = max(hi, r.y);
      }
    }
    return max(hi - lo, 0);
  });
}

AttnParams attn_params(const zero_attn_args& a);

}  // namespace zo
