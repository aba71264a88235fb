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
#include "zero_ops.h"

namespace zo {

constexpr int kAttnThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 64;  // rows of a staged tile

// A staged tile is 64 rows of D bf16 without gaps (the direct loads to shared
// memory write 64 lanes' 16 bytes one after another), and the 16-byte pieces of
// row r are stored at piece ^ swizzle(r).  The 8 rows of consecutive lanes'
// 16-byte reads, and the 4 rows of a transposing read, then fall on different
// banks: with 256-byte rows all start on the same bank and the 4 x 32 bytes of a
// transposing read need 4 different pairs of pieces; 128-byte rows alternate between
// two halves of the banks, 64- and 192-byte rows repeat after 4.
template <int D>
__device__ __forceinline__ constexpr int swizzle(int r) {
  return D == 128 ? (r & 7) << 1 : D == 64 ? r & 6 : (r >> 2) & 1;
}
template <int D>
constexpr int kTileBytes = kTile * D * 2;

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

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
  float* lse2;      // [B][Hq][tq64]  lse * log2(e), +inf for a query without keys
  float* delta;     // [B][Hq][tq64]  do . o
  int *qlo, *qhi;   // [B][tq64]      the keys a query sees; 0, 0 for none
  float* dpart;     // [B][Hq][query tiles][n_buckets]
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

// Hull of the lanes' non-empty ranges over a wave ({INT_MAX, 0}: none).
__device__ __forceinline__ int2 wave_hull(int2 r) {
  int lo = r.y > r.x ? r.x : 0x7FFFFFFF, hi = r.y;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    lo = min(lo, __shfl_xor(lo, d));
    hi = max(hi, __shfl_xor(hi, d));
  }
  return make_int2(lo, hi);
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
// one bit a sum.)
template <int D>
__device__ __forceinline__ bf16x8 frag_rows(const FragAt<D>& at, int t, int c) {
  const uint32_t x = (D == 64 || D == 128 ? at.rows ^ (c << 5) : at.rows + (c << 5)) + t * 64 * D;
  return *reinterpret_cast<const ZO_LDS bf16x8*>(x);
}

// Operand fragment, contraction along the column: columns 32 t + l % 32 and, of
// the 16 rows from 16 u, the 8 in the order in which a score result holds
// them.  A transposing read hands each of 16 lanes a column of the 4 x 16
// block whose rows those lanes address by fours.
template <int D>
__device__ __forceinline__ bf16x8 frag_cols(const FragAt<D>& at, int u, int t) {
  const uint32_t x = (D == 64 || D == 128 ? at.cols ^ (t << 6) : at.cols + (t << 6)) + u * 32 * D;
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

// Eight registers of a score result as an operand fragment.
__device__ __forceinline__ bf16x8 to_frag(const float* x) {
  bf16x8 f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = static_cast<bf16>(x[j]);
  return f;
}

// Clears the fragment's elements whose bit in `keep` is 0: rows that no owned
// row sees are weighted with 0, and whatever they hold (an uninitialised
// padding row's NaN, say) must not reach the product.
__device__ __forceinline__ bf16x8 keep_frag(bf16x8 f, uint32_t keep) {
  union {
    bf16x8 v;
    uint32_t u[4];
  } x;
  x.v = f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = ((keep >> (2 * j)) & 1u ? 0x0000FFFFu : 0u) |
                       ((keep >> (2 * j + 1)) & 1u ? 0xFFFF0000u : 0u);
    x.u[j] &= m;
  }
  return x.v;
}

// Whether any lane of this lane's half wave has the flag set.
__device__ __forceinline__ uint32_t any_in_half(bool f, int lane) {
  const uint64_t m = __ballot(f);
  const uint32_t half = lane >= 32 ? static_cast<uint32_t>(m >> 32) : static_cast<uint32_t>(m);
  return half != 0 ? 1u : 0u;
}

// Starts the loads of a tile of 64 rows, row0 .. + 63 of `base`, straight into
// shared memory (no registers on the way).  Rows outside [first, last) are
// replaced by a row inside: no owned row sees them.  wait_tile() ends them.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t tile, const bf16* base, int64_t stride, int row0,
                                          int first, int last, int wave, int lane) {
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    const int n = wave * (D / 32) + u;                 // of D / 8 loads of 64 pieces
    const int piece = n * 64 + lane;
    const int r = piece / (D / 8), c = (piece % (D / 8)) ^ swizzle<D>(r);
    const int row = min(max(row0 + r, first), last - 1);
    const bf16* src = base + row * stride + c * 8;
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)src,
        reinterpret_cast<ZO_LDS void*>(tile + n * 1024), 16, 0, 0);
  }
}

// The same for 64 words of a padded array, by one wave.
__device__ __forceinline__ void load_words(uint32_t to, const void* from, int lane) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)(static_cast<const uint32_t*>(from) + lane),
      reinterpret_cast<ZO_LDS void*>(to), 4, 0, 0);
}

// The calling thread's tile loads are done; the workgroup's after the barrier.
__device__ __forceinline__ void wait_tile() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
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

// The head's bias into shared memory.  A finite bias stays finite.
__device__ __forceinline__ void stage_bias(const AttnParams& p, int h, float* out, int tid) {
  const int span = bias_span(p.reach);
  for (int d = tid - span; d <= span; d += kAttnThreads) {
    const int64_t at = static_cast<int64_t>(bias_bucket(p, d)) * p.Hq + h;
    const float b = p.table_f32 ? static_cast<const float*>(p.table)[at]
                                : static_cast<float>(static_cast<const bf16*>(p.table)[at]);
    const float x = b * kLog2e;
    out[d + span] =
        __builtin_isinf(x) && !__builtin_isinf(b) ? __builtin_copysignf(-kLowest, b) : x;
  }
}

// Where a block of distances lies: all at or past one end of the reach (-1, 1),
// where the bias is one number, or not (0).
__device__ __forceinline__ int bias_side(int lowest, int highest, int reach) {
  return highest <= -reach ? -1 : lowest >= reach ? 1 : 0;
}

// Factors of the scores.  Without a cap a score in units of log2 is x * a.
// With one, cap tanh(y) = cap - 2 cap u, u = 1 / (exp(2 y) + 1): exp(2 y) is
// exp2(x * a) and the score c2 - 2 c2 u.  A negative scale is taken to q, so a > 0:
// the largest score is that of the largest x, and of the smallest u.  (A scale
// of 0 becomes one that vanishes beside any score.)
struct ScoreFactors {
  float a, c2;
  bool flip;
  __device__ __forceinline__ ScoreFactors(const AttnParams& p, bool cap) {
    const float s = fmaxf(fabsf(p.scale), 1e-30f) * kLog2e;
    a = cap ? fmaxf(2.f * s / p.cap, 1e-30f) : s;
    c2 = cap ? p.cap * kLog2e : 0.f;
    flip = p.scale < 0.f;
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
// heads of a key head together.
__device__ __forceinline__ int head_of_group(int x, int n) {
  return n % 8 == 0 ? (x % 8) * (n / 8) + x / 8 : x;
}

AttnParams attn_params(const zero_attn_args& a);

}  // namespace zo
