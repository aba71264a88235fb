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

// Row pitch, in elements, of a staged tile of D columns: D + 16 is an odd
// multiple of 8 banks of 4 bytes for every supported D, so the 8 rows that 16
// lanes' 16-byte reads take at a time, and the 4 rows of a transposing read,
// fall on different banks.
template <int D>
constexpr int kPitch = D + 16;

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
  float* lse2;      // [B][Hq][Tq]  lse * log2(e), +inf for a query without keys
  float* delta;     // [B][Hq][Tq]  do . o
  int2* qbounds;    // [B][tiles of 64 queries]  keys their queries see, as a hull
  float* dpart;     // [B][Hq][query tiles][n_buckets]
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

// Operand fragment of a row-major tile in shared memory, contraction along
// the row: rows row0 + l % 32, elements col0 + 8 (l / 32) .. + 7.
template <int PITCH>
__device__ __forceinline__ bf16x8 frag_rows(const bf16* tile, int row0, int col0, int lane) {
  return load8(tile + (row0 + (lane & 31)) * PITCH + col0 + 8 * (lane >> 5));
}

// Operand fragment of the same tile, contraction along the column: columns
// col0 + l % 32 and, of the 16 rows from row0, the 8 in the order in which a
// score result holds them.  A transposing read hands each of 16 lanes a
// column of the 4 x 16 block whose rows those lanes address by fours.
template <int PITCH>
__device__ __forceinline__ bf16x8 frag_cols(const bf16* tile, int row0, int col0, int lane) {
  const int i = lane & 15;
  const bf16* a = tile + (row0 + 4 * (lane >> 5) + (i >> 2)) * PITCH + col0 +
                  16 * ((lane >> 4) & 1) + 4 * (i & 3);
  using P = __attribute__((address_space(3))) s16x4*;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(a));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(a + 8 * PITCH));
  union {
    s16x4 s[2];
    bf16x8 v;
  } u;
  u.s[0] = lo;
  u.s[1] = hi;
  return u.v;
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

// A 64-row tile of D columns: global loads of a thread's 16-byte pieces (rows
// outside [first, last) read as 0) and their stores to shared memory.
template <int D>
struct Stage {
  static constexpr int kPieces = kTile * D / 8 / kAttnThreads;
  u32x4 r[kPieces];

  __device__ __forceinline__ void load(const bf16* base, int64_t stride, int row0, int first,
                                       int last, int tid) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int c = tid + u * kAttnThreads;
      const int row = row0 + c / (D / 8), col = (c % (D / 8)) * 8;
      r[u] = u32x4{0, 0, 0, 0};
      if (row >= first && row < last)
        r[u] = *reinterpret_cast<const u32x4*>(base + row * stride + col);
    }
  }
  __device__ __forceinline__ void store(bf16* tile, int tid) const {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int c = tid + u * kAttnThreads;
      const int row = c / (D / 8), col = (c % (D / 8)) * 8;
      *reinterpret_cast<u32x4*>(tile + row * kPitch<D> + col) = r[u];
    }
  }
};

// The head's bias by distance, times log2(e), into shared memory:
// out[d + reach].  A finite bias stays finite.
__device__ __forceinline__ void stage_bias(const AttnParams& p, int h, float* out, int tid) {
  for (int d = tid; d <= 2 * p.reach; d += kAttnThreads) {
    const int bucket = min(max(p.buckets[d], 0), p.n_buckets - 1);
    const int64_t at = static_cast<int64_t>(bucket) * p.Hq + h;
    const float b = p.table_f32 ? static_cast<const float*>(p.table)[at]
                                : static_cast<float>(static_cast<const bf16*>(p.table)[at]);
    const float x = b * kLog2e;
    out[d] = __builtin_isinf(x) && !__builtin_isinf(b) ? __builtin_copysignf(-kLowest, b) : x;
  }
}

// A raw product q.k as a score in units of log2: x = scale q.k, capped.
// `a` is scale * log2(e), or 2 scale log2(e) / cap with the cap, where
// cap tanh(y) = cap - 2 cap / (exp(2 y) + 1); `c2` is then cap log2(e).
template <bool CAP>
__device__ __forceinline__ float score2(float x, float a, float c2) {
  if constexpr (CAP) {
    const float e = exp2_hw(x * a);
    return __builtin_fmaf(rcp_hw(e + 1.f), -2.f * c2, c2);
  } else {
    return x * a;
  }
}


AttnParams attn_params(const zero_attn_args& a);

}  // namespace zo
