// zo_block_norm.hip -- the norm of a block's output, its gate, the residual sum
// and the next block's norm in one pass, forward and backward.
//
// Bound by memory: every row is read once, kept in registers across its norms'
// sums, and written once.  Forward, a row belongs to a wave where it has at most 1024 values (no
// barrier), to a workgroup beyond.  Backward, where a value takes some 30 operations
// and the sums over the tokens 16 registers a piece, the rows are spread over more threads;
// workgroups walk the rows and leave their sums in a row of the workspace, which a second kernel
// folds in order.
//
// Measured, bf16 with both norms and a gate by channel: forward of 16384 x 4096 91 to 94 us, 5.7 to
// 5.9 TB/s (all past the caches; written through them 98, read too 102); backward of 8192 x 4096 84 us, 4.8 TB/s,
// the fold 5 of them (loads through the caches 90; four barriers a row and the gate's sums of their own,
// twice the instructions: 104).  4097 x 1000, fp32 stream and a gate by token: backward 25 us.  8192 x
// 8192 backward 153 us, 5.3 TB/s; 4096 x 16384, where less is held, 192 us, 4.2 TB/s.
#include <algorithm>

#include "zo_device.h"
#include "zo_internal.h"
#include "zo_rows.h"

namespace zo {

// Workgroups of the backward pass at most, each of which leaves a row of parts for
// every gradient that is summed over the tokens.  (8192 x 4096: 84 us; 768 96, 1024 95: the parts
// grow, and not all run at once.)  One of 1024 threads fills a unit: 8192 x 8192 152 us with 256 of
// them, 162 with 512.  Fewer where each would have less than four rows: 500 x 4096 19 us, 23 with a
// row each.
constexpr int kBlockBwdGroups = 512, kBlockBwdLarge = 256, kBlockBwdFew = 256;

struct BlockParams {
  int64_t T;
  int C, post, gate_tokens, has_post_w, has_pre_w;
  float eps, offset, res_scale, branch_scale;
  const void *x, *y, *post_w, *gate, *pre_w;
  void *h, *z;
  const void *dh, *dz;
  void *dx, *dy, *dgate;
  int64_t x_s, y_s, gate_s, h_s, z_s, dh_s, dz_s, dx_s, dy_s, dgate_s;
  float* part;                     // [3][groups][C]: post_w, gate, pre_w; NULL: no sums wanted
  int want[3];
};

// Sums over a row's threads: a wave's lanes, or a workgroup's NT threads.
template <int NT>
struct RowSum {
  float* s;                        // [2][waves], used in turn
  int turn;
  __device__ __forceinline__ float operator()(float x) {
    x = join_lanes<64>(x, AddOp());
    if constexpr (NT > 64) {
      constexpr int kW = NT / 64;
      float* at = s + turn * kW;
      turn ^= 1;
      const int lane = threadIdx.x & 63;
      if (lane == 0) at[threadIdx.x >> 6] = x;
      __syncthreads();
      x = join_lanes<kW>(at[lane % kW], AddOp());
    }
    return x;
  }
};

// 1 / sqrt(mean(v^2) + eps), and where that mean is past binary32's ends, of v times a
// power of 2 (see far_root).  The same in all threads of the row.
template <int NT, int CH>
__device__ __forceinline__ float inverse_rms(RowSum<NT>& sum, const float (&v)[CH][8], float inv_c,
                                             float eps) {
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[k][j], v[k][j], sq);
  const float ms = __builtin_fmaf(sum(sq), inv_c, eps);
  float r = __builtin_amdgcn_rsqf(ms);
  if (__builtin_expect(far_mean(ms), 0)) {
    const float s = ms < 1.f ? 0x1p100f : 0x1p-100f;
    sq = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[k][j] * s, v[k][j] * s, sq);
    r = far_root(__builtin_fmaf(sum(sq), inv_c, eps * s * s), s);
  }
  return r;
}

// Row t of an array, as an address in scalar registers: its pieces' addresses are then an
// offset of 32 bits a lane, not 64 bits a lane for every array and piece.
template <typename T>
__device__ __forceinline__ const char* row_of(const void* base, int64_t t, int64_t stride) {
  const char* at = static_cast<const char*>(base) + t * stride * static_cast<int64_t>(sizeof(T));
  asm("" : "+s"(at));
  return at;
}
template <typename T>
__device__ __forceinline__ char* row_of(void* base, int64_t t, int64_t stride) {
  return const_cast<char*>(row_of<T>(static_cast<const void*>(base), t, stride));
}

// A piece's columns: 8 from c on, or, SPLIT, 4 from c on and 4 that are kHalf further, so that
// a wave's accesses of 16 bytes leave no gaps where values have 4 bytes (fp32, 8192 x 4096: forward 98
// us, 8 in a row 111; backward 152, 168).
template <typename E, typename R>
constexpr bool kSplit = sizeof(E) == 4 || sizeof(R) == 4;
template <bool SPLIT, int NT>
__device__ __forceinline__ int column(int tid, int k) {
  return SPLIT ? 8 * ((tid & ~63) + k * NT) + 4 * (tid & 63) : 8 * (tid + k * NT);
}

// A weight plus its offset, or 1 where there is none.
template <typename E, bool SPLIT>
__device__ __forceinline__ void weight8(const void* w, int has, float offset, int c, int C,
                                        float x[8]) {
  if (has) {
    load8<E, SPLIT>(w, c, C, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += offset;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
  }
}

// branch_scale times the gate, `gate` its row or NULL.
template <typename E, bool SPLIT>
__device__ __forceinline__ void gate8(const BlockParams& p, const char* gate, int c, float g[8]) {
  if (p.gate != nullptr) {
    load8<E, SPLIT>(gate, c, p.C, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= p.branch_scale;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = p.branch_scale;
  }
}

// A row whose root stands apart from its power takes that.
template <int CH>
__device__ __forceinline__ float with_power(float (&v)[CH][8], float r) {
  if (__builtin_expect(power_apart(r), 0)) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= far_power(r);
  }
  return fabsf(r);
}

// NT threads to a row, CH pieces of 8 values to a thread.
template <typename E, typename R, int NT, int CH, bool PAST>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_fwd_kernel(const BlockParams p) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  constexpr bool S = kSplit<E, R>;
  __shared__ float s[2 * NT / 64];
  RowSum<NT> sum{s, 0};
  const int tid = threadIdx.x % NT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + uniform(threadIdx.x / NT);
  if (t >= p.T) return;                        // (whole waves; with several rows no barrier)
  const float inv_c = 1.f / static_cast<float>(p.C);
  const char* gate = row_of<E>(p.gate, p.gate_tokens ? t : 0, p.gate_s);
  float h[CH][8], y[CH][8];
  bool on[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = column<S, NT>(tid, k);
    on[k] = c < p.C;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[k][j] = y[k][j] = 0.f;
    if (on[k]) {
      load8<R, S, true>(row_of<R>(p.x, t, p.x_s), c, p.C, h[k]);
      if (p.y != nullptr) load8<E, S, true>(row_of<E>(p.y, t, p.y_s), c, p.C, y[k]);
    }
  }
  if (p.y != nullptr) {
    const float r = p.post ? with_power(y, inverse_rms<NT, CH>(sum, y, inv_c, p.eps)) : 1.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = column<S, NT>(tid, k);
      if (!on[k]) continue;
      float w[8], g[8];
      weight8<E, S>(p.post_w, p.has_post_w, p.offset, c, p.C, w);
      gate8<E, S>(p, gate, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        h[k][j] = __builtin_fmaf(g[j], y[k][j] * r * w[j], h[k][j] * p.res_scale);
    }
  } else {
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[k][j] *= p.res_scale;
  }
  if (p.h != nullptr) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (on[k]) store8<R, S, PAST>(row_of<R>(p.h, t, p.h_s), column<S, NT>(tid, k), p.C, h[k]);
  }
  if (p.z == nullptr) return;
  const float r = with_power(h, inverse_rms<NT, CH>(sum, h, inv_c, p.eps));
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = column<S, NT>(tid, k);
    if (!on[k]) continue;
    float w[8];
    weight8<E, S>(p.pre_w, p.has_pre_w, p.offset, c, p.C, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[k][j] = h[k][j] * r * w[j];
    store8<E, S, PAST>(row_of<E>(p.z, t, p.z_s), c, p.C, h[k]);
  }
}

// A row behind a buffer descriptor: loads past its end, or of an array that is not there, give 0
// without a branch.  (ONCE: past the caches.)
template <typename T>
struct BufferRow {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ BufferRow(const void* base, int64_t t, int64_t stride, int C, bool on) {
    const char* at = row_of<T>(base, on ? t : 0, stride);
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0,
                                          on ? C * static_cast<int>(sizeof(T)) : 0, 0x00020000);
  }
  template <bool SPLIT, bool ONCE>
  __device__ __forceinline__ void load(int c, Vec8<T>& v) const {
    constexpr int kPast = ONCE ? 2 : 0;
    const int b = c * static_cast<int>(sizeof(T));
    if constexpr (sizeof(T) == 4) {
      constexpr int kNext = SPLIT ? 4 * kHalf : 16;
      v.a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, b, 0, kPast));
      v.b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, b + kNext, 0, kPast));
    } else if constexpr (SPLIT) {
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, b, 0, kPast));
      const u32x2 hi =
          __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, b + 2 * kHalf, 0, kPast));
      v.r = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      v.r = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, b, 0, kPast));
    }
  }
};

// What a thread's loads of a row fetch, CH pieces of each array.
template <typename E, typename R, int NT, int CH>
struct RawRow {
  Vec8<R> dh[CH], h[CH];
  Vec8<E> dz[CH], y[CH];
};

// Sums of up to four values over a row's threads at once.  Halves, then quarters of the wave
// take a value each by swaps between two registers, so a wave's 64 lanes are joined for
// all of them in 3 swaps and 7 additions; one barrier, and the sums are in scalar registers.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}
template <int G>
__device__ __forceinline__ float sum_lanes(float x) {      // of G consecutive lanes, G <= 16
  if constexpr (G >= 2) x = add_dpp<0xB1>(x);
  if constexpr (G >= 4) x = add_dpp<0x4E>(x);
  if constexpr (G >= 8) x = add_dpp<0x141>(x);
  if constexpr (G >= 16) x = add_dpp<0x140>(x);
  return x;
}
__device__ __forceinline__ float add_halves(float a, float b) {    // a's in the low 32 lanes
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_quarters(float a, float b) {  // a's in the even 16 lanes
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int NT, int N>
__device__ __forceinline__ void row_sums(float* s, int& turn, float (&x)[N]) {
  static_assert(N >= 1 && N <= 4);
  const int lane = threadIdx.x & 63;
  // lanes 0..15: x[0], 16..31: x[2], 32..47: x[1], 48..63: x[3]
  float v = add_halves(x[0], N > 1 ? x[N > 1 ? 1 : 0] : x[0]);
  const float w = N > 2 ? add_halves(x[N > 2 ? 2 : 0], N > 3 ? x[N > 3 ? 3 : 0] : x[N > 2 ? 2 : 0]) : v;
  v = sum_lanes<16>(add_quarters(v, w));
  if constexpr (NT > 64) {
    constexpr int kW = NT / 64;
    float* at = s + turn * (4 * kW);
    turn ^= 1;
    if ((lane & 15) == 0) at[(lane >> 4) * kW + (threadIdx.x % NT >> 6)] = v;
    __syncthreads();
    v = sum_lanes<kW>(at[(lane >> 4) * kW + lane % kW]);
  }
  constexpr int kAt[4] = {0, 32, 16, 48};
#pragma unroll
  for (int i = 0; i < N; ++i)
    x[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), kAt[i]));
}

// r = 1 / sqrt(mean(v^2) + eps), as far_root gives it, and m = mean(u v) of normed v, of a row whose
// mean square ms is past binary32's ends.  Rare: every wave reads the whole row again, and
// needs no barrier for it.  part(c, u, v) gives the values of column c.
template <typename Part>
__device__ __forceinline__ void far_norm(int C, float ms, float inv_c, float eps, float& r, float& m,
                                         Part part) {
  const float s = ms < 1.f ? 0x1p100f : 0x1p-100f;
  float vv = 0.f, uv = 0.f;
#pragma unroll 1
  for (int c = threadIdx.x & 63; c < C; c += 64) {
    float u, v;
    part(c, u, v);
    vv = __builtin_fmaf(v * s, v * s, vv);
    uv = __builtin_fmaf(u, v * s, uv);
  }
  vv = join_lanes<64>(vv, AddOp());
  uv = join_lanes<64>(uv, AddOp());
  const float mean = __builtin_fmaf(vv, inv_c, eps * s * s);
  r = far_root(mean, s);
  m = uv * inv_c * __builtin_amdgcn_rsqf(mean);
}

// Threads of a workgroup: four rows of up to 1024 values, two of up to 2048 (16384 x 2048: 73 us,
// with one 78), or one.
template <int NT>
constexpr int kBwdThreads = NT <= 128 ? 4 * NT : NT == 256 ? 512 : NT;

// Two barriers a row: h's and y's squares and u2 . h are summed first, u1 . y when
// gh is known.  What a row's loads fetched stays packed in registers, and is widened
// again for each use; the columns' weights are widened once.
//
// The gate's gradient and the first weight's come from one sum where the tokens share the
// gate: t = sum of gh yy gives branch_scale (post_w + offset) t and branch_scale gate t.
template <typename E, typename R, int NT, int CH, bool PAST>
__global__ __launch_bounds__(kBwdThreads<NT>) void block_norm_bwd_kernel(const BlockParams p) {
  constexpr int kRows = kBwdThreads<NT> / NT;
  __shared__ float s[NT > 64 ? kRows : 1][NT > 64 ? 8 * (NT / 64) : 1];
  __shared__ float fold[kRows > 1 ? kRows : 1][kRows > 1 ? NT * 8 : 1];
  // 16 waves to a unit leave each 128 registers: of the longest rows' two pieces dz, dh and the
  // weights are not held but read at each use, one piece after the other (y read again too: 225 us at
  // 4096 x 16384 for 192), and u1 and pre_w's sums wait in shared memory.
  constexpr bool kHold = NT < 1024 || CH == 1, S = kSplit<E, R> && kHold;
  constexpr int kHeld = kHold ? CH : 1;
  __shared__ f32x4 kept[kHold ? 1 : 2 * CH][kHold ? 1 : NT];
  __shared__ f32x4 kept_w2[kHold ? 1 : 2 * CH][kHold ? 1 : NT];
  const auto put = [&](auto& at, int k, const float x[8]) {
    at[2 * k][threadIdx.x] = f32x4{x[0], x[1], x[2], x[3]};
    at[2 * k + 1][threadIdx.x] = f32x4{x[4], x[5], x[6], x[7]};
  };
  const auto take = [&](auto& at, int k, float x[8]) {
    const f32x4 a = at[2 * k][threadIdx.x], b = at[2 * k + 1][threadIdx.x];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[4 + j] = b[j];
    }
  };
  const auto apart = [] {
    if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);
  };
  int turn = 0;
  const int tid = threadIdx.x % NT, row = uniform(threadIdx.x / NT);
  const float inv_c = 1.f / static_cast<float>(p.C);
  const bool use_y = p.y != nullptr && (p.post || p.gate != nullptr), use_z = p.dz != nullptr;
  const bool tokens = p.gate != nullptr && p.gate_tokens;
  // post_w and pre_w with the offset, and the gate times branch_scale; 0 behind the row's end
  const auto weights = [&](int k, float w1[8], float w2[8], float g[8]) {
    const int c = column<S, NT>(tid, k);
#pragma unroll
    for (int j = 0; j < 8; ++j) w1[j] = w2[j] = g[j] = 0.f;
    if (c < p.C) {
      weight8<E, S>(row_of<E>(p.post_w, 0, 0), p.has_post_w, p.offset, c, p.C, w1);
      weight8<E, S>(row_of<E>(p.pre_w, 0, 0), p.has_pre_w, p.offset, c, p.C, w2);
      if (tokens) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = p.branch_scale;
      } else {
        gate8<E, S>(p, row_of<E>(p.gate, 0, 0), c, g);
      }
    }
  };
  // of a piece: w2, and w1 times the gate (or branch_scale, where every token has its own)
  float held_w2[kHeld][8], held_gw[kHeld][8];
  const auto columns = [&](int k, float w2[8], float gw[8]) {
    float w1[8];
    weights(k, w1, w2, gw);
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[j] *= w1[j];
  };
  float sum_t[CH][8], sum_w2[kHeld][8];          // of gh yy (by a token's gate), of dz hh
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    if constexpr (kHold) columns(k, held_w2[k], held_gw[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_t[k][j] = sum_w2[kHold ? k : 0][j] = 0.f;
    if constexpr (!kHold) put(kept_w2, k, sum_w2[0]);
  }
  // A workgroup that has its unit to itself fetches the next row before it ends this one (8192 x
  // 8192: 162 us instead of 171; where two share a unit it gains nothing, 82 for 79 at 4096).
  constexpr bool kAhead = NT == 1024;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const auto row_at = [&](int64_t t0) { return t0 + row < p.T ? t0 + row : p.T - 1; };
  // (rows behind the last one: nothing is loaded or stored, but the barriers are met)
  const auto length = [&](int64_t t0) { return t0 + row < p.T ? p.C : 0; };
  RawRow<E, R, NT, CH> raw;
  const auto fetch = [&](int64_t t0, Vec8<E> (&y)[CH]) {
    const int64_t t = row_at(t0);
    const int C = length(t0);
    const BufferRow<R> at_h(p.h, t, p.h_s, C, use_z), at_dh(p.dh, t, p.dh_s, C, p.dh != nullptr);
    const BufferRow<E> at_dz(p.dz, t, p.dz_s, C, use_z), at_y(p.y, t, p.y_s, C, use_y);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = column<S, NT>(tid, k);
      at_h.template load<S, kHold>(c, raw.h[k]);
      if constexpr (kHold) at_dz.template load<S, kHold>(c, raw.dz[k]);
      at_y.template load<S, kHold>(c, y[k]);
      if constexpr (kHold) at_dh.template load<S, kHold>(c, raw.dh[k]);
    }
  };
  if constexpr (kAhead) fetch(static_cast<int64_t>(blockIdx.x) * kRows, raw.y);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < p.T; t0 += step) {
    const int64_t t = row_at(t0);
    const int C = length(t0);
    const char* gate = row_of<E>(p.gate, tokens ? t : 0, p.gate_s);
    if constexpr (!kAhead) fetch(t0, raw.y);
    const auto h_of = [&](int k, float x[8]) { raw.h[k].get(x); };
    const auto y_of = [&](int k, float x[8]) { raw.y[k].get(x); };
    const auto dh_of = [&](int k, float x[8]) {
      if constexpr (!kHold)
        BufferRow<R>(p.dh, t, p.dh_s, C, p.dh != nullptr)
            .template load<S, kHold>(column<S, NT>(tid, k), raw.dh[0]);
      raw.dh[kHold ? k : 0].get(x);
    };
    const auto dz_of = [&](int k, float x[8]) {
      if constexpr (!kHold)
        BufferRow<E>(p.dz, t, p.dz_s, C, use_z).template load<S, kHold>(column<S, NT>(tid, k), raw.dz[0]);
      raw.dz[kHold ? k : 0].get(x);
    };
    const auto columns_of = [&](int k, float w2[8], float gw[8]) {
      if constexpr (kHold) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w2[j] = held_w2[k][j];
          gw[j] = held_gw[k][j];
        }
      } else {
        columns(k, w2, gw);
      }
    };
    const auto u2_of = [&](int k, float x[8]) {
      float w2[8], gw[8];
      columns_of(k, w2, gw);
      dz_of(k, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= w2[j];
    };
    float sums[3] = {0.f, 0.f, 0.f};             // h^2, u2 h, y^2
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float h[8], u[8], y[8];
      h_of(k, h);
      u2_of(k, u);
      y_of(k, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[0] = __builtin_fmaf(h[j], h[j], sums[0]);
        sums[1] = __builtin_fmaf(u[j], h[j], sums[1]);
        sums[2] = __builtin_fmaf(y[j], y[j], sums[2]);
      }
      apart();
    }
    row_sums<NT, 3>(s[NT > 64 ? row : 0], turn, sums);
    const float ms2 = __builtin_fmaf(sums[0], inv_c, p.eps);
    const float ms1 = __builtin_fmaf(sums[2], inv_c, p.eps);
    float r2 = __builtin_amdgcn_rsqf(ms2), r1 = __builtin_amdgcn_rsqf(ms1);
    float m2 = sums[1] * inv_c * r2;             // mean(u2 hh)
    if (!use_z) {
      r2 = m2 = 0.f;
    } else if (__builtin_expect(far_mean(ms2), 0)) {
      far_norm(C, ms2, inv_c, p.eps, r2, m2, [&](int c, float& u, float& v) {
        u = value<E>(row_of<E>(p.dz, t, p.dz_s), c) *
            (p.has_pre_w ? value<E>(p.pre_w, c) + p.offset : 1.f);
        v = value<R>(row_of<R>(p.h, t, p.h_s), c);
      });
    }
    if (!p.post) {
      r1 = 1.f;
    } else if (__builtin_expect(far_mean(ms1), 0)) {
      float none;
      far_norm(C, ms1, inv_c, p.eps, r1, none, [&](int c, float& u, float& v) {
        u = 0.f;
        v = value<E>(row_of<E>(p.y, t, p.y_s), c);
      });
    }
    if (C == 0) r1 = r2 = m2 = 0.f;              // (with an eps of 0 they were infinite)
    const bool apart1 = power_apart(r1), apart2 = power_apart(r2);
    const float a2 = -fabsf(r2) * (m2 * far_power(r2));
    float u1[kHeld][8], dot[1] = {0.f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = column<S, NT>(tid, k);
      float gh[8], h[8], z[8], w2[8], gw[8];
      dh_of(k, gh);
      h_of(k, h);
      dz_of(k, z);
      columns_of(k, w2, gw);
      float* dw2 = sum_w2[kHold ? k : 0];
      if constexpr (!kHold) take(kept_w2, k, dw2);
#pragma unroll
      for (int j = 0; j < 8; ++j) w2[j] *= z[j];
      if (__builtin_expect(apart2, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] *= far_power(r2);
          w2[j] *= far_power(r2);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hh = h[j] * fabsf(r2);
        dw2[j] = __builtin_fmaf(z[j], hh, dw2[j]);
        gh[j] = __builtin_fmaf(a2, hh, __builtin_fmaf(fabsf(r2), w2[j], gh[j]));
      }
      if constexpr (!kHold) put(kept_w2, k, dw2);
      if (c < C && p.dx != nullptr) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = gh[j] * p.res_scale;
        store8<R, S, PAST>(row_of<R>(p.dx, t, p.dx_s), c, C, x);
      }
      // (where the longest rows' types differ no register is left to wait with it: read again)
      if constexpr (!kHold && sizeof(E) != sizeof(R)) columns_of(k, w2, gw);
      float* u = u1[kHold ? k : 0];
      float y[8];
      y_of(k, y);
      if (__builtin_expect(apart1, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= far_power(r1);
      }
      if (tokens) {
        float g[8], d[8];
        load8<E, S>(gate, c, C, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float yy = y[j] * fabsf(r1), v = gh[j] * gw[j];
          d[j] = v * yy;
          u[j] = v * g[j];
          sum_t[k][j] = __builtin_fmaf(gh[j] * g[j], yy, sum_t[k][j]);
          dot[0] = __builtin_fmaf(u[j], yy, dot[0]);
        }
        if (c < C && p.dgate != nullptr)
          store8<E, S, PAST>(row_of<E>(p.dgate, t, p.dgate_s), c, C, d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float yy = y[j] * fabsf(r1);
          u[j] = gh[j] * gw[j];
          sum_t[k][j] = __builtin_fmaf(gh[j], yy, sum_t[k][j]);
          dot[0] = __builtin_fmaf(u[j], yy, dot[0]);
        }
      }
      if constexpr (!kHold) put(kept, k, u);
      apart();
    }
    Vec8<E> next_y[CH];
    if constexpr (kAhead) fetch(t0 + step, next_y);
    float a1 = 0.f;                              // -r1 mean(u1 yy)
    if (p.dy != nullptr && p.post) {
      row_sums<NT, 1>(s[NT > 64 ? row : 0], turn, dot);
      a1 = -fabsf(r1) * (dot[0] * inv_c * far_power(r1));
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = column<S, NT>(tid, k);
      if (c >= C || p.dy == nullptr) continue;
      float* u = u1[kHold ? k : 0];
      if constexpr (!kHold) take(kept, k, u);
      if (p.post) {
        float y[8];
        y_of(k, y);
        if (__builtin_expect(apart1, 0)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[j] *= far_power(r1);
            u[j] *= far_power(r1);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = __builtin_fmaf(a1, y[j] * fabsf(r1), fabsf(r1) * u[j]);
      }
      store8<E, S, PAST>(row_of<E>(p.dy, t, p.dy_s), c, C, u);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int k = 0; k < CH; ++k) raw.y[k] = next_y[k];
    }
  }
  if (p.part == nullptr) return;
  // the parts of post_w's, the gate's and pre_w's gradient
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = column<S, NT>(tid, k);
    float w1[8], w2[8], g[8];
    weights(k, w1, w2, g);
    float* dw2 = sum_w2[kHold ? k : 0];
    if constexpr (!kHold) take(kept_w2, k, dw2);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (!p.want[q]) continue;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = q == 0 ? sum_t[k][j] * g[j]
               : q == 1 ? sum_t[k][j] * (p.branch_scale * w1[j]) : dw2[j];
      float* out = p.part + (static_cast<int64_t>(q) * gridDim.x + blockIdx.x) * p.C;
      if constexpr (kRows == 1) {
        store8<float, S>(out, c, p.C, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          fold[row][column<S, NT>(tid, 0) + j + (S && j >= 4 ? kHalf - 4 : 0)] = x[j];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * 8; i += kBwdThreads<NT>) {
          const int at = 8 * k * NT + i;
          float v = 0.f;
#pragma unroll
          for (int r = 0; r < kRows; ++r) v += fold[r][i];
          if (at < p.C) out[at] = v;
        }
        __syncthreads();
      }
    }
  }
}

// The workgroups' parts in order: 64 columns of one gradient (blockIdx.y: which) to a
// workgroup, every 16th part to a wave.
template <typename E>
__global__ __launch_bounds__(1024) void block_norm_fold_kernel(const float* part, int groups, int C,
                                                               void* dpost_w, void* dgate,
                                                               void* dpre_w) {
  __shared__ float sum[16][64];
  void* out = blockIdx.y == 0 ? dpost_w : blockIdx.y == 1 ? dgate : dpre_w;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  part += static_cast<int64_t>(blockIdx.y) * groups * C;
  float x = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) x += part[static_cast<int64_t>(g) * C + c];
  }
  sum[wave][lane] = x;
  __syncthreads();
  if (wave == 0 && c < C) {
    x = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) x += sum[w][lane];
    static_cast<E*>(out)[c] = static_cast<E>(x);
  }
}

namespace {

BlockParams block_params(const zero_block_norm_args& a) {
  BlockParams p = {};
  p.T = a.T;
  p.C = a.C;
  p.post = a.post_norm;
  p.gate_tokens = a.gate_tokens;
  p.has_post_w = a.post_w != nullptr;
  p.has_pre_w = a.pre_w != nullptr;
  p.eps = static_cast<float>(a.eps);
  p.offset = static_cast<float>(a.weight_offset);
  p.res_scale = static_cast<float>(a.res_scale);
  p.branch_scale = static_cast<float>(a.branch_scale);
  p.x = a.x;
  p.y = a.y;
  p.post_w = a.post_w;
  p.gate = a.gate;
  p.pre_w = a.pre_w;
  p.h = a.h;
  p.z = a.z;
  p.dh = a.dh;
  p.dz = a.dz;
  p.dx = a.dx;
  p.dy = a.dy;
  p.x_s = a.x_stride;
  p.y_s = a.y_stride;
  p.gate_s = a.gate_stride;
  p.h_s = a.h_stride;
  p.z_s = a.z_stride;
  p.dh_s = a.dh_stride;
  p.dz_s = a.dz_stride;
  p.dx_s = a.dx_stride;
  p.dy_s = a.dy_stride;
  p.dgate_s = a.dgate_stride;
  return p;
}

int rows_of(int C) { return C <= 1024 ? 4 : C <= 2048 ? 2 : 1; }

int bwd_groups(int64_t T, int C) {
  const int64_t n = (T + rows_of(C) - 1) / rows_of(C);
  const int64_t wanted = std::max<int64_t>(T / 4, std::min<int64_t>(n, kBlockBwdFew));
  return static_cast<int>(
      std::min({wanted, n, static_cast<int64_t>(C > 4096 ? kBlockBwdLarge : kBlockBwdGroups)}));
}

// From here on outputs go past the caches, which do not hold them until they are read.  (T x 4096 bf16,
// us, with both outputs' readers behind it: T = 16384 forward 171 instead of 191, backward 229 instead of 243;
// 12288, 192 MiB, 131 and 131, 174 and 179; 8192 92 instead of 86, 122 instead of 113.  The gradient of a
// gate by token does not count: with its reader too, backward at 8192, 10240 and 11264, 192 to 264 MiB of all three,
// past them 234, 280 and 304, through them 204, 269 and 298.)
constexpr int64_t kPastBytes = int64_t(192) << 20;

template <typename E, typename R, int NT, int CH>
void run_bwd(const BlockParams& p, hipStream_t s) {
  const int64_t bytes = (p.dx ? sizeof(R) : 0) + (p.dy ? sizeof(E) : 0);
  const auto fn = p.T * p.C * bytes >= kPastBytes ? block_norm_bwd_kernel<E, R, NT, CH, true>
                                                  : block_norm_bwd_kernel<E, R, NT, CH, false>;
  fn<<<bwd_groups(p.T, p.C), kBwdThreads<NT>, 0, s>>>(p);
}

template <typename E, typename R, int NT, int CH>
void run_fwd(const BlockParams& p, hipStream_t s) {
  constexpr int kThreads = NT < 256 ? 256 : NT, kRows = kThreads / NT;
  const int64_t bytes = (p.h ? sizeof(R) : 0) + (p.z ? sizeof(E) : 0);
  const auto fn = p.T * p.C * bytes >= kPastBytes ? block_norm_fwd_kernel<E, R, NT, CH, true>
                                                  : block_norm_fwd_kernel<E, R, NT, CH, false>;
  fn<<<static_cast<unsigned>((p.T + kRows - 1) / kRows), kThreads, 0, s>>>(p);
}

// By the row's length: forward the fewest threads that hold it with 16 values each (16384 x 4096: 98
// us, 8 values each 101, 32 each 107), backward with 8 (8192 x 4096: 84, 16 each 88; 4097 x 1000: 26,
// a wave with 16 each 28).
template <typename E, typename R>
hipError_t pick_block(const BlockParams& p, bool fwd, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  if (fwd) {
    if (p.C <= 512) run_fwd<E, R, 64, 1>(p, s);
    else if (p.C <= 1024) run_fwd<E, R, 64, 2>(p, s);
    else if (p.C <= 2048) run_fwd<E, R, 256, 1>(p, s);
    else if (p.C <= 4096) run_fwd<E, R, 256, 2>(p, s);
    else if (p.C <= 8192) run_fwd<E, R, 512, 2>(p, s);
    else run_fwd<E, R, 1024, 2>(p, s);
  } else {
    if (p.C <= 512) run_bwd<E, R, 64, 1>(p, s);
    else if (p.C <= 1024) run_bwd<E, R, 128, 1>(p, s);
    else if (p.C <= 2048) run_bwd<E, R, 256, 1>(p, s);
    else if (p.C <= 4096) run_bwd<E, R, 512, 1>(p, s);
    else if (p.C <= 8192) run_bwd<E, R, 1024, 1>(p, s);
    else run_bwd<E, R, 1024, 2>(p, s);
  }
  return hipGetLastError();
}

hipError_t pick_types(const zero_block_norm_args& a, const BlockParams& p, bool fwd,
                      hipStream_t s) {
  if (a.dtype == ZERO_F32) return pick_block<float, float>(p, fwd, s);
  return a.res_dtype == ZERO_F32 ? pick_block<bf16, float>(p, fwd, s)
                                 : pick_block<bf16, bf16>(p, fwd, s);
}

}  // namespace

size_t block_norm_workspace(int64_t T, int C) {
  return static_cast<size_t>(bwd_groups(T, C)) * 3 * C * sizeof(float);
}

hipError_t launch_block_norm_fwd(const zero_block_norm_args& a, hipStream_t s) {
  return pick_types(a, block_params(a), true, s);
}

hipError_t launch_block_norm_bwd(const zero_block_norm_args& a, hipStream_t s) {
  BlockParams p = block_params(a);
  void* shared_gate = a.gate_tokens ? nullptr : a.dgate;
  p.dgate = a.gate_tokens ? a.dgate : nullptr;
  p.want[0] = a.dpost_w != nullptr;
  p.want[1] = shared_gate != nullptr;
  p.want[2] = a.dpre_w != nullptr;
  const bool sums = p.want[0] || p.want[1] || p.want[2];
  p.part = sums ? static_cast<float*>(a.workspace) : nullptr;
  const hipError_t e = pick_types(a, p, false, s);
  if (e != hipSuccess || !sums) return e;
  const dim3 grid((a.C + 63) / 64, 3);
  const int groups = bwd_groups(a.T, a.C);
  if (a.dtype == ZERO_BF16)
    block_norm_fold_kernel<bf16>
        <<<grid, 1024, 0, s>>>(p.part, groups, a.C, a.dpost_w, shared_gate, a.dpre_w);
  else
    block_norm_fold_kernel<float>
        <<<grid, 1024, 0, s>>>(p.part, groups, a.C, a.dpost_w, shared_gate, a.dpre_w);
  return hipGetLastError();
}

}  // namespace zo
