// zo_block_norm.hip -- the norm of a block's output, its gate, the residual sum
// and the next block's norm in one pass, forward and backward.
//
// Bound by memory: every row is read once, kept in registers across its norms'
// sums, and written once.  A row belongs to a wave where it has at most 1024 values (no
// barrier), to a workgroup beyond.  Backward, workgroups walk the rows and keep the
// sums of the weights' and the gate's gradients for their own columns in registers; each
// leaves them in a row of the workspace, which a second kernel folds in order.
#include "zo_device.h"
#include "zo_internal.h"
#include "zo_rows.h"

namespace zo {

// Workgroups of the backward pass at most, each of which leaves a row of parts for
// every gradient that is summed over the tokens.
constexpr int kBlockBwdGroups = 512;

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
// power of 2.  The same in all threads of the row.
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
  if (far_mean(ms)) {
    const float s = ms < 1.f ? 0x1p100f : 0x1p-100f;
    sq = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[k][j] * s, v[k][j] * s, sq);
    r = s * __builtin_amdgcn_rsqf(__builtin_fmaf(sum(sq), inv_c, eps * s * s));
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

template <typename E>
__device__ __forceinline__ void load8(const void* p, int64_t at, float x[8]) {
  Vec8<E> v;
  v.load(p, at);
  v.get(x);
}

// A weight plus its offset, or 1 where there is none.
template <typename E>
__device__ __forceinline__ void weight8(const void* w, int has, float offset, int at, float x[8]) {
  if (has) {
    load8<E>(w, at, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] += offset;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 1.f;
  }
}

// branch_scale times the gate, `gate` its row or NULL.
template <typename E>
__device__ __forceinline__ void gate8(const BlockParams& p, const char* gate, int at, float g[8]) {
  if (p.gate != nullptr) {
    load8<E>(gate, at, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= p.branch_scale;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = p.branch_scale;
  }
}

// NT threads to a row, CH pieces of 8 values to a thread.
template <typename E, typename R, int NT, int CH>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_fwd_kernel(const BlockParams p) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
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
    const int c = 8 * (tid + k * NT);
    on[k] = c < p.C;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[k][j] = y[k][j] = 0.f;
    if (on[k]) {
      load8<R>(row_of<R>(p.x, t, p.x_s), c, h[k]);
      if (p.y != nullptr) load8<E>(row_of<E>(p.y, t, p.y_s), c, y[k]);
    }
  }
  if (p.y != nullptr) {
    const float r = p.post ? inverse_rms<NT, CH>(sum, y, inv_c, p.eps) : 1.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * (tid + k * NT);
      if (!on[k]) continue;
      float w[8], g[8];
      weight8<E>(p.post_w, p.has_post_w, p.offset, c, w);
      gate8<E>(p, gate, c, g);
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
      if (on[k]) Vec8<R>::store(row_of<R>(p.h, t, p.h_s), 8 * (tid + k * NT), h[k]);
  }
  if (p.z == nullptr) return;
  const float r = inverse_rms<NT, CH>(sum, h, inv_c, p.eps);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = 8 * (tid + k * NT);
    if (!on[k]) continue;
    float w[8];
    weight8<E>(p.pre_w, p.has_pre_w, p.offset, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[k][j] = h[k][j] * r * w[j];
    Vec8<E>::store(row_of<E>(p.z, t, p.z_s), c, h[k]);
  }
}

// Several sums over a row's threads at once: one barrier for all of them.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float* s, int& turn, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = join_lanes<64>(x[i], AddOp());
  if constexpr (NT > 64) {
    constexpr int kW = NT / 64;
    float* at = s + turn * (3 * kW);
    turn ^= 1;
    const int lane = threadIdx.x & 63;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) at[i * kW + (threadIdx.x >> 6)] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = join_lanes<kW>(at[i * kW + lane % kW], AddOp());
  }
}

// What the row's first sums leave of a norm: r = 1 / sqrt(ms) and mean(u v) r, of values
// scaled by s where ms is past binary32's ends.
template <int NT, int CH, typename U, typename V>
__device__ __forceinline__ void far_norm(float* s, int& turn, float ms, float inv_c, float eps,
                                         float& r, float& m, U u, V v) {
  const float f = ms < 1.f ? 0x1p100f : 0x1p-100f;
  float x[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float a[8], b[8];
    u(k, a);
    v(k, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[0] = __builtin_fmaf(b[j] * f, b[j] * f, x[0]);
      x[1] = __builtin_fmaf(a[j], b[j] * f, x[1]);
    }
  }
  row_sums<NT, 2>(s, turn, x);
  const float rf = __builtin_amdgcn_rsqf(__builtin_fmaf(x[0], inv_c, eps * f * f));
  r = f * rf;
  m = x[1] * inv_c * rf;
}

// Two barriers a row: h's and y's squares and u2 . h are summed first, u1 . y when
// gh is known.  What a row's loads fetched stays packed in registers, and is widened
// again for each use.
template <typename E, typename R, int NT, int CH>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_bwd_kernel(const BlockParams p) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  __shared__ float s[6 * NT / 64];
  __shared__ float fold[kRows > 1 ? kRows : 1][kRows > 1 ? NT * CH * 8 : 1];
  // 16 waves to a unit leave each 128 registers: two pieces of the longest rows are not
  // held from use to use but read again, and worked on one after the other; u1 waits in
  // shared memory.
  constexpr bool kHold = NT < 1024 || CH == 1;
  constexpr int kHeld = kHold ? CH : 1;
  __shared__ f32x4 kept[kHold ? 1 : 2 * CH][kHold ? 1 : NT];
  const auto apart = [] {
    if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);
  };
  int turn = 0;
  const int tid = threadIdx.x % NT, row = uniform(threadIdx.x / NT);
  const float inv_c = 1.f / static_cast<float>(p.C);
  float dw1[CH][8], dg[CH][8], dw2[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw1[k][j] = dg[k][j] = dw2[k][j] = 0.f;
  const bool use_y = p.y != nullptr && (p.post || p.gate != nullptr);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + row; t < p.T; t += step) {
    const char *at_dh = row_of<R>(p.dh, t, p.dh_s), *at_h = row_of<R>(p.h, t, p.h_s);
    const char *at_dz = row_of<E>(p.dz, t, p.dz_s), *at_y = row_of<E>(p.y, t, p.y_s);
    const char* gate = row_of<E>(p.gate, p.gate_tokens ? t : 0, p.gate_s);
    const char *post_w = row_of<E>(p.post_w, 0, 0), *pre_w = row_of<E>(p.pre_w, 0, 0);
    Vec8<R> raw_dh[kHeld], raw_h[kHeld];
    Vec8<E> raw_dz[kHeld], raw_y[kHeld];
    const auto fetch = [&](auto& raw, bool wanted, const char* at, int k) {
      const int c = 8 * (tid + k * NT);
      raw = {};
      if (wanted && c < p.C) raw.load(at, c);
    };
    const auto widen = [&](auto& raws, bool wanted, const char* at, int k, float x[8]) {
      if constexpr (!kHold) fetch(raws[0], wanted, at, k);
      raws[kHold ? k : 0].get(x);
    };
    const bool use_z = p.dz != nullptr;
    const auto dh_of = [&](int k, float x[8]) { widen(raw_dh, p.dh != nullptr, at_dh, k, x); };
    const auto h_of = [&](int k, float x[8]) { widen(raw_h, use_z, at_h, k, x); };
    const auto dz_of = [&](int k, float x[8]) { widen(raw_dz, use_z, at_dz, k, x); };
    const auto y_of = [&](int k, float x[8]) { widen(raw_y, use_y, at_y, k, x); };
    float sums[3] = {0.f, 0.f, 0.f};             // h^2, u2 h, y^2
    const auto u2_of = [&](int k, float x[8]) {
      float w[8];
      const int c = 8 * (tid + k * NT);
      dz_of(k, x);
      if (c < p.C && p.has_pre_w) {
        load8<E>(pre_w, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= w[j] + p.offset;
      }
    };
    if constexpr (kHold) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        fetch(raw_h[k], use_z, at_h, k);
        fetch(raw_dz[k], use_z, at_dz, k);
        fetch(raw_y[k], use_y, at_y, k);
        fetch(raw_dh[k], p.dh != nullptr, at_dh, k);
      }
    }
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
    row_sums<NT, 3>(s, turn, sums);
    const float ms2 = __builtin_fmaf(sums[0], inv_c, p.eps);
    const float ms1 = __builtin_fmaf(sums[2], inv_c, p.eps);
    float r2 = __builtin_amdgcn_rsqf(ms2), r1 = __builtin_amdgcn_rsqf(ms1);
    float m2 = sums[1] * inv_c * r2;             // mean(u2 hh)
    if (use_z && far_mean(ms2))
      far_norm<NT, CH>(s, turn, ms2, inv_c, p.eps, r2, m2, u2_of, h_of);
    if (!p.post) {
      r1 = 1.f;
    } else if (far_mean(ms1)) {
      float none;
      far_norm<NT, CH>(s, turn, ms1, inv_c, p.eps, r1, none, y_of, y_of);
    }
    float u1[kHeld][8], dot[1] = {0.f};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * (tid + k * NT);
      float gh[8];
      dh_of(k, gh);
      if (use_z) {
        float h[8], u[8], z[8];
        h_of(k, h);
        u2_of(k, u);
        dz_of(k, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hh = h[j] * r2;
          dw2[k][j] = __builtin_fmaf(z[j], hh, dw2[k][j]);
          gh[j] = __builtin_fmaf(r2, __builtin_fmaf(-m2, hh, u[j]), gh[j]);
        }
      }
      if (c < p.C && p.dx != nullptr) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = gh[j] * p.res_scale;
        Vec8<R>::store(row_of<R>(p.dx, t, p.dx_s), c, x);
      }
      float* u = u1[kHold ? k : 0];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = 0.f;
      if (c < p.C && p.y != nullptr) {
        float y[8], w[8], g[8];
        y_of(k, y);
        weight8<E>(post_w, p.has_post_w, p.offset, c, w);
        gate8<E>(p, gate, c, g);
        if (p.gate != nullptr) {
          float d[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            d[j] = p.branch_scale * gh[j] * (y[j] * r1 * w[j]);
            dg[k][j] += d[j];
          }
          if (p.dgate != nullptr) Vec8<E>::store(row_of<E>(p.dgate, t, p.dgate_s), c, d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float yy = y[j] * r1, du = gh[j] * g[j];
          dw1[k][j] = __builtin_fmaf(du, yy, dw1[k][j]);
          u[j] = du * w[j];
          dot[0] = __builtin_fmaf(u[j], yy, dot[0]);
        }
      }
      if constexpr (!kHold) {
        kept[2 * k][tid] = f32x4{u[0], u[1], u[2], u[3]};
        kept[2 * k + 1][tid] = f32x4{u[4], u[5], u[6], u[7]};
      }
      apart();
    }
    if (p.dy == nullptr) continue;
    float m1 = 0.f;                              // mean(u1 yy)
    if (p.post) {
      row_sums<NT, 1>(s, turn, dot);
      m1 = dot[0] * inv_c;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * (tid + k * NT);
      if (c >= p.C) continue;
      float* u = u1[kHold ? k : 0];
      if constexpr (!kHold) {
        const f32x4 a = kept[2 * k][tid], b = kept[2 * k + 1][tid];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u[j] = a[j];
          u[4 + j] = b[j];
        }
      }
      if (p.post) {
        float y[8];
        y_of(k, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = r1 * __builtin_fmaf(-m1, y[j] * r1, u[j]);
      }
      Vec8<E>::store(row_of<E>(p.dy, t, p.dy_s), c, u);
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (!p.want[q]) continue;
    float* out = p.part + (static_cast<int64_t>(q) * gridDim.x + blockIdx.x) * p.C;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = 8 * (tid + k * NT);
      const float* x = q == 0 ? dw1[k] : q == 1 ? dg[k] : dw2[k];
      if constexpr (kRows == 1) {
        if (c < p.C) Vec8<float>::store(out, c, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) fold[row][c + j] = x[j];
      }
    }
    if constexpr (kRows > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += 256) {
        float x = 0.f;
#pragma unroll
        for (int v = 0; v < kRows; ++v) x += fold[v][c];
        out[c] = x;
      }
      __syncthreads();
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

int rows_of(int C) { return C <= 1024 ? 4 : 1; }

int bwd_groups(int64_t T, int C) {
  const int64_t n = (T + rows_of(C) - 1) / rows_of(C);
  return static_cast<int>(n < kBlockBwdGroups ? n : kBlockBwdGroups);
}

template <typename E, typename R, int NT, int CH>
void run_bwd(const BlockParams& p, hipStream_t s) {
  block_norm_bwd_kernel<E, R, NT, CH>
      <<<bwd_groups(p.T, p.C), NT < 256 ? 256 : NT, 0, s>>>(p);
}

template <typename E, typename R, int NT, int CH>
void run_fwd(const BlockParams& p, hipStream_t s) {
  constexpr int kThreads = NT < 256 ? 256 : NT, kRows = kThreads / NT;
  block_norm_fwd_kernel<E, R, NT, CH>
      <<<static_cast<unsigned>((p.T + kRows - 1) / kRows), kThreads, 0, s>>>(p);
}

// By the row's length: forward the fewest threads that hold it with 16 values each;
// backward, where 24 sums a piece of 8 values stay in registers too, with 8 each.
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
    else if (p.C <= 1024) run_bwd<E, R, 64, 2>(p, s);
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
