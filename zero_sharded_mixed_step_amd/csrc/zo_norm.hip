// zo_norm.hip -- the RMS norm of query and key heads and the position
// rotation in one pass over the heads, forward and backward.
//
// Both are bound by memory: a row of D values is read once, kept in registers
// across the reduction, and written once.  A wave owns a token: G lanes share a
// head's row, 8 values each, so 64 / G heads are under way at a time, and the
// token's sines and cosines, formed once by the wave in binary64, serve all of
// its heads from registers.
#include "zo_device.h"
#include "zo_internal.h"

namespace zo {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;
constexpr int kMaxPairs = 128;
// Workgroups of the backward pass: each leaves one row of weight-gradient
// parts, which the fold kernel has to read again.
constexpr int kNormBwdGroups = 1024;

struct NormHeads {
  const void *x, *w, *dy;
  void *y, *dx;
  int H;
  int64_t x_t, x_h, y_t, y_h, dy_t, dy_h, dx_t, dx_h;
};

struct NormParams {
  NormHeads t[2];  // queries, keys
  const int32_t* pos;
  const double* inv_freq;
  int64_t T;
  int D, rot, interleaved;
  float eps;
  float* part;  // backward: [groups][2][D]
};

template <typename E>
struct Vec8;
template <>
struct Vec8<bf16> {
  u32x4 r;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    r = *reinterpret_cast<const u32x4*>(static_cast<const bf16*>(p) + at);
  }
  __device__ __forceinline__ void get(float x[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16_bits_to_f32(r[j]);
      x[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static void store(void* p, int64_t at, const float x[8]) {
    bf16x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<bf16>(x[j]);
    *reinterpret_cast<bf16x8*>(static_cast<bf16*>(p) + at) = v;
  }
};
template <>
struct Vec8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void get(float x[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[4 + j] = b[j];
    }
  }
  __device__ __forceinline__ static void store(void* p, int64_t at, const float x[8]) {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    q[0] = f32x4{x[0], x[1], x[2], x[3]};
    q[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
};

// What a lane needs to turn its 8 values: cosines, signed sines (of its own
// member of each pair), and where the other members are.
struct Turn {
  float c[8], s[8];
  int lane_step;     // pairs half a rotation apart: the partner's lane, relative
  bool interleaved;  // pairs inside the lane

  // out = x cos + partner * signed sin, with sign -1 for the way back
  template <bool BACK>
  __device__ __forceinline__ void apply(const float x[8], float y[8], int lane) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float other = interleaved ? x[j ^ 1] : __shfl(x[j], lane + lane_step);
      y[j] = __builtin_fmaf(BACK ? -s[j] : s[j], other, x[j] * c[j]);
    }
  }
};

// Sine and cosine of the token's angles, by the wave, then each lane's share.
__device__ __forceinline__ void make_turn(const NormParams& p, int64_t t, int lane, int chunk,
                                          float* cs, Turn& turn) {
  const int pairs = p.rot / 2;
  if (pairs > 0 && t < p.T) {
    const double at = static_cast<double>(p.pos[t]) * 0.15915494309189535;  // 1 / 2 pi
    for (int i = lane; i < pairs; i += 64) {
      const double rev = at * p.inv_freq[i];
      float s, c;
      sincospif(2.f * static_cast<float>(rev - rint(rev)), &s, &c);
      cs[i] = c;
      cs[kMaxPairs + i] = s;
    }
  }
  __syncthreads();
  const int d0 = 8 * chunk;
  turn.interleaved = p.interleaved || pairs == 0;
  turn.lane_step = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    turn.c[j] = 1.f;
    turn.s[j] = 0.f;
  }
  if (d0 < p.rot) {
    if (p.interleaved) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        turn.c[j] = cs[(d0 + j) / 2];
        const float s = cs[kMaxPairs + (d0 + j) / 2];
        turn.s[j] = j & 1 ? s : -s;
      }
    } else {
      const bool second = d0 >= pairs;
      turn.lane_step = second ? -pairs / 8 : pairs / 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = d0 + j - (second ? pairs : 0);
        turn.c[j] = cs[i];
        turn.s[j] = second ? cs[kMaxPairs + i] : -cs[kMaxPairs + i];
      }
    }
  }
}

template <int G>
__device__ __forceinline__ float sum_row(float x) {
  return join_lanes<G>(x, AddOp());
}

template <typename E>
__device__ __forceinline__ void load_weight(const void* w, int at, bool active, float out[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = 1.f;
  if (w != nullptr && active) {
    Vec8<E> v;
    v.load(w, at);
    v.get(out);
  }
}

template <typename E, int G>
__global__ __launch_bounds__(kNormThreads) void norm_fwd_kernel(const NormParams p) {
  constexpr int kHeads = 64 / G, kU = 2;  // heads at a time, times two in flight
  __shared__ float cs[kNormWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = lane % G, sub = lane / G;
  const bool active = 8 * chunk < p.D;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kNormWaves + wave;
  Turn turn;
  make_turn(p, t, lane, chunk, cs[wave], turn);
  if (t >= p.T) return;
  const float inv_d = 1.f / static_cast<float>(p.D);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const NormHeads& a = p.t[which];
    float w[8];
    load_weight<E>(a.w, 8 * chunk, active, w);
    for (int h0 = 0; h0 < a.H; h0 += kHeads * kU) {
      Vec8<E> raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * kHeads + sub;
        raw[u] = Vec8<E>{};
        if (h < a.H && active) raw[u].load(a.x, t * a.x_t + h * a.x_h + 8 * chunk);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * kHeads + sub;
        float x[8], y[8], sq = 0.f;
        raw[u].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(x[j], x[j], sq);
        sq = sum_row<G>(sq);
        const float r = 1.f / sqrtf(__builtin_fmaf(sq, inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
        turn.apply<false>(x, y, lane);
        if (h < a.H && active) Vec8<E>::store(a.y, t * a.y_t + h * a.y_h + 8 * chunk, y);
      }
    }
  }
}

template <typename E, int G>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(const NormParams p) {
  constexpr int kHeads = 64 / G;
  __shared__ float cs[kNormWaves][2 * kMaxPairs];
  __shared__ float fold[kNormWaves][2][8 * G];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = lane % G, sub = lane / G;
  const bool active = 8 * chunk < p.D;
  const float inv_d = 1.f / static_cast<float>(p.D);
  float w[2][8], dw[2][8];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    load_weight<E>(p.t[which].w, 8 * chunk, active, w[which]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[which][j] = 0.f;
  }
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kNormWaves; t0 < p.T;
       t0 += static_cast<int64_t>(gridDim.x) * kNormWaves) {
    const int64_t t = t0 + wave;
    Turn turn;
    make_turn(p, t, lane, chunk, cs[wave], turn);
    if (t < p.T) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const NormHeads& a = p.t[which];
        for (int h0 = 0; h0 < a.H; h0 += kHeads) {
          const int h = h0 + sub;
          const bool on = h < a.H && active;
          Vec8<E> rx{}, rg{};
          if (on) {
            rx.load(a.x, t * a.x_t + h * a.x_h + 8 * chunk);
            rg.load(a.dy, t * a.dy_t + h * a.dy_h + 8 * chunk);
          }
          float x[8], g[8], u[8], sq = 0.f, ux = 0.f;
          rx.get(x);
          rg.get(u);
          turn.apply<true>(u, g, lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sq = __builtin_fmaf(x[j], x[j], sq);
            u[j] = g[j] * w[which][j];
            ux = __builtin_fmaf(u[j], x[j], ux);
          }
          sq = sum_row<G>(sq);
          ux = sum_row<G>(ux);
          const float r = 1.f / sqrtf(__builtin_fmaf(sq, inv_d, p.eps));
          const float k = ux * inv_d * r * r;             // mean(u xhat) r
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (on) dw[which][j] = __builtin_fmaf(g[j], x[j] * r, dw[which][j]);
            u[j] = r * __builtin_fmaf(-k, x[j], u[j]);
          }
          if (on) Vec8<E>::store(a.dx, t * a.dx_t + h * a.dx_h + 8 * chunk, u);
        }
      }
    }
    __syncthreads();                                      // before the next token's angles
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = dw[which][j];
#pragma unroll
      for (int d = G; d < 64; d <<= 1) x += __shfl_xor(x, d);
      if (sub == 0) fold[wave][which][8 * chunk + j] = x;
    }
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * p.D; k += kNormThreads) {
    const int which = k >= p.D, d = k - which * p.D;
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kNormWaves; ++v) x += fold[v][which][d];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * p.D + k] = x;
  }
}

// dw: the workgroups' parts, 8 columns to a workgroup.
template <typename E>
__global__ __launch_bounds__(256) void norm_fold_kernel(const float* part, int groups, int D,
                                                        void* dwq, void* dwk) {
  __shared__ float sum[32][9];
  const int col = threadIdx.x % 8, r0 = threadIdx.x / 8, k = blockIdx.x * 8 + col;
  float x = 0.f;
  for (int r = r0; r < groups; r += 32) x += part[static_cast<int64_t>(r) * 2 * D + k];
  sum[r0][col] = x;
  __syncthreads();
  if (threadIdx.x < 8) {
    x = 0.f;
    for (int r = 0; r < 32; ++r) x += sum[r][col];
    void* out = k < D ? dwq : dwk;
    if (out != nullptr) static_cast<E*>(out)[k % D] = static_cast<E>(x);
  }
}

namespace {

NormParams norm_params(const zero_qk_norm_rope_args& a) {
  NormParams p = {};
  const auto heads = [](const void* x, const void* w, void* y, const void* dy, void* dx, int H,
                        const int64_t* xs, const int64_t* ys, const int64_t* dys,
                        const int64_t* dxs) {
    return NormHeads{x, w, dy, y, dx, H, xs[0], xs[1], ys[0], ys[1], dys[0], dys[1], dxs[0], dxs[1]};
  };
  p.t[0] = heads(a.q, a.wq, a.yq, a.dyq, a.dq, a.Hq, a.q_stride, a.yq_stride, a.dyq_stride,
                 a.dq_stride);
  p.t[1] = heads(a.k, a.wk, a.yk, a.dyk, a.dk, a.Hk, a.k_stride, a.yk_stride, a.dyk_stride,
                 a.dk_stride);
  p.pos = a.pos;
  p.inv_freq = a.inv_freq;
  p.T = a.T;
  p.D = a.D;
  p.rot = a.rot_dim;
  p.interleaved = a.interleaved;
  p.eps = static_cast<float>(a.eps);
  return p;
}

int bwd_groups(int64_t T) {
  const int64_t n = (T + kNormWaves - 1) / kNormWaves;
  return static_cast<int>(n < kNormBwdGroups ? n : kNormBwdGroups);
}

template <typename E, int G>
hipError_t run_norm(const NormParams& p, bool fwd, hipStream_t s) {
  if (fwd) {
    const unsigned grid = static_cast<unsigned>((p.T + kNormWaves - 1) / kNormWaves);
    norm_fwd_kernel<E, G><<<grid, kNormThreads, 0, s>>>(p);
  } else if (p.T > 0) {
    norm_bwd_kernel<E, G><<<bwd_groups(p.T), kNormThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t pick_norm(const NormParams& p, bool fwd, hipStream_t s) {
  if (p.D <= 32) return run_norm<E, 4>(p, fwd, s);
  if (p.D <= 64) return run_norm<E, 8>(p, fwd, s);
  if (p.D <= 128) return run_norm<E, 16>(p, fwd, s);
  return run_norm<E, 32>(p, fwd, s);
}

}  // namespace

size_t qk_norm_rope_workspace(int64_t T, int D) {
  return static_cast<size_t>(bwd_groups(T)) * 2 * D * sizeof(float);
}

hipError_t launch_qk_norm_rope_fwd(const zero_qk_norm_rope_args& a, hipStream_t s) {
  const NormParams p = norm_params(a);
  return a.dtype == ZERO_BF16 ? pick_norm<bf16>(p, true, s) : pick_norm<float>(p, true, s);
}

hipError_t launch_qk_norm_rope_bwd(const zero_qk_norm_rope_args& a, hipStream_t s) {
  NormParams p = norm_params(a);
  const bool weights = a.dwq != nullptr || a.dwk != nullptr;
  p.part = weights ? static_cast<float*>(a.workspace) : nullptr;
  const hipError_t e =
      a.dtype == ZERO_BF16 ? pick_norm<bf16>(p, false, s) : pick_norm<float>(p, false, s);
  if (e != hipSuccess || !weights) return e;
  const unsigned grid = 2 * a.D / 8;
  if (a.dtype == ZERO_BF16)
    norm_fold_kernel<bf16><<<grid, 256, 0, s>>>(p.part, bwd_groups(a.T), a.D, a.dwq, a.dwk);
  else
    norm_fold_kernel<float><<<grid, 256, 0, s>>>(p.part, bwd_groups(a.T), a.D, a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace zo
