// zo_norm.hip -- the RMS norm of query and key heads and the position
// rotation in one pass over the heads, forward and backward.
//
// Both are bound by memory: a row of D values is read once, kept in registers
// across the reduction, and written once.  A wave owns a token: G lanes share a
// head's row, 8 values each, so 64 / G heads are under way at a time, and the
// token's sines and cosines, formed once by the wave in binary64, serve all of
// its heads from registers.  (A workgroup to a token instead of a wave: 106 us
// instead of 67 for the forward pass of 16384 tokens, as more lanes wait for the angles.)
//
// Measured, 40 heads of 128 in bf16: forward of 16384 tokens 67 us, 5.0 TB/s (fp32: 133 us, 5.0);
// backward of 8192 tokens 60 us, 4.2 TB/s.
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
  float* part;  // backward: [2][groups][D]
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

// The value of the lane half a group of G away.
template <int G>
__device__ __forceinline__ float across(float x) {
  const uint32_t v = __float_as_uint(x);
  if constexpr (G == 4) return __uint_as_float(dpp_move<0x4E>(v));                     // 2 3 0 1
  if constexpr (G == 8) return __uint_as_float(dpp_move<0x1B>(dpp_move<0x141>(v)));    // 8 mirrored, 4 mirrored
  if constexpr (G == 16) return __uint_as_float(dpp_move<0x128>(v));                   // turned by 8
  if constexpr (G == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
  }
}

// What a lane needs to turn its 8 values: cosines, signed sines (of its own
// member of each pair), and where the other members are.
enum class Partner { kInside, kAcross, kLane };  // in the lane; half the group away; lane_step away
struct Turn {
  float c[8], s[8];
  int lane_step;
  Partner partner;

  // out = x cos + partner * signed sin, with sign -1 for the way back
  template <bool BACK, int G>
  __device__ __forceinline__ void apply(const float x[8], float y[8], int lane) const {
    float other[8];
    if (partner == Partner::kInside) {
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = x[j ^ 1];
    } else if (partner == Partner::kAcross) {
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = across<G>(x[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = __shfl(x[j], lane + lane_step);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(BACK ? -s[j] : s[j], other[j], x[j] * c[j]);
  }
};

// Sine and cosine of the token's angles, by the wave, then each lane's share.
template <int G>
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
  turn.partner = p.interleaved || pairs == 0 ? Partner::kInside
                 : p.rot == 8 * G            ? Partner::kAcross
                                             : Partner::kLane;
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

// Whether a row's mean square plus eps is near the ends of binary32 (the reciprocal root takes
// no subnormal numbers): of values below 1e-15 with an eps below 1e-30, or above 1e15.
__device__ __forceinline__ bool far_mean(float v) { return !(v >= 1e-30f && v <= 1e30f); }

// 1 / sqrt(mean(x^2) + eps) of such a row, from x times a power of 2.
template <int G>
__device__ __forceinline__ float far_inverse_rms(const float x[8], float v, float inv_d, float eps) {
  const float s = v < 1.f ? 0x1p100f : 0x1p-100f;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j] * s, x[j] * s, sum);
  return s * __builtin_amdgcn_rsqf(__builtin_fmaf(sum_row<G>(sum), inv_d, eps * s * s));
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
  constexpr int kHeads = 64 / G, kU = 4;  // heads at a time, times four in flight
  __shared__ float cs[kNormWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = lane % G, sub = lane / G;
  const bool active = 8 * chunk < p.D;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kNormWaves + wave;
  Turn turn;
  make_turn<G>(p, t, lane, chunk, cs[wave], turn);
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
        const float ms = __builtin_fmaf(sq, inv_d, p.eps);
        float r = __builtin_amdgcn_rsqf(ms);
        if (__any(h < a.H && far_mean(ms))) {             // (by the wave)
          const float fr = far_inverse_rms<G>(x, ms, inv_d, p.eps);
          r = far_mean(ms) ? fr : r;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
        turn.template apply<false, G>(x, y, lane);
        if (h < a.H && active) Vec8<E>::store(a.y, t * a.y_t + h * a.y_h + 8 * chunk, y);
      }
    }
  }
}

// Queries and keys go to workgroups of their own (blockIdx.y): one weight and one
// row of its gradient to keep.
template <typename E, int G>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(const NormParams p) {
  constexpr int kHeads = 64 / G, kU = 2;
  __shared__ float cs[kNormWaves][2 * kMaxPairs];
  __shared__ float fold[kNormWaves][8 * G];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = lane % G, sub = lane / G;
  const bool active = 8 * chunk < p.D;
  const float inv_d = 1.f / static_cast<float>(p.D);
  const NormHeads& a = p.t[blockIdx.y];
  float w[8], dw[8];
  load_weight<E>(a.w, 8 * chunk, active, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kNormWaves;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kNormWaves; t0 < p.T && a.H > 0; t0 += step) {
    const int64_t t = t0 + wave;
    Turn turn;
    make_turn<G>(p, t, lane, chunk, cs[wave], turn);
    for (int h0 = 0; h0 < a.H && t < p.T; h0 += kHeads * kU) {
      Vec8<E> rx[kU], rg[kU];
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        const int h = h0 + v * kHeads + sub;
        rx[v] = rg[v] = Vec8<E>{};
        if (h < a.H && active) {
          rx[v].load(a.x, t * a.x_t + h * a.x_h + 8 * chunk);
          rg[v].load(a.dy, t * a.dy_t + h * a.dy_h + 8 * chunk);
        }
      }
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        const int h = h0 + v * kHeads + sub;
        const bool on = h < a.H && active;
        float x[8], g[8], u[8], sq = 0.f, ux = 0.f;
        rx[v].get(x);
        rg[v].get(u);
        turn.template apply<true, G>(u, g, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sq = __builtin_fmaf(x[j], x[j], sq);
          u[j] = g[j] * w[j];
          ux = __builtin_fmaf(u[j], x[j], ux);
        }
        sq = sum_row<G>(sq);
        ux = sum_row<G>(ux);
        const float ms = __builtin_fmaf(sq, inv_d, p.eps);
        float r = __builtin_amdgcn_rsqf(ms);
        float k = ux * inv_d * r * r;                     // mean(u xhat) r
        if (__any(h < a.H && far_mean(ms))) {             // (by the wave)
          const float fr = far_inverse_rms<G>(x, ms, inv_d, p.eps);
          float t = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) t = __builtin_fmaf(u[j], x[j] * fr, t);
          t = sum_row<G>(t);
          r = far_mean(ms) ? fr : r;
          k = far_mean(ms) ? t * inv_d * fr : k;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (on) dw[j] = __builtin_fmaf(g[j], x[j] * r, dw[j]);
          u[j] = r * __builtin_fmaf(-k, x[j], u[j]);
        }
        if (on) Vec8<E>::store(a.dx, t * a.dx_t + h * a.dx_h + 8 * chunk, u);
      }
    }
    __syncthreads();                                      // before the next token's angles
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float x = dw[j];
#pragma unroll
    for (int d = G; d < 64; d <<= 1) x += __shfl_xor(x, d);
    if (sub == 0) fold[wave][8 * chunk + j] = x;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kNormWaves; ++v) x += fold[v][d];
    p.part[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * p.D + d] = x;
  }
}

// dw: the workgroups' parts, 8 columns of one weight to a workgroup (blockIdx.y:
// which), 128 threads to a column.
template <typename E>
__global__ __launch_bounds__(1024) void norm_fold_kernel(const float* part, int groups, int D,
                                                         void* dwq, void* dwk) {
  __shared__ float sum[16][8];
  const int lane = threadIdx.x & 63, col = lane % 8, d = blockIdx.x * 8 + col;
  part += static_cast<int64_t>(blockIdx.y) * groups * D + d;
  float x = 0.f;
#pragma unroll 8
  for (int r = threadIdx.x / 8; r < groups; r += 128) x += part[static_cast<int64_t>(r) * D];
#pragma unroll
  for (int k = 8; k < 64; k <<= 1) x += __shfl_xor(x, k);
  if (lane < 8) sum[threadIdx.x / 64][col] = x;
  __syncthreads();
  void* out = blockIdx.y == 0 ? dwq : dwk;
  if (threadIdx.x < 8 && out != nullptr) {
    x = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) x += sum[r][col];
    static_cast<E*>(out)[d] = static_cast<E>(x);
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
    norm_bwd_kernel<E, G><<<dim3(bwd_groups(p.T), 2), kNormThreads, 0, s>>>(p);
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
  const dim3 grid(a.D / 8, 2);
  if (a.dtype == ZERO_BF16)
    norm_fold_kernel<bf16><<<grid, 1024, 0, s>>>(p.part, bwd_groups(a.T), a.D, a.dwq, a.dwk);
  else
    norm_fold_kernel<float><<<grid, 1024, 0, s>>>(p.part, bwd_groups(a.T), a.D, a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace zo
