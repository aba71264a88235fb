// zo_policy.hip -- the clipped policy loss with a KL term, on sampled tokens.
//
// Bound by memory, as the distillation loss: the logits are read once and their
// gradient is written once.  A workgroup owns a row and keeps it in registers (packed
// as it came) between the maximum, the sum and the gradient; of a row too long for that the
// rest is kept in shared memory, and what is beyond that too is read twice, for its maximum and sum
// and for its gradient.  The backward pass needs no row-wide sum, so a row is cut into pieces over
// workgroups.
//
// The sampled token is left out of the sum and added to it in binary64: with rest the sum of
// the others' powers and own its own, lp = -log(1 + rest / own) and 1 - q_a = rest /
// total keep their digits however sure the student is of the token.  What follows from lp
// (ratio, clipping, KL term) is some binary64 operations a row.
//
// The forward's gradient is written past the caches: alone the kernel takes 4 to 20 % less (8192 x 50257
// bf16: 310 us, through them 322; 2048 x 50257: 72, 93), and with the gradient's reader behind it as long
// as before (587 and 587, 162 and 161).
//
// Measured: 8192 x 50257 bf16, the loss alone 187 us, 4.4 TB/s, with the gradient 312 us, 5.3 TB/s of
// logits read and gradient written (350 with the library's logarithms and exponentials in binary64,
// which one thread works on while the row waits; 626 where the gradient's rows start elsewhere between 16
// bytes than the logits'); the backward alone, 1024 x 131072 fp32, 160 to 164 us, 6.6 TB/s (172 with
// loads through the caches).
#include <algorithm>

#include "zo_device.h"
#include "zo_internal.h"
#include "zo_rows.h"

namespace zo {

struct PolicyParams {
  int64_t N, V;
  double inv_tau, low, high, kl_coef, grad_scale;   // low, high: the ratio's borders
  const void* z;
  const int32_t* action;
  const float *adv, *old_lp, *ref_lp, *weight;
  float *loss, *stats;
  void* dz;
  int64_t z_stride, dz_stride;
  int seg, in_place;                                // backward: chunks of a piece
  int kept;                                         // forward: chunks in shared memory
};

// The row's coefficient in the gradient, grad_scale w g / tau, within binary32: where it
// is past its ends a probability of 0 must still give 0.
__device__ __forceinline__ float coefficient(const PolicyParams& p, float w, double g) {
  const double c = p.grad_scale * static_cast<double>(w) * p.inv_tau *
                   (g > -kLowest ? -static_cast<double>(kLowest)
                                 : g < kLowest ? static_cast<double>(kLowest) : g);
  return c > -static_cast<double>(kLowest) ? -kLowest
         : c < static_cast<double>(kLowest) ? kLowest : static_cast<float>(c);
}

// Logarithm and exponential of the row's numbers in binary64 with some 1e-12 of relative error,
// by their series: one thread works on them while the row waits, and the library's, whose
// last digits nobody needs here, take several times the steps.
//
// log(1 + x), -0.3 < x < 0.42, with the relative error kept for small x: 2 artanh(v)
// with v = x / (2 + x), |v| < 0.175.
__device__ __forceinline__ double log_near(double x) {
  const double v = x / (2.0 + x), q = v * v;
  double s = 1.0 / 15;
  s = __builtin_fma(s, q, 1.0 / 13);
  s = __builtin_fma(s, q, 1.0 / 11);
  s = __builtin_fma(s, q, 1.0 / 9);
  s = __builtin_fma(s, q, 1.0 / 7);
  s = __builtin_fma(s, q, 1.0 / 5);
  s = __builtin_fma(s, q, 1.0 / 3);
  return __builtin_fma(s * q, 2.0 * v, 2.0 * v);
}

// log x, 2^-1000 < x < 2^1000.
__device__ __forceinline__ double log_of(double x) {
  const double m = __builtin_amdgcn_frexp_mant(x);
  const bool low = m < 0.70710678118654752;
  const double f = low ? m + m : m;            // in [0.7, 1.42)
  const int k = __builtin_amdgcn_frexp_exp(x) - (low ? 1 : 0);
  return __builtin_fma(static_cast<double>(k), 0.69314718055994531, log_near(f - 1.0));
}

// e^x - 1 - x for x = k log 2 + t: (2^k (1 + t + w) - 1) - x with w = e^t - 1 - t by
// Taylor, |t| < 0.35, and w itself where k is 0.  Also gives e^x.
__device__ __forceinline__ double exp_series(double x, double& beyond) {
  if (!(x > -745.0)) {                         // (a NaN too)
    const double e = x <= -745.0 ? 0.0 : x;
    beyond = e - 1.0 - x;
    return e;
  }
  if (x > 710.0) {
    beyond = __builtin_huge_val();
    return beyond;
  }
  const double k = __builtin_rint(x * 1.4426950408889634);
  const double t = __builtin_fma(-k, 1.9082149292705877e-10,
                                 __builtin_fma(-k, 0.69314718036912382, x));
  double w = 1.0 / 39916800;                   // 1 / 11!
  w = __builtin_fma(w, t, 1.0 / 3628800);
  w = __builtin_fma(w, t, 1.0 / 362880);
  w = __builtin_fma(w, t, 1.0 / 40320);
  w = __builtin_fma(w, t, 1.0 / 5040);
  w = __builtin_fma(w, t, 1.0 / 720);
  w = __builtin_fma(w, t, 1.0 / 120);
  w = __builtin_fma(w, t, 1.0 / 24);
  w = __builtin_fma(w, t, 1.0 / 6);
  w = __builtin_fma(w, t, 0.5);
  w = w * t * t;
  const double e = __builtin_amdgcn_ldexp(1.0 + (t + w), static_cast<int>(k));
  beyond = k == 0.0 ? w : e - 1.0 - x;
  return e;
}

// The lanes' 16 bytes straight to shared memory, lane l's to to[l].
template <typename T>
__device__ __forceinline__ void load_to_lds(T* to, const void* from) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)from,
      (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

struct PolicyRow {
  double loss, g, kl;
};

// Loss (before the row's weight), its derivative by lp, and the KL term.
__device__ __forceinline__ PolicyRow policy_row(const PolicyParams& p, int64_t n, double lp) {
  const double A = p.adv[n];
  double none;
  const double r = p.old_lp != nullptr ? exp_series(lp - static_cast<double>(p.old_lp[n]), none)
                   : lp != lp          ? lp : 1.0;
  const double bound = r < p.low ? p.low : r > p.high ? p.high : r;   // (a NaN stays)
  PolicyRow o;
  const double free_ = r * A, held = bound * A;
  o.loss = -(held < free_ ? held : free_);
  const bool clipped = (A > 0.0 && r > p.high) || (A < 0.0 && r < p.low);
  o.g = clipped ? 0.0 : -free_;
  o.kl = 0.0;
  if (p.ref_lp != nullptr) {
    const double e = static_cast<double>(p.ref_lp[n]) - lp;
    exp_series(e, o.kl);
    o.loss += p.kl_coef * o.kl;
    o.g -= p.kl_coef * (o.kl + e);
  }
  return o;
}

// Where logits over tau log 2 are so far from 0, a row is formed from differences.
constexpr float kFar = 0x1p20f;

// Forward: loss and statistics, and the gradient if asked for.  The row stays in registers, CH
// chunks to a thread.  LONG: what is beyond them stays in shared memory, p.kept chunks, and what is
// beyond those is read once for its maximum and sum together and again for the gradient.
template <typename E, int NT, int CH, bool LONG>
__global__ __launch_bounds__(NT, CH <= 8 ? 8 : 4) void policy_fwd_kernel(const PolicyParams p) {
  constexpr int kN = Chunk<E>::kN, kW = NT / 64;
  using Raw = decltype(Chunk<E>::r);
  extern __shared__ __align__(16) char beyond[];
  Raw* const kept = reinterpret_cast<Raw*>(beyond);
  __shared__ float tops[kW];
  __shared__ double sums[kW];
  __shared__ float row[2];                     // the gradient's coefficient, and 1 / total
  // two of the chunks that the first wave holds, while one of its lanes works on the row's
  // numbers: with 8 there are no registers for both
  constexpr bool kStash = CH == 8;
  __shared__ Raw stash[kStash ? 2 * 64 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int64_t n = blockIdx.x;
  const Row<E> in(p.z, n * p.z_stride, p.V), out(p.dz, n * p.dz_stride, p.V);
  const int chunks = in.chunks();
  const int32_t action = static_cast<int32_t>(uniform(p.action[n]));
  const bool named = action >= 0 && action < p.V;
  const int own_chunk = named ? (action + in.shift) / kN : -1, own_e = (action + in.shift) % kN;
  float own_z = 0.f;
  if (named) own_z = static_cast<float>(in.p[action]);
  const float k2 = static_cast<float>(p.inv_tau * 1.4426950408889634);
  const int kept_end = LONG ? min(chunks, CH * NT + p.kept) : 0;
  if constexpr (LONG) {
    for (int c0 = CH * NT + wave * 64; c0 < kept_end; c0 += NT) {
      const int c = c0 + lane;
      if (c >= kept_end) continue;
      if (in.whole(c))
        load_to_lds(kept + (c0 - CH * NT), in.p + static_cast<int64_t>(c) * kN - in.shift);
      else
        kept[c - CH * NT] = in.load(c).r;
    }
  }
  const auto chunk_max = [&](const Chunk<E>& x, float a) {
#pragma unroll
    for (int e = 0; e < kN; ++e) a = fmaxf(a, x.get(e));
    return a;
  };
  // the powers of a chunk but for the sampled token's
  const auto chunk_sum = [&](const Chunk<E>& x, int c, const auto& power) {
    float s = 0.f;
    if (c == own_chunk) {
#pragma unroll
      for (int e = 0; e < kN; ++e) s += e == own_e ? 0.f : power(x.get(e));
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) s += power(x.get(e));
    }
    return s;
  };
  // exp((z - m) / tau) = 2^(z k2 - m2), with m2 the rounded m k2: the same in every term, and put
  // right in the logarithm of the sum (see base)
  float rest_m = -kInf, rest_m2 = 0.f, rest_sum = 0.f;
  if constexpr (LONG) {
    constexpr int kAtOnce = 4;
    for (int c = kept_end + tid; c < chunks; c += kAtOnce * NT) {
      Chunk<E> x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        x[k].fill_lowest();
        if (c + k * NT < chunks) x[k] = in.load(c + k * NT);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float top = chunk_max(x[k], -kInf);
        if (top > rest_m) {
          // (not of a chunk that is masked by the lowest value alone, whose product may be past
          // binary32; the row of one that is so far above 0 is read again, see far)
          const float m2 = top * k2;
          if (fabsf(m2) <= 2.f * kFar) {
            if (rest_sum > 0.f) rest_sum *= exp2_hw(rest_m2 - m2);
            rest_m2 = m2;
          }
          rest_m = top;
        }
        rest_sum += chunk_sum(x[k], c + k * NT,
                              [&](float z) { return exp2_hw(__builtin_fmaf(z, k2, -rest_m2)); });
      }
    }
  }
  Chunk<E> held[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    held[c].fill_lowest();
    if (tid + c * NT < chunks) held[c] = in.load(tid + c * NT);
  }
  float m = rest_m, sum = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) m = chunk_max(held[c], m);
  const auto each_kept = [&](const auto& f) {    // (a lane reads what its own wave has put there)
    if constexpr (LONG) {
#pragma unroll 1
      for (int c = CH * NT + tid; c < kept_end; c += NT) {
        Chunk<E> x;
        x.r = kept[c - CH * NT];
        f(x, c);
      }
    }
  };
  if constexpr (LONG) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    each_kept([&](const Chunk<E>& x, int) { m = chunk_max(x, m); });
  }
  m = join_lanes<64>(m, MaxOp());
  if (lane == 0) tops[wave] = m;
  __syncthreads();
  m = join_lanes<kW>(tops[lane % kW], MaxOp());
  const bool low = m == -kInf;
  if (low) m = 0.f;                            // nothing but -inf: a sum of 0, not of NaN
  keep_packed(held);
  // Where the rounding of m2 would outweigh the powers (or m k2 is past binary32), they are formed
  // from the difference z - m: such a row is read again.
  const bool far = !(fabsf(m) * k2 <= kFar);
  const float m2 = far ? 0.f : m * k2;
  const auto power = [&](float z) { return exp2_hw(__builtin_fmaf(z, k2, -m2)); };
  const auto power_far = [&](float z) { return exp2_hw((z - m) * k2); };
  if (far) {
#pragma unroll 1
    for (int c = tid; c < chunks; c += NT) sum += chunk_sum(in.load(c), c, power_far);
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (tid + c * NT < chunks) sum += chunk_sum(held[c], tid + c * NT, power);
    each_kept([&](const Chunk<E>& x, int c) { sum += chunk_sum(x, c, power); });
    if constexpr (LONG) sum += rest_sum > 0.f ? rest_sum * exp2_hw(rest_m2 - m2) : rest_sum;
  }
  keep_packed(held);
  const double part = join_lanes<64>(static_cast<double>(sum), AddOp());
  if (lane == 0) sums[wave] = part;
  __syncthreads();
  const double rest = join_lanes<kW>(sums[lane % kW], AddOp());
  const auto row_numbers = [&] {
    const float w = p.weight ? p.weight[n] : 1.f;
    // x / tau less the powers' base: what m2 and k2 were rounded by comes back here
    const double base = static_cast<double>(m) * p.inv_tau +
                        (far ? 0.0 : static_cast<double>(m2) - static_cast<double>(m) * k2) *
                            0.6931471805599453;
    const double x = static_cast<double>(own_z) * p.inv_tau - base;
    double none;
    const double own = named ? exp_series(x, none) : 0.0, total = rest + own;
    PolicyRow o{0.0, 0.0, 0.0};
    double lse = -__builtin_huge_val(), lp = 0.0, others = 1.0, log_total = 0.0;
    const bool empty = low && total == 0.0;    // (a NaN has no part in a maximum, but in the sum)
    const bool live = named && !empty;
    // (the largest logit's power is about 1, so the total is no less; where the token has
    // most of it, lp = -log(1 + rest / own))
    if (!empty) {
      log_total = log_of(total);
      lse = base + log_total;
    }
    if (live) {
      const double q = rest / own;
      lp = q < 0.4 ? -log_near(q) : x - log_total;
      others = rest / total;
      o = policy_row(p, n, lp);
    }
    p.loss[n] = live && w != 0.f ? static_cast<float>(o.loss * static_cast<double>(w)) : 0.f;
    float* stats = p.stats + 4 * n;
    stats[0] = static_cast<float>(lse);
    stats[1] = static_cast<float>(lp);
    stats[2] = static_cast<float>(o.g);
    stats[3] = static_cast<float>(o.kl);
    const float c = w != 0.f ? coefficient(p, w, o.g) : 0.f;
    row[0] = c;
    row[1] = static_cast<float>(1.0 / total);
    if (p.dz != nullptr) tops[0] = c * static_cast<float>(others);   // the sampled token's gradient
  };
  if (wave == 0) {
    if constexpr (kStash) {
#pragma unroll
      for (int c = 0; c < 2; ++c) stash[c * 64 + lane] = held[c].r;
      asm volatile("" ::: "memory");
    }
    if (lane == 0) row_numbers();
    if constexpr (kStash) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int c = 0; c < 2; ++c) held[c].r = stash[c * 64 + lane];
    }
  }
  if (p.dz == nullptr) return;
  __syncthreads();
  const float c0 = row[0], own_grad = tops[0];
  if (c0 == 0.f) {
    const float zero[kN] = {};
    for (int c = tid; c < chunks; c += NT) out.template store<true>(c, in.shift, zero);
    return;
  }
  const float factor = -c0 * row[1];
  const auto grad = [&](const Chunk<E>& x, int c, const auto& power) {
    float y[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) y[e] = power(x.get(e)) * factor;
    if (c == own_chunk) {
#pragma unroll
      for (int e = 0; e < kN; ++e) y[e] = e == own_e ? own_grad : y[e];
    }
    out.template store<true>(c, in.shift, y);
  };
  if (far) {
#pragma unroll 1
    for (int c = tid; c < chunks; c += NT) grad(in.load(c), c, power_far);
    return;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (tid + c * NT < chunks) grad(held[c], tid + c * NT, power);
  each_kept([&](const Chunk<E>& x, int c) { grad(x, c, power); });
  if constexpr (LONG) {
    constexpr int kAtOnce = 4;
    for (int c = kept_end + tid; c < chunks; c += kAtOnce * NT) {
      Chunk<E> x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        x[k].fill_lowest();
        if (c + k * NT < chunks) x[k] = in.load(c + k * NT);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (c + k * NT < chunks) grad(x[k], c + k * NT, power);
    }
  }
}

// Backward from saved statistics: a piece of a row to a workgroup.  q_j = exp(z_j / tau - lse), or
// exp((z_j - z_a) / tau + lp) where lse is so large that its rounding and those of z_j / tau, some
// 2^-24 of it each, would show beside the gradient's own: 2^-19 of an fp32 q at 32 (where its own exponential
// is off by as much), an eighth of a rounding to bf16 at 2048.  In place one workgroup then has the
// whole row, as the gradient is written over z_a (1024 x 131072 fp32 about 100, so that all rows are such: 277
// us, about 0 188; to another place 168 and 168).
template <typename E>
constexpr float kFarLse = sizeof(E) == 4 ? 0x1p5f : 0x1p11f;
template <typename E, int NT>
__global__ __launch_bounds__(NT) void policy_bwd_kernel(const PolicyParams p) {
  constexpr int kN = Chunk<E>::kN;
  const int64_t n = blockIdx.y;
  const Row<E> in(p.z, n * p.z_stride, p.V), out(p.dz, n * p.dz_stride, p.V);
  const int c0 = blockIdx.x * p.seg;
  int c1 = min(c0 + p.seg, in.chunks());
  if (c0 >= c1) return;
  const float w = p.weight ? p.weight[n] : 1.f;
  const float lse = p.stats[4 * n], lp = p.stats[4 * n + 1], g = p.stats[4 * n + 2];
  const int32_t action = static_cast<int32_t>(uniform(p.action[n]));
  const bool named = action >= 0 && action < p.V;
  const int own_chunk = named ? (action + in.shift) / kN : -1, own_e = (action + in.shift) % kN;
  const float c = w != 0.f && named ? coefficient(p, w, g) : 0.f;
  const bool live = c != 0.f;
  const float inv_tau = static_cast<float>(p.inv_tau);
  float shift = 0.f, base = lse;
  if (live && fabsf(lse) > kFarLse<E> && fabsf(lp) < fabsf(lse)) {
    if (p.in_place) {
      if (blockIdx.x > 0) return;
      c1 = in.chunks();
    }
    shift = static_cast<float>(in.p[action]);
    base = -lp;
    if (p.in_place) __syncthreads();
  }
  const auto prob = [&](float z) { return exp2_hw(__builtin_fmaf(z - shift, inv_tau, -base) * kLog2e); };
  constexpr int kAtOnce = 4;                           // loads under way, a thread
  for (int cc = c0 + threadIdx.x; cc < c1; cc += kAtOnce * NT) {
    Chunk<E> x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      x[k].fill_lowest();
      if (live && cc + k * NT < c1) x[k] = in.template load<true>(cc + k * NT);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int at = cc + k * NT;
      if (at >= c1) continue;
      float y[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) y[e] = live ? -c * prob(x[k].get(e)) : 0.f;
      if (live && at == own_chunk) {
        const float own = c * static_cast<float>(-expm1(static_cast<double>(lp)));
#pragma unroll
        for (int e = 0; e < kN; ++e) y[e] = e == own_e ? own : y[e];
      }
      out.store(at, in.shift, y);
    }
  }
}

namespace {

template <typename E, int NT, int CH>
hipError_t run_fwd(const PolicyParams& p, hipStream_t s) {
  policy_fwd_kernel<E, NT, CH, false><<<static_cast<unsigned>(p.N), NT, 0, s>>>(p);
  return hipGetLastError();
}

// Rows beyond 8192 chunks.  Two workgroups fill a unit's registers, and what they keep in
// shared memory its 160 KiB (written through the caches, 4096 x 80000 bf16: 256 us, one with 16 chunks a
// thread 309; 2048 x 128000: 222, 247; 9000 kept, so that one workgroup runs on a unit: 256, 256; 2048 x
// 200000: 382 us and 1024 x 131072 fp32 270 us, everything read in three passes 515 and 360.  Past them:
// 233, 201, 328 and 222).
template <typename E>
hipError_t run_fwd_long(const PolicyParams& q, int64_t chunks, hipStream_t s) {
  constexpr int NT = 1024, CH = 8, kKept = 4800;
  PolicyParams p = q;
  p.kept = static_cast<int>(std::min<int64_t>(chunks - NT * CH, kKept));
  const auto fn = policy_fwd_kernel<E, NT, CH, true>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kKept * 16);
  if (e != hipSuccess) return e;
  fn<<<static_cast<unsigned>(p.N), NT, p.kept * 16, s>>>(p);
  return hipGetLastError();
}

// By the length of the row: 8 chunks a thread, in the fewest threads that hold it, so that all
// rows under way fill the card's registers (bf16 with the gradient, still written through the caches:
// 16384 x 4001 65 us, 256 threads with 2 chunks each 81; 4096 x 8200 33, 1024 with 2 45; 4096 x 20000
// 67, 1024 with 4 76).
// Rows of fewer than 4096 bf16 or 2048 fp32 values, 128 threads with 4.
template <typename E>
hipError_t pick_fwd(const PolicyParams& p, hipStream_t s) {
  const int64_t chunks = (p.V + Chunk<E>::kN - 1) / Chunk<E>::kN + 1;
  if (chunks <= 128 * 4) return run_fwd<E, 128, 4>(p, s);
  if (chunks <= 128 * 8) return run_fwd<E, 128, 8>(p, s);
  if (chunks <= 256 * 8) return run_fwd<E, 256, 8>(p, s);
  if (chunks <= 512 * 8) return run_fwd<E, 512, 8>(p, s);
  if (chunks <= 1024 * 8) return run_fwd<E, 1024, 8>(p, s);
  return run_fwd_long<E>(p, chunks, s);
}

template <typename E>
hipError_t run_bwd(const PolicyParams& p, hipStream_t s) {
  constexpr int NT = 256;
  const int chunks = static_cast<int>((p.V + Chunk<E>::kN - 1) / Chunk<E>::kN + 1);
  for (int64_t n0 = 0; n0 < p.N; n0 += 65535) {
    PolicyParams q = p;
    const int64_t rows = p.N - n0 < 65535 ? p.N - n0 : 65535;
    q.seg = NT * (Chunk<E>::kN == 4 ? 2 : 4);    // (the distillation loss's pieces)
    q.z = static_cast<const E*>(p.z) + n0 * p.z_stride;
    q.dz = static_cast<E*>(p.dz) + n0 * p.dz_stride;
    q.action = p.action + n0;
    q.weight = p.weight ? p.weight + n0 : nullptr;
    q.stats = p.stats + 4 * n0;
    policy_bwd_kernel<E, NT>
        <<<dim3((chunks + q.seg - 1) / q.seg, static_cast<unsigned>(rows)), NT, 0, s>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_policy(const zero_policy_args& a, bool forward, hipStream_t s) {
  PolicyParams p = {};
  p.N = a.N;
  p.V = a.V;
  p.inv_tau = 1.0 / a.temperature;
  p.low = 1.0 - a.clip_low;
  p.high = 1.0 + a.clip_high;
  p.kl_coef = a.kl_coef;
  p.grad_scale = a.grad_scale;
  p.z = a.logits;
  p.action = a.action;
  p.adv = a.advantage;
  p.old_lp = a.old_logp;
  p.ref_lp = a.ref_logp;
  p.weight = a.row_weight;
  p.loss = a.loss;
  p.stats = a.stats;
  p.dz = a.dlogits;
  p.z_stride = a.logits_stride;
  p.dz_stride = a.dlogits_stride;
  p.in_place = a.logits == a.dlogits;
  if (forward) return a.dtype == ZERO_BF16 ? pick_fwd<bf16>(p, s) : pick_fwd<float>(p, s);
  return a.dtype == ZERO_BF16 ? run_bwd<bf16>(p, s) : run_bwd<float>(p, s);
}

}  // namespace zo
