// zo_distill.hip -- the distillation loss against a teacher's top logits.
//
// Bound by memory: the logits are read once and their gradient is written
// once.  A workgroup owns a row; the forward pass keeps it in registers
// (packed as it came) between the maximum, the sums and the gradient, or, when
// the row is too long for that, reads it again.  The backward pass needs no
// row-wide sum, so a row is cut into pieces over workgroups.
//
// Rows may start at any element (an odd vocabulary makes every other row of a
// bf16 matrix misaligned): a row is taken as 16-byte chunks counted from the
// aligned address at or below its start, and its first and last chunk are
// loaded and stored element by element.
//
// The teacher's K entries and everything of them is formed in binary64: the
// tail's mass is a difference from 1.  The entries' positions are marked in a
// bit map in shared memory, so that the sum outside them is a sum of its own and
// no difference of large numbers, and about its own maximum where it is far below the row's.
//
// Measured: 8192 x 50257 bf16 with the gradient 312 us, 5.3 TB/s of logits read and
// gradient written, the loss alone 206 us, 4.0 TB/s; the backward alone, 1024 x 131072 fp32,
// 168 us, 6.4 TB/s, 2048 x 50257 bf16 76 us, 5.4.
#include "zo_device.h"
#include "zo_internal.h"

namespace zo {

// How far below 0 c = 1 - pT / qT goes in a row's statistics; from there on the 1 has no
// place in it, and log(pT / qT), which is above 1 where c never is, stands there instead.
constexpr double kMostC = 1 << 24;

struct DistillParams {
  int64_t N, V;
  int K, tail;
  double inv_tau, tau;
  double grad_scale;
  const void* z;
  const int32_t* idx;
  const void* val;
  const float* tlse;
  const float* weight;
  float *loss, *stats;
  void* dz;
  int64_t z_stride, dz_stride;
  int seg;  // backward: chunks of a piece
};

template <typename E>
struct Chunk;
template <>
struct Chunk<bf16> {
  static constexpr int kN = 8;
  u32x4 r;
  __device__ __forceinline__ float get(int e) const {
    return e & 1 ? __uint_as_float(r[e >> 1] & 0xFFFF0000u) : bf16_bits_to_f32(r[e >> 1]);
  }
  __device__ __forceinline__ void fill_lowest() {  // -inf
    r = u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
  }
  __device__ __forceinline__ void put_raw(int e, bf16 x) {
    union {
      bf16 b;
      uint16_t u;
    } c;
    c.b = x;
    const uint32_t bits = c.u;
    r[e >> 1] = e & 1 ? (r[e >> 1] & 0x0000FFFFu) | (bits << 16) : (r[e >> 1] & 0xFFFF0000u) | bits;
  }
};
template <>
struct Chunk<float> {
  static constexpr int kN = 4;
  f32x4 r;
  __device__ __forceinline__ float get(int e) const { return r[e]; }
  __device__ __forceinline__ void fill_lowest() { r = f32x4{-kInf, -kInf, -kInf, -kInf}; }
  __device__ __forceinline__ void put_raw(int e, float x) { r[e] = x; }
};

template <typename E>
__device__ __forceinline__ float value(const void* p, int64_t at) {
  return static_cast<float>(static_cast<const E*>(p)[at]);
}

// A row as aligned chunks: chunk c holds elements c * kN - shift .. + kN - 1.
template <typename E>
struct Row {
  static constexpr int kN = Chunk<E>::kN;
  E* p;       // element 0
  int shift;
  int64_t V;
  __device__ __forceinline__ Row(const void* base, int64_t at, int64_t v)
      : p(const_cast<E*>(static_cast<const E*>(base)) + at), V(v) {
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(E)) % kN);
  }
  __device__ __forceinline__ int chunks() const {
    return static_cast<int>((V + shift + kN - 1) / kN);
  }
  __device__ __forceinline__ bool whole(int c) const {
    const int64_t e0 = static_cast<int64_t>(c) * kN - shift;
    return e0 >= 0 && e0 + kN <= V;
  }
  __device__ __forceinline__ Chunk<E> load(int c) const {
    Chunk<E> x;
    const int64_t e0 = static_cast<int64_t>(c) * kN - shift;
    if (whole(c)) {
      x.r = *reinterpret_cast<const decltype(x.r)*>(p + e0);
    } else {
      x.fill_lowest();
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (e0 + e >= 0 && e0 + e < V) x.put_raw(e, p[e0 + e]);
    }
    return x;
  }
  // y as this row's elements that chunk c of a row shifted by `from` holds
  __device__ __forceinline__ void store(int c, int from, const float y[kN]) const {
    const int64_t e0 = static_cast<int64_t>(c) * kN - from;
    if (from == shift && e0 >= 0 && e0 + kN <= V) {
      Chunk<E> x;
      if constexpr (sizeof(E) == 2) {
        union {
          bf16x8 b;
          u32x4 u;
        } v;
#pragma unroll
        for (int e = 0; e < kN; ++e) v.b[e] = static_cast<bf16>(y[e]);
        x.r = v.u;
      } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) x.r[e] = y[e];
      }
      *reinterpret_cast<decltype(x.r)*>(p + e0) = x.r;
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (e0 + e >= 0 && e0 + e < V) p[e0 + e] = static_cast<E>(y[e]);
    }
  }
};

// Between the passes over a held row: its values are unpacked again in the next
// pass, not carried over as twice the registers.
template <typename E, int CH>
__device__ __forceinline__ void keep_packed(Chunk<E> (&held)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) asm volatile("" : "+v"(held[c].r));
}

// The teacher's side of a row, in shared memory: p[k], the student's logit
// z[k] (of entries in [from, to)) and idx[k], -1 for an absent entry; and what
// the row needs of them.  All of it is one wave's work, wave-wide sums and no
// barrier, so that the workgroup's others are at the row meanwhile.
struct Teacher {
  float* p;
  float* z;
  int* idx;
  double* sums;  // mass: sum of p; cross: sum of p (log p - z / tau); how many entries
};

template <typename E>
__device__ __forceinline__ void load_teacher(const DistillParams& p, int64_t n, const E* z,
                                             int64_t from, int64_t to, int lane, const Teacher& t) {
  float mx = -kInf;
  int entries = 0;
  for (int k = lane; k < p.K; k += 64) {
    const int i = p.idx[n * p.K + k];
    const bool ok = i >= 0 && i < p.V;
    t.idx[k] = ok ? i : -1;
    t.z[k] = ok && i >= from && i < to ? static_cast<float>(z[i]) : 0.f;
    const float v = ok ? value<E>(p.val, n * p.K + k) : -kInf;
    t.p[k] = v;
    entries += ok;
    mx = MaxOp()(mx, v);
  }
  double base;
  if (p.tlse != nullptr) {
    base = p.tlse[n];
  } else {
    mx = join_lanes<64>(mx, MaxOp());
    const double m = static_cast<double>(mx) * p.inv_tau;
    double s = 0.0;
    for (int k = lane; k < p.K; k += 64)
      if (t.idx[k] >= 0) s += exp(static_cast<double>(t.p[k]) * p.inv_tau - m);
    base = m + log(join_lanes<64>(s, AddOp()));
  }
  double mass = 0.0, cross = 0.0;
  for (int k = lane; k < p.K; k += 64) {
    double pk = 0.0;
    if (t.idx[k] >= 0) {
      const double lp = static_cast<double>(t.p[k]) * p.inv_tau - base;
      pk = exp(lp);
      mass += pk;
      if (pk != 0.0) cross += pk * (lp - static_cast<double>(t.z[k]) * p.inv_tau);
    }
    t.p[k] = static_cast<float>(pk);
  }
  mass = join_lanes<64>(mass, AddOp());
  cross = join_lanes<64>(cross, AddOp());
  entries = join_lanes<64>(entries, AddOp());
  if (lane == 0) {
    t.sums[0] = mass;
    t.sums[1] = cross;
    t.sums[2] = entries;
  }
}

__device__ __forceinline__ float prob(float z, float inv_tau, float lse) {
  return exp2_hw(__builtin_fmaf(z, inv_tau, -lse) * kLog2e);
}

// Writes the gradient of the row's entries over what the row's pass wrote.
template <typename E, int NT, typename Prob>
__device__ __forceinline__ void store_entries(const DistillParams& p, const Row<E>& out,
                                              const Teacher& t, float scale, int64_t from,
                                              int64_t to, Prob prob_of) {
  __syncthreads();                       // orders the workgroup's stores
  for (int k = threadIdx.x; k < p.K; k += NT) {
    const int i = t.idx[k];
    if (i >= from && i < to)
      out.p[i] = static_cast<E>(scale * (prob_of(t.z[k]) - t.p[k]));
  }
}

// Shared memory of the kernels: the waves' parts of the maximum and of the two sums, the
// teacher's, and the bit map.
template <int NT>
struct DistillShared {
  double* sum;   // [2][waves]
  float* top;    // [waves]
  Teacher t;
  uint32_t* bits;
  __device__ __forceinline__ DistillShared(char* smem, int K) {
    sum = reinterpret_cast<double*>(smem);
    t.sums = sum + 2 * (NT / 64);
    top = reinterpret_cast<float*>(t.sums + 4);
    bits = reinterpret_cast<uint32_t*>(top + NT / 64);         // 16-byte aligned, as is smem
    t.p = reinterpret_cast<float*>(bits);
    t.z = t.p + K;
    t.idx = reinterpret_cast<int*>(t.z + K);
    bits += (3 * K + 3) & ~3;
  }
  static size_t bytes(int K, int64_t bit_words) {
    return 2 * (NT / 64) * 8 + 4 * 8 + (NT / 64) * 4 + ((3 * K + 3) & ~3) * 4 + bit_words * 4;
  }
};

__host__ __device__ constexpr int64_t bit_words(int64_t V, int n) { return ((V + n) / 128 + 1) * 4; }

// Forward: loss and statistics, and the gradient if asked for.  CH > 0: the
// row stays in registers, CH chunks to a thread; CH = 0: it is read again.
// The workgroup's last wave first does the teacher's work and marks the
// entries, while the others load the row; two barriers, of the maximum and of
// the sums, come before the gradient.  64 registers a thread, two rows to a
// compute unit, one loading while the other computes.
template <typename E, int NT, int CH>
__global__ __launch_bounds__(NT, CH <= 8 ? 8 : 4) void distill_fwd_kernel(
    const DistillParams p) {
  constexpr int kN = Chunk<E>::kN, kW = NT / 64;
  constexpr int kHeld = CH > 0 ? CH : 1;
  extern __shared__ __align__(16) char smem[];
  const DistillShared<NT> sh(smem, p.K);
  const Teacher& t = sh.t;
  uint32_t* bits = sh.bits;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = blockIdx.x;
  const Row<E> in(p.z, n * p.z_stride, p.V), out(p.dz, n * p.dz_stride, p.V);
  const int chunks = in.chunks();
  const float w = p.weight ? p.weight[n] : 1.f;
  const float k2 = static_cast<float>(p.inv_tau * 1.4426950408889634);

  if (wave == kW - 1) {
    if (p.tail)
      for (int64_t i = 4 * lane; i < bit_words(p.V, kN); i += 256)
        *reinterpret_cast<u32x4*>(bits + i) = u32x4{0, 0, 0, 0};
    load_teacher<E>(p, n, in.p, 0, p.V, lane, t);
    if (p.tail)                            // (the wave's own writes: in order)
      for (int k = lane; k < p.K; k += 64)
        if (t.idx[k] >= 0) {
          const int64_t e = t.idx[k] + in.shift;
          atomicOr(&bits[e >> 5], 1u << (e & 31));
        }
  }
  Chunk<E> held[kHeld];
  if constexpr (CH > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      held[c].fill_lowest();
      if (tid + c * NT < chunks) held[c] = in.load(tid + c * NT);
    }
  }

  float m = -kInf, sum = 0.f, rest = 0.f;
  const auto chunk_max = [&](const Chunk<E>& x, float a) {
#pragma unroll
    for (int e = 0; e < kN; ++e) a = fmaxf(a, x.get(e));
    return a;
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) m = chunk_max(held[c], m);
  } else {
    for (int c = tid; c < chunks; c += NT) m = chunk_max(in.load(c), m);
  }
  m = join_lanes<64>(m, MaxOp());
  if (lane == 0) sh.top[wave] = m;
  __syncthreads();
  m = join_lanes<kW>(sh.top[lane % kW], MaxOp());
  if (m == -kInf) m = 0.f;               // nothing but -inf: a sum of 0, not of NaN
  if constexpr (CH > 0) keep_packed(held);

  // exp((z - m) / tau) = 2^(z k2 - m2), with m2 the rounded m k2: the same in
  // every term, and put right in the logarithm of the sum (see base_of)
  const float m2 = m * k2;
  const auto power = [&](float z) { return exp2_hw(__builtin_fmaf(z, k2, -m2)); };
  const auto marks = [&](int c) {        // of the chunk's elements, the teacher's
    const int64_t e = static_cast<int64_t>(c) * kN;
    return (bits[e >> 5] >> (e & 31)) & ((1u << kN) - 1);
  };
  const auto chunk_sum = [&](const Chunk<E>& x, int c) {
    const uint32_t marked = p.tail ? marks(c) : 0;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kN; ++e) s += power(x.get(e));
    sum += s;
    rest += marked != 0 ? 0.f : s;
    if (marked != 0) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (!((marked >> e) & 1u)) rest += power(x.get(e));
    }
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (tid + c * NT < chunks) chunk_sum(held[c], tid + c * NT);
  } else {
    for (int c = tid; c < chunks; c += NT) chunk_sum(in.load(c), c);
  }
  if constexpr (CH > 0) keep_packed(held);
  const double part = join_lanes<64>(static_cast<double>(sum), AddOp());
  const double part_rest = join_lanes<64>(static_cast<double>(rest), AddOp());
  if (lane == 0) {
    sh.sum[wave] = part;
    sh.sum[kW + wave] = part_rest;
  }
  __syncthreads();
  const double total = join_lanes<kW>(sh.sum[lane % kW], AddOp());
  const double outside = p.tail ? join_lanes<kW>(sh.sum[kW + lane % kW], AddOp()) : 0.0;
  // With a tail, gradients outside the entries are z's power times c / total; where the
  // entries lead so far that 1 has no place in c = 1 - pT / qT, minus pT times the softmax of
  // the outside alone, about its own maximum: below the row's its powers, and c, would
  // leave binary32.  (Uniform, and rare: an ordinary row takes one comparison.)
  double mass = 0.0, coef = 1.0, out_mass = outside;
  float m_out = m, m_out2 = m2;
  bool sure = false;
  if (p.tail) {
    // (no token is left for a tail where the entries are the whole vocabulary)
    mass = t.sums[0] < 1.0 && t.sums[2] < static_cast<double>(p.V) ? 1.0 - t.sums[0] : 0.0;
    if (mass > 0.0) coef = 1.0 - mass * (total / outside);
    sure = coef < -kMostC;
  }
  if (sure) {
    const auto out_max = [&](const Chunk<E>& x, int c, float a) {
      const uint32_t marked = marks(c);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (!((marked >> e) & 1u)) a = fmaxf(a, x.get(e));
      return a;
    };
    const auto out_sum = [&](const Chunk<E>& x, int c) {
      const uint32_t marked = marks(c);
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (!((marked >> e) & 1u)) a += exp2_hw(__builtin_fmaf(x.get(e), k2, -m_out2));
      return a;
    };
    float mo = -kInf;
    if constexpr (CH > 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (tid + c * NT < chunks) mo = out_max(held[c], tid + c * NT, mo);
    } else {
      for (int c = tid; c < chunks; c += NT) mo = out_max(in.load(c), c, mo);
    }
    mo = join_lanes<64>(mo, MaxOp());
    if (lane == 0) sh.top[wave] = mo;
    __syncthreads();
    mo = join_lanes<kW>(sh.top[lane % kW], MaxOp());
    m_out = mo == -kInf ? 0.f : mo;
    m_out2 = m_out * k2;
    float part_out = 0.f;
    if constexpr (CH > 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (tid + c * NT < chunks) part_out += out_sum(held[c], tid + c * NT);
    } else {
      for (int c = tid; c < chunks; c += NT) part_out += out_sum(in.load(c), c);
    }
    const double wave_out = join_lanes<64>(static_cast<double>(part_out), AddOp());
    if (lane == 0) sh.sum[wave] = wave_out;
    __syncthreads();
    out_mass = join_lanes<kW>(sh.sum[lane % kW], AddOp());
    if (out_mass == 0.0 && mass <= (1.0 + fabs(static_cast<double>(p.tlse[n]))) * 0x1p-23) {
      // the student's vocabulary ends with the entries, and so does the teacher's but for
      // its logarithm's rounding
      sure = false;
      mass = 0.0;
      coef = 1.0;
      m_out2 = m2;
    }
  }
  // a row without weight, or with nothing to be compared with: statistics only
  const bool live = w != 0.f && (t.sums[2] != 0.0 || p.tail);
  if (p.dz != nullptr) {
    const float scale = static_cast<float>(p.grad_scale * p.tau * static_cast<double>(w));
    if (live) {
      const float inv = static_cast<float>(1.0 / total);
      const float other =
          sure ? -scale * static_cast<float>(mass / out_mass) : static_cast<float>(coef) * scale * inv;
      const auto grad = [&](const Chunk<E>& x, int c) {
        float y[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) y[e] = exp2_hw(__builtin_fmaf(x.get(e), k2, -m_out2)) * other;
        out.store(c, in.shift, y);
      };
      if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (tid + c * NT < chunks) grad(held[c], tid + c * NT);
      } else {
        for (int c = tid; c < chunks; c += NT) grad(in.load(c), c);
      }
      store_entries<E, NT>(p, out, t, scale, 0, p.V, [&](float z) { return power(z) * inv; });
    } else {
      const float zero[kN] = {};
      for (int c = tid; c < chunks; c += NT) out.store(c, in.shift, zero);
    }
  }
  // the logarithms come last: in binary64 they take registers that the held row
  // leaves only now
  if (tid == 0) {
    // of powers 2^(z k2 - x2) about x: x / tau, less what x2 and k2 were rounded by (k2's
    // rounding alone moves a sum about 0 by 6e-4 at x / tau = 1e4)
    const auto base_of = [&](float x, float x2) {
      return static_cast<double>(x) * p.inv_tau +
             (static_cast<double>(x2) - static_cast<double>(x) * k2) * 0.6931471805599453;
    };
    const double lse = base_of(m, m2) + log(total);
    double loss = t.sums[1] + t.sums[0] * lse;
    if (mass > 0.0) {
      const double ratio = log(mass) - (base_of(m_out, m_out2) + log(out_mass)) + lse;   // of pT / qT
      loss += mass * ratio;
      if (sure) coef = ratio;
    }
    p.loss[n] = live ? static_cast<float>(loss * p.tau * p.tau * static_cast<double>(w)) : 0.f;
    p.stats[2 * n] = static_cast<float>(lse);
    p.stats[2 * n + 1] = static_cast<float>(coef);
  }
}

// Backward from saved statistics: a piece of a row to a workgroup.
template <typename E, int NT>
__global__ __launch_bounds__(NT) void distill_bwd_kernel(const DistillParams p) {
  constexpr int kN = Chunk<E>::kN;
  extern __shared__ __align__(16) char smem[];
  const DistillShared<NT> sh(smem, p.K);
  const Teacher& t = sh.t;

  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t n = blockIdx.y;
  const Row<E> in(p.z, n * p.z_stride, p.V), out(p.dz, n * p.dz_stride, p.V);
  const int c0 = blockIdx.x * p.seg, c1 = min(c0 + p.seg, in.chunks());
  if (c0 >= c1) return;
  const float w = p.weight ? p.weight[n] : 1.f;
  const float inv_tau = static_cast<float>(p.inv_tau);
  // (only this piece's logits are read: in place, others may be gradients already)
  const int64_t from = max(static_cast<int64_t>(c0) * kN - in.shift, int64_t(0));
  const int64_t to = static_cast<int64_t>(c1) * kN - in.shift;
  if (tid >= NT - 64 && w != 0.f) load_teacher<E>(p, n, in.p, from, to, lane, t);
  const float lse = p.stats[2 * n], c = p.stats[2 * n + 1];
  const float scale = static_cast<float>(p.grad_scale * p.tau * static_cast<double>(w));
  // (above 1: log(pT / qT), and the gradient outside is minus exp(z / tau - lse + it))
  const bool sure = c > 1.f;
  const float other = sure ? -scale : c * scale;
  const float lse_out = sure ? static_cast<float>(static_cast<double>(lse) - c) : lse;
  // without a tail a row may have no entry; in place, the entries' logits come first
  if (w != 0.f && (!p.tail || p.z == p.dz)) __syncthreads();
  const bool live = w != 0.f && (p.tail || t.sums[2] != 0.0);
  constexpr int kAtOnce = 4;                           // loads under way, a thread
  for (int cc = c0 + tid; cc < c1; cc += kAtOnce * NT) {
    Chunk<E> x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      x[k].fill_lowest();
      if (live && cc + k * NT < c1) x[k] = in.load(cc + k * NT);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      float y[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) y[e] = live ? other * prob(x[k].get(e), inv_tau, lse_out) : 0.f;
      if (cc + k * NT < c1) out.store(cc + k * NT, in.shift, y);
    }
  }
  if (live)
    store_entries<E, NT>(p, out, t, scale, from, to,
                         [&](float z) { return prob(z, inv_tau, lse); });
}

namespace {

template <typename E, int NT, int CH>
hipError_t run_fwd(const DistillParams& p, hipStream_t s) {
  const size_t lds =
      DistillShared<NT>::bytes(p.K, p.tail ? bit_words(p.V, Chunk<E>::kN) : 0);
  const auto fn = distill_fwd_kernel<E, NT, CH>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds));
  if (e != hipSuccess) return e;
  fn<<<static_cast<unsigned>(p.N), NT, lds, s>>>(p);
  return hipGetLastError();
}

// By the length of the row: held in registers where it fits (8192 x 50257 with the
// gradient, bf16: 312 us, read again 516), in the fewest that hold it, and short rows by
// smaller workgroups (4096 x 4001: 23 us, by 1024 threads 51).
template <typename E>
hipError_t pick_fwd(const DistillParams& p, hipStream_t s) {
  const int64_t chunks = (p.V + Chunk<E>::kN - 1) / Chunk<E>::kN + 1;
  if (chunks <= 256 * 2) return run_fwd<E, 256, 2>(p, s);
  if (chunks <= 256 * 4) return run_fwd<E, 256, 4>(p, s);
  if (chunks <= 1024 * 2) return run_fwd<E, 1024, 2>(p, s);
  if (chunks <= 1024 * 4) return run_fwd<E, 1024, 4>(p, s);
  if (chunks <= 1024 * 8) return run_fwd<E, 1024, 8>(p, s);
  if (chunks <= 1024 * 16) return run_fwd<E, 1024, 16>(p, s);
  return run_fwd<E, 1024, 0>(p, s);
}

template <typename E>
hipError_t run_bwd(DistillParams p, hipStream_t s) {
  constexpr int NT = 256;
  const int chunks = static_cast<int>((p.V + Chunk<E>::kN - 1) / Chunk<E>::kN + 1);
  // A piece is 2 (fp32) or 4 (bf16) chunks of 16 bytes a thread: short enough that a row's
  // loads are spread over many workgroups, long enough for what each does for the teacher's
  // entries.  1024 x 131072 fp32: 169 us, with 4, 8 and 16 chunks 194, 190 and 200;
  // 2048 x 50257 bf16: 76 us, with 2, 8 and 16 chunks 83, 88 and 98.
  p.seg = NT * (Chunk<E>::kN == 4 ? 2 : 4);
  const size_t lds = DistillShared<NT>::bytes(p.K, 0);
  for (int64_t n0 = 0; n0 < p.N; n0 += 65535) {
    DistillParams q = p;
    const int64_t rows = p.N - n0 < 65535 ? p.N - n0 : 65535;
    q.z = static_cast<const E*>(p.z) + n0 * p.z_stride;
    q.dz = static_cast<E*>(p.dz) + n0 * p.dz_stride;
    q.idx = p.idx + n0 * p.K;
    q.val = static_cast<const E*>(p.val) + n0 * p.K;
    q.tlse = p.tlse ? p.tlse + n0 : nullptr;
    q.weight = p.weight ? p.weight + n0 : nullptr;
    q.stats = p.stats + 2 * n0;
    distill_bwd_kernel<E, NT>
        <<<dim3((chunks + p.seg - 1) / p.seg, static_cast<unsigned>(rows)), NT, lds, s>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_distill(const zero_distill_args& a, bool forward, hipStream_t s) {
  DistillParams p = {};
  p.N = a.N;
  p.V = a.V;
  p.K = a.K;
  p.tail = a.teacher_lse != nullptr;
  p.tau = a.temperature;
  p.inv_tau = 1.0 / a.temperature;
  p.grad_scale = a.grad_scale;
  p.z = a.logits;
  p.idx = a.teacher_idx;
  p.val = a.teacher_val;
  p.tlse = a.teacher_lse;
  p.weight = a.row_weight;
  p.loss = a.loss;
  p.stats = a.stats;
  p.dz = a.dlogits;
  p.z_stride = a.logits_stride;
  p.dz_stride = a.dlogits_stride;
  if (forward) return a.dtype == ZERO_BF16 ? pick_fwd<bf16>(p, s) : pick_fwd<float>(p, s);
  return a.dtype == ZERO_BF16 ? run_bwd<bf16>(p, s) : run_bwd<float>(p, s);
}

}  // namespace zo
