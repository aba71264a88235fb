// zo_attn_fwd.hip -- attention, forward: one pass over the keys with the
// running maximum and sum of the softmax.
//
// A workgroup owns 128 queries of one head, 32 to a wave, whose q fragments
// stay in registers; tiles of 64 keys and values are loaded straight into shared
// memory, one tile ahead of use.  (Two tiles ahead: 184 instead of 164 us at 64
// columns, 226 and 222 at 96, 115 and 117 at 32: the shared memory is worth more as room
// for a third workgroup on the compute unit.)  Per tile a wave forms
// S^T = K Q^T, updates its statistics and adds V^T P^T to the output accumulators.
// The accumulators are rescaled only when the maximum has grown by more than a factor of 2^8
// in any row, which binary32 has room for.
//
// Two waves a SIMD, of two workgroups, overlap one's products with the other's score work,
// which takes more issue than the products: an exponential a score, and with a cap one more and
// a reciprocal, at a quarter of the rate of other instructions.  Measured on 4096 queries and
// keys, 32 heads, no mask: 940 to 990 TFLOP/s at 128 columns (770 to 810 capped), 890 to 920 at
// 96, 815 to 840 at 64 (the card's clock differs from day to day).  Documents and few heads add
// idle units: counted at 4096 keys in two documents, 32 on 8 heads, cap, units are busy 79 % of
// the kernel, at 8 x 1024 tokens, 12 heads of 64, bias, 51 %.
// Splitting the keys for a single token (choose_split), 4 x 12 heads on 5003 keys: 19 us, 3.2
// TB/s of k and v.
#include "zo_attn.h"
#include "zo_internal.h"

namespace zo {

// One tile of 64 keys for a wave's 32 queries.
template <int D, int CAP, bool BIAS>
__device__ __forceinline__ void attn_fwd_tile(const AttnParams& p, const FragAt<D>& kt,
                                              const FragAt<D>& vt, const bf16x8 (&qf)[D / 16],
                                              f32x16 (&acc)[D / 32], float& m, float& l, int2 rng,
                                              int k0, int i0, const ScoreFactors& f,
                                              const float* bias, int lane) {
  // x; with a cap up to kUCap u; with a larger one, or a bias, the score
  float s[2][16];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    f32x16 x;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) x = mfma(frag_rows<D>(kt, t, c), qf[c], x);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[t][r] = CAP != kNoCap ? f.u_of(x[r]) : x[r];
      if constexpr (CAP == kAnyCap) s[t][r] = f.any_cap(x[r], s[t][r]);
    }
  }
  if constexpr (BIAS) {
    const auto add_bias = [&](float x, float c) {
      return CAP == kByU     ? __builtin_fmaf(x, -2.f * f.c2, f.c2 + c)
             : CAP == kNoCap ? __builtin_fmaf(x, f.a, c)
                             : x + c;
    };
    const int d0 = k0 - (i0 + p.off);    // distances span d0 - 31 .. d0 + 63
    const int side = bias_side(d0 - 31, d0 + kTile - 1, p.reach);
    if (side != 0) {
      const float c = bias[side < 0 ? 0 : 2 * bias_span(p.reach)];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[t][r] = add_bias(s[t][r], c);
    } else {
      const float* row = bias + d0 - (lane & 31) + 4 * (lane >> 5) + bias_span(p.reach);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float c = row[32 * t + 8 * (r >> 2) + (r & 3)];
          s[t][r] = add_bias(s[t][r], c);
        }
    }
  }
  constexpr bool kU = CAP == kByU && !BIAS;   // s holds u: the smallest is the largest score
  constexpr bool kScore = BIAS || CAP == kAnyCap;
  if (!__all(rng.x <= k0 && rng.y >= k0 + kTile)) {    // not every query sees every key
    const uint32_t n = rng.y - rng.x;
    const int from = k0 + 4 * (lane >> 5) - rng.x;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t j = from + 32 * t + 8 * (r >> 2) + (r & 3);
        s[t][r] = j < n ? s[t][r] : (kU ? kInf : -kInf);
      }
  }
  float mx = s[0][0];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) mx = kU ? fminf(mx, s[t][r]) : fmaxf(mx, s[t][r]);
  if constexpr (kU)
    mx = __builtin_fmaf(mx, -2.f * f.c2, f.c2);
  else if constexpr (!kScore)
    mx *= f.a;
  mx = max_halves(mx);
  // The reference of the exponentials moves only when it is 2^8 too low: p, its
  // sum and the outputs carry the factor in their exponents, at no loss.
  if (__any(mx > m + 8.f)) {
    const float mn = fmaxf(m, mx), g = exp2_hw(m - mn);
    m = mn;
    l *= g;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] *= g;
  }
  // (A tile's p are summed before the row's sum takes them: term by term, equal terms round the
  // same way each time, and of 2^17 keys at 0.7 of the largest the sum is 3e-4 off.)
  const float shift = kU ? f.c2 - m : -m;
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = s[g >> 1][8 * (g & 1) + j];
      if constexpr (kScore)
        e[j] = exp2_hw(x - m);
      else
        e[j] = exp2_hw(__builtin_fmaf(x, kU ? -2.f * f.c2 : f.a, shift));
      sum += e[j];
    }
    const bf16x8 pf = to_frag(e);
#pragma unroll
    for (int t = 0; t < D / 32; ++t) {
      acc[t] = mfma(frag_cols<D>(vt, g, t), pf, acc[t]);
    }
  }
  l += sum;
}

template <int D, int CAP, bool BIAS, bool SPLIT>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_fwd_kernel(const AttnParams p) {
  constexpr int kRows = 32 * kWaves, kBufs = 2, kTiles = 2 * kBufs;
  extern __shared__ __align__(1024) char smem[];      // [kBufs] tiles of K, of V
  const uint32_t tiles = lds_address(smem);
  int2* ranges = reinterpret_cast<int2*>(smem + kTiles * kTileBytes<D>);  // [kRows]
  int* hull = reinterpret_cast<int*>(ranges + kRows);                // [kWaves][2]
  float* bias = reinterpret_cast<float*>(hull + 2 * kWaves);

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bh = head_of_group(blockIdx.x, gridDim.x), b = bh / p.Hq, h = bh % p.Hq;
  const int hk = h / p.group;
  BiasStage bs;
  if constexpr (BIAS) bs.buckets(p, tid);
  const int tile = query_tile(p, place(), b, reinterpret_cast<int*>(ranges), tid, 2 * kUnits);
  const int i0 = tile * kRows + wave * 32;
  const int i = i0 + (lane & 31);
  const ScoreFactors f(p, CAP);
  const FragAt<D> at(lane);

  const int2 rng = key_range(p, b, i);
  const int2 wh = wave_hull(rng);
  if (lane == 0) {
    hull[2 * wave] = wh.x;
    hull[2 * wave + 1] = wh.y;
  }
  if (lane < 32) ranges[wave * 32 + lane] = rng;
  if constexpr (BIAS) bs.values(p, h);
  __syncthreads();
  int first = 0x7FFFFFFF, last = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    first = min(first, hull[2 * w]);
    last = max(last, hull[2 * w + 1]);
  }
  first = __builtin_amdgcn_readfirstlane(min(first, last));
  last = __builtin_amdgcn_readfirstlane(last);
  int k0 = first & ~(kTile - 1), kend = last;
  if constexpr (SPLIT) {
    k0 = max(k0, static_cast<int>(blockIdx.z) * p.tiles_per_split * kTile);
    kend = min(kend, (static_cast<int>(blockIdx.z) + 1) * p.tiles_per_split * kTile);
  }

  const TileLoad<D> kl(p.k + b * p.ks.b + hk * p.ks.h, p.ks.t, first, last, wave, lane);
  const TileLoad<D> vl(p.v + b * p.vs.b + hk * p.vs.h, p.vs.t, first, last, wave, lane);
  const auto stage = [&](int buf, int row0) {
    kl.start(tiles + buf * kTileBytes<D>, row0, wave, lane);
    vl.start(tiles + (kBufs + buf) * kTileBytes<D>, row0, wave, lane);
  };
#pragma unroll
  for (int n = 0; n < kBufs - 1; ++n)
    if (k0 + n * kTile < kend) stage(n, k0 + n * kTile);
  bf16x8 qf[D / 16];
  {
    const bf16* q = p.q + b * p.qs.b + static_cast<int64_t>(min(i, p.Tq - 1)) * p.qs.t + h * p.qs.h;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) qf[c] = signed_frag(load8(q + 16 * c + 8 * half), f.flip);
  }
  f32x16 acc[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
  float m = kLowest, l = 0.f;
  if constexpr (BIAS) bs.store(p, h, bias, tid);
  const bool gaps = p.ranges && has_gaps(ranges, last, tid);
  wait_tile();
  // Turns in which the wave has nothing to see have a loop of their own: a
  // branch inside one loop copied the accumulators to other registers every turn.
  // Every wave goes through the same number of turns, each with its barrier.
  int buf = 0;
  const auto turn = [&](auto work) {
    const int ahead = k0 + (kBufs - 1) * kTile;
    if (ahead < kend) stage((buf + kBufs - 1) % kBufs, ahead);
    if (gaps) {
      const uint64_t seen = seen_keys(ranges, k0, reinterpret_cast<uint32_t*>(hull), tid);
      clear_rows<D>(tiles + buf * kTileBytes<D>, tiles + (kBufs + buf) * kTileBytes<D>, seen, tid);
      __syncthreads();
    }
    work();
    // (One wait in two places: where the compiler has a single one it moves work across it, 287
    // us instead of 277 at 4096 keys, 32 heads of 128, no mask.)
    if (ahead < kend)
      wait_tile();
    else
      wait_tile();
    k0 += kTile;
    buf = buf + 1 == kBufs ? 0 : buf + 1;
  };
  const auto sees = [&] { return wh.x < k0 + kTile && wh.y > k0; };
  while (k0 < kend) {
    while (k0 < kend && !sees()) turn([] {});
    while (k0 < kend && sees())
      turn([&] {
        attn_fwd_tile<D, CAP, BIAS>(p, at.in(tiles + buf * kTileBytes<D>),
                                    at.in(tiles + (kBufs + buf) * kTileBytes<D>), qf, acc, m, l, rng,
                                    k0, i0, f, bias, lane);
      });
  }

  l += __shfl_xor(l, 32);
  if (i >= p.Tq) return;
  const int64_t row = static_cast<int64_t>(bh) * p.Tq + i;
  if constexpr (SPLIT) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hq * p.Tq;
    float* out = p.osplit + (blockIdx.z * rows + row) * D;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const f32x4 x = {acc[t][r], acc[t][r + 1], acc[t][r + 2], acc[t][r + 3]};
        *reinterpret_cast<f32x4*>(out + 32 * t + result_row(r, lane)) = x;
      }
    if (half == 0) {
      float* st = p.osplit + p.splits * rows * D + 2 * (blockIdx.z * rows + row);
      st[0] = m;
      st[1] = l;
    }
  } else {
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);     // NaN stays NaN
    bf16* o = p.o + b * p.os.b + static_cast<int64_t>(i) * p.os.t + h * p.os.h;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        bf16x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = static_cast<bf16>(acc[t][r + e] * inv);
        *reinterpret_cast<bf16x4*>(o + 32 * t + result_row(r, lane)) = x;
      }
    if (half == 0) p.lse[row] = l == 0.f ? -kInf : (m + log2_hw(l)) * kLn2;
  }
}

// Joins the parts of split rows: a wave to a row.  Lane z takes part z's
// statistics, so that all of their loads are under way at once.
constexpr int kMaxSplits = 64;

template <int D>
__global__ __launch_bounds__(64) void attn_join_kernel(const AttnParams p) {
  constexpr int kN = (D + 63) / 64;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hq * p.Tq;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x;
  const float* st = p.osplit + p.splits * rows * D + 2 * row;
  float mine = kLowest, l = 0.f;
  if (lane < p.splits) {
    mine = st[2 * rows * lane];
    l = st[2 * rows * lane + 1];
  }
  float m = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float f = exp2_hw(mine - m);
  l *= f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  float x[kN];
#pragma unroll
  for (int c = 0; c < kN; ++c) x[c] = 0.f;
  for (int z0 = 0; z0 < p.splits; z0 += 8) {       // 8 loads under way at a time
    float part[8][kN];
#pragma unroll
    for (int z = 0; z < 8; ++z)
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        part[z][c] = 0.f;
        if (z0 + z < p.splits && lane + 64 * c < D)
          part[z][c] = p.osplit[((z0 + z) * rows + row) * D + lane + 64 * c];
      }
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      const float fz = __shfl(f, z0 + z);          // (of a part that is not there: times 0)
#pragma unroll
      for (int c = 0; c < kN; ++c) x[c] = __builtin_fmaf(fz, part[z][c], x[c]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const int64_t bh = row / p.Tq;
  const int i = static_cast<int>(row % p.Tq);
  bf16* o = p.o + (bh / p.Hq) * p.os.b + i * p.os.t + (bh % p.Hq) * p.os.h;
#pragma unroll
  for (int c = 0; c < kN; ++c)
    if (lane + 64 * c < D) o[lane + 64 * c] = static_cast<bf16>(x[c] * inv);
  if (lane == 0) p.lse[row] = l == 0.f ? -kInf : (m + log2_hw(l)) * kLn2;
}

namespace {

// Keys are split over workgroups where the query tiles alone leave compute
// units idle: 20 us instead of 102 for one token of 4 x 12 heads on 5003 keys.
struct Split {
  int n, tiles_each;
};

Split choose_split(int B, int Tq, int Tk, int Hq) {
  const int64_t groups = static_cast<int64_t>(B) * Hq * ((Tq + 127) / 128);
  const int tiles = (Tk + kTile - 1) / kTile;
  int64_t n = 512 / (groups > 0 ? groups : 1);
  if (n > tiles / 4) n = tiles / 4;        // at least 4 tiles to a part
  if (n > kMaxSplits) n = kMaxSplits;
  if (n < 2) return {1, tiles};
  const int each = static_cast<int>((tiles + n - 1) / n);
  return {(tiles + each - 1) / each, each};
}

template <int D, int CAP, bool BIAS>
hipError_t run_fwd(const AttnParams& p, hipStream_t s) {
  const size_t lds = 2 * 2 * kTileBytes<D> + 128 * sizeof(int2) + 2 * kWaves * sizeof(int) +
                     (BIAS ? bias_entries(p.reach) * sizeof(float) : 0);
  const dim3 grid(p.B * p.Hq, (p.Tq + 127) / 128, p.splits);
  if (p.splits > 1) {
    const auto fn = attn_fwd_kernel<D, CAP, BIAS, true>;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                       hipFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(lds));
    if (e != hipSuccess) return e;
    fn<<<grid, kAttnThreads, lds, s>>>(p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = static_cast<int64_t>(p.B) * p.Hq * p.Tq;
    attn_join_kernel<D><<<static_cast<unsigned>(rows), 64, 0, s>>>(p);
  } else {
    const auto fn = attn_fwd_kernel<D, CAP, BIAS, false>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
    fn<<<grid, kAttnThreads, lds, s>>>(p);
  }
  return hipGetLastError();
}

template <int D, int CAP>
hipError_t pick_fwd(const AttnParams& p, hipStream_t s) {
  return p.table ? run_fwd<D, CAP, true>(p, s) : run_fwd<D, CAP, false>(p, s);
}

template <int D>
hipError_t pick_fwd(const AttnParams& p, hipStream_t s) {
  switch (cap_form(p.cap)) {
    case kNoCap: return pick_fwd<D, kNoCap>(p, s);
    case kByU: return pick_fwd<D, kByU>(p, s);
    default: return pick_fwd<D, kAnyCap>(p, s);
  }
}

}  // namespace

size_t attn_fwd_workspace(int B, int Tq, int Tk, int Hq, int Hk, int D) {
  (void)Hk;
  const Split sp = choose_split(B, Tq, Tk, Hq);
  return sp.n > 1 ? static_cast<size_t>(sp.n) * B * Hq * Tq * (D + 2) * sizeof(float) : 0;
}

hipError_t launch_attn_fwd(const zero_attn_args& a, hipStream_t s) {
  AttnParams p = attn_params(a);
  const Split sp = choose_split(a.B, a.Tq, a.Tk, a.Hq);
  p.splits = sp.n;
  p.tiles_per_split = sp.tiles_each;
  p.osplit = static_cast<float*>(a.workspace);
  switch (a.D) {
    case 32: return pick_fwd<32>(p, s);
    case 64: return pick_fwd<64>(p, s);
    case 96: return pick_fwd<96>(p, s);
    default: return pick_fwd<128>(p, s);
  }
}

AttnParams attn_params(const zero_attn_args& a) {
  AttnParams p = {};
  p.B = a.B;
  p.Tq = a.Tq;
  p.Tk = a.Tk;
  p.Hq = a.Hq;
  p.Hk = a.Hk;
  p.group = a.Hq / a.Hk;
  p.causal = a.causal;
  p.off = a.Tk - a.Tq;
  p.scale = static_cast<float>(a.scale);
  p.cap = static_cast<float>(a.cap);
  p.q = static_cast<const bf16*>(a.q);
  p.k = static_cast<const bf16*>(a.k);
  p.v = static_cast<const bf16*>(a.v);
  p.ranges = a.ranges;
  p.table = a.bias_table;
  p.buckets = a.bias_buckets;
  p.table_f32 = a.bias_dtype == ZERO_F32;
  p.n_buckets = a.n_buckets;
  p.reach = a.bias_table ? a.reach : 0;
  p.o = static_cast<bf16*>(a.o);
  p.lse = a.lse;
  p.d_o = static_cast<const bf16*>(a.d_o);
  p.dq = static_cast<bf16*>(a.dq);
  p.dk = static_cast<bf16*>(a.dk);
  p.dv = static_cast<bf16*>(a.dv);
  p.dtable = a.dbias_table;
  const auto st = [](const int64_t* x) { return Strides3{x[0], x[1], x[2]}; };
  p.qs = st(a.q_stride);
  p.ks = st(a.k_stride);
  p.vs = st(a.v_stride);
  p.os = st(a.o_stride);
  p.dos = st(a.do_stride);
  p.dqs = st(a.dq_stride);
  p.dks = st(a.dk_stride);
  p.dvs = st(a.dv_stride);
  return p;
}

// Document runs of a batch row, found by a workgroup: every thread takes a
// run of consecutive tokens; the start of the document that a segment's first
// token continues, and the end of the one its last token begins or continues,
// come from a scan over the segments.
__global__ __launch_bounds__(1024) void attn_ranges_kernel(const int32_t* doc,
                                                           const int32_t* prefix, int T,
                                                           int causal, int2* ranges) {
  __shared__ int last_start[1024], first_start[1024];
  const int tid = threadIdx.x;
  doc += static_cast<int64_t>(blockIdx.x) * T;
  ranges += static_cast<int64_t>(blockIdx.x) * T;
  if (prefix) prefix += static_cast<int64_t>(blockIdx.x) * T;
  const int each = (T + 1023) / 1024;
  const int lo = static_cast<int>(min(static_cast<int64_t>(tid) * each, static_cast<int64_t>(T)));
  const int hi = min(lo + each, T);
  int ls = -1, fs = T;                     // starts of documents inside [lo, hi)
  for (int t = lo; t < hi; ++t)
    if (t == 0 || doc[t] != doc[t - 1]) {
      ls = t;
      if (fs == T) fs = t;
    }
  last_start[tid] = ls;
  first_start[tid] = fs;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {     // running maximum from the left, minimum from the right
    const int a = tid >= d ? last_start[tid - d] : -1;
    const int b = tid + d < 1024 ? first_start[tid + d] : T;
    __syncthreads();
    last_start[tid] = max(last_start[tid], a);
    first_start[tid] = min(first_start[tid], b);
    __syncthreads();
  }
  int start = tid > 0 ? last_start[tid - 1] : 0;
  const int after = tid < 1023 ? first_start[tid + 1] : T;   // first start beyond the segment
  int end = -1;
  for (int t = lo; t < hi; ++t) {
    if (t == 0 || doc[t] != doc[t - 1]) {
      start = t;
      end = -1;
    }
    if (end < 0) {
      end = t + 1;
      while (end < hi && doc[end] == doc[t]) ++end;
      if (end == hi) end = after;
    }
    int2 r = make_int2(start, end);
    if (causal) {
      int see = t + 1;
      if (prefix) {
        const int64_t reach = static_cast<int64_t>(start) + prefix[t];
        if (reach > see) see = static_cast<int>(min(reach, static_cast<int64_t>(end)));
      }
      r.y = min(see, end);
    }
    if (doc[t] < 0) r = make_int2(0, 0);
    ranges[t] = r;
  }
}

hipError_t launch_attn_ranges(const int32_t* doc, const int32_t* prefix, int B, int T, int causal,
                              int32_t* ranges, hipStream_t s) {
  attn_ranges_kernel<<<B, 1024, 0, s>>>(doc, prefix, T, causal, reinterpret_cast<int2*>(ranges));
  return hipGetLastError();
}

}  // namespace zo
