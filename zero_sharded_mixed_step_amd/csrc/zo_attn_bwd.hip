// zo_attn_bwd.hip -- attention, backward, with no atomics: one kernel owns
// keys and walks the queries (dk, dv), one owns queries and walks the keys (dq
// and the bias gradient).  Scores are formed again from q, k and the saved
// lse in both: 7 matrix products instead of the 5 of a kernel that adds dq
// through memory, for gradients that have one fixed order of summation.
//
// A first kernel leaves delta = do . o and the lse in units of log2 in the
// workspace, and the ranges, clipped, all padded to whole tiles of 64 queries.
#include "zo_attn.h"
#include "zo_internal.h"

namespace zo {

// 64 queries of one (batch, head): 4 threads to a row.
__global__ __launch_bounds__(256) void attn_bwd_prepare_kernel(const AttnParams p, int D) {
  const int bh = blockIdx.x, b = bh / p.Hq, h = bh % p.Hq;
  const int tid = threadIdx.x, sub = tid & 3;
  const int i = blockIdx.y * 64 + (tid >> 2);
  float sum = 0.f;
  const int2 r = key_range(p, b, i);
  if (r.y > r.x) {
    const bf16* o = p.o + b * p.os.b + static_cast<int64_t>(i) * p.os.t + h * p.os.h;
    const bf16* g = p.d_o + b * p.dos.b + static_cast<int64_t>(i) * p.dos.t + h * p.dos.h;
    for (int c = sub * 8; c < D; c += 32) {
      const bf16x8 x = load8(o + c), y = load8(g + c);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        sum = __builtin_fmaf(static_cast<float>(x[e]), static_cast<float>(y[e]), sum);
    }
  }
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
  if (sub == 0) {
    const int64_t row = static_cast<int64_t>(bh) * p.tq64 + i;
    p.delta[row] = sum;
    float lse = -kInf;
    if (r.y > r.x) lse = p.lse[static_cast<int64_t>(bh) * p.Tq + i];
    p.lse2[row] = lse != -kInf ? lse * kLog2e : kInf;
    if (h == 0) {
      p.qlo[static_cast<int64_t>(b) * p.tq64 + i] = r.x;
      p.qhi[static_cast<int64_t>(b) * p.tq64 + i] = r.y;
    }
  }
}

// One score's p, ds and dx, from the raw product x, dp, and base = bias - lse2 (plus c2
// with a cap).  With a cap, u = (1 - tanh) / 2 and dx is a quarter of ds (1 -
// tanh^2) = 4 ds u (1 - u): the 4 goes into the gradients' final scale.
template <bool CAP>
__device__ __forceinline__ void grad_score(float x, float base, float dp, float delta,
                                           const ScoreFactors& f, float& pr, float& ds,
                                           float& dx) {
  if constexpr (CAP) {
    const float u = rcp_hw(exp2_hw(x * f.a) + 1.f);
    pr = exp2_hw(__builtin_fmaf(u, -2.f * f.c2, base));
    ds = pr * (dp - delta);
    dx = ds * __builtin_fmaf(-u, u, u);
  } else {
    pr = exp2_hw(__builtin_fmaf(x, f.a, base));
    ds = pr * (dp - delta);
    dx = ds;
  }
}

// ---------------------------------------------------------------- dk, dv ---

// One tile of 64 queries for a wave's 32 keys.  FULL: every query sees every key.
template <int D, bool CAP, bool BIAS, bool FULL>
__device__ __forceinline__ void attn_dkv_tile(const AttnParams& p, const FragAt<D>& qt,
                                              const FragAt<D>& gt, const float* stat,
                                              const bf16x8 (&kf)[D / 16],
                                              const bf16x8 (&vf)[D / 16], f32x16 (&dk)[D / 32],
                                              f32x16 (&dv)[D / 32], int j, int jw, int i0,
                                              const ScoreFactors& f, const float* bias, int lane) {
  const int half = lane >> 5;
  const int* lo = reinterpret_cast<const int*>(stat) + 2 * kTile;
  const int* hi = lo + kTile;
#pragma unroll
  for (int s = 0; s < 2; ++s) {          // 32 queries at a time
    f32x16 x, dp;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) x = mfma(frag_rows<D>(qt, s, c), kf[c], x);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dp = mfma(frag_rows<D>(gt, s, c), vf[c], dp);
    const int d0 = jw - (i0 + 32 * s + p.off);         // distances span d0 - 31 .. d0 + 31
    const int side = BIAS ? bias_side(d0 - 31, d0 + 31, p.reach) : 1;
    const float* row = bias + d0 + (lane & 31) - 4 * half + bias_span(p.reach);
    const float end = BIAS ? bias[side < 0 ? 0 : 2 * bias_span(p.reach)] : 0.f;
    float pr[16], dx[16];
    uint32_t keep[2] = {0, 0};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 32 * s + 8 * g + 4 * half;
      const f32x4 lse = *reinterpret_cast<const f32x4*>(stat + at);
      const f32x4 del = *reinterpret_cast<const f32x4*>(stat + kTile + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * g + e;
        float base = (CAP ? f.c2 : 0.f) - lse[e];
        if constexpr (BIAS) base += side != 0 ? end : row[-(8 * g + e)];
        float ds;
        grad_score<CAP>(x[r], base, dp[r], del[e], f, pr[r], ds, dx[r]);
        if constexpr (!FULL) {
          const bool seen = j >= lo[at + e] && j < hi[at + e];
          pr[r] = seen ? pr[r] : 0.f;
          dx[r] = seen ? dx[r] : 0.f;
          keep[r >> 3] |= any_in_half(seen, lane) << (r & 7);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16x8 pf = to_frag(pr + 8 * u), xf = to_frag(dx + 8 * u);
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        bf16x8 of = frag_cols<D>(gt, 2 * s + u, t);
        if constexpr (!FULL) of = keep_frag(of, keep[u]);
        dv[t] = mfma(of, pf, dv[t]);
      }
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        bf16x8 qf = frag_cols<D>(qt, 2 * s + u, t);
        if constexpr (!FULL) qf = keep_frag(qf, keep[u]);
        dk[t] = mfma(qf, xf, dk[t]);
      }
    }
  }
}

// A workgroup owns 128 keys of one key head, 32 to a wave, and walks tiles of
// 64 queries of the query heads that share it, or of a part of them.
template <int D, bool CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, D >= 96 ? 1 : 2) void attn_dkv_kernel(const AttnParams p) {
  constexpr int kStat = 4 * kTile * 4;                 // lse2, delta, lo, hi of a tile
  extern __shared__ __align__(1024) char smem[];       // [2] tiles of q, of do
  const uint32_t tiles = lds_address(smem);
  char* stats = smem + 4 * kTileBytes<D>;              // [2] kStat
  int* span = reinterpret_cast<int*>(stats + 2 * kStat);             // [kWaves][2]
  float* bias = reinterpret_cast<float*>(span + 2 * kWaves);

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bx = head_of_group(blockIdx.x, gridDim.x);
  const int part = bx % p.parts, bk = bx / p.parts, b = bk / p.Hk, hk = bk % p.Hk;
  const int j0 = blockIdx.y * 128;                     // the workgroup's first key
  const int jw = j0 + wave * 32, j = jw + (lane & 31);
  const int* qlo = p.qlo + static_cast<int64_t>(b) * p.tq64;
  const int* qhi = p.qhi + static_cast<int64_t>(b) * p.tq64;
  const ScoreFactors f(p, CAP);
  const FragAt<D> at(lane);
  const int heads = p.group / p.parts, h0 = hk * p.group + part * heads;

  // the tiles of queries that see any of the keys lie in [qa, qb)
  int qa = 0x7FFFFFFF, qb = 0;
  for (int i = tid; i < p.tq64; i += kAttnThreads) {
    const int lo = qlo[i], hi = qhi[i];
    if (lo < j0 + 128 && hi > j0 && hi > lo) {
      qa = min(qa, i / kTile);
      qb = max(qb, i / kTile + 1);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    qa = min(qa, __shfl_xor(qa, d));
    qb = max(qb, __shfl_xor(qb, d));
  }
  if (lane == 0) {
    span[2 * wave] = qa;
    span[2 * wave + 1] = qb;
  }
  if constexpr (BIAS) stage_bias(p, h0, bias, tid);    // (a bias goes with one head a workgroup)
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    qa = min(qa, span[2 * w]);
    qb = max(qb, span[2 * w + 1]);
  }
  qb = __builtin_amdgcn_readfirstlane(qb);
  qa = __builtin_amdgcn_readfirstlane(min(qa, qb));
  const int turns = (qb - qa) * heads;

  int head = 0, qi = qa;                               // of the next tile to stage
  const auto stage = [&](int buf) {
    const int64_t bh = static_cast<int64_t>(b) * p.Hq + h0 + head;
    const bf16* qg = p.q + b * p.qs.b + (h0 + head) * p.qs.h;
    const bf16* og = p.d_o + b * p.dos.b + (h0 + head) * p.dos.h;
    load_tile<D>(tiles + buf * kTileBytes<D>, qg, p.qs.t, qi * kTile, 0, p.Tq, wave, lane);
    load_tile<D>(tiles + (2 + buf) * kTileBytes<D>, og, p.dos.t, qi * kTile, 0, p.Tq, wave, lane);
    const uint32_t to = tiles + 4 * kTileBytes<D> + buf * kStat + wave * kTile * 4;
    const int i0 = qi * kTile;
    const void* from = wave == 0   ? static_cast<const void*>(p.lse2 + bh * p.tq64 + i0)
                       : wave == 1 ? static_cast<const void*>(p.delta + bh * p.tq64 + i0)
                       : wave == 2 ? static_cast<const void*>(qlo + i0)
                                   : static_cast<const void*>(qhi + i0);
    load_words(to, from, lane);
    if (++qi == qb) {
      qi = qa;
      ++head;
    }
  };
  if (turns > 0) stage(0);
  bf16x8 kf[D / 16], vf[D / 16];
  {
    const int64_t jj = min(j, p.Tk - 1);
    const bf16* k = p.k + b * p.ks.b + jj * p.ks.t + hk * p.ks.h;
    const bf16* v = p.v + b * p.vs.b + jj * p.vs.t + hk * p.vs.h;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      kf[c] = signed_frag(load8(k + 16 * c + 8 * half), f.flip);
      vf[c] = load8(v + 16 * c + 8 * half);
    }
  }
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[t][r] = dv[t][r] = 0.f;
  wait_tile();

  int n = 0, buf = 0, i0 = qa * kTile;                 // of the tile at hand
  const auto stat_of = [&] { return reinterpret_cast<const float*>(stats + buf * kStat); };
  const auto turn = [&](auto full) {
    if (n + 1 < turns) stage(buf ^ 1);
    const float* stat = stat_of();
    bool some = full.value;
    if constexpr (!full.value) {
      const int lo = reinterpret_cast<const int*>(stat)[2 * kTile + lane];
      const int hi = reinterpret_cast<const int*>(stat)[3 * kTile + lane];
      some = __any(lo < jw + 32 && hi > jw && hi > lo) != 0;
    }
    if (some) {
      const FragAt<D> qt = at.in(tiles + buf * kTileBytes<D>);
      const FragAt<D> gt = at.in(tiles + (2 + buf) * kTileBytes<D>);
      attn_dkv_tile<D, CAP, BIAS, full.value>(p, qt, gt, stat, kf, vf, dk, dv, j, jw, i0, f, bias,
                                              lane);
    }
    wait_tile();
    ++n;
    buf ^= 1;
    i0 = i0 + kTile == qb * kTile ? qa * kTile : i0 + kTile;
  };
  const auto sees_all = [&] {
    const int* stat = reinterpret_cast<const int*>(stat_of());
    return __all(stat[2 * kTile + lane] <= jw && stat[3 * kTile + lane] >= jw + 32) != 0;
  };
  while (n < turns) {
    while (n < turns && !sees_all()) turn(Bool<false>());
    while (n < turns && sees_all()) turn(Bool<true>());
  }

  if (j >= p.Tk) return;
  const float ks = p.scale * (CAP ? 4.f : 1.f);
  if (p.parts > 1) {
    const int64_t rows = static_cast<int64_t>(p.parts) * p.B * p.Hk * p.Tk;
    float* ok = p.kvpart + ((static_cast<int64_t>(part) * p.B * p.Hk + bk) * p.Tk + j) * D;
    float* ov = ok + rows * D;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        f32x4 x, y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = dk[t][r + e] * ks;
          y[e] = dv[t][r + e];
        }
        *reinterpret_cast<f32x4*>(ok + 32 * t + result_row(r, lane)) = x;
        *reinterpret_cast<f32x4*>(ov + 32 * t + result_row(r, lane)) = y;
      }
    return;
  }
  bf16* ok = p.dk + b * p.dks.b + static_cast<int64_t>(j) * p.dks.t + hk * p.dks.h;
  bf16* ov = p.dv + b * p.dvs.b + static_cast<int64_t>(j) * p.dvs.t + hk * p.dvs.h;
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      bf16x4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = static_cast<bf16>(dk[t][r + e] * ks);
        y[e] = static_cast<bf16>(dv[t][r + e]);
      }
      *reinterpret_cast<bf16x4*>(ok + 32 * t + result_row(r, lane)) = x;
      *reinterpret_cast<bf16x4*>(ov + 32 * t + result_row(r, lane)) = y;
    }
}

// dk and dv from the parts, in the order of the heads: 8 values to a thread.
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(const AttnParams p, int D) {
  const int64_t n = static_cast<int64_t>(p.B) * p.Hk * p.Tk * D;      // of one part
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (at >= n) return;
  const int d = static_cast<int>(at % D);
  const int64_t row = at / D, j = row % p.Tk, bk = row / p.Tk, b = bk / p.Hk, hk = bk % p.Hk;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float* from = p.kvpart + which * p.parts * n + at;
    f32x4 x = *reinterpret_cast<const f32x4*>(from), y = *reinterpret_cast<const f32x4*>(from + 4);
    for (int k = 1; k < p.parts; ++k) {
      x += *reinterpret_cast<const f32x4*>(from + k * n);
      y += *reinterpret_cast<const f32x4*>(from + k * n + 4);
    }
    bf16x8 out;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = static_cast<bf16>(x[e]);
      out[4 + e] = static_cast<bf16>(y[e]);
    }
    bf16* to = which == 0 ? p.dk + b * p.dks.b + j * p.dks.t + hk * p.dks.h
                          : p.dv + b * p.dvs.b + j * p.dvs.t + hk * p.dvs.h;
    *reinterpret_cast<bf16x8*>(to + d) = out;
  }
}

// ------------------------------------------------ dq and the bias gradient ---

// One tile of 64 keys for a wave's 32 queries.  `mine`: the half wave's sums of ds by
// distance (nullptr: not wanted), at distance 0 - lane; `ends`: of the distances past the reach.
template <int D, bool CAP, bool BIAS, bool FULL>
__device__ __forceinline__ void attn_dq_tile(const AttnParams& p, const FragAt<D>& kt,
                                             const FragAt<D>& vt, const bf16x8 (&qf)[D / 16],
                                             const bf16x8 (&of)[D / 16], f32x16 (&dq)[D / 32],
                                             int2 rng, float lse2, float delta, int k0, int i0,
                                             const ScoreFactors& f, const float* bias,
                                             uint32_t mine, float (&ends)[2], int lane) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    f32x16 x, dp;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) x = mfma(frag_rows<D>(kt, s, c), qf[c], x);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dp = mfma(frag_rows<D>(vt, s, c), of[c], dp);
    const int d0 = k0 + 32 * s - (i0 + p.off);         // distances span d0 - 31 .. d0 + 31
    const int side = BIAS ? bias_side(d0 - 31, d0 + 31, p.reach) : 1;
    const int from = d0 - (lane & 31) + 4 * (lane >> 5) + bias_span(p.reach);
    const float end = BIAS ? bias[side < 0 ? 0 : 2 * bias_span(p.reach)] : 0.f;
    const float base0 = (CAP ? f.c2 : 0.f) - lse2;
    float dx[16], all = 0.f;
    uint32_t keep[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int to = 8 * (r >> 2) + (r & 3);
      float base = base0, pr, ds;
      if constexpr (BIAS) base += side != 0 ? end : bias[from + to];
      grad_score<CAP>(x[r], base, dp[r], delta, f, pr, ds, dx[r]);
      if constexpr (!FULL) {
        const int j = k0 + 32 * s + result_row(r, lane);
        const bool seen = j >= rng.x && j < rng.y;
        ds = seen ? ds : 0.f;
        dx[r] = seen ? dx[r] : 0.f;
        keep[r >> 3] |= any_in_half(seen, lane) << (r & 7);
      }
      if constexpr (BIAS) {
        if (side != 0)
          all += ds;
        else
          __builtin_amdgcn_ds_faddf(reinterpret_cast<ZO_LDS float*>(mine + 4 * (from + to)), ds, 0,
                                    0, false);
      }
    }
    if constexpr (BIAS) ends[0] += side < 0 ? all : 0.f;
    if constexpr (BIAS) ends[1] += side > 0 ? all : 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16x8 xf = to_frag(dx + 8 * u);
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        bf16x8 kf = frag_cols<D>(kt, 2 * s + u, t);
        if constexpr (!FULL) kf = keep_frag(kf, keep[u]);
        dq[t] = mfma(kf, xf, dq[t]);
      }
    }
  }
}

// A workgroup owns 128 queries of one head, 32 to a wave, and walks tiles of
// 64 keys.  With the bias, sums of ds by distance are kept per half wave in
// shared memory: the 32 lanes of a half wave hold 32 consecutive queries, so
// at one key row their distances, and the addresses they add to, all differ,
// and every address has one writer at a time, in program order.  Blocks that
// lie past the reach share a bucket and are summed in two registers instead.
template <int D, bool CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_dq_kernel(const AttnParams p) {
  extern __shared__ __align__(1024) char smem[];       // [2] tiles of k, of v
  const uint32_t tiles = lds_address(smem);
  int* hull = reinterpret_cast<int*>(smem + 4 * kTileBytes<D>);      // [kWaves][2]
  float* past = reinterpret_cast<float*>(hull + 2 * kWaves);         // [kWaves][2]
  float* bias = past + 2 * kWaves;                                   // [entries]
  const int entries = BIAS ? bias_entries(p.reach) : 0;
  float* hist = bias + entries;                                      // [8][entries]

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bh = head_of_group(blockIdx.x, gridDim.x), b = bh / p.Hq, h = bh % p.Hq;
  const int hk = h / p.group;
  const int tile = gridDim.y - 1 - blockIdx.y;
  const int i0 = tile * 128 + wave * 32;
  const int i = i0 + (lane & 31);
  const ScoreFactors f(p, CAP);
  const FragAt<D> at(lane);

  const int2 rng = key_range(p, b, i);
  const int2 wh = wave_hull(rng);
  if (lane == 0) {
    hull[2 * wave] = wh.x;
    hull[2 * wave + 1] = wh.y;
  }
  float ends[2] = {0.f, 0.f};
  uint32_t mine = 0;
  if constexpr (BIAS) {
    stage_bias(p, h, bias, tid);
    for (int d = tid; d < 8 * entries; d += kAttnThreads) hist[d] = 0.f;
    mine = lds_address(hist + (2 * wave + half) * entries);
  }
  __syncthreads();
  int first = 0x7FFFFFFF, last = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    first = min(first, hull[2 * w]);
    last = max(last, hull[2 * w + 1]);
  }
  first = __builtin_amdgcn_readfirstlane(min(first, last));
  last = __builtin_amdgcn_readfirstlane(last);

  const bf16* kg = p.k + b * p.ks.b + hk * p.ks.h;
  const bf16* vg = p.v + b * p.vs.b + hk * p.vs.h;
  const auto stage = [&](int buf, int row0) {
    load_tile<D>(tiles + buf * kTileBytes<D>, kg, p.ks.t, row0, first, last, wave, lane);
    load_tile<D>(tiles + (2 + buf) * kTileBytes<D>, vg, p.vs.t, row0, first, last, wave, lane);
  };
  int k0 = first & ~(kTile - 1);
  if (k0 < last) stage(0, k0);
  bf16x8 qf[D / 16], of[D / 16];
  {
    const int64_t ii = min(i, p.Tq - 1);
    const bf16* q = p.q + b * p.qs.b + ii * p.qs.t + h * p.qs.h;
    const bf16* o = p.d_o + b * p.dos.b + ii * p.dos.t + h * p.dos.h;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qf[c] = signed_frag(load8(q + 16 * c + 8 * half), f.flip);
      of[c] = load8(o + 16 * c + 8 * half);
    }
  }
  const int64_t row = static_cast<int64_t>(bh) * p.tq64 + min(i, p.tq64 - 1);
  const float lse2 = p.lse2[row], delta = p.delta[row];
  f32x16 dq[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[t][r] = 0.f;
  wait_tile();

  int buf = 0;
  const auto turn = [&](auto full) {
    if (k0 + kTile < last) stage(buf ^ 1, k0 + kTile);
    if (full.value || (wh.x < k0 + kTile && wh.y > k0)) {
      const FragAt<D> kt = at.in(tiles + buf * kTileBytes<D>);
      const FragAt<D> vt = at.in(tiles + (2 + buf) * kTileBytes<D>);
      attn_dq_tile<D, CAP, BIAS, full.value>(p, kt, vt, qf, of, dq, rng, lse2, delta, k0, i0, f,
                                             bias, mine, ends, lane);
    }
    wait_tile();
    k0 += kTile;
    buf ^= 1;
  };
  const auto sees_all = [&] { return __all(rng.x <= k0 && rng.y >= k0 + kTile) != 0; };
  while (k0 < last) {
    while (k0 < last && !sees_all()) turn(Bool<false>());
    while (k0 < last && sees_all()) turn(Bool<true>());
  }

  if (i < p.Tq) {
    const float ks = p.scale * (CAP ? 4.f : 1.f);
    bf16* o = p.dq + b * p.dqs.b + static_cast<int64_t>(i) * p.dqs.t + h * p.dqs.h;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        bf16x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = static_cast<bf16>(dq[t][r + e] * ks);
        *reinterpret_cast<bf16x4*>(o + 32 * t + result_row(r, lane)) = x;
      }
  }
  if constexpr (BIAS) {
    if (p.dtable == nullptr) return;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      ends[0] += __shfl_xor(ends[0], d);
      ends[1] += __shfl_xor(ends[1], d);
    }
    if (lane == 0) {
      past[2 * wave] = ends[0];
      past[2 * wave + 1] = ends[1];
    }
    __syncthreads();
    for (int d = tid; d < entries; d += kAttnThreads) {    // by distance, in the bias' place
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) x += hist[w * entries + d];
      if (d == 0) x += past[0] + past[2] + past[4] + past[6];
      if (d == entries - 1) x += past[1] + past[3] + past[5] + past[7];
      bias[d] = x;
      hist[d] = __int_as_float(bias_bucket(p, d - bias_span(p.reach)));   // (its own entry)
    }
    __syncthreads();
    float* out = p.dpart + (static_cast<int64_t>(bh) * gridDim.y + tile) * p.n_buckets;
    for (int bucket = wave; bucket < p.n_buckets; bucket += kWaves) {
      float x = 0.f;
      for (int d = lane; d < entries; d += 64)
        x += __float_as_int(hist[d]) == bucket ? bias[d] : 0.f;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
      if (lane == 0) out[bucket] = x;
    }
  }
}

// dbias_table[bucket][h]: the parts of all batch rows and query tiles, a
// workgroup to an element.
__global__ __launch_bounds__(256) void attn_dtable_kernel(const AttnParams p, int tiles) {
  __shared__ float part[256];
  const int h = blockIdx.x, bucket = blockIdx.y, tid = threadIdx.x;
  float x = 0.f;
  for (int64_t n = tid; n < static_cast<int64_t>(p.B) * tiles; n += 256) {
    const int64_t b = n / tiles, t = n % tiles;
    x += p.dpart[((b * p.Hq + h) * tiles + t) * p.n_buckets + bucket];
  }
  part[tid] = x;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if (tid < w) part[tid] += part[tid + w];
    __syncthreads();
  }
  if (tid == 0) {
    const int64_t at = static_cast<int64_t>(bucket) * p.Hq + h;
    if (p.table_f32)
      static_cast<float*>(p.dtable)[at] = part[0];
    else
      static_cast<bf16*>(p.dtable)[at] = static_cast<bf16>(part[0]);
  }
}

namespace {

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

int up64(int n) { return (n + kTile - 1) / kTile * kTile; }

// In how many parts a key head's query heads are taken: enough for two
// workgroups to a compute unit, and one head each with a bias (whose table in
// shared memory is one head's).
int choose_parts(int B, int Tk, int Hq, int Hk, bool bias) {
  const int group = Hq / Hk;
  if (bias) return group;
  const int64_t groups = static_cast<int64_t>(B) * Hk * ((Tk + 127) / 128);
  int parts = 1;
  while (parts < group && (group % parts != 0 || groups * parts < 512)) ++parts;
  return parts;
}

template <typename F>
hipError_t launch_lds(F fn, dim3 grid, size_t lds, const AttnParams& p, hipStream_t s) {
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds));
  if (e != hipSuccess) return e;
  fn<<<grid, kAttnThreads, lds, s>>>(p);
  return hipGetLastError();
}

template <int D, bool CAP, bool BIAS>
hipError_t run_bwd(const AttnParams& p, hipStream_t s) {
  const size_t n = BIAS ? bias_entries(p.reach) : 0;
  const int tiles = (p.Tq + 127) / 128;
  const size_t staged = 4 * kTileBytes<D>;
  hipError_t e = hipSuccess;
  if (p.B > 0 && p.Tk > 0) {
    e = launch_lds(attn_dkv_kernel<D, CAP, BIAS>, dim3(p.B * p.Hk * p.parts, (p.Tk + 127) / 128),
                   staged + 8 * kTile * 4 + 2 * kWaves * 4 + n * 4, p, s);
    if (e != hipSuccess) return e;
    if (p.parts > 1) {
      const int64_t pieces = static_cast<int64_t>(p.B) * p.Hk * p.Tk * D / 8;
      attn_dkv_join_kernel<<<static_cast<unsigned>((pieces + 255) / 256), 256, 0, s>>>(p, D);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (p.B > 0 && p.Tq > 0)
    e = launch_lds(attn_dq_kernel<D, CAP, BIAS>, dim3(p.B * p.Hq, tiles),
                   staged + 4 * kWaves * 4 + 9 * n * 4, p, s);
  if (e != hipSuccess) return e;
  if (BIAS && p.dtable) {
    attn_dtable_kernel<<<dim3(p.Hq, p.n_buckets), 256, 0, s>>>(p, tiles);
    e = hipGetLastError();
  }
  return e;
}

template <int D>
hipError_t pick_bwd(const AttnParams& p, hipStream_t s) {
  if (p.cap > 0.f)
    return p.table ? run_bwd<D, true, true>(p, s) : run_bwd<D, true, false>(p, s);
  return p.table ? run_bwd<D, false, true>(p, s) : run_bwd<D, false, false>(p, s);
}

// The workspace, in order; returns its size.
size_t lay_out(AttnParams& p, int D, int n_buckets, char* base) {
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    char* x = base + at;
    at += up16(bytes);
    return x;
  };
  const size_t rows = static_cast<size_t>(p.B) * p.tq64, parts = p.parts > 1 ? p.parts : 0;
  p.lse2 = reinterpret_cast<float*>(take(rows * p.Hq * 4));
  p.delta = reinterpret_cast<float*>(take(rows * p.Hq * 4));
  p.qlo = reinterpret_cast<int*>(take(rows * 4));
  p.qhi = reinterpret_cast<int*>(take(rows * 4));
  p.dpart = reinterpret_cast<float*>(
      take(static_cast<size_t>(p.B) * p.Hq * ((p.Tq + 127) / 128) * n_buckets * 4));
  p.kvpart = reinterpret_cast<float*>(take(2 * parts * p.B * p.Hk * p.Tk * D * 4));
  return at;
}

}  // namespace

size_t attn_bwd_workspace(int B, int Tq, int Tk, int Hq, int Hk, int D, int n_buckets) {
  AttnParams p = {};
  p.B = B;
  p.Tq = Tq;
  p.tq64 = up64(Tq);
  p.Tk = Tk;
  p.Hq = Hq;
  p.Hk = Hk;
  p.parts = choose_parts(B, Tk, Hq, Hk, n_buckets > 0);
  return lay_out(p, D, n_buckets, nullptr);
}

hipError_t launch_attn_bwd(const zero_attn_args& a, hipStream_t s) {
  AttnParams p = attn_params(a);
  p.tq64 = up64(a.Tq);
  p.parts = choose_parts(a.B, a.Tk, a.Hq, a.Hk, a.bias_table != nullptr);
  lay_out(p, a.D, a.bias_table ? a.n_buckets : 0, static_cast<char*>(a.workspace));
  if (a.B > 0 && a.Tq > 0) {
    attn_bwd_prepare_kernel<<<dim3(a.B * a.Hq, p.tq64 / 64), 256, 0, s>>>(p, a.D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (a.D) {
    case 32: return pick_bwd<32>(p, s);
    case 64: return pick_bwd<64>(p, s);
    case 96: return pick_bwd<96>(p, s);
    default: return pick_bwd<128>(p, s);
  }
}

}  // namespace zo
