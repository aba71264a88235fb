// zo_attn_bwd.hip -- attention, backward, with no atomics: one kernel owns
// keys and walks the queries (dk, dv), one owns queries and walks the keys (dq
// and the bias gradient).  Scores are formed again from q, k and the saved
// lse in both: 7 matrix products instead of the 5 of a kernel that adds dq
// through memory, for gradients that have one fixed order of summation.
//
// A first kernel leaves delta = do . o, minus the lse in units of log2 and the
// ranges, clipped, in the workspace, all padded to whole tiles of 64 queries, and
// which tiles of queries see a tile of keys.
//
// Measured, counting 5 products: 670 TFLOP/s at 128 columns, 705 at 96 and 620 at 64 (4096 keys,
// 16 heads, no mask), 405 with a cap, 32 heads on 8 of 128 and documents of 1325 and 2671
// tokens (465 us).  No unit is near full there: in the keys' kernel the matrix units are busy 22 %
// of the time, vector issue is about a third of the busy time, waves wait 30 % of it, and units
// are idle 22 % (512 uneven workgroups on 256).  What costs is work that follows on itself: a
// block's products, its scores (an exponential each, with a cap one more and a reciprocal, at a
// quarter of the rate of other instructions), the gradients' products.
#include "zo_attn.h"
#include "zo_internal.h"

#include <type_traits>

namespace zo {

// The bits 0 .. n - 1 (n from below 0 to above 64).
__device__ __forceinline__ uint64_t bits_below(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
}

// A row's lse from which on down the row takes no part: every key that it sees has a bias
// that masks it.
constexpr float kLseLost = -16777216.f;

// What sees a tile of 128 keys (p.tile), by a workgroup.
__device__ __forceinline__ void key_tile_words(const AttnParams& p, int b, int t, int tid) {
  __shared__ int words[kWaves][kTileWords];
  const int j0 = 128 * t, wave = tid >> 6;
  int qa = 0x7FFFFFFF, qb = 0;
  uint64_t seen_lo = 0, seen_hi = 0;
  for (int i0 = tid; i0 < p.Tq; i0 += 8 * kAttnThreads) {  // 8 loads under way at a time
    int2 r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = key_range(p, b, i0 + k * kAttnThreads);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int lo = max(r[k].x - j0, 0), hi = min(r[k].y - j0, 128);
      if (lo < hi) {
        const int t = (i0 + k * kAttnThreads) / kTile;
        qa = min(qa, t);
        qb = max(qb, t + 1);
        seen_lo |= bits_below(hi) & ~bits_below(lo);
        seen_hi |= bits_below(hi - 64) & ~bits_below(lo - 64);
      }
    }
  }
  const uint32_t mine[4] = {static_cast<uint32_t>(seen_lo), static_cast<uint32_t>(seen_lo >> 32),
                            static_cast<uint32_t>(seen_hi), static_cast<uint32_t>(seen_hi >> 32)};
  qa = join_lanes<64>(qa, MinOp());
  qb = join_lanes<64>(qb, MaxOp());
  uint32_t all[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) all[w] = join_lanes<64>(mine[w], OrOp());
  if ((tid & 63) == 0) {
    words[wave][0] = qa;
    words[wave][1] = qb;
    for (int w = 0; w < 4; ++w) words[wave][2 + w] = all[w];
  }
  __syncthreads();
  if (tid < kTileWords) {
    int x = words[0][tid];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const int y = words[w][tid];
      x = tid == 0 ? min(x, y) : tid == 1 ? max(x, y) : x | y;
    }
    p.tile[(static_cast<int64_t>(b) * ((p.Tk + 127) / 128) + t) * kTileWords + tid] = x;
  }
}

// 64 queries of one (batch, head): 4 threads to a row.  The workgroups before those of
// the queries, `before` a head, take tiles of 128 keys, the heads of a batch row in turn.
__global__ __launch_bounds__(256) void attn_bwd_prepare_kernel(const AttnParams p, int D, int before) {
  const int bh = blockIdx.x, b = bh / p.Hq, h = bh % p.Hq;
  const int tid = threadIdx.x, sub = tid & 3;
  if (static_cast<int>(blockIdx.y) < before) {
    const int t = blockIdx.y * p.Hq + h;
    if (128 * t < p.Tk) key_tile_words(p, b, t, tid);
    return;
  }
  const int i = (blockIdx.y - before) * 64 + (tid >> 2);
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
  sum = join_lanes<4>(sum, AddOp());
  if (sub == 0) {
    const int64_t row = static_cast<int64_t>(bh) * p.tq64 + i;
    p.delta[row] = sum;
    float lse = -kInf;
    if (r.y > r.x) lse = p.lse[static_cast<int64_t>(bh) * p.Tq + i];
    // (below kLseLost binary32 has no place for the log of a sum beside the scores: exp(s - lse)
    // would be any power of 2^64)
    p.base[row] = lse < kLseLost ? -kInf
                                 : (cap_form(p.cap) == kByU ? p.cap * kLog2e : 0.f) - lse * kLog2e;
    if (h == 0) {
      p.qlo[static_cast<int64_t>(b) * p.tq64 + i] = r.x;
      p.qhi[static_cast<int64_t>(b) * p.tq64 + i] = r.y;
    }
  }
}

// One score's p, ds and dx, from the raw product x, dp - delta, and base = bias - lse (in log2,
// plus c2 with a cap up to kUCap).  With a cap, u = (1 - tanh) / 2 and dx is a quarter of ds
// (1 - tanh^2) = 4 ds u (1 - u): the 4 goes into the gradients' final scale.
template <int CAP>
__device__ __forceinline__ void grad_score(float x, float base, float dp_delta,
                                           const ScoreFactors& f, float& pr, float& ds,
                                           float& dx) {
  if constexpr (CAP != kNoCap) {
    const float u = f.u_of(x);
    pr = exp2_hw(CAP == kByU ? __builtin_fmaf(u, -2.f * f.c2, base) : f.any_cap(x, u) + base);
    ds = pr * dp_delta;
    dx = ds * __builtin_fmaf(-u, u, u);
  } else {
    pr = exp2_hw(__builtin_fmaf(x, f.a, base));
    ds = pr * dp_delta;
    dx = ds;
  }
}

// ---------------------------------------------------------------- dk, dv ---

// The registers of one wave a SIMD for 128 columns, and for 96 with a bias: k, v, dk and
// dv alone take 192 or 144 of the 256 that two waves leave each, and the rest does not fit.
// (Where it does, two waves: 358 us instead of 425 at 96 columns, 275 instead of 333 at
// 64; 4096 keys, 16 heads.)
// A large cap's series has no place beside another wave either: 64 to 128 columns went to
// scratch.
template <int D, int CAP, bool BIAS>
constexpr bool kDkvAlone = D > 96 || (D > 64 && BIAS) || CAP == kAnyCap;

// One tile of 64 queries, do's behind q's, for a wave's 32 keys: two blocks of 32
// queries, of 4 D / 16 matrix instructions and 16 scores a lane each.  A wave that has
// its SIMD for itself overlaps the two by itself: the second block's scores are
// multiplied while the first's are worked on, and the first's gradients while the
// second's are.
template <int D, int CAP, bool BIAS>
struct DkvTile {
  static constexpr bool kOverlap = kDkvAlone<D, CAP, BIAS>;
  static constexpr int kG = kBuffers<D, kDkvAlone<D, CAP, BIAS>> * kTileBytes<D>;  // from q's tile to do's
  static constexpr int kC = D / 16, kT = D / 32;
  const AttnParams& p;
  const ScoreFactors& f;
  const float* bias;
  const bf16x8 (&kf)[kC], (&vf)[kC];
  f32x16 (&dk)[kT], (&dv)[kT];
  int j, jw, i0, lane;
  FragAt<D> qt;
  uint32_t quads, words;

  struct Block {
    f32x16 x, dp;                        // the raw scores; do . v
    bf16x8 pf[2], xf[2];                 // p, dx as operands
    bf16x8 q[kC], g[kC];                 // rows of q, do
    bf16x8 qc[2 * kT], gc[2 * kT];       // columns of q, do
  };

  __device__ __forceinline__ f32x4 quad(int array, int at) const {  // words at + 4 half .. + 3
    return *reinterpret_cast<const ZO_LDS f32x4*>(quads + 4 * (array * kTile + at));
  }
  __device__ __forceinline__ int word(int array, int at) const {    // word at + l % 32
    return *reinterpret_cast<const ZO_LDS int*>(words + 4 * (array * kTile + at));
  }
  __device__ __forceinline__ void rows(Block& k, int s) const {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      k.q[c] = frag_rows<D>(qt, s, c);
      k.g[c] = frag_rows<D>(qt, s, c, kG);
    }
  }
  __device__ __forceinline__ void cols(Block& k, int s) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        k.gc[u * kT + t] = frag_cols<D>(qt, 2 * s + u, t, kG);
        k.qc[u * kT + t] = frag_cols<D>(qt, 2 * s + u, t);
      }
  }
  __device__ __forceinline__ void multiply(Block& k) const {
#pragma unroll
    for (int r = 0; r < 16; ++r) k.x[r] = k.dp[r] = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      k.x = mfma(k.q[c], kf[c], k.x);
      k.dp = mfma(k.g[c], vf[c], k.dp);
    }
  }
  __device__ __forceinline__ void add(const Block& k) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        dv[t] = mfma(k.gc[u * kT + t], k.pf[u], dv[t]);
        dk[t] = mfma(k.qc[u * kT + t], k.xf[u], dk[t]);
      }
  }
  __device__ __forceinline__ bool block_full(int s) const {
    return __all(word(2, 32 * s) <= jw && word(3, 32 * s) >= jw + 32);
  }
  template <bool FULL>
  __device__ __forceinline__ void scores(Block& k, int s) const {
    const int d0 = jw - (i0 + 32 * s + p.off);         // distances span d0 - 31 .. d0 + 31
    const int side = BIAS ? bias_side(d0 - 31, d0 + 31, p.reach) : 1;
    const float* row = bias + d0 + (lane & 31) - 4 * (lane >> 5) + bias_span(p.reach);
    const float end = BIAS ? bias[side < 0 ? 0 : 2 * bias_span(p.reach)] : 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float pr[8], dx[8];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int at = 32 * s + 16 * u + 8 * g;
        const f32x4 base4 = quad(0, at), del = quad(1, at);
        bool out[4] = {};
        if (!FULL) {
          const f32x4 lo = quad(2, at), hi = quad(3, at);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[e] = static_cast<int>(j < __float_as_int(lo[e])) |
                     static_cast<int>(j >= __float_as_int(hi[e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 4 * g + e, r = 8 * u + n;
          float base = base4[e], ds;
          if constexpr (BIAS) base += side != 0 ? end : row[-(16 * u + 8 * g + e)];
          float x = k.x[r], dp_delta = k.dp[r] - del[e];
          // p = 0, whatever score and dp are.  (Three selections before the exponentials and not
          // two behind them, for which the comparisons' results would wait in registers: 465 us
          // instead of 479, 4001 keys, 32 on 8 heads of 128, cap, prefixes.)
          if (!FULL) {
            base = out[e] ? -kInf : base;
            x = out[e] ? 0.f : x;
            dp_delta = out[e] ? 0.f : dp_delta;
          }
          grad_score<CAP>(x, base, dp_delta, f, pr[n], ds, dx[n]);
        }
      }
      k.pf[u] = to_frag(pr);
      k.xf[u] = to_frag(dx);
    }
  }
  // (FIRST reads, then matrix instructions with what fits beside each)
  template <int FIRST, int READS, int BESIDE>
  static __device__ __forceinline__ void interleave() {
    __builtin_amdgcn_sched_group_barrier(0x100, FIRST, 0);
#pragma unroll
    for (int n = 0; n < 2 * kC; ++n) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, BESIDE, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // Holds the operands' making where it stands: it would be moved down to their use.
  static __device__ __forceinline__ void here(Block& k) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      arrived(k.pf[u]);
      arrived(k.xf[u]);
    }
  }
  // FULL: every query of the tile sees all of the wave's keys.  The next tile is staged
  // in three places.
  template <bool FULL, typename S0, typename S1, typename S2>
  __device__ __forceinline__ void overlapped(S0 stage0, S1 stage1, S2 stage2) const {
    Block a, b;
    rows(a, 0);
    __builtin_amdgcn_sched_barrier(0);
    stage0();
    multiply(a);
    __builtin_amdgcn_sched_barrier(0);
    rows(b, 1);
    multiply(b);
    scores<FULL>(a, 0);
    here(a);
    if (!FULL) arrived(b.x), arrived(b.dp);
    interleave<FULL ? 4 : 8, FULL ? 2 : 3, FULL ? 20 : 26>();
    stage1();
    cols(a, 0);
    add(a);
    scores<FULL>(b, 1);
    here(b);
    interleave<FULL ? 8 : 16, FULL ? 3 : 4, FULL ? 20 : 26>();
    stage2();
    cols(b, 1);
    add(b);
    interleave<8, 2, 20>();
  }
  __device__ __forceinline__ void any() const {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Block a;
      rows(a, s);
      multiply(a);
      if (block_full(s))
        scores<true>(a, s);
      else
        scores<false>(a, s);
      cols(a, s);
      add(a);
    }
  }
};

// Which tile of 128 keys a workgroup takes: the most often seen first (see query_tile).
__device__ __forceinline__ int key_tile(const AttnParams& p, const Place& w, int b, int* scratch,
                                        int tid, int at_once) {
  const int n = w.ny, y = w.y;
  if (!p.ranges || p.Tq == 0 || n < kMinRanked || n > kMaxRanked || w.nx * n <= at_once) return y;
  return tile_of_rank(y, n, scratch, tid, [&](int t) {
    const int* words = p.tile + (static_cast<int64_t>(b) * n + t) * kTileWords;
    return max(words[1] - words[0], 0);
  });
}

// A workgroup owns 128 keys of one key head, 32 to a wave, and walks tiles of
// 64 queries of the query heads that share it, or of a part of them.
template <int D, int CAP, bool BIAS>
__device__ __forceinline__ void attn_dkv(const AttnParams& p, const Place& w, char* smem) {
  constexpr int kBufs = kBuffers<D, kDkvAlone<D, CAP, BIAS>>, kTiles = 2 * kBufs;
  constexpr int kAhead = (kBufs - 2) * (2 * TileLoad<D>::kLoads + 1);
  constexpr int kStat = 4 * kTile * 4;                 // base, delta, lo, hi of a tile
  // smem: [kBufs] tiles of q, of do
  const uint32_t tiles = lds_address(smem);
  char* stats = smem + kTiles * kTileBytes<D>;         // [kBufs] kStat
  float* bias = reinterpret_cast<float*>(stats + kBufs * kStat);

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bx = head_of_group(w.x, w.nx);
  const int part = bx % p.parts, bk = bx / p.parts, b = bk / p.Hk, hk = bk % p.Hk;
  BiasStage bs;                                        // (a bias goes with one head a workgroup)
  if constexpr (BIAS) bs.buckets(p, tid);
  const int j0 = key_tile(p, w, b, reinterpret_cast<int*>(smem), tid,
                          kDkvAlone<D, CAP, BIAS> ? kUnits : 2 * kUnits) * 128;   // its first key
  const int jw = j0 + wave * 32, j = jw + (lane & 31);
  const int* qlo = p.qlo + static_cast<int64_t>(b) * p.tq64;
  const int* qhi = p.qhi + static_cast<int64_t>(b) * p.tq64;
  const ScoreFactors f(p, CAP);
  const FragAt<D> at(lane);
  const int heads = p.group / p.parts, h0 = hk * p.group + part * heads;

  if constexpr (BIAS) bs.values(p, h0);
  const int* words = p.tile + (static_cast<int64_t>(b) * w.ny + j0 / 128) * kTileWords;
  int qa = 0, qb = 0;
  uint32_t wave_sees = 0;
  if (p.Tq > 0) {                                      // (without queries there is no workspace)
    qb = uniform(words[1]);
    qa = uniform(min(words[0], qb));
    wave_sees = uniform(words[2 + wave]);
  }
  const int turns = (qb - qa) * heads;

  TileLoad<D> ql(p.q + b * p.qs.b + h0 * p.qs.h, p.qs.t, 0, p.Tq, wave, lane);
  TileLoad<D> ol(p.d_o + b * p.dos.b + h0 * p.dos.h, p.dos.t, 0, p.Tq, wave, lane);
  int qi = qa;                                         // the next tile to stage
  // of the tile's words a wave loads an array of its own
  const int64_t first_head = (static_cast<int64_t>(b) * p.Hq + h0) * p.tq64;
  const uint32_t* words_at = wave == 0   ? reinterpret_cast<const uint32_t*>(p.base + first_head)
                             : wave == 1 ? reinterpret_cast<const uint32_t*>(p.delta + first_head)
                             : wave == 2 ? reinterpret_cast<const uint32_t*>(qlo)
                                         : reinterpret_cast<const uint32_t*>(qhi);
  const int words_step = wave < 2 ? p.tq64 : 0;
  const auto stage_words = [&](int buf, bool on) {
    lds_load4(tiles + kTiles * kTileBytes<D> + buf * kStat + wave * kTile * 4,
              buffer_at(words_at + qi * kTile, static_cast<uint32_t>(on) * kTile * 4), lane * 4);
    const bool end = qi + 1 == qb;
    qi = end ? qa : qi + 1;
    words_at += end ? words_step : 0;
    ql.base += end ? p.qs.h : 0;
    ol.base += end ? p.dos.h : 0;
  };
  const auto stage = [&](int buf) {
    ql.start(tiles + buf * kTileBytes<D>, qi * kTile, wave, lane);
    ol.start(tiles + (kBufs + buf) * kTileBytes<D>, qi * kTile, wave, lane);
    stage_words(buf, true);
  };
#pragma unroll
  for (int k = 0; k < kBufs - 1; ++k)
    if (k < turns) stage(k);
  bf16x8 kf[D / 16], vf[D / 16];
  {
    const int64_t jj = min(j, p.Tk - 1);
    const bf16* k = p.k + b * p.ks.b + jj * p.ks.t + hk * p.ks.h;
    const bf16* v = p.v + b * p.vs.b + jj * p.vs.t + hk * p.vs.h;
    // (a key that no query sees may hold anything)
    const bool seen = (wave_sees >> (lane & 31)) & 1;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      kf[c] = vf[c] = bf16x8{};
      if (seen) {
        kf[c] = signed_frag(load8(k + 16 * c + 8 * half), f.flip);
        vf[c] = load8(v + 16 * c + 8 * half);
      }
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      arrived(kf[c]);
      arrived(vf[c]);
    }
  }
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[t][r] = dv[t][r] = 0.f;
  if constexpr (BIAS) bs.store(p, h0, bias, tid);
  wait_tile();

  int n = 0, buf = 0, i0 = qa * kTile;                 // of the tile at hand
  const auto stat_of = [&] { return reinterpret_cast<const float*>(stats + buf * kStat); };
  const auto word = [&](int k) { return reinterpret_cast<const int*>(stat_of())[k * kTile + lane]; };
  // (A tile's loads, issued in one go by four waves, hold each of them up for most of
  // the 500 cycles that the 32 KiB of 128 columns take to pass: `work` that issues them
  // by itself does so in three places.)
  const auto turn = [&](auto work, bool by_itself = false) {
    const bool more = n + kBufs - 1 < turns;
    if (more && !by_itself) stage((buf + kBufs - 1) % kBufs);
    // a query that sees nothing (padding) may hold anything: cleared, since a weight of 0
    // does not stop a NaN
    const uint64_t seeing = __ballot(word(3) > word(2));
    if (~seeing != 0) {
      clear_rows<D>(tiles + buf * kTileBytes<D>, tiles + (kBufs + buf) * kTileBytes<D>, seeing, tid);
      __syncthreads();
    }
    work();
    if (more)
      wait_tile<kAhead>();
    else
      wait_tile();
    ++n;
    buf = buf + 1 == kBufs ? 0 : buf + 1;
    i0 = i0 + kTile == qb * kTile ? qa * kTile : i0 + kTile;
  };
  const auto seen = [&] { return __any(word(2) < jw + 32 && word(3) > jw) != 0; };
  const auto full = [&] { return __all(word(2) <= jw && word(3) >= jw + 32) != 0; };
  using Tile = DkvTile<D, CAP, BIAS>;
  const auto tile = [&] {
    // the lane's places in the tile's words (opaque: one register each, not one a use)
    const uint32_t stat = tiles + kTiles * kTileBytes<D> + buf * kStat;
    uint32_t quads = stat + 16 * half, words = stat + 4 * (lane & 31);
    asm volatile("" : "+v"(quads), "+v"(words));
    return Tile{p, f, bias, kf, vf, dk, dv, j, jw, i0, lane, at.in(tiles + buf * kTileBytes<D>), quads,
                words};
  };
  const bool near = ql.near && ol.near;
  const auto overlapped = [&](auto is_full) {
    return [&] {
      const bool more = n + kBufs - 1 < turns;
      const int to = (buf + kBufs - 1) % kBufs;
      tile().template overlapped<decltype(is_full)::value>(
          [&] { ql.start_near(tiles + to * kTileBytes<D>, qi * kTile, more, wave); },
          [&] { ol.start_near(tiles + (kBufs + to) * kTileBytes<D>, qi * kTile, more, wave); },
          [&] { stage_words(to, more); });
    };
  };
  while (n < turns) {
    while (n < turns && !seen()) turn([] {});
    if constexpr (Tile::kOverlap) {
      while (n < turns && near && full()) turn(overlapped(std::true_type()), true);
      while (n < turns && near && seen() && !full()) turn(overlapped(std::false_type()), true);
    }
    while (n < turns && !(Tile::kOverlap && near) && seen()) turn([&] { tile().any(); });
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

template <int D, int CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, (kDkvAlone<D, CAP, BIAS> ? 1 : 2)) void attn_dkv_kernel(const AttnParams p) {
  extern __shared__ __align__(1024) char smem[];
  attn_dkv<D, CAP, BIAS>(p, place(), smem);
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

// Adds a 32 x 32 block's ds, summed along its diagonals, to the wave's sums by
// distance at `mine`, of which entry `at` is that of the diagonal through the
// block's corner.  The block is written to shared memory with every row (key)
// turned by its number, so that entry (j - i) mod 32 of row j is that of query i; lane
// c + 32 h then sums column c over the rows at or below the main diagonal (h = 0:
// distance c) or above it (h = 1: distance c - 32).  Adding each value to its
// distance by an atomic in shared memory took ten times as long: those go a
// lane at a time.
constexpr int kDiagWords = 32 * 32;                    // of a wave, before its sums
__device__ __forceinline__ void add_diagonals(const float (&ds)[16], uint32_t mine, int at,
                                              int lane) {
  using F = ZO_LDS float*;
  const uint32_t block = mine - 4 * kDiagWords;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int j = result_row(r, lane);
    *reinterpret_cast<F>(block + 4 * (32 * j + ((j - lane) & 31))) = ds[r];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int c = lane & 31;
  const bool above = lane >= 32;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float x = *reinterpret_cast<F>(block + 4 * (32 * j + c));
    sum += (j < c) == above ? x : 0.f;
  }
  const F to = reinterpret_cast<F>(mine + 4 * (at + c - (above ? 32 : 0)));
  *to += sum;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One tile of 64 keys for a wave's 32 queries.  `mine`: the wave's sums of ds by
// distance, in shared memory; `ends`: of the distances past the reach.
template <int D, int CAP, bool BIAS>
__device__ __forceinline__ void attn_dq_tile(const AttnParams& p, const FragAt<D>& kt,
                                             const FragAt<D>& vt, const bf16x8 (&qf)[D / 16],
                                             const bf16x8 (&of)[D / 16], f32x16 (&dq)[D / 32],
                                             int2 rng, float base0, float delta, int k0, int i0,
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
    float base[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      base[r] = base0;
      if constexpr (BIAS) base[r] += side != 0 ? end : bias[from + 8 * (r >> 2) + (r & 3)];
    }
    if (!__all(rng.x <= k0 + 32 * s && rng.y >= k0 + 32 * s + 32)) {
      const uint32_t n = rng.y - rng.x;
      const int first = k0 + 32 * s + 4 * (lane >> 5) - rng.x;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t j = first + 8 * (r >> 2) + (r & 3);
        base[r] = j < n ? base[r] : -kInf;               // p = 0, whatever x and dp are
        x[r] = j < n ? x[r] : 0.f;
        dp[r] = j < n ? dp[r] : delta;
      }
    }
    float dx[16], ds[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float pr;
      grad_score<CAP>(x[r], base[r], dp[r] - delta, f, pr, ds[r], dx[r]);
    }
    float all = 0.f;
    if constexpr (BIAS) {
      if (side != 0) {
#pragma unroll
        for (int r = 0; r < 16; ++r) all += ds[r];
      } else {
        add_diagonals(ds, mine, d0 + bias_span(p.reach), lane);
      }
    }
    if constexpr (BIAS) ends[0] += side < 0 ? all : 0.f;
    if constexpr (BIAS) ends[1] += side > 0 ? all : 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16x8 xf = to_frag(dx + 8 * u);
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        dq[t] = mfma(frag_cols<D>(kt, 2 * s + u, t), xf, dq[t]);
      }
    }
  }
}

// A workgroup owns 128 queries of one head, 32 to a wave, and walks tiles of
// 64 keys.  With the bias, sums of ds by distance are kept per wave in shared
// memory; blocks that lie past the reach share a bucket and are summed in two
// registers instead.
template <int D, int CAP, bool BIAS>
constexpr bool kDqAlone = (D > 96 && BIAS) || CAP == kAnyCap;

template <int D, int CAP, bool BIAS>
__device__ __forceinline__ void attn_dq(const AttnParams& p, const Place& w, char* smem) {
  constexpr int kBufs = kBuffers<D, kDqAlone<D, CAP, BIAS>>, kTiles = 2 * kBufs;
  constexpr int kAhead = (kBufs - 2) * 2 * TileLoad<D>::kLoads;
  // smem: [kBufs] tiles of k, of v
  const uint32_t tiles = lds_address(smem);
  int2* ranges = reinterpret_cast<int2*>(smem + kTiles * kTileBytes<D>);  // [128]
  int* hull = reinterpret_cast<int*>(ranges + 128);                  // [kWaves][2]
  float* past = reinterpret_cast<float*>(hull + 2 * kWaves);         // [kWaves][2]
  float* bias = past + 2 * kWaves;                                   // [entries]
  const int entries = BIAS ? bias_entries(p.reach) : 0;
  const int hist_words = kDiagWords + entries;                       // a block, then the sums
  float* hist = bias + entries;                                      // [kWaves][hist_words]

  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bh = head_of_group(w.x, w.nx), b = bh / p.Hq, h = bh % p.Hq;
  const int hk = h / p.group;
  BiasStage bs;
  if constexpr (BIAS) bs.buckets(p, tid);
  const int tile = query_tile(p, w, b, reinterpret_cast<int*>(ranges), tid, kDqAlone<D, CAP, BIAS> ? kUnits : 2 * kUnits);
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
  if (lane < 32) ranges[wave * 32 + lane] = rng;
  if constexpr (BIAS) bs.values(p, h);
  float ends[2] = {0.f, 0.f};
  uint32_t mine = 0;
  if constexpr (BIAS) {
    for (int d = lane; d < entries; d += 64) hist[wave * hist_words + kDiagWords + d] = 0.f;
    mine = lds_address(hist + wave * hist_words + kDiagWords);
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

  const TileLoad<D> kl(p.k + b * p.ks.b + hk * p.ks.h, p.ks.t, first, last, wave, lane);
  const TileLoad<D> vl(p.v + b * p.vs.b + hk * p.vs.h, p.vs.t, first, last, wave, lane);
  const auto stage = [&](int buf, int row0) {
    kl.start(tiles + buf * kTileBytes<D>, row0, wave, lane);
    vl.start(tiles + (kBufs + buf) * kTileBytes<D>, row0, wave, lane);
  };
  int k0 = first & ~(kTile - 1);
#pragma unroll
  for (int n = 0; n < kBufs - 1; ++n)
    if (k0 + n * kTile < last) stage(n, k0 + n * kTile);
  bf16x8 qf[D / 16], of[D / 16];
  {
    const int64_t ii = min(i, p.Tq - 1);
    const bf16* q = p.q + b * p.qs.b + ii * p.qs.t + h * p.qs.h;
    const bf16* o = p.d_o + b * p.dos.b + ii * p.dos.t + h * p.dos.h;
    // (a query that sees nothing may hold anything)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qf[c] = of[c] = bf16x8{};
      if (rng.y > rng.x) {
        qf[c] = signed_frag(load8(q + 16 * c + 8 * half), f.flip);
        of[c] = load8(o + 16 * c + 8 * half);
      }
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      arrived(qf[c]);
      arrived(of[c]);
    }
  }
  const int64_t row = static_cast<int64_t>(bh) * p.tq64 + min(i, p.tq64 - 1);
  float base0 = p.base[row], delta = p.delta[row];
  arrived(base0);
  arrived(delta);
  f32x16 dq[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[t][r] = 0.f;
  if constexpr (BIAS) bs.store(p, h, bias, tid);
  const bool gaps = p.ranges && has_gaps(ranges, last, tid);
  wait_tile();

  int buf = 0;
  const auto turn = [&](auto work) {
    const int ahead = k0 + (kBufs - 1) * kTile;
    if (ahead < last) stage((buf + kBufs - 1) % kBufs, ahead);
    if (gaps) {
      const uint64_t seen = seen_keys(ranges, k0, reinterpret_cast<uint32_t*>(hull), tid);
      clear_rows<D>(tiles + buf * kTileBytes<D>, tiles + (kBufs + buf) * kTileBytes<D>, seen, tid);
      __syncthreads();
    }
    work();
    if (ahead < last)
      wait_tile<kAhead>();
    else
      wait_tile();
    k0 += kTile;
    buf = buf + 1 == kBufs ? 0 : buf + 1;
  };
  const auto sees = [&] { return wh.x < k0 + kTile && wh.y > k0; };
  while (k0 < last) {
    while (k0 < last && !sees()) turn([] {});
    while (k0 < last && sees())
      turn([&] {
        attn_dq_tile<D, CAP, BIAS>(p, at.in(tiles + buf * kTileBytes<D>),
                                   at.in(tiles + (kBufs + buf) * kTileBytes<D>), qf, of, dq, rng, base0,
                                   delta, k0, i0, f, bias, mine, ends, lane);
      });
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
    ends[0] = join_lanes<64>(ends[0], AddOp());
    ends[1] = join_lanes<64>(ends[1], AddOp());
    if (lane == 0) {
      past[2 * wave] = ends[0];
      past[2 * wave + 1] = ends[1];
    }
    __syncthreads();
    float* out = p.dpart + (static_cast<int64_t>(bh) * w.ny + tile) * entries;
    for (int d = tid; d < entries; d += kAttnThreads) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) x += hist[w * hist_words + kDiagWords + d];
      if (d == 0) x += past[0] + past[2] + past[4] + past[6];
      if (d == entries - 1) x += past[1] + past[3] + past[5] + past[7];
      out[d] = x;
    }
  }
}

template <int D, int CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, (kDqAlone<D, CAP, BIAS> ? 1 : 2)) void attn_dq_kernel(
    const AttnParams p) {
  extern __shared__ __align__(1024) char smem[];
  attn_dq<D, CAP, BIAS>(p, place(), smem);
}

// Both in one launch, where both run two workgroups to a compute unit: the second's
// workgroups fill the places that the last of the first leave (118 us instead of 121:
// 8 x 1024 tokens, 12 heads of 64, bias).  `kv` and `q`: the two grids, of which the launch
// takes the workgroups from `first` on.
template <int D, int CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_grads_kernel(const AttnParams p, int2 kv, int2 q,
                                                                    int first) {
  extern __shared__ __align__(1024) char smem[];
  const int id = first + blockIdx.x, behind = id - kv.x * kv.y;
  if (behind < 0)
    attn_dkv<D, CAP, BIAS>(p, Place{id % kv.x, id / kv.x, kv.x, kv.y}, smem);
  else
    attn_dq<D, CAP, BIAS>(p, Place{behind % q.x, behind / q.x, q.x, q.y}, smem);
}

// The sums by distance over all batch rows and query tiles: 64 distances of a head
// to a workgroup, 16 threads to a distance.
__global__ __launch_bounds__(1024) void attn_dsum_kernel(const AttnParams p, int tiles) {
  __shared__ float sums[16][64];
  const int entries = bias_entries(p.reach), rows = p.B * tiles;
  const int h = blockIdx.x, lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int d = blockIdx.y * 64 + lane;
  float x = 0.f;
  if (d < entries)
    for (int n0 = g; n0 < rows; n0 += 64) {            // 4 loads under way at a time
      float part[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int n = n0 + 16 * u;
        part[u] = 0.f;
        if (n < rows) {
          const int64_t b = n / tiles, t = n % tiles;
          part[u] = p.dpart[((b * p.Hq + h) * tiles + t) * entries + d];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) x += part[u];
    }
  sums[g][lane] = x;
  __syncthreads();
  if (g == 0 && d < entries) {
    x = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) x += sums[k][lane];
    p.dsum[static_cast<int64_t>(h) * entries + d] = x;
  }
}

// dbias_table[.][h]: the sums by distance, by bucket; a wave to a bucket.
__global__ __launch_bounds__(1024) void attn_dtable_kernel(const AttnParams p) {
  extern __shared__ float sums[];                      // [entries], then bucket ids
  const int h = blockIdx.x, tid = threadIdx.x, lane = tid & 63, entries = bias_entries(p.reach);
  int* bucket = reinterpret_cast<int*>(sums + entries);
  for (int d = tid; d < entries; d += 1024) {
    sums[d] = p.dsum[static_cast<int64_t>(h) * entries + d];
    bucket[d] = bias_bucket(p, d - bias_span(p.reach));
  }
  __syncthreads();
  for (int k = tid >> 6; k < p.n_buckets; k += 16) {
    float x = 0.f;
#pragma unroll 4
    for (int d = lane; d < entries; d += 64) x += bucket[d] == k ? sums[d] : 0.f;
    x = join_lanes<64>(x, AddOp());
    if (lane == 0) {
      const int64_t at = static_cast<int64_t>(k) * p.Hq + h;
      if (p.table_f32)
        static_cast<float*>(p.dtable)[at] = x;
      else
        static_cast<bf16*>(p.dtable)[at] = static_cast<bf16>(x);
    }
  }
}

namespace {

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

int up64(int n) { return (n + kTile - 1) / kTile * kTile; }

// In how many parts a key head's query heads are taken: enough for two
// workgroups to a compute unit (457 us instead of 701 in one part: 4001 keys, 32 heads on
// 8), and one head each with a bias (whose table in shared memory is one head's).
int choose_parts(int B, int Tk, int Hq, int Hk, bool bias) {
  const int group = Hq / Hk;
  if (bias) return group;
  const int64_t groups = static_cast<int64_t>(B) * Hk * ((Tk + 127) / 128);
  int parts = 1;
  while (parts < group && (group % parts != 0 || groups * parts < 512)) ++parts;
  return parts;
}

template <typename... A>
hipError_t launch_lds(void (*fn)(A...), dim3 grid, size_t lds, hipStream_t s, A... args) {
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds));
  if (e != hipSuccess) return e;
  fn<<<grid, kAttnThreads, lds, s>>>(args...);
  return hipGetLastError();
}

template <int D, int CAP, bool BIAS>
hipError_t run_bwd(const AttnParams& p, hipStream_t s) {
  const size_t n = BIAS ? bias_entries(p.reach) : 0;
  const size_t dkv_bufs = kBuffers<D, kDkvAlone<D, CAP, BIAS>>, dq_bufs = kBuffers<D, kDqAlone<D, CAP, BIAS>>;
  const size_t kv_lds = dkv_bufs * (2 * kTileBytes<D> + 4 * kTile * 4) + n * 4;
  const size_t q_lds = dq_bufs * 2 * kTileBytes<D> + 128 * 8 + 4 * kWaves * 4 +
                       (BIAS ? n + kWaves * (kDiagWords + n) : 0) * sizeof(float);
  const int tiles = (p.Tq + 127) / 128;
  const int2 kv = make_int2(p.B * p.Hk * p.parts, (p.Tk + 127) / 128);
  const int2 q = make_int2(p.B * p.Hq, tiles);
  hipError_t e = hipSuccess;
  if constexpr (kDkvAlone<D, CAP, BIAS> || kDqAlone<D, CAP, BIAS>) {
    if (kv.x > 0 && kv.y > 0) e = launch_lds(attn_dkv_kernel<D, CAP, BIAS>, dim3(kv.x, kv.y), kv_lds, s, p);
    if (e != hipSuccess) return e;
    if (q.x > 0 && q.y > 0) e = launch_lds(attn_dq_kernel<D, CAP, BIAS>, dim3(q.x, q.y), q_lds, s, p);
  } else {
    const int64_t both = static_cast<int64_t>(kv.x) * kv.y + static_cast<int64_t>(q.x) * q.y;
    constexpr int64_t kMost = 1 << 23;                 // (256 threads each, below 2^32)
    if (both > 0x7FFFFFFF) return hipErrorInvalidConfiguration;      // (hundreds of GiB of rows)
    for (int64_t first = 0; first < both && e == hipSuccess; first += kMost)
      e = launch_lds(attn_grads_kernel<D, CAP, BIAS>,
                     dim3(static_cast<unsigned>(both - first < kMost ? both - first : kMost)),
                     kv_lds > q_lds ? kv_lds : q_lds, s, p, kv, q, static_cast<int>(first));
  }
  if (e != hipSuccess) return e;
  if (p.parts > 1 && kv.x > 0 && kv.y > 0) {
    const int64_t pieces = static_cast<int64_t>(p.B) * p.Hk * p.Tk * D / 8;
    attn_dkv_join_kernel<<<static_cast<unsigned>((pieces + 255) / 256), 256, 0, s>>>(p, D);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (BIAS && p.dtable) {                              // (the sum over an empty batch is 0)
    attn_dsum_kernel<<<dim3(p.Hq, static_cast<unsigned>((n + 63) / 64)), 1024, 0, s>>>(p, tiles);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    attn_dtable_kernel<<<p.Hq, 1024, 2 * n * sizeof(float), s>>>(p);
    e = hipGetLastError();
  }
  return e;
}

template <int D, int CAP>
hipError_t pick_bwd(const AttnParams& p, hipStream_t s) {
  return p.table ? run_bwd<D, CAP, true>(p, s) : run_bwd<D, CAP, false>(p, s);
}

template <int D>
hipError_t pick_bwd(const AttnParams& p, hipStream_t s) {
  switch (cap_form(p.cap)) {
    case kNoCap: return pick_bwd<D, kNoCap>(p, s);
    case kByU: return pick_bwd<D, kByU>(p, s);
    default: return pick_bwd<D, kAnyCap>(p, s);
  }
}

// The workspace, in order; returns its size.
size_t lay_out(AttnParams& p, int D, size_t entries, char* base) {
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    char* x = base + at;
    at += up16(bytes);
    return x;
  };
  const size_t rows = static_cast<size_t>(p.B) * p.tq64, parts = p.parts > 1 ? p.parts : 0;
  p.base = reinterpret_cast<float*>(take(rows * p.Hq * 4));
  p.delta = reinterpret_cast<float*>(take(rows * p.Hq * 4));
  p.qlo = reinterpret_cast<int*>(take(rows * 4));
  p.qhi = reinterpret_cast<int*>(take(rows * 4));
  p.tile = reinterpret_cast<int*>(
      take(p.Tq > 0 ? static_cast<size_t>(p.B) * ((p.Tk + 127) / 128) * kTileWords * sizeof(int) : 0));
  p.dpart = reinterpret_cast<float*>(
      take(static_cast<size_t>(p.B) * p.Hq * ((p.Tq + 127) / 128) * entries * 4));
  p.dsum = reinterpret_cast<float*>(take(p.Hq * entries * 4));
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
  // (for any reach up to the largest: the size goes by the buckets)
  return lay_out(p, D, n_buckets > 0 ? bias_entries(ZERO_ATTN_MAX_REACH) : 0, nullptr);
}

hipError_t launch_attn_bwd(const zero_attn_args& a, hipStream_t s) {
  AttnParams p = attn_params(a);
  p.tq64 = up64(a.Tq);
  p.parts = choose_parts(a.B, a.Tk, a.Hq, a.Hk, a.bias_table != nullptr);
  lay_out(p, a.D, a.bias_table ? bias_entries(p.reach) : 0, static_cast<char*>(a.workspace));
  if (a.B > 0 && a.Tq > 0) {
    const int before = ((a.Tk + 127) / 128 + a.Hq - 1) / a.Hq;
    attn_bwd_prepare_kernel<<<dim3(a.B * a.Hq, p.tq64 / 64 + before), 256, 0, s>>>(p, a.D,
                                                                                        before);
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
