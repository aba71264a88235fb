// zo_attn_bwd.hip -- attention, backward, with no atomics: one kernel owns
// keys and walks the queries (dk, dv), one owns queries and walks the keys (dq
// and the bias gradient).  Scores are formed again from q, k and the saved
// lse in both: 7 matrix products instead of the 5 of a kernel that adds dq
// through memory, for gradients that have one fixed order of summation.
//
// A first kernel leaves delta = do . o and the lse in units of log2 in the
// workspace, and for every 64 queries the hull of the keys they see.
#include "zo_attn.h"
#include "zo_internal.h"

namespace zo {

// 64 queries of one (batch, head): 4 threads to a row.
__global__ __launch_bounds__(256) void attn_bwd_prepare_kernel(const AttnParams p, int D) {
  const int bh = blockIdx.x, b = bh / p.Hq, h = bh % p.Hq;
  const int tid = threadIdx.x, sub = tid & 3;
  const int i = blockIdx.y * 64 + (tid >> 2);
  float sum = 0.f;
  int2 r = key_range(p, b, i);
  if (i < p.Tq && r.y > r.x) {
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
  if (i < p.Tq && sub == 0) {
    const int64_t row = static_cast<int64_t>(bh) * p.Tq + i;
    p.delta[row] = sum;
    const float lse = p.lse[row];
    p.lse2[row] = r.y > r.x && lse != -kInf ? lse * kLog2e : kInf;
  }
  if (h == 0) {
    __shared__ int2 part[4];
    const int2 w = wave_hull(r);
    if ((tid & 63) == 0) part[tid >> 6] = w;
    __syncthreads();
    if (tid == 0) {
      int2 x = part[0];
#pragma unroll
      for (int k = 1; k < 4; ++k) x = make_int2(min(x.x, part[k].x), max(x.y, part[k].y));
      p.qbounds[static_cast<int64_t>(b) * gridDim.y + blockIdx.y] = x;
    }
  }
}

// p and dx of one element from the raw product x = q.k, its bias, dp and the
// row's statistics; ds (before the cap's derivative) for the bias gradient.
template <bool CAP>
__device__ __forceinline__ void grad_score(float x, float bias, float dp, float lse2, float delta,
                                           float a, float c2, float& pr, float& ds, float& dx) {
  if constexpr (CAP) {
    const float u = rcp_hw(exp2_hw(x * a) + 1.f);            // (1 - tanh) / 2
    pr = exp2_hw(__builtin_fmaf(u, -2.f * c2, c2) + (bias - lse2));
    ds = pr * (dp - delta);
    dx = ds * (4.f * u * (1.f - u));                         // 1 - tanh^2
  } else {
    pr = exp2_hw(__builtin_fmaf(x, a, bias - lse2));
    ds = pr * (dp - delta);
    dx = ds;
  }
}

// ---------------------------------------------------------------- dk, dv ---

// A workgroup owns 128 keys of one key head, 32 to a wave, and walks tiles of
// 64 queries of every query head that shares it.
template <int D, bool CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads) void attn_dkv_kernel(const AttnParams p) {
  constexpr int P = kPitch<D>;
  extern __shared__ __align__(16) char smem[];
  bf16* qt = reinterpret_cast<bf16*>(smem);            // [kTile][P]
  bf16* gt = qt + kTile * P;                           // [kTile][P]
  float* stat = reinterpret_cast<float*>(gt + kTile * P);   // [2][kTile]
  int2* rows = reinterpret_cast<int2*>(stat + 2 * kTile);   // [kTile]
  float* bias = reinterpret_cast<float*>(rows + kTile);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
  const int b = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk;
  const int j0 = blockIdx.y * 128;                     // the workgroup's first key
  const int jw = j0 + wave * 32, j = jw + (lane & 31);
  const int qtiles = (p.Tq + kTile - 1) / kTile;

  bf16x8 kf[D / 16], vf[D / 16];
  {
    const int64_t jj = min(j, p.Tk - 1);
    const bf16* k = p.k + b * p.ks.b + jj * p.ks.t + hk * p.ks.h;
    const bf16* v = p.v + b * p.vs.b + jj * p.vs.t + hk * p.vs.h;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      kf[c] = load8(k + 16 * c + 8 * half);
      vf[c] = load8(v + 16 * c + 8 * half);
    }
  }
  const float c2 = CAP ? p.cap * kLog2e : 0.f;
  const float a = CAP ? 2.f * p.scale * kLog2e / p.cap : p.scale * kLog2e;

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[t][r] = dv[t][r] = 0.f;

  for (int g = 0; g < p.group; ++g) {
    const int h = hk * p.group + g;
    const int64_t bh = static_cast<int64_t>(b) * p.Hq + h;
    const bf16* qg = p.q + b * p.qs.b + h * p.qs.h;
    const bf16* og = p.d_o + b * p.dos.b + h * p.dos.h;
    if constexpr (BIAS) {
      __syncthreads();
      stage_bias(p, h, bias, tid);
    }
    for (int qi = 0; qi < qtiles; ++qi) {
      const int2 hull = p.qbounds[static_cast<int64_t>(b) * qtiles + qi];
      if (hull.x >= j0 + 128 || hull.y <= j0) continue;        // the same for the whole workgroup
      const int i0 = qi * kTile;
      __syncthreads();
      {
        Stage<D> sq, so;
        sq.load(qg, p.qs.t, i0, 0, p.Tq, tid);
        so.load(og, p.dos.t, i0, 0, p.Tq, tid);
        sq.store(qt, tid);
        so.store(gt, tid);
        if (tid < kTile) {
          const int i = i0 + tid;
          rows[tid] = key_range(p, b, i);
          stat[tid] = i < p.Tq ? p.lse2[bh * p.Tq + i] : kInf;
          stat[kTile + tid] = i < p.Tq ? p.delta[bh * p.Tq + i] : 0.f;
        }
      }
      __syncthreads();
      if (hull.x >= jw + 32 || hull.y <= jw) continue;
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {                            // 32 queries at a time
        const int is = i0 + 32 * s;
        const int2 mine = rows[32 * s + (lane & 31)];
        if (!__any(mine.x < jw + 32 && mine.y > jw)) continue;
        const bool full = __all(mine.x <= jw && mine.y >= jw + 32);
        f32x16 x, dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          x = mfma(frag_rows<P>(qt, 32 * s, 16 * c, lane), kf[c], x);
          dp = mfma(frag_rows<P>(gt, 32 * s, 16 * c, lane), vf[c], dp);
        }
        float pr[16], dx[16];
        uint32_t keep[2] = {0xFFu, 0xFFu};
        if (!full) keep[0] = keep[1] = 0;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int row = 8 * r4 + 4 * half + 32 * s;
          const f32x4 lse = *reinterpret_cast<const f32x4*>(stat + row);
          const f32x4 del = *reinterpret_cast<const f32x4*>(stat + kTile + row);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 4 * r4 + e;
            float bb = 0.f;
            if constexpr (BIAS) {
              const int d = j - (i0 + row + e + p.off);
              bb = bias[min(max(d, -p.reach), p.reach) + p.reach];
            }
            float ds;
            grad_score<CAP>(x[r], bb, dp[r], lse[e], del[e], a, c2, pr[r], ds, dx[r]);
            if (!full) {
              const int2 see = rows[row + e];
              const bool seen = j >= see.x && j < see.y;
              pr[r] = seen ? pr[r] : 0.f;
              dx[r] = seen ? dx[r] : 0.f;
              keep[r >> 3] |= any_in_half(seen, lane) << (r & 7);
            }
          }
        }
        (void)is;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bf16x8 pf = to_frag(pr + 8 * u), xf = to_frag(dx + 8 * u);
#pragma unroll
          for (int t = 0; t < D / 32; ++t) {
            bf16x8 of = frag_cols<P>(gt, 32 * s + 16 * u, 32 * t, lane);
            bf16x8 qf = frag_cols<P>(qt, 32 * s + 16 * u, 32 * t, lane);
            if (keep[u] != 0xFFu) {
              of = keep_frag(of, keep[u]);
              qf = keep_frag(qf, keep[u]);
            }
            dv[t] = mfma(of, pf, dv[t]);
            dk[t] = mfma(qf, xf, dk[t]);
          }
        }
      }
    }
  }
  if (j >= p.Tk) return;
  bf16* ok = p.dk + b * p.dks.b + static_cast<int64_t>(j) * p.dks.t + hk * p.dks.h;
  bf16* ov = p.dv + b * p.dvs.b + static_cast<int64_t>(j) * p.dvs.t + hk * p.dvs.h;
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      bf16x4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = static_cast<bf16>(dk[t][r + e] * p.scale);
        y[e] = static_cast<bf16>(dv[t][r + e]);
      }
      *reinterpret_cast<bf16x4*>(ok + 32 * t + result_row(r, lane)) = x;
      *reinterpret_cast<bf16x4*>(ov + 32 * t + result_row(r, lane)) = y;
    }
}

// ------------------------------------------------ dq and the bias gradient ---

// A workgroup owns 128 queries of one head, 32 to a wave, and walks tiles of
// 64 keys.  With the bias, sums of ds by distance are kept per half wave in
// shared memory: the 32 lanes of a half wave hold 32 consecutive queries, so
// at one key row their distances, and the addresses they add to, all differ,
// and every address has one writer at a time, in program order.  Distances
// past the reach share a bucket and are summed in two registers instead.
template <int D, bool CAP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads) void attn_dq_kernel(const AttnParams p) {
  constexpr int P = kPitch<D>;
  extern __shared__ __align__(16) char smem[];
  bf16* kt = reinterpret_cast<bf16*>(smem);            // [kTile][P]
  bf16* vt = kt + kTile * P;                           // [kTile][P]
  int* hull = reinterpret_cast<int*>(vt + kTile * P);  // [kWaves][2]
  float* bias = reinterpret_cast<float*>(hull + 2 * kWaves);      // [2 reach + 1]
  float* hist = bias + (BIAS ? 2 * p.reach + 1 : 0);              // [8][2 reach + 1]
  float* ends = hist + (BIAS ? 8 * (2 * p.reach + 1) : 0);        // [2][256]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
  const int bh = blockIdx.x, b = bh / p.Hq, h = bh % p.Hq;
  const int hk = h / p.group;
  const int tile = gridDim.y - 1 - blockIdx.y;
  const int i0 = tile * 128 + wave * 32;
  const int i = i0 + (lane & 31);
  const int64_t row = static_cast<int64_t>(bh) * p.Tq + min(i, p.Tq - 1);

  const int2 rng = key_range(p, b, i);
  const int2 wh = wave_hull(rng);
  if (lane == 0) {
    hull[2 * wave] = wh.x;
    hull[2 * wave + 1] = wh.y;
  }
  float* mine = hist;
  float low = 0.f, high = 0.f;
  if constexpr (BIAS) {
    stage_bias(p, h, bias, tid);
    for (int d = tid; d < 8 * (2 * p.reach + 1); d += kAttnThreads) hist[d] = 0.f;
    mine = hist + (2 * wave + half) * (2 * p.reach + 1) + p.reach;
  }
  bf16x8 qf[D / 16], of[D / 16];
  {
    const int64_t ii = min(i, p.Tq - 1);
    const bf16* q = p.q + b * p.qs.b + ii * p.qs.t + h * p.qs.h;
    const bf16* o = p.d_o + b * p.dos.b + ii * p.dos.t + h * p.dos.h;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qf[c] = load8(q + 16 * c + 8 * half);
      of[c] = load8(o + 16 * c + 8 * half);
    }
  }
  const float lse2 = p.lse2[row], delta = p.delta[row];
  const float c2 = CAP ? p.cap * kLog2e : 0.f;
  const float a = CAP ? 2.f * p.scale * kLog2e / p.cap : p.scale * kLog2e;
  __syncthreads();
  int first = 0x7FFFFFFF, last = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    first = min(first, hull[2 * w]);
    last = max(last, hull[2 * w + 1]);
  }
  if (first > last) first = last;

  const bf16* kg = p.k + b * p.ks.b + hk * p.ks.h;
  const bf16* vg = p.v + b * p.vs.b + hk * p.vs.h;
  f32x16 dq[D / 32];
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[t][r] = 0.f;

  for (int k0 = first & ~(kTile - 1); k0 < last; k0 += kTile) {
    __syncthreads();
    {
      Stage<D> sk, sv;
      sk.load(kg, p.ks.t, k0, first, last, tid);
      sv.load(vg, p.vs.t, k0, first, last, tid);
      sk.store(kt, tid);
      sv.store(vt, tid);
    }
    __syncthreads();
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      const int ks = k0 + 32 * s;
      if (wh.x >= ks + 32 || wh.y <= ks) continue;
      const bool full = __all(rng.x <= ks && rng.y >= ks + 32);
      f32x16 x, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = dp[r] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        x = mfma(frag_rows<P>(kt, 32 * s, 16 * c, lane), qf[c], x);
        dp = mfma(frag_rows<P>(vt, 32 * s, 16 * c, lane), of[c], dp);
      }
      float dx[16];
      uint32_t keep[2] = {0xFFu, 0xFFu};
      if (!full) keep[0] = keep[1] = 0;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int j = ks + result_row(r, lane);
        const int d = j - (i + p.off);
        float bb = 0.f, pr, ds;
        if constexpr (BIAS) bb = bias[min(max(d, -p.reach), p.reach) + p.reach];
        grad_score<CAP>(x[r], bb, dp[r], lse2, delta, a, c2, pr, ds, dx[r]);
        if (!full) {
          const bool seen = j >= rng.x && j < rng.y;
          ds = seen ? ds : 0.f;
          dx[r] = seen ? dx[r] : 0.f;
          keep[r >> 3] |= any_in_half(seen, lane) << (r & 7);
        }
        if constexpr (BIAS) {
          if (d <= -p.reach)
            low += ds;
          else if (d >= p.reach)
            high += ds;
          else
            unsafeAtomicAdd(mine + d, ds);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8 xf = to_frag(dx + 8 * u);
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          bf16x8 kf = frag_cols<P>(kt, 32 * s + 16 * u, 32 * t, lane);
          if (keep[u] != 0xFFu) kf = keep_frag(kf, keep[u]);
          dq[t] = mfma(kf, xf, dq[t]);
        }
      }
    }
  }
  if (i < p.Tq) {
    bf16* o = p.dq + b * p.dqs.b + static_cast<int64_t>(i) * p.dqs.t + h * p.dqs.h;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        bf16x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = static_cast<bf16>(dq[t][r + e] * p.scale);
        *reinterpret_cast<bf16x4*>(o + 32 * t + result_row(r, lane)) = x;
      }
  }
  if constexpr (BIAS) {
    if (p.dtable == nullptr) return;
    const int n = 2 * p.reach + 1;
    ends[tid] = low;
    ends[256 + tid] = high;
    __syncthreads();
    for (int d = tid; d < n; d += kAttnThreads) {      // one sum by distance, in bias' place
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) x += hist[w * n + d];
      bias[d] = x;
    }
    for (int w = 128; w > 0; w >>= 1) {
      if (tid < w) {
        ends[tid] += ends[tid + w];
        ends[256 + tid] += ends[256 + tid + w];
      }
      __syncthreads();
    }
    if (tid == 0) {
      bias[0] += ends[0];
      bias[2 * p.reach] += ends[256];
    }
    __syncthreads();
    if (tid < p.n_buckets) {
      float x = 0.f;
      for (int d = 0; d < n; ++d)
        if (min(max(p.buckets[d], 0), p.n_buckets - 1) == tid) x += bias[d];
      p.dpart[(static_cast<int64_t>(bh) * gridDim.y + tile) * p.n_buckets + tid] = x;
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
  const size_t n = 2 * p.reach + 1;
  const int tiles = (p.Tq + 127) / 128;
  const size_t staged = 2 * sizeof(bf16) * kTile * kPitch<D>;
  hipError_t e = hipSuccess;
  if (p.B > 0 && p.Tk > 0)
    e = launch_lds(attn_dkv_kernel<D, CAP, BIAS>, dim3(p.B * p.Hk, (p.Tk + 127) / 128),
                   staged + kTile * 16 + (BIAS ? n * sizeof(float) : 0), p, s);
  if (e != hipSuccess) return e;
  if (p.B > 0 && p.Tq > 0)
    e = launch_lds(attn_dq_kernel<D, CAP, BIAS>, dim3(p.B * p.Hq, tiles),
                   staged + 2 * kWaves * sizeof(int) + (BIAS ? (9 * n + 512) * sizeof(float) : 0),
                   p, s);
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

}  // namespace

size_t attn_bwd_workspace(int B, int Tq, int Tk, int Hq, int Hk, int D, int n_buckets) {
  (void)Tk;
  (void)Hk;
  (void)D;
  const size_t rows = static_cast<size_t>(B) * Hq * Tq;
  return 2 * up16(rows * sizeof(float)) +
         up16(static_cast<size_t>(B) * ((Tq + kTile - 1) / kTile) * sizeof(int2)) +
         up16(static_cast<size_t>(B) * Hq * ((Tq + 127) / 128) * n_buckets * sizeof(float));
}

hipError_t launch_attn_bwd(const zero_attn_args& a, hipStream_t s) {
  AttnParams p = attn_params(a);
  const size_t rows = static_cast<size_t>(a.B) * a.Hq * a.Tq;
  char* w = static_cast<char*>(a.workspace);
  p.lse2 = reinterpret_cast<float*>(w);
  w += up16(rows * sizeof(float));
  p.delta = reinterpret_cast<float*>(w);
  w += up16(rows * sizeof(float));
  p.qbounds = reinterpret_cast<int2*>(w);
  w += up16(static_cast<size_t>(a.B) * ((a.Tq + kTile - 1) / kTile) * sizeof(int2));
  p.dpart = reinterpret_cast<float*>(w);
  if (a.B > 0 && a.Tq > 0) {
    attn_bwd_prepare_kernel<<<dim3(a.B * a.Hq, (a.Tq + 63) / 64), 256, 0, s>>>(p, a.D);
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
