// zo_grads.hip -- the exact global norm of the gradients of many tensors, and
// their unscaling and clipping.
//
// Both stream the tensors once.  The addresses travel in the kernels' arguments, as many
// as 4 KiB hold to a launch, and every tensor is cut into tiles of 8192 elements, so that
// one launch covers tensors of any sizes.  A tensor may start at any element: the
// hardware's unaligned loads fetch 8 elements at a time from there.
//
// The norm is the optimizer step's fixed-point sum of squares (zs_device.h), so it is the
// same for any grid and order and adds up with other accumulators.  Each workgroup leaves
// its digits in a row of the workspace, and one workgroup adds them up.
//
// Bound by memory, and by the host's checks and launches where there is little of it.  Measured, 194
// tensors, 150.5 million values in bf16: the norm 59 us, 5.1 TB/s, its fold 5, the clipping 101 us, 5.9
// TB/s of reads and writes; both as they follow on each other 165.  10 tensors, 267000 values: 17 us.
#include <type_traits>

#include "zo_internal.h"
#include "zs_device.h"

namespace zo {

using zs::kDigits;
using zs::kVec;

constexpr int kGradThreads = 256;
constexpr int kGradTile = 8192;               // elements of a tile: 4 chunks of 8 a thread
constexpr int kTileChunks = kGradTile / kVec / kGradThreads;
constexpr int kNormGroups = 1024;             // workgroups at most
constexpr uint32_t kClipGroups = 2048;
constexpr int kWords = kDigits + 1;           // digits, then the non-finite count
static_assert(kTileChunks == 4, "a quad's lanes convert a group each");

// Tensors of one launch.  first[i] is tensor i's first tile; info[i] holds the elements of
// its last tile, and kBf16In and kBf16Out.  (Words, as scalar loads have no smaller: a byte
// would come by a vector load, whose wait waits for the tile's loads too.)
constexpr uint32_t kTail = 0xFFFF, kBf16In = 1u << 16, kBf16Out = 1u << 17;
template <int N>
struct TensorTable {
  int count;
  uint32_t first[N + 1];
  uint32_t info[N];
  const void* grad[N];

  // The tensor of a tile.
  __device__ __forceinline__ int find(uint32_t tile) const {
    int at = 0, step = 1;
    while (step < N) step <<= 1;
    for (; step > 0; step >>= 1)
      if (at + step < count && first[at + step] <= tile) at += step;
    return at;
  }
};
constexpr int kNormTensors = 240, kClipTensors = 160;

struct GradNormParams {
  TensorTable<kNormTensors> t;
  uint32_t tiles;
  float inv_scale;
  int add;                                    // to what earlier launches of the call left
  uint64_t* part;                             // [groups][kWords]
};
struct GradClipParams {
  TensorTable<kClipTensors> t;
  void* out[kClipTensors];
  uint32_t tiles;
  float inv_scale;
  int lead;                                   // whether this launch writes the scalars
  const zero_norm_acc* accs;
  int n_accs, check_overflow;
  double max_norm;
  float *norm_out, *coef_out;
  int32_t* skipped_out;
};
static_assert(sizeof(GradNormParams) <= 4096 && sizeof(GradClipParams) <= 4096,
              "kernel arguments");

// What a thread holds of a tile: chunks of W elements.  The tensor's start may lie at any
// element.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

template <bool BF16, int W>
struct RawTile {
  static constexpr int kWidth = W, kChunks = kGradTile / W / kGradThreads;
  static constexpr int kWide = BF16 ? 8 : 4;         // elements of 16 bytes
  static constexpr int kPieces = (W + kWide - 1) / kWide;
  zs::u32x4 v[kChunks][kPieces];                     // (8 bytes in the first two words)

  // A thread's chunk u of a tile starts at element (u * 256 + thread) * W.
  __device__ __forceinline__ static int chunk_at(int u) {
    return (u * kGradThreads + static_cast<int>(threadIdx.x)) * W;
  }

  __device__ __forceinline__ void load(const char* tile) {
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      if constexpr (BF16 && W == 8) {
        v[u][0] = reinterpret_cast<const u32x4_any*>(tile)[chunk_at(u) / 8];
      } else if constexpr (BF16) {
        const u32x2_any x = reinterpret_cast<const u32x2_any*>(tile)[chunk_at(u) / 4];
        v[u][0] = zs::u32x4{x[0], x[1], 0, 0};
      } else {
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
          v[u][h] = __builtin_bit_cast(
              zs::u32x4, reinterpret_cast<const f32x4_any*>(tile)[chunk_at(u) / 4 + h]);
      }
    }
  }

  // Of a tile of n elements: those behind it are +0.
  __device__ __forceinline__ void load_some(const char* tile, int n) {
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = chunk_at(u);
#pragma unroll
      for (int h = 0; h < kPieces; ++h) v[u][h] = zs::u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (c + j >= n) continue;
        if constexpr (BF16)
          v[u][0][j / 2] |=
              static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(tile)[c + j]) << (16 * (j & 1));
        else
          v[u][j / 4][j & 3] = reinterpret_cast<const uint32_t*>(tile)[c + j];
      }
    }
  }

  __device__ __forceinline__ void widen(int u, float scale, float x[W]) const {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (BF16) {
        const uint32_t h = v[u][0][j / 2];
        x[j] = __uint_as_float(j & 1 ? h & 0xFFFF0000u : h << 16) * scale;
      } else {
        x[j] = __uint_as_float(v[u][j / 4][j & 3]) * scale;
      }
    }
  }
};

// Works on one tile: use(raw, tensor, info, first element, elements).
template <bool BF16, int W, typename Use>
__device__ __forceinline__ void with_tile(const void* tensor, int i, uint32_t info, int64_t e0,
                                          int n, Use use) {
  const char* base = static_cast<const char*>(tensor) + e0 * (BF16 ? 2 : 4);
  RawTile<BF16, W> raw;
  if (n == kGradTile) raw.load(base);
  else raw.load_some(base, n);
  use(raw, i, info, e0, n);
}

// A workgroup's tiles, one of every gridDim.x; with CLIP a tensor's last tile comes first, and
// chunks are of 4 elements where either side is fp32: 16 bytes, so that a wave's accesses leave no
// gaps (60 tensors of 4096 x 4096, fp32: 1540 us, in chunks of 8 1900; bf16 to fp32 1160, 1540).
template <bool CLIP, int N, typename Use>
__device__ __forceinline__ void walk(const TensorTable<N>& t, uint32_t tiles, Use use) {
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int i = t.find(tile);
    const uint32_t info = t.info[i], first = t.first[i], last = t.first[i + 1] - 1;
    const uint32_t inside = CLIP ? last - tile : tile - first;
    const int64_t e0 = static_cast<int64_t>(inside) * kGradTile;
    const int n = inside == last - first ? static_cast<int>(info & kTail) : kGradTile;
    if (!(info & kBf16In)) {
      with_tile<false, CLIP ? 4 : 8>(t.grad[i], i, info, e0, n, use);
      continue;
    }
    if constexpr (CLIP) {
      if (!(info & kBf16Out)) {
        with_tile<true, 4>(t.grad[i], i, info, e0, n, use);
        continue;
      }
    }
    with_tile<true, 8>(t.grad[i], i, info, e0, n, use);
  }
}

// The four group sums that a thread's quad has of a tile.  Squares of finite binary32
// values sum to less than 2^261 in binary64, so only a value that is not finite makes the
// chunk's sum infinite or NaN: they are looked for (zs::chunk_sumsq) only then.  Elements
// behind the tensor's end are +0.
template <bool BF16>
__device__ __forceinline__ void tile_sums(const RawTile<BF16, kVec>& r, float scale,
                                          double s4[kTileChunks], uint32_t& nonfinite) {
#pragma unroll
  for (int u = 0; u < kTileChunks; ++u) {
    float g[kVec];
    r.widen(u, scale, g);
    double a = 0.0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const double x = static_cast<double>(g[j]);
      a = __builtin_fma(x, x, a);
    }
    if (!__builtin_isfinite(a)) a = zs::chunk_sumsq(g, nonfinite);
    s4[u] = zs::quad_group_sum(a);
  }
}

__global__ __launch_bounds__(kGradThreads) void grads_norm_kernel(const GradNormParams p) {
  __shared__ uint64_t s_digit[kDigits][kGradThreads];
  __shared__ uint64_t s_part[kGradThreads / 64][kWords];
  const int tid = threadIdx.x, quad_lane = tid & 3;
#pragma unroll
  for (int k = 0; k < kDigits; ++k) s_digit[k][tid] = 0;
  uint32_t nonfinite = 0;
  walk<false>(p.t, p.tiles, [&](const auto& raw, int, uint32_t, int64_t, int) {
    double s4[kTileChunks];
    tile_sums(raw, p.inv_scale, s4, nonfinite);
    // every lane of a quad holds the four group sums: lane q converts group q
    const double S = quad_lane == 0 ? s4[0] : quad_lane == 1 ? s4[1] : quad_lane == 2 ? s4[2] : s4[3];
    int base;
    uint32_t p0, p1, p2;
    zs::fixed_point_split(S, base, p0, p1, p2);
    if (p0 != 0) s_digit[base][tid] += p0;
    if (p1 != 0) s_digit[base + 1][tid] += p1;
    if (p2 != 0) s_digit[base + 2][tid] += p2;
  });
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    uint64_t v = k < kDigits ? s_digit[k < kDigits ? k : 0][tid] : nonfinite;
    if (__ballot(v != 0) != 0) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    }
    if (lane == 0) s_part[wave][k] = v;
  }
  __syncthreads();
  if (tid < kWords) {
    uint64_t v = 0;
#pragma unroll
    for (int w = 0; w < kGradThreads / 64; ++w) v += s_part[w][tid];
    uint64_t* out = p.part + static_cast<int64_t>(blockIdx.x) * kWords + tid;
    *out = p.add ? *out + v : v;
  }
}

// Adds the workgroups' rows to the accumulator: 64 threads to each of its words.
constexpr int kFoldThreads = 64 * kWords;
__global__ __launch_bounds__(kFoldThreads) void grads_fold_kernel(const uint64_t* part, int groups,
                                                                 zero_norm_acc* acc, int add) {
  __shared__ uint64_t s[64][kWords];
  const int k = threadIdx.x % kWords, r = threadIdx.x / kWords;
  uint64_t v = 0;
#pragma unroll 4
  for (int g = r; g < groups; g += 64) v += part[static_cast<int64_t>(g) * kWords + k];
  s[r][k] = v;
  __syncthreads();
  if (r == 0) {
    v = 0;
#pragma unroll 8
    for (int i = 0; i < 64; ++i) v += s[i][k];
    uint64_t* out = k < kDigits ? &acc->digit[k] : &acc->nonfinite;
    *out = add ? *out + v : v;
  }
  if (threadIdx.x < 2 && !add) acc->reserved[threadIdx.x] = 0;
}

// -------------------------------------------------------------- clipping ---

// Past the caches: what the norm left in them of the gradients is read back from there,
// which plain stores of the outputs would push out.  194 tensors of 301 MB, norm and
// clipping: 175 us instead of 207; from the last tile to the first, so that the clipping
// begins with what the norm read last, 168.
template <bool BF16, int W>
__device__ __forceinline__ void store_chunk(void* base, int c, int left, const float x[W]) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + c;
    uint32_t w[W / 2];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      const __bf16 lo = static_cast<__bf16>(x[2 * j]), hi = static_cast<__bf16>(x[2 * j + 1]);
      w[j] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, lo)) |
             static_cast<uint32_t>(__builtin_bit_cast(uint16_t, hi)) << 16;
    }
    if (left >= W) {
      if constexpr (W == 8)
        __builtin_nontemporal_store(u32x4_any{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_any*>(p));
      else
        __builtin_nontemporal_store(u32x2_any{w[0], w[1]}, reinterpret_cast<u32x2_any*>(p));
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < left) p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
  } else {
    static_assert(W == 4);
    float* p = static_cast<float*>(base) + c;
    if (left >= W) {
      __builtin_nontemporal_store(f32x4_any{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4_any*>(p));
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (j < left) p[j] = x[j];
    }
  }
}

template <bool OUT, bool IN, int W>
__device__ __forceinline__ void clip_tile(const RawTile<IN, W>& r, int n, float scale, float coef,
                                          void* out) {
#pragma unroll
  for (int u = 0; u < RawTile<IN, W>::kChunks; ++u) {
    const int c = RawTile<IN, W>::chunk_at(u);
    float g[W];
    r.widen(u, scale, g);
#pragma unroll
    for (int j = 0; j < W; ++j) g[j] *= coef;
    if (n == kGradTile) store_chunk<OUT, W>(out, c, W, g);
    else store_chunk<OUT, W>(out, c, n - c, g);
  }
}

// zs::fixed_to_double, operation for operation: RNE_binary64(X * 2^-128).  Its words are
// chosen by comparisons, not by an index, so they stay in registers: every workgroup waits for
// this number.
__device__ __forceinline__ double fixed_value(const uint32_t w[zs::kSumWords]) {
  constexpr int kN = zs::kSumWords;
  int word = -1;
  uint32_t high = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if (w[k] != 0u) {
      word = k;
      high = w[k];
    }
  if (word < 0) return 0.0;
  const int top = 32 * word + (31 - __clz(static_cast<int>(high)));
  if (top <= 52)
    return __builtin_amdgcn_ldexp(static_cast<double>(static_cast<uint64_t>(w[1]) << 32 | w[0]),
                                  -128);
  const int s = top - 52, i = s >> 5, off = s & 31;    // lowest kept bit
  const int half = (s - 1) >> 5, half_bit = (s - 1) & 31;
  uint32_t w0 = 0, w1 = 0, w2 = 0, wh = 0, sticky = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    w0 = k == i ? w[k] : w0;
    w1 = k == i + 1 ? w[k] : w1;
    w2 = k == i + 2 ? w[k] : w2;
    wh = k == half ? w[k] : wh;
    sticky |= k < half ? w[k] : 0u;
  }
  sticky |= wh & ((1u << half_bit) - 1u);
  const uint64_t lo = static_cast<uint64_t>(w1) << 32 | w0, hi = w2;
  uint64_t mant = (off ? lo >> off | hi << (64 - off) : lo) & ((1ull << 53) - 1ull);
  if (((wh >> half_bit) & 1u) && (sticky != 0u || (mant & 1ull))) ++mant;   // (2^53 is exact too)
  return __builtin_amdgcn_ldexp(static_cast<double>(mant), s - 128);
}

// The step's gate (zs::evaluate_gate, operation for operation) with the norm that it comes
// from: infinite where a value is not finite.
__device__ __forceinline__ zs::Gate gate_and_norm(const GradClipParams& p, double& norm) {
  zs::Gate g{1.0f, 0};
  norm = 0.0;
  if (p.n_accs <= 0) return g;
  uint32_t w[zs::kSumWords];
  uint64_t nonfinite;
  zs::acc_total(p.accs, p.n_accs, w, nonfinite);
  norm = nonfinite > 0 ? __builtin_huge_val() : __builtin_sqrt(fixed_value(w));
  if (p.check_overflow && nonfinite > 0) {
    g.skip = 1;
  } else if (p.max_norm > 0.0) {
    const double c = p.max_norm / (norm + 1e-6);
    g.coef = c < 1.0 ? static_cast<float>(c) : 1.0f;
  }
  return g;
}

// (At least four workgroups to a unit: with the registers that the compiler takes by itself three,
// and 194 tensors of 301 MB take 169 us for both passes, not 165.)
__global__ __launch_bounds__(kGradThreads, 4) void grads_clip_kernel(const GradClipParams p) {
  __shared__ zs::Gate s_gate;
  if (threadIdx.x == 0) {
    double norm;
    const zs::Gate g = gate_and_norm(p, norm);
    s_gate = g;
    if (p.lead && blockIdx.x == 0) {
      if (p.skipped_out != nullptr) *p.skipped_out = g.skip;
      if (p.coef_out != nullptr) *p.coef_out = g.skip ? 0.f : g.coef;
      if (p.norm_out != nullptr) *p.norm_out = static_cast<float>(norm);
    }
  }
  __syncthreads();
  if (s_gate.skip) return;
  const float coef = s_gate.coef;
  walk<true>(p.t, p.tiles, [&](const auto& raw, int i, uint32_t info, int64_t e0, int n) {
    if (coef == 1.f && p.inv_scale == 1.f && p.out[i] == p.t.grad[i]) return;
    const bool out = info & kBf16Out;
    char* to = static_cast<char*>(p.out[i]) + e0 * (out ? 2 : 4);
    constexpr int kW = std::remove_reference_t<decltype(raw)>::kWidth;
    if constexpr (kW == 8) {
      clip_tile<true>(raw, n, p.inv_scale, coef, to);
    } else {
      if (out) clip_tile<true>(raw, n, p.inv_scale, coef, to);
      else clip_tile<false>(raw, n, p.inv_scale, coef, to);
    }
  });
}

namespace {

uint32_t tiles_of(int64_t n) { return static_cast<uint32_t>((n + kGradTile - 1) / kGradTile); }

// Puts tensors that have elements into the table, from `from` on (with `out` from there
// back), as many as fit it and as have fewer than 2^31 tiles together; the next tensor to take.
template <int N>
int64_t fill_table(const zero_grads_args& a, int64_t from, TensorTable<N>& t, void** out,
                   uint32_t& tiles) {
  const int64_t step = out != nullptr ? -1 : 1;
  t.count = 0;
  tiles = 0;
  for (; from >= 0 && from < a.count; from += step) {
    const int64_t n = a.sizes[from];
    if (n == 0) continue;
    const uint32_t more = tiles_of(n);
    if (t.count == N || (t.count > 0 && tiles + static_cast<uint64_t>(more) > (1u << 31))) break;
    const int i = t.count++;
    t.first[i] = tiles;
    t.info[i] = static_cast<uint32_t>((n - 1) % kGradTile + 1) |
                (a.dtypes[from] == ZERO_BF16 ? kBf16In : 0u);
    t.grad[i] = a.grads[from];
    if (out != nullptr) {
      out[i] = a.outs[from];
      t.info[i] |= a.out_dtypes[from] == ZERO_BF16 ? kBf16Out : 0u;
    }
    tiles += more;
  }
  t.first[t.count] = tiles;
  return from;
}

}  // namespace

size_t grads_workspace() { return kNormGroups * kWords * sizeof(uint64_t); }

hipError_t launch_grads_norm(const zero_grads_args& a, hipStream_t s) {
  GradNormParams p;
  p.inv_scale = static_cast<float>(a.inv_scale);
  p.part = static_cast<uint64_t*>(a.workspace);
  // all launches of a call have the same workgroups, whose rows they add to
  uint64_t all = 0;
  for (int64_t i = 0; i < a.count; ++i) all += tiles_of(a.sizes[i]);
  const int groups = all < kNormGroups ? static_cast<int>(all) : kNormGroups;
  p.add = 0;
  for (int64_t from = 0; from < a.count;) {
    from = fill_table(a, from, p.t, nullptr, p.tiles);
    if (p.tiles == 0) break;
    grads_norm_kernel<<<groups, kGradThreads, 0, s>>>(p);
    p.add = 1;
  }
  if (groups == 0 && a.add) return hipSuccess;
  grads_fold_kernel<<<1, kFoldThreads, 0, s>>>(p.part, groups, a.acc, a.add);
  return hipGetLastError();
}

hipError_t launch_grads_clip(const zero_grads_args& a, hipStream_t s) {
  GradClipParams p;
  p.inv_scale = static_cast<float>(a.inv_scale);
  p.accs = a.accs;
  p.n_accs = a.n_accs;
  p.check_overflow = a.check_overflow;
  p.max_norm = a.max_norm;
  p.norm_out = a.norm_out;
  p.coef_out = a.coef_out;
  p.skipped_out = a.skipped_out;
  p.lead = 1;
  for (int64_t from = a.count - 1; p.lead || from >= 0;) {
    from = fill_table(a, from, p.t, p.out, p.tiles);
    if (p.tiles == 0 && !p.lead) break;
    const uint32_t grid = p.tiles < 1 ? 1 : p.tiles < kClipGroups ? p.tiles : kClipGroups;
    grads_clip_kernel<<<grid, kGradThreads, 0, s>>>(p);
    p.lead = 0;
  }
  return hipGetLastError();
}

}  // namespace zo
