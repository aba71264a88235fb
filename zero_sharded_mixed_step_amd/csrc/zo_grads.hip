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
#include <type_traits>

#include "zo_internal.h"
#include "zs_device.h"

namespace zo {

using zs::kDigits;
using zs::kVec;

constexpr int kGradThreads = 256;
constexpr int kGradTile = 8192;               // elements of a tile: 4 chunks of 8 a thread
constexpr int kTileChunks = kGradTile / kVec / kGradThreads;
constexpr int kNormGroups = 1024;             // workgroups of the norm at most
constexpr int kWords = kDigits + 1;           // digits, then the non-finite count
static_assert(kTileChunks == 4, "a quad's lanes convert a group each");

// Tensors of one launch.  first[i] is tensor i's first tile; its last tile holds tail[i]
// elements.
template <int N>
struct TensorTable {
  int count;
  uint32_t first[N + 1];
  uint16_t tail[N];
  uint8_t type[N];                            // bit 0: bf16 gradients, bit 1: bf16 outputs
  const void* grad[N];

  // The tensor of a tile, from tensor `at` on.
  __device__ __forceinline__ int find(uint32_t tile, int at) const {
    int step = 1;
    while (step < N) step <<= 1;
    for (; step > 0; step >>= 1)
      if (at + step < count && first[at + step] <= tile) at += step;
    return at;
  }
};
constexpr int kNormTensors = 256, kClipTensors = 160;

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

// Eight elements from any element on; those from `left` on read as +0.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

struct Raw8 {
  zs::u32x4 a, b;
};
__device__ __forceinline__ Raw8 load_any(const void* base, bool is_bf16, int64_t e0, int left) {
  Raw8 r{};
  if (is_bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + e0;
    if (left >= kVec) {
      r.a = *reinterpret_cast<const u32x4_any*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < left) r.a[j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
    }
  } else {
    const float* p = static_cast<const float*>(base) + e0;
    if (left >= kVec) {
      const f32x4_any x = *reinterpret_cast<const f32x4_any*>(p);
      const f32x4_any y = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.a[j] = __float_as_uint(x[j]);
        r.b[j] = __float_as_uint(y[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < left) (j < 4 ? r.a : r.b)[j & 3] = __float_as_uint(p[j]);
    }
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw8& r, bool is_bf16, float x[kVec]) {
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const uint32_t h = r.a[j / 2];
    const float b = __uint_as_float(j & 1 ? h & 0xFFFF0000u : h << 16);
    x[j] = is_bf16 ? b : __uint_as_float((j < 4 ? r.a : r.b)[j & 3]);
  }
}

// A thread's chunk u of a tile starts at element (u * 256 + thread) * 8.
__global__ __launch_bounds__(kGradThreads) void grads_norm_kernel(const GradNormParams p) {
  __shared__ uint64_t s_digit[kDigits][kGradThreads];
  __shared__ uint64_t s_part[kGradThreads / 64][kWords];
  const int tid = threadIdx.x, quad_lane = tid & 3;
#pragma unroll
  for (int k = 0; k < kDigits; ++k) s_digit[k][tid] = 0;
  uint32_t nonfinite = 0;
  int at = 0;
  for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    at = p.t.find(tile, at);
    const uint32_t inside = tile - p.t.first[at];
    const int n = tile + 1 == p.t.first[at + 1] ? p.t.tail[at] : kGradTile;
    const bool is_bf16 = p.t.type[at] & 1;
    const int64_t e0 = static_cast<int64_t>(inside) * kGradTile;
    Raw8 raw[kTileChunks];
#pragma unroll
    for (int u = 0; u < kTileChunks; ++u) {
      const int c = (u * kGradThreads + tid) * kVec;
      raw[u] = load_any(p.t.grad[at], is_bf16, e0 + c, n - c);
    }
    double s4[kTileChunks];
#pragma unroll
    for (int u = 0; u < kTileChunks; ++u) {
      float g[kVec];
      widen(raw[u], is_bf16, g);
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[j] *= p.inv_scale;
      // (elements behind the tensor's end are +0: an inv_scale is finite)
      s4[u] = zs::quad_group_sum(zs::chunk_sumsq(g, nonfinite));
    }
    // every lane of a quad holds the four group sums: lane q converts group q
    const double S = quad_lane == 0 ? s4[0] : quad_lane == 1 ? s4[1] : quad_lane == 2 ? s4[2] : s4[3];
    int base;
    uint32_t p0, p1, p2;
    zs::fixed_point_split(S, base, p0, p1, p2);
    if (p0 != 0) s_digit[base][tid] += p0;
    if (p1 != 0) s_digit[base + 1][tid] += p1;
    if (p2 != 0) s_digit[base + 2][tid] += p2;
  }
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

__device__ __forceinline__ void store_any(void* base, bool is_bf16, int64_t e0, int left,
                                          const float x[kVec]) {
  if (is_bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + e0;
    zs::u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __bf16 lo = static_cast<__bf16>(x[2 * j]), hi = static_cast<__bf16>(x[2 * j + 1]);
      w[j] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, lo)) |
             static_cast<uint32_t>(__builtin_bit_cast(uint16_t, hi)) << 16;
    }
    if (left >= kVec) {
      *reinterpret_cast<u32x4_any*>(p) = w;
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < left) p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
  } else {
    float* p = static_cast<float*>(base) + e0;
    if (left >= kVec) {
      *reinterpret_cast<f32x4_any*>(p) = f32x4_any{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_any*>(p + 4) = f32x4_any{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < left) p[j] = x[j];
    }
  }
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
  norm = nonfinite > 0 ? __builtin_huge_val() : __builtin_sqrt(zs::fixed_to_double(w));
  if (p.check_overflow && nonfinite > 0) {
    g.skip = 1;
  } else if (p.max_norm > 0.0) {
    const double c = p.max_norm / (norm + 1e-6);
    g.coef = c < 1.0 ? static_cast<float>(c) : 1.0f;
  }
  return g;
}

__global__ __launch_bounds__(kGradThreads) void grads_clip_kernel(const GradClipParams p) {
  __shared__ zs::Gate s_gate;
  const int tid = threadIdx.x;
  if (tid == 0) {
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
  int at = 0;
  for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    at = p.t.find(tile, at);
    if (coef == 1.f && p.inv_scale == 1.f && p.out[at] == p.t.grad[at]) continue;
    const uint32_t inside = tile - p.t.first[at];
    const int n = tile + 1 == p.t.first[at + 1] ? p.t.tail[at] : kGradTile;
    const bool in_bf16 = p.t.type[at] & 1, out_bf16 = p.t.type[at] & 2;
    const int64_t e0 = static_cast<int64_t>(inside) * kGradTile;
    Raw8 raw[kTileChunks];
#pragma unroll
    for (int u = 0; u < kTileChunks; ++u) {
      const int c = (u * kGradThreads + tid) * kVec;
      raw[u] = load_any(p.t.grad[at], in_bf16, e0 + c, n - c);
    }
#pragma unroll
    for (int u = 0; u < kTileChunks; ++u) {
      const int c = (u * kGradThreads + tid) * kVec;
      float g[kVec];
      widen(raw[u], in_bf16, g);
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[j] = g[j] * p.inv_scale * coef;
      store_any(p.out[at], out_bf16, e0 + c, n - c, g);
    }
  }
}

namespace {

uint32_t tiles_of(int64_t n) { return static_cast<uint32_t>((n + kGradTile - 1) / kGradTile); }

// Puts tensors [from, ...) that have elements into the table, as many as fit it and as have
// fewer than 2^31 tiles together; the next tensor to take.
template <int N>
int64_t fill_table(const zero_grads_args& a, int64_t from, TensorTable<N>& t, void** out,
                   uint32_t& tiles) {
  t.count = 0;
  tiles = 0;
  for (; from < a.count; ++from) {
    const int64_t n = a.sizes[from];
    if (n == 0) continue;
    const uint32_t more = tiles_of(n);
    if (t.count == N || (t.count > 0 && tiles + static_cast<uint64_t>(more) > (1u << 31))) break;
    const int i = t.count++;
    t.first[i] = tiles;
    t.tail[i] = static_cast<uint16_t>((n - 1) % kGradTile + 1);
    t.grad[i] = a.grads[from];
    t.type[i] = a.dtypes[from] == ZERO_BF16 ? 1 : 0;
    if (out != nullptr) {
      out[i] = a.outs[from];
      t.type[i] |= a.out_dtypes[from] == ZERO_BF16 ? 2 : 0;
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
  for (int64_t from = 0; p.lead || from < a.count;) {
    from = fill_table(a, from, p.t, p.out, p.tiles);
    if (p.tiles == 0 && !p.lead) break;
    const uint32_t grid = p.tiles < 1 ? 1 : p.tiles < 4096 ? p.tiles : 4096;
    grads_clip_kernel<<<grid, kGradThreads, 0, s>>>(p);
    p.lead = 0;
  }
  return hipGetLastError();
}

}  // namespace zo
