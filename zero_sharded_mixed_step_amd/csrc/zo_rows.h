// zo_rows.h -- rows of values as the memory-bound operators take them: eight
// values of an aligned row, or, where a row may start at any element, 16-byte
// chunks counted from the aligned address at or below its start, whose first and
// last are loaded and stored element by element.
#pragma once

#include "zo_device.h"

namespace zo {

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
  // (past the caches)
  __device__ __forceinline__ static void store_once(void* p, int64_t at, const float x[8]) {
    bf16x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<bf16>(x[j]);
    __builtin_nontemporal_store(v, reinterpret_cast<bf16x8*>(static_cast<bf16*>(p) + at));
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
  __device__ __forceinline__ static void store_once(void* p, int64_t at, const float x[8]) {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, q);
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, q + 1);
  }
};

// Eight columns of a row of C from c on, or, SPLIT, four and four that are kHalf further, so that a
// wave's accesses of 16 bytes leave no gaps where values have 4 bytes.  0 behind the row's end.
// (ONCE: past the caches.)
constexpr int kHalf = 256;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <bool ONCE, typename V>
__device__ __forceinline__ V load_as(const void* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool SPLIT, bool ONCE>
__device__ __forceinline__ void load_raw8(const bf16* p, int c, int C, Vec8<bf16>& v) {
  v.r = u32x4{0, 0, 0, 0};
  if constexpr (SPLIT) {
    if (c < C) {
      const u32x2 x = load_as<ONCE, u32x2>(p + c);
      v.r[0] = x[0];
      v.r[1] = x[1];
    }
    if (c + kHalf < C) {
      const u32x2 x = load_as<ONCE, u32x2>(p + c + kHalf);
      v.r[2] = x[0];
      v.r[3] = x[1];
    }
  } else if (c < C) {
    v.r = load_as<ONCE, u32x4>(p + c);
  }
}
template <bool SPLIT, bool ONCE>
__device__ __forceinline__ void load_raw8(const float* p, int c, int C, Vec8<float>& v) {
  v.a = v.b = f32x4{0.f, 0.f, 0.f, 0.f};
  if (c < C) v.a = load_as<ONCE, f32x4>(p + c);
  if ((SPLIT ? c + kHalf : c) < C) v.b = load_as<ONCE, f32x4>(p + c + (SPLIT ? kHalf : 4));
}
template <typename T, bool SPLIT, bool ONCE = false>
__device__ __forceinline__ void load8(const void* p, int c, int C, float x[8]) {
  Vec8<T> v;
  load_raw8<SPLIT, ONCE>(static_cast<const T*>(p), c, C, v);
  v.get(x);
}

template <bool ONCE, typename V>
__device__ __forceinline__ void store_as(void* p, V v) {
  if constexpr (ONCE) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}
template <bool ONCE>
__device__ __forceinline__ void store4(float* p, const float x[4]) {
  store_as<ONCE>(p, f32x4{x[0], x[1], x[2], x[3]});
}
template <bool ONCE>
__device__ __forceinline__ void store4(bf16* p, const float x[4]) {
  bf16x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = static_cast<bf16>(x[j]);
  store_as<ONCE>(p, v);
}
template <typename T, bool SPLIT, bool ONCE = false>
__device__ __forceinline__ void store8(void* p, int c, int C, const float x[8]) {
  T* const at = static_cast<T*>(p) + c;
  if constexpr (SPLIT) {
    if (c < C) store4<ONCE>(at, x);
    if (c + kHalf < C) store4<ONCE>(at + kHalf, x + 4);
  } else if (c < C) {
    if constexpr (ONCE) Vec8<T>::store_once(at, 0, x);
    else Vec8<T>::store(at, 0, x);
  }
}

// Whether a row's mean square plus eps is near the ends of binary32 (the reciprocal root takes
// no subnormal numbers): of values below 1e-15 with an eps below 1e-30, or above 1e15.
__device__ __forceinline__ bool far_mean(float v) { return !(v >= 1e-30f && v <= 1e30f); }

// 1 / sqrt of such a row's mean from `mean`, that of its values times `power` (2^100 or 2^-100).  Where
// it is no normal number (values below 2^-127 or above 2^126) power and root stay apart, as infinity
// times 0 would be no number: minus the root, and the values take far_power of it.
__device__ __forceinline__ float far_root(float mean, float power) {
  const float root = __builtin_amdgcn_rsqf(mean), r = root * power;
  return r >= 0x1p-126f && r < kInf ? r : -root;
}
__device__ __forceinline__ bool power_apart(float r) {               // (of a value that all lanes have)
  return static_cast<int32_t>(uniform(__float_as_uint(r))) < 0;
}
__device__ __forceinline__ float far_power(float r) {
  return r >= 0.f ? 1.f : r < -1.f ? 0x1p100f : 0x1p-100f;
}

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
  // (ONCE: past the caches)
  template <bool ONCE = false>
  __device__ __forceinline__ Chunk<E> load(int c) const {
    Chunk<E> x;
    const int64_t e0 = static_cast<int64_t>(c) * kN - shift;
    if (whole(c)) {
      const auto* at = reinterpret_cast<const decltype(x.r)*>(p + e0);
      if constexpr (ONCE) x.r = __builtin_nontemporal_load(at);
      else x.r = *at;
    } else {
      x.fill_lowest();
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (e0 + e >= 0 && e0 + e < V) x.put_raw(e, p[e0 + e]);
    }
    return x;
  }
  // y as this row's elements that chunk c of a row shifted by `from` holds: one by one where this row
  // is shifted otherwise (a gradient whose rows start elsewhere between 16 bytes than the logits':
  // 8192 x 50257 bf16 626 us for 313)
  template <bool ONCE = false>
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
      auto* at = reinterpret_cast<decltype(x.r)*>(p + e0);
      if constexpr (ONCE) __builtin_nontemporal_store(x.r, at);
      else *at = x.r;
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

}  // namespace zo
