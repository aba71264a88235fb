// zo_device.h -- device building blocks shared by the training operators:
// element types, wave reductions and the matrix-core fragments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zo {

typedef __bf16 bf16;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.402823466e+38f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t low16) {
  return __uint_as_float(low16 << 16);
}

__device__ __forceinline__ uint32_t uniform(uint32_t x) {
  return __builtin_amdgcn_readfirstlane(x);
}

// Joins a 32- or 64-bit value over groups of G consecutive lanes (all of them get the
// result) by moves between registers: neighbours, pairs, mirrored halves of 8 and
// of 16 lanes (the halves are uniform by then), then rows of 16 and halves of the
// wave swapped.  A shuffle through the shared-memory crossbar takes some 100 cycles
// where one of these takes 8.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false);
}
template <typename T, typename Move>
__device__ __forceinline__ T move_words(T x, Move move) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, move(__builtin_bit_cast(uint32_t, x)));
  } else {
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint64_t lo = move(static_cast<uint32_t>(v)), hi = move(static_cast<uint32_t>(v >> 32));
    return __builtin_bit_cast(T, hi << 32 | lo);
  }
}
template <int G, typename T, typename Op>
__device__ __forceinline__ T join_lanes(T x, Op op) {
  static_assert((sizeof(T) == 4 || sizeof(T) == 8) && G <= 64);
  if constexpr (G >= 2) x = op(x, move_words(x, dpp_move<0xB1>));    // lanes 1 0 3 2
  if constexpr (G >= 4) x = op(x, move_words(x, dpp_move<0x4E>));    // lanes 2 3 0 1
  if constexpr (G >= 8) x = op(x, move_words(x, dpp_move<0x141>));   // 8 lanes mirrored
  if constexpr (G >= 16) x = op(x, move_words(x, dpp_move<0x140>));  // 16 lanes mirrored
  if constexpr (G >= 32)
    x = op(move_words(x, [](uint32_t v) {
             return __builtin_amdgcn_permlane16_swap(v, v, false, false)[0];
           }),
           move_words(x, [](uint32_t v) {
             return __builtin_amdgcn_permlane16_swap(v, v, false, false)[1];
           }));
  if constexpr (G >= 64)
    x = op(move_words(x, [](uint32_t v) {
             return __builtin_amdgcn_permlane32_swap(v, v, false, false)[0];
           }),
           move_words(x, [](uint32_t v) {
             return __builtin_amdgcn_permlane32_swap(v, v, false, false)[1];
           }));
  return x;
}

struct AddOp {
  template <typename X>
  __device__ __forceinline__ X operator()(X a, X b) const {
    return a + b;
  }
};
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const {
    return a > b || a != a ? a : b;      // a NaN stays
  }
  __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};
struct MinOp {
  __device__ __forceinline__ int operator()(int a, int b) const { return min(a, b); }
};
struct OrOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a | b; }
};

}  // namespace zo
