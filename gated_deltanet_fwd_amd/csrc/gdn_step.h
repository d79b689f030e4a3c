// What the serving steps' kernels share: rows in registers, sums over lanes by swaps, states as buffers.
#pragma once
#include "gdn_device.h"

namespace gdn {

constexpr unsigned MAX_GRID_Y = 65535;

template <typename T, int N> // N elements of a row; rows are 16-byte aligned, no more
struct Vec {
  typedef T type __attribute__((ext_vector_type(N), aligned(N * sizeof(T) < 16 ? N * sizeof(T) : 16)));
};

template <typename T, int N>
__device__ __forceinline__ void unpack(const typename Vec<T, N>::type& r, float* v) {
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = (float)r[e];
}

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// The lane-swap instructions exchange the odd 16-lane rows (swap16) or the upper half (swap32) of x
// with the even rows or the lower half of y.
struct Pair {
  float x, y;
};
__device__ __forceinline__ Pair swap16(float x, float y) {
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  return {__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, (unsigned)s[1])};
}
__device__ __forceinline__ Pair swap32(float x, float y) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
  return {__builtin_bit_cast(float, (unsigned)s[0]), __builtin_bit_cast(float, (unsigned)s[1])};
}
// x in a register of its own (with one value as both operands the compiler folds a swap away)
__device__ __forceinline__ float copy_of(float x) {
  asm("" : "+v"(x));
  return x;
}

// cache policies of a buffer access: non-temporal; non-temporal and written through
constexpr int NT = 2, WRITE_THROUGH = 19;

} // namespace gdn
