// q8_common.cuh — how bf16 values find their power-of-two e4m3 scale, shared by the
// quantising write and the split of the attention's queries.
#pragma once

#include <cstdint>

namespace ddt {

// Larger of m and |x|, for each of two packed bf16 values; NaN if either is.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(d) : "r"(m), "r"(x));
  return d;
}

__device__ __forceinline__ uint32_t max_of_halves(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Smallest e with amax <= 448 * 2^e for the bits of a finite bf16 magnitude: 448 = 1.75 *
// 2^8, so e is amax's exponent less 8, one more when its significand exceeds 1.75.
__device__ __forceinline__ int e4m3_exponent(uint32_t amax_bits) {
  return static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u);
}

__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace ddt
