// q8_common.cuh — shared by the kernels of the paged 8-bit cache: how bf16 values find
// their power-of-two e4m3 scale (the quantising write, the split of the attention's
// queries), and the cluster barrier in two halves.
#pragma once

#include <cstdint>

namespace ddt {

// The larger magnitude of two packed bf16 values each, under some sign; NaN if either is.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The larger of the two halves' magnitudes.
__device__ __forceinline__ uint32_t max_of_halves(uint32_t m) { return max(m & 0x7fffu, (m >> 16) & 0x7fffu); }

// Smallest e with amax <= 448 * 2^e for the bits of a finite bf16 magnitude: 448 = 1.75 *
// 2^8, so e is amax's exponent less 8, one more when its significand exceeds 1.75.
__device__ __forceinline__ int e4m3_exponent(uint32_t amax_bits) {
  return static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u);
}

__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Cluster barrier in two halves: what a CTA wrote (or read) before its arrival lies
// before what any CTA does after its wait.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace ddt
