// Key bounds of a block, and the 8-bit codes with power-of-two scales that
// hold them and the queries scored against them (bounds.cu, select.cu).
//
// For one block and kv head: hi_d and lo_d, the largest and smallest key
// element d over the block's rows, so that
//   q . k <= sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d)
// for every key k of the block.  They are stored as codes in [-127, 127] of
// the unit 2^e, e the smallest exponent in [-40, 40] with absmax <= 127 2^e:
// hi rounded up and lo rounded down, so the bound still holds.  With a query
// coded the same way the sum is one of whole numbers, below 2^24 in absolute
// value, times a power of two: exact in fp32 in any order, so scores, ties and
// with them the selected blocks do not depend on how the sum is split.  Half
// the bytes of bf16 bounds, and they are what the scoring pass reads.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace pkv {

constexpr int kBoundExpMin = -40, kBoundExpMax = 40;

// e for an absmax given by its fp32 bit pattern (sign bit clear): 127 is
// 1.984375 * 2^6.  Zeros and subnormals clamp to the smallest e, infinities
// and NaN to the largest.
__device__ __forceinline__ int bound_exponent(uint32_t absmax) {
  const int e = (int)(absmax >> 23) - 133 + ((absmax & 0x7FFFFFu) > 0x7E0000u);
  return min(kBoundExpMax, max(kBoundExpMin, e));
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Products, maxima and conversions with subnormals kept, whatever the
// fast-math flags; the maxima propagate NaN.
__device__ __forceinline__ float mul_ieee(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Codes of hi (rounded up) and lo (rounded down) in units 1 / inv, a power of
// two.  The product is exact but where it lies below the range of fp32: rounded the
// code's way there too, it does not become 0.  A NaN takes the outermost code.
__device__ __forceinline__ int code_up(float x, float inv) {
  float y;
  int c;
  asm("mul.rp.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(inv));
  asm("cvt.rpi.s32.f32 %0, %1;" : "=r"(c) : "f"(y));
  return x != x ? 127 : min(127, max(-127, c));
}
__device__ __forceinline__ int code_down(float x, float inv) {
  float y;
  int c;
  asm("mul.rm.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(inv));
  asm("cvt.rmi.s32.f32 %0, %1;" : "=r"(c) : "f"(y));
  return x != x ? -127 : min(127, max(-127, c));
}

}  // namespace pkv
