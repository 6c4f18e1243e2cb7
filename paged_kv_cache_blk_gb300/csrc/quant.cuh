// Quantisation of one token row's heads for int8 pools, shared by the
// quantising scatter (copy_kernels.cu), the rotary append (rope.cu) and the
// fused decode step (decode.cu), so all store the same bytes.
//
// One warp per (token, kv head), VPL = head_dim / 32 values per lane:
// absmax of the head (fp32, a warp max over the |x| bit patterns), scale =
// absmax / 127 and code = round_half_even(x / scale), both divisions IEEE
// fp32 with subnormals kept (div.rn.f32 without .ftz, whatever the fast-math
// flags), codes clamped to [-127, 127].  A zero absmax stores scale 0 and
// codes 0.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace pkv {

__device__ __forceinline__ float div_ieee(float a, float b) {
  float r;
  asm("div.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int VPL>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* src, float (&x)[VPL]) {
  if constexpr (VPL == 8) {
    const uint4 r = *reinterpret_cast<const uint4*>(src);
    x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z); x[5] = bf16_hi(r.z); x[6] = bf16_lo(r.w); x[7] = bf16_hi(r.w);
  } else if constexpr (VPL == 4) {
    const uint2 r = *reinterpret_cast<const uint2*>(src);
    x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
  } else if constexpr (VPL == 2) {
    const uint32_t r = *reinterpret_cast<const uint32_t*>(src);
    x[0] = bf16_lo(r); x[1] = bf16_hi(r);
  } else {
    x[0] = __uint_as_float((uint32_t)(*reinterpret_cast<const uint16_t*>(src)) << 16);
  }
}

// Code of x in a head whose absmax has the bit pattern `absmax`.
__device__ __forceinline__ int quantise_value(float x, uint32_t absmax, float scale) {
  return absmax == 0 ? 0 : min(127, max(-127, __float2int_rn(div_ieee(x, scale))));
}

// The same codes for 4 N values of a head, as stored bytes (code + 128), four a
// word.  x / scale is first taken as x * (1 / scale): an approximate reciprocal
// (1 ulp, 2^-23) and two roundings of 2^-24 of a value up to 127, the IEEE
// quotient one more: together below 2^-14,
// so both round to the same code unless the value lies that near a half-way
// point, and only such elements are divided (bf16 rows have exact half-way
// points, one element in 300).  Scales whose reciprocal is not an
// ordinary number divide always.
template <int N>
__device__ __forceinline__ void quantise_bytes(const float* x, uint32_t absmax, float scale,
                                               uint32_t (&w)[N]) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  const bool exact = !(scale > 7.9e-31f && scale < 1.2e30f);
  uint32_t b[4 * N];
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) {
    // adding 1.5 * 2^23 + 128 leaves the rounded code + 128 in the low byte
    const float t = x[i] * inv;
    const float r = t + 12583040.f;
    b[i] = __float_as_uint(r);
    if (exact || fabsf(t - (r - 12583040.f)) > 0.5f - 0x1p-14f)
      b[i] = (uint32_t)(quantise_value(x[i], absmax, scale) + 128);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                       __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
}

// Quantise one head (VPL values per lane); returns the scale, codes in c.
template <int VPL>
__device__ __forceinline__ float quantise_head(const float (&x)[VPL], int (&c)[VPL]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  m = __reduce_max_sync(0xffffffffu, m);
  const float scale = div_ieee(__uint_as_float(m), 127.f);
#pragma unroll
  for (int i = 0; i < VPL; ++i) c[i] = quantise_value(x[i], m, scale);
  return scale;
}

// Codes are stored offset binary: the byte of code c is c + 128.
template <int VPL>
__device__ __forceinline__ void store_codes(char* dst, const int (&c)[VPL]) {
  uint32_t w[(VPL + 3) / 4] = {};
#pragma unroll
  for (int i = 0; i < VPL; ++i) w[i / 4] |= (uint32_t)((c[i] + 128) & 0xFF) << (8 * (i % 4));
  if constexpr (VPL == 8) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else if constexpr (VPL == 4) {
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else if constexpr (VPL == 2) {
    *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w[0];
  } else {
    *reinterpret_cast<uint8_t*>(dst) = (uint8_t)w[0];
  }
}

}  // namespace pkv
