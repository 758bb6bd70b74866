// The numbers of a cache in 4 bits: 16 neighbouring channels of a row share a
// scale s, a byte whose bits moved up by 7 are a binary16, and each stands for
// (code - 8) s.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace h3 {
namespace {

constexpr uint32_t kScaleMax = 0xD7;  // 3840; bytes above it stand for NaN

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte > kScaleMax ? __int_as_float(0x7FFFFFFF) : __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// The largest of 8 bf16 values without their signs, as bits (a NaN is larger than an infinity).
__device__ __forceinline__ uint32_t abs_max8(const uint32_t* n) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(n[0] & kAbs, n[1] & kAbs), __vmaxu2(n[2] & kAbs, n[3] & kAbs));
  return max(m & 0xFFFFu, m >> 16);
}
// The same of two times 8 values, in the lower and the upper half.
__device__ __forceinline__ uint32_t abs_max8_pair(const uint32_t* n, const uint32_t* m) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t x = __vmaxu2(__vmaxu2(n[0] & kAbs, n[1] & kAbs), __vmaxu2(n[2] & kAbs, n[3] & kAbs));
  const uint32_t y = __vmaxu2(__vmaxu2(m[0] & kAbs, m[1] & kAbs), __vmaxu2(m[2] & kAbs, m[3] & kAbs));
  return __vmaxu2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
}

// How a group is stored whose largest value is `top` (bf16 bits).
//   scale: top / 7 rounded to 5 exponent and 3 mantissa bits.  A quotient of an 8-bit significand and 7 lies half way
//     between two such numbers or at least 2^-8 of itself away, so the product with 1 / 7, a few steps of float32 off, is
//     put back on the halves by rounding it to 8 steps.
//   codes: |x| / s is a quotient of an 8-bit and a 4-bit significand, so it either lies half way between two integers or is
//     at least 2^-9 of itself away from there: taken 2^-13 too large, which is more than its float32 error, halves are
//     rounded away from zero and nothing else is.  The rounding is the addition of 1.5 * 2^23, whose bits are taken
//     off the packed codes at the end.  Between the least normal and the largest scale |x| / s is below 7.5.
constexpr float kRoundCode = 12582912.0f + 8.0f;             // and the codes' 8
constexpr uint32_t kRoundBits = 0x4B400000u * 0x11111111u;  // of 12582912, in all eight places

// Both maxima of a pair lie in [2^-11, 2^14): their scales are normal and below the largest one.
__device__ __forceinline__ bool plain_maxima(uint32_t tops) {
  return __vmaxu2(__vminu2(tops, 0x467F467Fu), 0x3A003A00u) == tops;
}
// The scale of such a group, `top` as float bits, and the codes of 8 of its values.
__device__ __forceinline__ uint32_t plain_codes(const uint32_t* n, uint32_t top, uint32_t& codes) {
  const uint32_t u = (__float_as_uint(__uint_as_float(top) * (1.0f / 7.0f)) + 4u) & ~7u;
  const uint32_t r = u + 0x7FFFFu + ((u >> 20) & 1u);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__uint_as_float(r & 0xFFF00000u)));
  inv *= 1.0f + 0x1p-13f;
  codes = 0u - kRoundBits;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __uint_as_float(e & 1 ? n[e >> 1] & 0xFFFF0000u : n[e >> 1] << 16);
    codes += __float_as_uint(fmaf(x, inv, kRoundCode)) << (4 * e);
  }
  return (r >> 20) - (112u << 3);
}
// Any group's scale, and the codes of 8 of its values.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  if (top >= 0x7F80u) return 0xFFu;
  const float t = fminf(__uint_as_float(top << 16) * (1.0f / 7.0f), 3840.0f);
  const uint32_t u = (__float_as_uint(t) + 4u) & ~7u;
  if (u < 0x38800000u) return static_cast<uint32_t>(__float2int_rn(__uint_as_float(u) * 0x1p17f));  // below 2^-14
  return ((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
}
__device__ __forceinline__ uint32_t codes_of(uint32_t n0, uint32_t n1, uint32_t n2, uint32_t n3, uint32_t scale) {
  if (scale == 0u || scale == 0xFFu) return 0x88888888u;
  const float inv = __fdividef(1.0f + 0x1p-13f, scale_value(scale));
  uint32_t codes = 0;
#pragma unroll 1
  for (int e = 7; e >= 0; --e) {
    const uint32_t w = e < 2 ? n0 : e < 4 ? n1 : e < 6 ? n2 : n3;
    const float x = __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    codes = codes * 16u + __float_as_uint(fminf(fmaxf(x * inv, -8.0f), 7.0f) + kRoundCode);
  }
  return codes - kRoundBits;
}

}  // namespace
}  // namespace h3
