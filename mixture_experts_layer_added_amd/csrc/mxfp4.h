// MXFP4 as the kernels use it: E2M1 codes (sign, two bits of exponent, one of mantissa: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6), two a byte with the even element in the low four bits, and one E8M0 scale,
// 2^(code - 127), per 32 elements; scale code 255 is NaN and makes its whole block NaN.
#pragma once
#include "launch_added.h"

namespace moe {

constexpr int kMxBlock = 32;

// Scale code of a block from the bits of its largest magnitude m 2^x, 1 <= m < 2: the smallest
// scale for which that value still lies inside the codes' range, whose last value is 6.  At
// 2^(x-2) it becomes 4 m: rounding to nearest takes it to 6 up to (not with) 4 m = 7, and the two
// neighbours of stochastic rounding need 4 m <= 6; beyond that the next power of two is taken.
// The integer maximum of the bits of |x| puts an infinity above every number and a NaN above
// that, so either of them makes the block NaN.
template <bool kRandom>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t bits) {
  const uint32_t e = bits >> 23, m = bits & 0x7fffffu;
  if (bits == 0) return 127;  // a block of zeros: scale 1
  if (e == 255) return 255;
  return e < 2 ? 0 : e - 2 + (kRandom ? m > 0x400000u : m >= 0x600000u);
}
// 2^(code - 127); code 0 is 2^-127, not a normal number; code 255 (NaN) has no use as a divisor
__device__ __forceinline__ float mx_scale(uint32_t code) {
  return __uint_as_float(code ? code << 23 : 0x400000u);
}

// Codes of two values over scale s, to nearest even, in byte kByte of w.  The conversion divides
// exactly (s is a power of two) and treats s = 2^-127 as such.
template <int kByte>
__device__ __forceinline__ uint32_t mx_pack2(uint32_t w, float a, float b, float s) {
  return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, s, kByte);
}
__device__ __forceinline__ uint32_t mx_pack8(const float* v, float s) {
  uint32_t w = 0;
  w = mx_pack2<0>(w, v[0], v[1], s);
  w = mx_pack2<1>(w, v[2], v[3], s);
  w = mx_pack2<2>(w, v[4], v[5], s);
  return mx_pack2<3>(w, v[6], v[7], s);
}

// Code of v under scale code sc, rounded to one of its two neighbours by a random byte r: up where
// the fraction between them, in 256ths, passes r + 1/2, so that the mean over all r is v within 1/512
// of a step.
__device__ __forceinline__ uint32_t mx_code_random(float v, uint32_t sc, uint32_t r) {
  const float a = __builtin_fabsf(v) * mx_scale(254 - sc);
  const bool b2 = a >= 2.0f, b4 = a >= 4.0f;
  const float f = a * (b4 ? 0.5f : b2 ? 1.0f : 2.0f), low = __builtin_floorf(f);
  const uint32_t m = (uint32_t)low + ((f - low) * 256.0f > (float)r + 0.5f);
  return (m + (b4 ? 4u : b2 ? 2u : 0u)) | (__float_as_uint(v) >> 31 << 3);
}
// Eight codes at once, for v that were bf16 (those below 1 need no more than 22 bits of fraction).  The
// conversion adds the seed to the fraction below the code and cuts: with 255 - r in the seed's top
// byte and 0x7fffff behind it the code is the upper one where the fraction passes r + 1/2.  Compared
// with the definition for every finite bf16 inside the range of every scale, and every byte
// (tests/test_gpu_mxfp4_random_all.py).  Of each conversion only the low four bits are used: the
// second value of a pair takes other bits of the seed, and what the register held before is not kept.
// r is given as 255 - r.
__device__ __forceinline__ uint32_t mx_pack8_random(const float* v, uint32_t sc, uint2 r) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = mx_scale(sc);
  auto code = [&](float x, uint32_t bytes, uint32_t i) {
    const f32x2 p = {x, x};
    const uint32_t seed = __builtin_amdgcn_perm(bytes, 0x007fffffu, (4 + i) << 24 | 0x020100u);
    return (uint32_t)__builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(
        0u, __builtin_shufflevector(p, p, 0, -1), seed, s, 0);
  };
  auto join = [&](int first) {  // codes first, first + 2, + 4, + 6 in the low halves of four bytes
    const uint32_t a = __builtin_amdgcn_perm(code(v[first + 2], r.x, first + 2),
                                             code(v[first], r.x, first), 0x0c0c0400u);
    const uint32_t b = __builtin_amdgcn_perm(code(v[first + 6], r.y, first + 2),
                                             code(v[first + 4], r.y, first), 0x0c0c0400u);
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
  };
  const uint32_t even = join(0), odd = join(1) << 4;
  return (even & 0x0f0f0f0fu) | (odd & 0xf0f0f0f0u);
}

// D += B A over one block of 64 of k: 32 x 32 outputs, lane l holds 32 codes (16 bytes) of row
// l % 32 of either operand and the scale of those in byte kOb / kOa of its scale register.  The
// result's lane holds row l % 32 of A and rows 8 (i/4) + 4 (l/32) + i%4 of B, i = 0 .. 15.
template <int kOb, int kOa>
__device__ __forceinline__ f32x16 mx_mfma32(const u32x4& b, const u32x4& a, const f32x16& c,
                                            uint32_t sb, uint32_t sa) {
  const i32x8 x = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, kOb, (int)sb, kOa,
                                                         (int)sa);
}

}  // namespace moe
