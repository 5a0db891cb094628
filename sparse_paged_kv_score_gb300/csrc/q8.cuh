// The 8-bit cache format: one scale s for a sub-block of 16 tokens and 128 dims of a head (K and V apart), a power of
// two, and a byte u = c + 128 for a value (c + 1/2) s with the code c = floor(x / s) in [-128, 127].  With a the largest
// magnitude of the sub-block's rows and E = floor(log2 a):  s = 2^(E - 6), at least 2^-126; 0 for a = 0, NaN where a
// value is not finite.
//   - |value - x| <= s / 2 <= max(a / 128, 2^-127), for every x of the sub-block.
//   - The mean of value - x is 0 for numbers anywhere between two codes.  bf16 numbers of at least s lie g apart, s / g of them to
//     a code: floors are taken of 0, g, .. s - g beyond it, (s - g) / 2 on average, so they come back g / 2 high, whatever their sign.
//     N(0, 1) rows in bf16: +0.0022 in the mean beside an error of 0.0105 rms; in fp32 3e-6.
//   - Floors compose: floor(floor(x / s) / 2^k) = floor(x / (2^k s)).  A sub-block whose scale grows as rows are added
//     holds what it would hold had they all come at once, so appends may be cut into calls in any way.
//   - (c + 1/2) s = (2 c + 1) s / 2 has 8 significant bits: exact in bf16, and 16 of them sum exactly in fp32.
// (One fp32 scale and codes rounded to nearest would halve the error at best, where a is a power of two, and would lose
// both properties: a growing scale rounds the codes again.)
//
// A page-head is 16416 contiguous bytes, in the order in which a lane of the decode attention takes them:
//   [0, 8192)      key codes, 8 tokens to 1024 bytes: token t's dims 32 c + 16 j .. + 15 at 512 j + 64 (t % 8) + 16 c
//   [8192, 16384)  value codes, 8 tokens to 1024 bytes: tokens t, t + 1 (t even) and dims 16 b + 8 j .. + 7 at
//                  512 j + 64 b + 16 ((t % 8) / 2), the two tokens' bytes of a dim side by side
//   [16384, 16416) the key scales of the four sub-blocks, their value scales (fp32)
// so that 16-byte load j of lane 4 r + c gives key r's dims 32 c + 16 j .., or values 2c and 2c + 1's dims 16 r + 8 j ..
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace spkv {

constexpr int kQ8Page = 16416;      // bytes of a page-head
constexpr int kQ8V = 8192;          // value codes
constexpr int kQ8KScale = 16384;
constexpr int kQ8VScale = 16400;

// Byte of token t, dim d.
__host__ __device__ __forceinline__ int q8_k_code(int t, int d) {
  return (t >> 3) * 1024 + ((d >> 4) & 1) * 512 + (t & 7) * 64 + (d >> 5) * 16 + (d & 15);
}
__host__ __device__ __forceinline__ int q8_v_code(int t, int d) {
  return kQ8V + (t >> 3) * 1024 + ((d >> 3) & 1) * 512 + (d >> 4) * 64 + ((t & 7) >> 1) * 16 + (d & 7) * 2 + (t & 1);
}

// Scale, as bits, of a sub-block whose largest magnitude has the bits a (a NaN's are the largest).  Scales are ordered
// as their bits are, 0 first and NaN last.
constexpr uint32_t kQ8NaN = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t q8_scale(uint32_t a) {
  if (a == 0) return 0;
  if (a >= 0x7F800000u) return kQ8NaN;
  return static_cast<uint32_t>(max(static_cast<int>(a >> 23) - 6, 1)) << 23;
}
// 1 / s of a scale; 0 for 0 and NaN.
__device__ __forceinline__ float q8_inverse(uint32_t s) {
  return s == 0 || s >= 0x7F800000u ? 0.f : __uint_as_float((254u << 23) - s);
}
// Bytes of four values under a scale's inverse: floor(x / s) + 128, from one fused product and sum rounded down (so that a
// negative number too small for fp32 gives -1).  1.5 * 2^23: the sum's last bits are the integer's.
__device__ __forceinline__ uint32_t q8_bytes(float4 x, float inverse) {
  constexpr float kMagic = 12582912.f + 128.f;
  const uint32_t a = __float_as_uint(__fmaf_rd(x.x, inverse, kMagic)), b = __float_as_uint(__fmaf_rd(x.y, inverse, kMagic));
  const uint32_t c = __float_as_uint(__fmaf_rd(x.z, inverse, kMagic)), d = __float_as_uint(__fmaf_rd(x.w, inverse, kMagic));
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Powers of two by which codes under scale `was` shrink under scale `is` >= was (8 leaves only their sign).
__device__ __forceinline__ int q8_shift(uint32_t was, uint32_t is) {
  return is >= 0x7F800000u ? 0 : min(8, static_cast<int>((is - was) >> 23));
}
// floor(c / 2^k) of four codes: floor((u - 128) / 2^k) + 128 = (u + 128 (2^k - 1)) >> k, two bytes at a time.
__device__ __forceinline__ uint32_t q8_shrink(uint32_t w, int k) {
  const uint32_t add = 0x00800080u * ((1u << k) - 1u);
  const uint32_t lo = (((w & 0x00FF00FFu) + add) >> k) & 0x00FF00FFu;
  const uint32_t hi = ((((w >> 8) & 0x00FF00FFu) + add) >> k) & 0x00FF00FFu;
  return lo | hi << 8;
}

// Bytes 0 and 1 (2 and 3) of w as the f16 pair of their codes: 0x6400 | u is 1024 + u.
__device__ __forceinline__ uint32_t q8_f16(uint32_t magic) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(magic), "r"(0xE480E480u));   // - 1152
  return d;
}
__device__ __forceinline__ uint32_t q8_f16_lo(uint32_t w) { return q8_f16(__byte_perm(w, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t q8_f16_hi(uint32_t w) { return q8_f16(__byte_perm(w, 0x64646464u, 0x4342)); }

}  // namespace spkv
