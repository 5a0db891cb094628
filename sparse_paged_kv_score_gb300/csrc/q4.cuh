// The 4-bit cache format: e2m1 codes, one e4m3 scale for 16 dims of a token-head, one fp32 scale g
// for a kv head; value = code * scale * g.  A page-head is 9216 contiguous bytes, laid out in the
// order in which a warp of the decode attention takes it into matrix fragments:
//   [0, 4096)     key codes: token t at 64 t, byte b holds dims 2b (low nibble) and 2b + 1
//   [4096, 8192)  value codes: 8 tokens x 8 blocks of 16 dims, block-major: (t / 8) * 512 +
//                 block * 64 + (t % 8) * 8, eight bytes (16 dims)
//   [8192, 8704)  key scales: lane (t % 8, block / 2), then t / 16, (t / 8) % 2, block % 2
//   [8704, 9216)  value scales: lane (block, (t % 8) / 2), then t / 16, (t / 8) % 2, t % 2
// so one 16-byte load of lane 4 r + c gives keys r's dims 32 c .. 32 c + 31, values 2c and 2c + 1's
// block r, and all four 16-token tiles' scales of those.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace spkv {

constexpr int kQ4Page = 9216;        // bytes of a page-head
constexpr int kQ4V = 4096;           // value codes
constexpr int kQ4KScale = 8192;
constexpr int kQ4VScale = 8704;
constexpr int kQ4Block = 16;         // dims that share a scale

__host__ __device__ __forceinline__ int q4_k_code(int t) { return t * 64; }
// Block `blk` (16 dims, 8 bytes) of token t's value.
__host__ __device__ __forceinline__ int q4_v_code(int t, int blk) {
  return kQ4V + (t >> 3) * 512 + blk * 64 + (t & 7) * 8;
}
__host__ __device__ __forceinline__ int q4_k_scale(int t, int blk) {
  return kQ4KScale + (4 * (t & 7) + (blk >> 1)) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (blk & 1);
}
__host__ __device__ __forceinline__ int q4_v_scale(int t, int blk) {
  return kQ4VScale + (4 * blk + ((t & 7) >> 1)) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
}

// The four bytes of w (two e2m1 codes each, the low nibble first) as four f16 pairs.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Two e4m3 scales (low byte first) as an f16 pair.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
  uint32_t o;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o) : "h"(static_cast<uint16_t>(two)));
  return o;
}
// a, b as two e2m1 codes in one byte (a in the low nibble); nearest even, saturating.
__device__ __forceinline__ uint32_t f32_to_e2m1(float a, float b) {
  uint32_t o;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(o) : "f"(a), "f"(b));
  return o;
}
// x as an e4m3 byte; nearest even, saturating (NaN gives 0x7F).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t o;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(o) : "f"(0.f), "f"(x));
  return o & 0xFFu;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  const uint32_t h = e4m3_to_f16(byte);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}
// The code in the low nibble of n as fp32.
__device__ __forceinline__ float e2m1_to_f32(uint32_t n) {
  const uint32_t mag = n & 7u;
  // 1.m * 2^(e-1) for e > 0, m / 2 for e = 0
  const float v = mag < 2 ? 0.5f * mag : __uint_as_float(((mag >> 1) + 126u) << 23 | (mag & 1u) << 22);
  return n & 8u ? -v : v;
}

// The scale byte of a block whose largest magnitude is amax (its bits, so that a NaN counts as the
// largest), for the head's scale g: e4m3(amax / (6 g)).
__device__ __forceinline__ uint32_t q4_scale_byte(uint32_t amax_bits, float g) {
  return f32_to_e4m3(__fdiv_rn(__uint_as_float(amax_bits), __fmul_rn(6.0f, g)));
}

// Largest magnitude's bits over N values.
template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&x)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// N values of a block as codes, two a byte, dim order; d = scale * g.  A block whose scale is zero
// or NaN holds zero codes (its values are 0, or NaN by the scale).
// A code is x / d, rounded to fp32 and then to e2m1.  With r = 1 / d to half a step (2^-24), x r (1 -+ 2^-21) and
// the products' own roundings leave fp32(x / d) between the two products, and rounding to fewer bits keeps the
// order: where both round alike that is the code.  Only else is x divided (6000 rows in and out 45.9 -> 44.4 us).
template <int N>
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[N], float d) {
  if (!(d > 0.f)) return 0;
  const bool near = d >= 0x1p-100f && d <= 0x1p100f;   // else bounds that do not meet
  const float r = __frcp_rn(d);
  const float lo = near ? __fmul_rn(r, 1.f - 0x1p-21f) : 0.f;
  const float hi = near ? __fmul_rn(r, 1.f + 0x1p-21f) : __int_as_float(0x7F800000);
  uint32_t w = 0, up = 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    w |= f32_to_e2m1(__fmul_rn(x[i], lo), __fmul_rn(x[i + 1], lo)) << (4 * i);
    up |= f32_to_e2m1(__fmul_rn(x[i], hi), __fmul_rn(x[i + 1], hi)) << (4 * i);
  }
  if (w == up) return w;
  w = 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) w |= f32_to_e2m1(__fdiv_rn(x[i], d), __fdiv_rn(x[i + 1], d)) << (4 * i);
  return w;
}

// Four codes (the low 16 bits of c) times their scale, exact.
__device__ __forceinline__ float4 q4_values(uint32_t c, float scale) {
  uint32_t h[4];
  e2m1_to_f16(c, h);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

}  // namespace spkv
