// The 4-bit KV format (RPA_DTYPE_FP4_E2M1) on the device.
//
// A row of D dimensions is D / 16 blocks.  A dimension is an e2m1 code (sign,
// two exponent bits of bias 1, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6),
// two to a byte, the even dimension in the low half; a block has one unsigned
// scale byte of five exponent bits (bias 15) and three mantissa bits, which
// are the f16 bits of the scale shifted right by 7: a scale is read with one
// shift.  Scales stop at 10240, so that a code times its scale (six
// significant bits at most, magnitudes 2^-18 to 61440) is exact in f16, and
// exact in bf16 too; byte 255 reads as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace rpa {
namespace kv4 {

constexpr float kMaxScale = 10240.f;

// The scale byte for a block whose largest magnitude is `amax` (finite): the
// nearest scale to amax / 6, ties to even.  The division is correctly rounded,
// and no float next to a midpoint of two scales divides onto it (the midpoint
// times 6 has at most 7 significant bits), so this equals rounding the exact
// quotient.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float t = fminf(__fdiv_rn(amax, 6.f), kMaxScale);
  if (t < 6.103515625e-5f)  // below 2^-14: steps of 2^-17
    return static_cast<uint32_t>(__float2int_rn(t * 131072.f));
  const uint32_t b = __float_as_uint(t);
  return ((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// Two codes (low half first) of two floats: round to nearest even, at most 6.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n mov.b32 %0, {t, 0, 0, 0};\n}\n"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// A block of 16 floats -> codes (element 0 in the lowest four bits) and the
// scale byte.  x / s is computed as x r with r ~ 1 / s and one correction by
// the exact remainder, which gives the quotient itself wherever it is
// representable (the ties between codes are), so a tie goes to the even code.
__device__ __forceinline__ uint32_t encode_block(const float (&x)[16], uint2& codes) {
  uint32_t top = 0;  // largest magnitude as bits: NaN > infinity > finite
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  codes = make_uint2(0u, 0u);
  if (top >= 0x7f800000u) return 255u;
  const uint32_t byte = scale_byte(__uint_as_float(top));
  const float s = scale_value(byte);
  const float r = byte ? __frcp_rn(s) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float q = x[i + k] * r;
      v[k] = fmaf(fmaf(-q, s, x[i + k]), r, q);
    }
    w[i >> 3] |= encode2(v[0], v[1]) << (4 * (i & 7));
  }
  codes = make_uint2(w[0], w[1]);
  return byte;
}

// Eight codes -> four f16x2 of two consecutive elements each (exact).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two scale bytes -> f16x2, `lo` in the low half.
__device__ __forceinline__ uint32_t scale_pair(uint32_t lo, uint32_t hi) {
  return (lo | (hi << 16)) << 7;
}

// A block's values: codes times the scale, as f16x2 pairs (exact).
__device__ __forceinline__ void decode_block(uint2 codes, uint32_t byte, uint32_t (&h)[8]) {
  uint32_t a[4], b[4];
  decode8(codes.x, a);
  decode8(codes.y, b);
  const uint32_t s = scale_pair(byte, byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = hmul2(a[i], s);
    h[4 + i] = hmul2(b[i], s);
  }
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace kv4
}  // namespace rpa
