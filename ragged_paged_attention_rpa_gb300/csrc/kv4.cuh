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

// Division of row indices below 2^31 by a head count: one wide product and a
// shift (a 64-bit division by a variable costs some 50 instructions, a tenth of
// what a thread of the cache's kernels runs).
struct HeadDiv {
  uint32_t magic, shift;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (__umulhi(n, magic) + n) >> shift;
  }
};
inline HeadDiv head_div(int32_t heads) {
  uint32_t shift = 0;
  while ((1ll << shift) < heads) ++shift;
  return {static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - heads)) / heads + 1), shift};
}

// x / d from r ~ 1 / d by one correction with the exact remainder: the quotient
// itself where it is representable, and otherwise within little more than half
// a step of it.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}

// The scale byte for a block whose largest magnitude is `amax` (finite): the
// nearest scale to amax / 6, ties to even.  A midpoint of two scales times 6
// has at most 7 significant bits, so it divides back onto the midpoint, and the
// floats next to it are more than half a step away: this equals rounding the
// exact quotient.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float t = fminf(quotient(amax, 6.f, 1.f / 6.f), kMaxScale);
  if (t < 6.103515625e-5f)  // below 2^-14: steps of 2^-17
    return static_cast<uint32_t>(__float2int_rn(t * 131072.f));
  const uint32_t b = __float_as_uint(t);
  return ((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// The top bits of the bytes of w that are 255 (scales that read as NaN); and w
// without those bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u;
}
__device__ __forceinline__ uint32_t without_nan(uint32_t w, uint32_t nan) { return w & ~((nan >> 7) * 255u); }

// The blocks of a row of D dimensions that read as NaN, a bit each, from its
// scale bytes.
template <int D>
__device__ __forceinline__ uint32_t nan_blocks(const uint8_t* scales) {
  uint32_t blocks = 0;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t nan = nan_bytes(__ldg(reinterpret_cast<const uint32_t*>(scales) + i));
    blocks |= ((nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) | (nan >> 28 & 8u)) << (4 * i);
  }
  return blocks;
}

// Eight codes (lowest four bits first) of eight floats: round to nearest even,
// at most 6.
__device__ __forceinline__ uint32_t encode8(const float* x) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Largest magnitude of three floats, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// A block of 16 floats -> codes (element 0 in the lowest four bits) and the
// scale byte.  x / s by `quotient`: one that is a midpoint of two magnitudes is
// representable and stays one, so the conversion's tie goes to the even code,
// and no other lands on it (as for the scale).
__device__ __forceinline__ uint32_t encode_block(const float (&x)[16], uint2& codes) {
  float t[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) t[i] = max_abs3(x[3 * i], x[3 * i + 1], x[3 * i + 2]);
  const float top = max_abs3(max_abs3(t[0], t[1], t[2]), max_abs3(t[3], t[4], x[15]), 0.f);
  codes = make_uint2(0u, 0u);
  if (!(top < INFINITY)) return 255u;
  const uint32_t byte = scale_byte(top);
  const float s = scale_value(byte);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  if (byte == 0) r = 0.f;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = quotient(x[i], s, r);
  codes = make_uint2(encode8(v), encode8(v + 8));
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

// 32 bytes from or to global memory: one access where they are 32-byte aligned
// (two 16-byte ones, 32 bytes apart between lanes, touch every sector twice:
// the read of 8192 rows of 16 heads of 256 took 37.5 us with them, 25.7 us so).
__device__ __forceinline__ void load32(const void* src, bool whole, uint32_t (&w)[8]) {
  if (whole) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(src));
  } else {
    const uint4* p = static_cast<const uint4*>(src);
    const uint4 a = __ldg(p), b = __ldg(p + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* dst, bool whole, const uint32_t (&w)[8]) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* p = static_cast<uint4*>(dst);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A block's values as 16 bf16 (exact: six significant bits).
__device__ __forceinline__ void decode_block_bf16(uint2 codes, uint32_t byte, uint32_t (&w)[8]) {
  uint32_t h[8];
  decode_block(codes, byte, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = half2_floats(h[i]);
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace kv4
}  // namespace rpa
