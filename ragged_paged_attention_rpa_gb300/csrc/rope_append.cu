// Rotation of q and k by given positions, and the cache write of k and v at given
// slots, in one pass over the rows.
//
// Dimensions x, y of a pair i turn by a = pos * inv_freq[i]:
//   x cos a - y sin a,  y cos a + x sin a.
// The angle in turns, pos * inv_freq / 2 pi, is wanted modulo 1 only, so the factor
// inv_freq / 2 pi is taken modulo 1 too (a position is a whole number) as a 64-bit
// fraction F; pos * F modulo 2^64 is then one wrapping product and exact.  F comes
// from a product of two floats and two floats' worth of 1 / 2 pi, the rounding
// error kept by an FMA: 48 bits of it are right.  Its upper two bits, rounded, are quarter
// turns; of the rest, signed, 24 bits go through sincospif, and eight more by their
// first derivatives (a page of e4m3 shows it: a sine off by 2^-22 rounds twice as many
// values to the other neighbour as one off by 2^-24).
//
// A lane holds two octets of a row, so that both dimensions of every pair are its
// own: octets u and u + R / 16 of the rotated part, or of the rest (R the rotated
// dimensions; neighbouring pairs lie within an octet).  D / 16 lanes hold a row, a
// warp 2 to 8 rows at once; the lanes that hold the same pairs of these rows share
// out the sines and exchange them by shuffles.  A warp takes a token's rows, or a
// part of them where there are too few tokens to fill the GPU.
//
// HBM-bound: every row is read once and written once.  8192 tokens of 32 + 2 x 16 rows of
// 256, the pages e4m3: 470 MB in 79 us, 5.9 TB/s (0.87 of a plain copy; the lanes'
// conversions keep the schedulers 48% busy); bf16 pages 83.5 us, 6.4 TB/s; fp32 rows and
// pages 164 us, 6.6 TB/s.  1024 tokens of 8 + 2 rows: 5.6 us, a launch
// and two dependent reads (positions and rows, then the stores) for 10 MB.
#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kWarps = 4;
// CTAs an SM holds at least, which sets the registers: 8192 tokens of 64 rows of 256
// take 83 us with 5 of them and 4 rows (2 of fp32) in flight a lane, 86 with 4 and 6, 90
// with 6 and 3 or 2, 102 with 8 and 2.
constexpr int kMinCtas = 5;

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  const int32_t* pos;
  const int64_t* slots;
  const float* freq;
  void* q_out;
  void* k_pages;
  void* v_pages;
  const float* k_scale;
  const float* v_scale;
  unsigned char* ws;
  int64_t pool_slots;
  int32_t tokens, hq, hkv, rotary, chunks, rows;  // a warp takes `rows` of a token's rows
  bool pairs, whole;  // whole: fp32 rows are 32-byte aligned
};

// Eight elements of a row as they lie in memory, as floats, and back.
template <typename T>
struct Octet;
template <>
struct Octet<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) { u = *reinterpret_cast<const uint4*>(src); }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Octet<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = *reinterpret_cast<const float4*>(src);
    b = reinterpret_cast<const float4*>(src)[1];
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* dst, bool, const float (&x)[8], float, float) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* dst, bool whole, const float (&x)[8], float, float) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
  kv4::store32(dst, whole, w);
}
// e4m3: x / s to the nearest, at most 448, NaN as NaN.  x r by one correction with the
// exact remainder (as kv4::quotient), except where it passes the range of 32 bits, as an
// infinite x does: the remainder of an infinity is NaN.
__device__ __forceinline__ void store8(uint8_t* dst, bool, const float (&x)[8], float s, float r) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = x[4 * i + j], q = v * r;
      y[j] = fabsf(q) < INFINITY ? fmaf(fmaf(-q, s, v), r, q) : q;
    }
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}\n"
        : "=r"(w[i])
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// f / 2 pi modulo 1, in 2^-64: of |f|, negated modulo 1 where f < 0 (one less a small fraction
// would not fit 24 bits).
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr float kHi = 0.15915493667125702f, kLo = 6.4206382432985265e-09f;  // 1 / 2 pi
  const float a = fabsf(f);
  const float hi = a * kHi, lo = fmaf(a, kLo, fmaf(a, kHi, -hi));
  const float part = hi - floorf(hi);  // exact, in [0, 1): hi >= 0
  const float rest = lo - rintf(lo);     // |lo| passes 1 only for |f| beyond 2^26
  const uint64_t turn = __float2ull_rz(part * 18446744073709551616.f) +
                        static_cast<uint64_t>(__float2ll_rn(rest * 18446744073709551616.f));
  return f < 0.f ? uint64_t{0} - turn : turn;
}

// Sine and cosine of a / 2^64 turns.
__device__ __forceinline__ void turned(uint64_t a, float& s, float& c) {
  const uint32_t quarter = static_cast<uint32_t>((a + (uint64_t{1} << 61)) >> 62);
  // The rest, |rest| <= 2^29, over 2^31 half turns.
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(a >> 32) - (quarter << 30));
  const float x = __int2float_rn(rest);
  const float e = static_cast<float>(rest - __float2int_rn(x)) * 1.4629180792671596e-9f;  // pi / 2^31
  float s0, c0;
  sincospif(x * 4.656612873077393e-10f, &s0, &c0);
  const float s1 = fmaf(c0, e, s0), c1 = fmaf(-s0, e, c0);
  s = quarter & 1 ? c1 : s1;
  c = quarter & 1 ? s1 : c1;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

template <int D, typename T, typename KV>
__global__ void __launch_bounds__(32 * kWarps, kMinCtas) append_rope_kernel(const AppendParams p) {
  constexpr int kLanes = D / 16;          // of a row
  constexpr int kRows = 32 / kLanes;      // rows of a warp
  constexpr int kMine = 8 / kRows;        // sines and cosines a lane works out
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;  // rows a lane loads before it stores one
  const int lane = threadIdx.x & 31, u = lane % kLanes, sub = lane / kLanes;
  const int32_t R = p.rotary, heads = p.hq + 2 * p.hkv;
  const bool turns = u < R / 16;
  // The lane's two octets.
  const int32_t first = turns ? 8 * u : R + 8 * (u - R / 16);
  const int32_t second = first + (turns ? R / 2 : (D - R) / 2);
  const int64_t items = static_cast<int64_t>(p.tokens) * p.chunks;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); w < items;
       w += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int32_t t = static_cast<int32_t>(w / p.chunks);
    const int32_t r0 = static_cast<int32_t>(w - static_cast<int64_t>(t) * p.chunks) * p.rows;
    const int32_t r1 = min(heads, r0 + p.rows);
    // The first rows are on their way while the sines are worked out.
    Octet<T> raw[kBatch][2];
    auto load = [&](int32_t rb) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int32_t r = rb + b * kRows;
        if (r >= r1) continue;
        const T* src = r < p.hq ? static_cast<const T*>(p.q) + t * p.qs + static_cast<int64_t>(r) * D
                       : r < p.hq + p.hkv
                           ? static_cast<const T*>(p.k) + t * p.ks + static_cast<int64_t>(r - p.hq) * D
                           : static_cast<const T*>(p.v) + t * p.vs + static_cast<int64_t>(r - p.hq - p.hkv) * D;
        raw[b][0].load(src + first);
        raw[b][1].load(src + second);
      }
    };
    load(r0 + sub);
    int64_t slot = -1;
    if (r1 > p.hq) slot = __ldg(p.slots + t);
    // Pair e of the lane (e < 4 in the first octet of neighbouring pairs) is pair
    // 8 u + e, or 4 u + e and R / 4 + 4 u + e - 4.
    float cs[8], sn[8];
    if (R > 0) {
      const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(__ldg(p.pos + t)));
      float c[kMine], s[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = sub * kMine + i;
        c[i] = 1.f;
        s[i] = 0.f;
        if (turns) {
          const int32_t pair = !p.pairs ? 8 * u + e : (e < 4 ? 4 * u + e : R / 4 + 4 * u + e - 4);
          const float f = __ldg(p.freq + pair), nan = f - f;  // 0, or NaN where f is no number
          turned(pos * turn_fraction(f), s[i], c[i]);
          s[i] += nan;
          c[i] += nan;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int from = e / kMine * kLanes + u;
        cs[e] = __shfl_sync(0xffffffffu, c[e % kMine], from);
        sn[e] = __shfl_sync(0xffffffffu, s[e % kMine], from);
      }
    }
    if (slot >= p.pool_slots) {
      if (lane == 0 && p.ws) report_error(p.ws, RPA_DEVERR_PAGE_ID, t);
      slot = -1;
    }
    for (int32_t rb = r0 + sub; rb < r1;) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int32_t r = rb + b * kRows;
        if (r >= r1) continue;
        float x[8], y[8];
        raw[b][0].floats(x);
        raw[b][1].floats(y);
        if (turns && r < p.hq + p.hkv) {
          if (!p.pairs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float a = x[e], o = y[e];
              x[e] = fmaf(a, cs[e], -o * sn[e]);
              y[e] = fmaf(o, cs[e], a * sn[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = x[2 * e], o = x[2 * e + 1];
              x[2 * e] = fmaf(a, cs[e], -o * sn[e]);
              x[2 * e + 1] = fmaf(o, cs[e], a * sn[e]);
              const float a2 = y[2 * e], o2 = y[2 * e + 1];
              y[2 * e] = fmaf(a2, cs[4 + e], -o2 * sn[4 + e]);
              y[2 * e + 1] = fmaf(o2, cs[4 + e], a2 * sn[4 + e]);
            }
          }
        }
        if (r < p.hq) {
          T* dst = static_cast<T*>(p.q_out) + (static_cast<int64_t>(t) * p.hq + r) * D;
          store8(dst + first, p.whole, x, 1.f, 1.f);
          store8(dst + second, p.whole, y, 1.f, 1.f);
        } else if (slot >= 0) {
          const bool is_k = r < p.hq + p.hkv;
          const int32_t g = is_k ? r - p.hq : r - p.hq - p.hkv;
          KV* dst = static_cast<KV*>(is_k ? p.k_pages : p.v_pages) + (slot * p.hkv + g) * D;
          float s = 1.f, inv = 1.f;
          if constexpr (sizeof(KV) == 1) {
            s = __ldg((is_k ? p.k_scale : p.v_scale) + g);
            // Row and scale 2^64 times as large where the reciprocal could be infinite, or
            // the remainder too small for 32 bits.
            if (s < 0x1p-64f) {
              s *= 0x1p64f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] *= 0x1p64f;
                y[e] *= 0x1p64f;
              }
            }
            inv = 1.f / s;
          }
          store8(dst + first, p.whole, x, s, inv);
          store8(dst + second, p.whole, y, s, inv);
        }
      }
      rb += kBatch * kRows;
      load(rb);
    }
  }
}

// A token's rows are split between warps while these are one wave (1024 tokens of 10
// rows in two parts: 4.9 us; in three, a wave and a little: 6.3).
constexpr int64_t kWave = 152 * kMinCtas * kWarps;

template <int D, typename T, typename KV>
int launch_t(AppendParams& p, cudaStream_t s) {
  constexpr int kRows = 32 / (D / 16);
  const int32_t heads = p.hq + 2 * p.hkv, most = (heads + kRows - 1) / kRows;
  const int32_t want = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(most, kWave / p.tokens)));
  p.rows = (most + want - 1) / want * kRows;
  p.chunks = (heads + p.rows - 1) / p.rows;
  const int64_t warps = static_cast<int64_t>(p.tokens) * p.chunks;
  const int grid = static_cast<int>(std::min<int64_t>((warps + kWarps - 1) / kWarps, 1 << 20));
  append_rope_kernel<D, T, KV><<<grid, 32 * kWarps, 0, s>>>(p);
  return static_cast<int>(cudaGetLastError());
}

template <int D>
int launch_d(AppendParams& p, bool f32, cudaStream_t s) {
  if (p.k_scale) return f32 ? launch_t<D, float, uint8_t>(p, s) : launch_t<D, __nv_bfloat16, uint8_t>(p, s);
  return f32 ? launch_t<D, float, float>(p, s) : launch_t<D, __nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace

int launch_append_rope(const AppendArgs& a, void* stream) {
  if (a.tokens == 0 || a.hq + a.hkv == 0) return 0;
  AppendParams p{a.q, a.k, a.v, a.q_stride, a.k_stride, a.v_stride, a.positions, a.slot_map, a.inv_freq,
                 a.q_out, a.k_pages, a.v_pages, a.k_scale, a.v_scale, a.workspace, a.pool_slots,
                 a.tokens, a.hq, a.hkv, a.rotary_dim, 1, 1, a.interleaved, false};
  p.whole = ((reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_pages) |
              reinterpret_cast<uintptr_t>(a.v_pages)) & 31) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int e = static_cast<int>(cudaErrorInvalidValue);
  switch (a.head_dim) {
    case 64: e = launch_d<64>(p, a.f32, s); break;
    case 128: e = launch_d<128>(p, a.f32, s); break;
    case 256: e = launch_d<256>(p, a.f32, s); break;
    default: break;
  }
  if (e) return e;
  trace_mark(RPA_KERNEL_APPEND_ROPE, stream);
  return 0;
}

}  // namespace rpa
