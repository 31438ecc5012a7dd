// The 4-bit KV cache's write and read: rows of K and V to codes and scales in
// their pages, and back.
//
// A page holds, for each KV head, page_size rows of D / 2 code bytes, and in a
// second array page_size rows of D / 16 scale bytes ([page][head][slot][...]):
// one head's part of a page is one contiguous run, which is how attention
// fetches it.  Row (t, h) of a step goes to (page, slot) = slot_map[t] divided
// by the page size; a negative entry leaves its row out (padding).
//
// One thread per block of 16 dimensions, of K and of V: neighbouring threads
// take neighbouring blocks, so a warp reads 512 consecutive elements of each.
// HBM-bound: at bf16 a row costs 2 bytes an element on one side and 0.5625 on
// the other.  8192 tokens of 16 heads of 256 (172 MB either way): written in
// 28.3 us (6.1 TB/s; the encoding keeps the schedulers 64% busy), read in 25.7 us
// (6.7 TB/s).  A grid split in two, K and V apart, was slower.  A decode step's
// 512 rows take 2 us, a launch's latency.
#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kThreads = 128;

struct Kv4CacheParams {
  const void* k_rows;  // the read's are written
  const void* v_rows;
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_scales;
  uint8_t* v_scales;
  const int64_t* slot_map;
  unsigned char* ws;  // error word (may be null)
  int64_t blocks;     // tokens * heads * blocks a row
  int64_t pool_slots;
  int32_t heads, bpr_shift, page_shift;  // blocks a row = 1 << bpr_shift
  kv4::HeadDiv by_heads;
  bool whole;         // k_rows and v_rows are 32-byte aligned
};

// Block i of an array of rows, as floats and back.
__device__ __forceinline__ void load16(const __nv_bfloat16* rows, int64_t i, bool whole, float (&x)[16]) {
  uint32_t w[8];
  kv4::load32(rows + i * 16, whole, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load16(const float* rows, int64_t i, bool whole, float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
    kv4::load32(rows + i * 16 + 8 * h, whole, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[8 * h + j] = __uint_as_float(w[j]);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* rows, int64_t i, bool whole, uint2 codes, uint32_t byte) {
  uint32_t w[8];
  kv4::decode_block_bf16(codes, byte, w);
  kv4::store32(rows + i * 16, whole, w);
}
__device__ __forceinline__ void store16(float* rows, int64_t i, bool whole, uint2 codes, uint32_t byte) {
  uint32_t h[8];
  kv4::decode_block(codes, byte, h);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = kv4::half2_floats(h[4 * q + j]);
      w[2 * j] = __float_as_uint(f.x);
      w[2 * j + 1] = __float_as_uint(f.y);
    }
    kv4::store32(rows + i * 16 + 8 * q, whole, w);
  }
}

// Block index in the pool of block `b` of head h of token t, or -1 (padding,
// or a slot outside the pool, which sets the error word).
__device__ __forceinline__ int64_t pool_block(const Kv4CacheParams& p, int64_t i) {
  const uint32_t row = static_cast<uint32_t>(i >> p.bpr_shift);  // below 2^31
  const int32_t b = static_cast<int32_t>(i) & ((1 << p.bpr_shift) - 1);
  const uint32_t t = p.by_heads(row);
  const uint32_t h = row - t * p.heads;
  const int64_t slot = __ldg(p.slot_map + t);
  if (slot < 0) return -1;
  if (slot >= p.pool_slots) {
    if (p.ws) report_error(p.ws, RPA_DEVERR_PAGE_ID, static_cast<int32_t>(t));
    return -1;
  }
  const int64_t page = slot >> p.page_shift;
  const int64_t in = slot & ((1 << p.page_shift) - 1);
  return ((((page * p.heads + h) << p.page_shift) + in) << p.bpr_shift) + b;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4CacheParams p) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.blocks; i += step) {
    float k[16], v[16];
    load16(static_cast<const T*>(p.k_rows), i, p.whole, k);
    load16(static_cast<const T*>(p.v_rows), i, p.whole, v);
    const int64_t dst = pool_block(p, i);
    if (dst < 0) continue;
    uint2 kc, vc;
    const uint32_t ks = kv4::encode_block(k, kc), vs = kv4::encode_block(v, vc);
    reinterpret_cast<uint2*>(p.k_pages)[dst] = kc;
    reinterpret_cast<uint2*>(p.v_pages)[dst] = vc;
    p.k_scales[dst] = static_cast<uint8_t>(ks);
    p.v_scales[dst] = static_cast<uint8_t>(vs);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4CacheParams p) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.blocks; i += step) {
    const int64_t src = pool_block(p, i);
    if (src < 0) continue;
    const uint2 kc = reinterpret_cast<const uint2*>(p.k_pages)[src];
    const uint2 vc = reinterpret_cast<const uint2*>(p.v_pages)[src];
    const uint32_t ks = p.k_scales[src], vs = p.v_scales[src];
    store16(static_cast<T*>(const_cast<void*>(p.k_rows)), i, p.whole, kc, ks);
    store16(static_cast<T*>(const_cast<void*>(p.v_rows)), i, p.whole, vc, vs);
  }
}

}  // namespace

int launch_kv4_cache(const Kv4CacheArgs& a, void* stream) {
  Kv4CacheParams p;
  p.k_rows = a.k_rows;
  p.v_rows = a.v_rows;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.whole = ((reinterpret_cast<uintptr_t>(a.k_rows) | reinterpret_cast<uintptr_t>(a.v_rows)) & 31) == 0;
  p.slot_map = a.slot_map;
  p.ws = a.workspace;
  p.heads = a.hkv;
  int shift = 0;
  while ((16 << shift) < a.head_dim) ++shift;
  p.bpr_shift = shift;
  p.blocks = (static_cast<int64_t>(a.tokens) * a.hkv) << shift;
  if (p.blocks == 0) return 0;
  p.by_heads = kv4::head_div(a.hkv);
  shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  p.page_shift = shift;
  p.pool_slots = static_cast<int64_t>(a.num_pages) << shift;
  const int grid = static_cast<int>(std::min<int64_t>((p.blocks + kThreads - 1) / kThreads, 152 * 64));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = a.elem_bytes == 4;
  if (a.read)
    f32 ? kv4_read_kernel<float><<<grid, kThreads, 0, s>>>(p)
        : kv4_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  else
    f32 ? kv4_write_kernel<float><<<grid, kThreads, 0, s>>>(p)
        : kv4_write_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  trace_mark(a.read ? RPA_KERNEL_KV4_READ : RPA_KERNEL_KV4_WRITE, stream);
  return 0;
}

}  // namespace rpa
