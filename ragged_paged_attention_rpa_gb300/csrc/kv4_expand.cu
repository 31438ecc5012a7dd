// 4-bit pages widened to bf16 for the tensor-core prefill.
//
// A prompt's keys are used by every query block: widening them in the prefill
// kernel would convert each key once per block (128 x D codes per 128-key tile
// against 128 x 128 exponentials: at D = 256 more work than the softmax).  So
// the keys the sequences' queries see are widened once, to scratch pages in
// the workspace ([page][slot][head][dim], the bf16 pool's layout) with a page
// table of their own, and the prefill runs on those.  The values are exact in
// bf16 (six significant bits).  A block of V that reads as NaN becomes zeros (in
// the product it would reach the rows that do not see its key, 0 times NaN) and
// sets a word of the header, on which the prefill's epilogue looks the scales up
// for each row.  The prefill takes maxima of the products before it scales them,
// which wants a positive logit scale: for a negative one K's signs are turned.
//
// One thread per 16 dimensions of K and of V; HBM-bound: 0.5625 bytes an
// element read, 2 written (and the prefill reads them back from L2 or HBM).  A
// prompt's 8192 keys of 16 heads of 256 (172 MB) take 27.7 us, 6.2 TB/s.
#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kThreads = 256;

struct ExpandList {
  int32_t n, page_end;  // sequences; one past the last scratch page
  Plan::Kv4Expand s[kKv4ExpandSeqs];
};

struct ExpandParams {
  const uint2* k;
  const uint2* v;
  const uint8_t* ks;
  const uint8_t* vs;
  uint4* k_out;
  uint4* v_out;
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  int32_t* table_out;
  unsigned char* ws;
  uint32_t k_signs;  // turned in K's codes
  int32_t hkv, bpr_shift, page_shift, mpps, num_pages;
  kv4::HeadDiv by_heads;
};

__global__ void __launch_bounds__(kThreads)
kv4_expand_kernel(const ExpandParams p, const __grid_constant__ ExpandList list) {
  const int32_t first = list.s[0].page0;
  // Rows (key, head) of the scratch pages: below 2^31, since 2^31 of them would
  // be 512 GB of bf16 K and V.
  const int64_t rows = (static_cast<int64_t>(list.page_end - first) << p.page_shift) * p.hkv;
  const int64_t row0 = (static_cast<int64_t>(first) << p.page_shift) * p.hkv;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  bool v_nan = false;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < rows << p.bpr_shift; i += step) {
    const uint32_t row = static_cast<uint32_t>(i >> p.bpr_shift);
    const int32_t b = static_cast<int32_t>(i) & ((1 << p.bpr_shift) - 1);
    const uint32_t key_row = p.by_heads(row);
    const int32_t h = static_cast<int32_t>(row - key_row * p.hkv);
    const int32_t scratch = first + static_cast<int32_t>(key_row >> p.page_shift);
    const int32_t in = static_cast<int32_t>(key_row) & ((1 << p.page_shift) - 1);
    int lo = 0, hi = list.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (list.s[mid].page0 <= scratch) lo = mid; else hi = mid - 1;
    }
    const Plan::Kv4Expand& e = list.s[lo];
    const int32_t slot = e.slot0 + (scratch - e.page0);
    const int64_t at = static_cast<int64_t>(e.seq) * p.mpps + slot;
    const int32_t page = __ldg(p.page_table + at);
    const bool ok = page >= 0 && page < p.num_pages;
    if (in == 0 && h == 0 && b == 0) {
      p.table_out[at] = ok ? scratch : -1;
      if (!ok) report_error(p.ws, RPA_DEVERR_PAGE_ID, e.seq);
      // (What is widened goes by the plan's lengths, the prefill by the device's.)
      if (scratch == e.page0) {
        const int32_t q0 = p.cu_q_lens[e.seq], q1 = p.cu_q_lens[e.seq + 1];
        if (q0 != e.q0 || q1 - q0 != e.q_len || p.kv_lens[e.seq] != e.hi) report_error(p.ws, RPA_DEVERR_LENGTHS, e.seq);
      }
    }
    const int32_t key = (slot << p.page_shift) + in;
    if (!ok || key < e.lo || key >= e.hi) continue;
    const int64_t src = ((((static_cast<int64_t>(page) * p.hkv + h) << p.page_shift) + in) << p.bpr_shift) + b;
    const int64_t dst = 2 * ((row0 << p.bpr_shift) + i);
    const uint2 kc = __ldg(p.k + src), vc = __ldg(p.v + src);
    const uint32_t ks = __ldg(p.ks + src), vs = __ldg(p.vs + src);
    v_nan |= vs == 255u;
    uint32_t w[8];  // the workspace's arrays are 256-byte aligned
    kv4::decode_block_bf16(make_uint2(kc.x ^ p.k_signs, kc.y ^ p.k_signs), ks, w);
    kv4::store32(p.k_out + dst, true, w);
    kv4::decode_block_bf16(vc, vs == 255u ? 0u : vs, w);
    kv4::store32(p.v_out + dst, true, w);
  }
  if (v_nan) *reinterpret_cast<int32_t*>(p.ws + kKv4NanOff) = 1;
}

}  // namespace

int launch_kv4_expand(const Plan& plan, const Args& a, void* stream) {
  ExpandParams p;
  p.k = static_cast<const uint2*>(a.k_pages);
  p.v = static_cast<const uint2*>(a.v_pages);
  p.ks = a.k_block_scales;
  p.vs = a.v_block_scales;
  p.k_out = reinterpret_cast<uint4*>(a.workspace + plan.off_kv4_k);
  p.v_out = reinterpret_cast<uint4*>(a.workspace + plan.off_kv4_v);
  p.page_table = a.page_table;
  p.cu_q_lens = a.cu_q_lens;
  p.kv_lens = a.kv_lens;
  p.table_out = reinterpret_cast<int32_t*>(a.workspace + plan.off_kv4_table);
  p.ws = a.workspace;
  p.k_signs = a.sm_scale < 0.f ? 0x88888888u : 0u;
  p.hkv = plan.hkv;
  p.by_heads = kv4::head_div(plan.hkv);
  int shift = 0;
  while ((16 << shift) < plan.d) ++shift;
  p.bpr_shift = shift;
  shift = 0;
  while ((1 << shift) < plan.p) ++shift;
  p.page_shift = shift;
  p.mpps = plan.mpps;
  p.num_pages = plan.num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ExpandList& list = thread_staging<ExpandList>();  // copied into the launch parameters
  const size_t n = plan.kv4_expand.size();
  for (size_t off = 0; off < n; off += kKv4ExpandSeqs) {
    list.n = static_cast<int32_t>(std::min<size_t>(kKv4ExpandSeqs, n - off));
    for (int i = 0; i < list.n; ++i) list.s[i] = plan.kv4_expand[off + i];
    list.page_end = off + list.n < n ? plan.kv4_expand[off + list.n].page0 : plan.kv4_scratch_pages;
    const int64_t blocks = (static_cast<int64_t>(list.page_end - list.s[0].page0) << p.page_shift) * p.hkv
                           << p.bpr_shift;
    const int grid = static_cast<int>(std::min<int64_t>((blocks + kThreads - 1) / kThreads, plan.num_sms * 64));
    kv4_expand_kernel<<<grid, kThreads, 0, s>>>(p, list);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return static_cast<int>(e);
    trace_mark(RPA_KERNEL_KV4_EXPAND, stream);
  }
  return 0;
}

}  // namespace rpa
