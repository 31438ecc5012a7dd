// Attention of drafted trees on CUDA cores: the fp32 debug build, and shapes that
// the tensor-core kernel does not take.  fp32 throughout.
//
// One CTA per (node, query head); its warps take the keys by turns of 32, look up
// which of them the node sees and fold in one after the other: a lane holds D / 32
// dimensions, the score is a sum over the warp, the running maximum, sum and output
// stay in registers.  The warps' states merge in shared memory at the end.  Not
// tuned: every node reads its keys for itself (6 nodes of 4 heads of 64 after 700 keys: 53
// us, 8.3 on tensor cores).
#include "tree.cuh"

namespace rpa {
namespace {

constexpr int kWarps = 8;

struct TreeSimtParams {
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  const uint64_t* mask;
  const int32_t* positions;
  unsigned char* ws;
  int32_t hq, hkv, page_size, page_shift, mpps, num_pages, words;
  float scale_log2;
};

template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarps)
tree_simt_kernel(const T* q, const T* k_pages, const T* v_pages, T* out, const TreeSimtParams p,
                 const __grid_constant__ TreeSeqs<kTreeSeqsLarge> seqs) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t t = seqs.s[0].q0 + static_cast<int32_t>(blockIdx.x), h = blockIdx.y;
  int lo_s = 0, hi_s = seqs.n - 1;
  while (lo_s < hi_s) {
    const int mid = (lo_s + hi_s + 1) >> 1;
    if (seqs.s[mid].q0 <= t) lo_s = mid; else hi_s = mid - 1;
  }
  const TreeSeq s = seqs.s[lo_s];
  if (threadIdx.x == 0 && h == 0 && t == s.q0) tree_check_lengths(s, p.cu_q_lens, p.kv_lens, p.ws);
  const int32_t g = h / (p.hq / p.hkv);
  const int32_t first = tree_first_key(s, p.positions, t, p.ws);
  const uint64_t* row = p.mask + static_cast<int64_t>(t) * p.words;
  const int32_t* table = p.page_table + static_cast<int64_t>(s.seq) * p.mpps;
  float x[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = to_float(q[(static_cast<int64_t>(t) * p.hq + h) * D + 32 * e + lane]);
    o[e] = 0.f;
  }
  // From the window's first key or the first node, whichever is earlier: the window bounds the
  // context alone.
  for (int32_t k0 = (min(first, s.len - s.nodes) & ~31) + 32 * warp; k0 < s.len; k0 += 32 * kWarps) {
    for (uint32_t bits = tree_sees32(s, row, first, k0); bits; bits &= bits - 1) {
      const int32_t key = k0 + __ffs(bits) - 1;
      const int32_t page = __ldg(table + (key >> p.page_shift));
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) report_error(p.ws, RPA_DEVERR_PAGE_ID, s.seq);
        continue;
      }
      const int64_t at =
          ((static_cast<int64_t>(page) * p.page_size + (key & (p.page_size - 1))) * p.hkv + g) * D + lane;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(x[e], to_float(k_pages[at + 32 * e]), dot);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      const float sc = dot * p.scale_log2;
      const float m_new = fmaxf(m, sc);
      // (A score of -inf weighs nothing; a NaN goes on.)
      const float f = m == m_new ? 1.f : fast_exp2(m - m_new), w = sc == -INFINITY ? 0.f : fast_exp2(sc - m_new);
      l = fmaf(l, f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, to_float(v_pages[at + 32 * e]), o[e] * f);
      m = m_new;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][32 * e + lane] = o[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (s_l[w] == 0.f) continue;
      const float f = s_m[w] == top ? 1.f : fast_exp2(s_m[w] - top);
      sum = fmaf(f, s_l[w], sum);
      acc = fmaf(f, s_o[w][d], acc);
    }
    out[(static_cast<int64_t>(t) * p.hq + h) * D + d] = from_float<T>(sum == 0.f ? 0.f : acc / sum);
  }
}

template <int D, typename T>
int launch_t(const Plan& plan, const Args& a, cudaStream_t stream) {
  TreeSimtParams p{a.page_table, a.cu_q_lens, a.kv_lens, a.tree_mask, a.positions, a.workspace,
                   plan.hq, plan.hkv, plan.p, 0, plan.mpps, plan.num_pages, plan.tree_words,
                   a.sm_scale * 1.4426950408889634f};
  while ((1 << p.page_shift) < plan.p) ++p.page_shift;
  auto& list = thread_staging<TreeSeqs<kTreeSeqsLarge>>();
  for (const TreeLaunch& l : plan.tree_launches) {
    list.n = l.seq_end - l.seq_begin;
    int64_t nodes = 0;
    for (int32_t i = 0; i < list.n; ++i) {
      list.s[i] = plan.tree_seqs[l.seq_begin + i];
      nodes += list.s[i].nodes;
    }
    tree_simt_kernel<D, T><<<dim3(static_cast<unsigned>(nodes), plan.hq), 32 * kWarps, 0, stream>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k_pages), static_cast<const T*>(a.v_pages),
        static_cast<T*>(a.out), p, list);
    if (cudaError_t e = cudaGetLastError()) return static_cast<int>(e);
    trace_mark(RPA_KERNEL_TREE_ATTN, stream);
  }
  return 0;
}

}  // namespace

int launch_tree_simt(const Plan& plan, const Args& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = plan.dtype == RPA_DTYPE_F32;
  switch (plan.d) {
    case 64: return f32 ? launch_t<64, float>(plan, a, s) : launch_t<64, __nv_bfloat16>(plan, a, s);
    case 128: return f32 ? launch_t<128, float>(plan, a, s) : launch_t<128, __nv_bfloat16>(plan, a, s);
    case 256: return f32 ? launch_t<256, float>(plan, a, s) : launch_t<256, __nv_bfloat16>(plan, a, s);
    default: return static_cast<int>(cudaErrorInvalidValue);
  }
}

}  // namespace rpa
