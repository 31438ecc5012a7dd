// Drafted trees beside their attention: masks and positions from the nodes'
// parents, and the rows of an accepted path moved together in the cache.
//
// build_tree: with depth(i) = 0 for a node that follows the context and
// depth(parent) + 1 otherwise, positions = C + depth, and bit j of row i says
// whether node j is i or an ancestor of it.  A request is one CTA: its parents go
// to shared memory, a thread walks from its node to the root.  Parents come
// before their children, so the walk meets the mask's words from the last to the
// first and keeps one at a time.
//
// commit_tree: row k of the path takes the K and V of node path[k] >= k.  A thread
// owns 16 bytes of the row and goes down the path, eight nodes read before eight
// are written: a later node's source lies behind every place written so far, so
// nothing is lost where source and destination rows overlap.
//
// Both move kilobytes: their time is a launch and a few dependent reads.
#include <algorithm>

#include "common.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = 64 * kTreeMaxWords;

struct BuildTreeParams {
  const int32_t* parents;
  const int32_t* cu;
  const int32_t* kv;
  const int32_t* window;
  unsigned long long* mask;
  int32_t* positions;
  unsigned char* ws;
  int32_t total_q, words;
};

__global__ void __launch_bounds__(kThreads) build_tree_kernel(const BuildTreeParams p) {
  __shared__ int16_t parent[kMaxNodes];
  const int32_t s = blockIdx.x;
  const int32_t q0 = __ldg(p.cu + s), q1 = __ldg(p.cu + s + 1), len = __ldg(p.kv + s);
  const int32_t w = p.window ? __ldg(p.window + s) : 0;
  // (In 64 bits: lengths that cannot be used may be anything.)
  const int64_t n64 = static_cast<int64_t>(q1) - q0;
  if (q0 < 0 || n64 < 0 || q1 > p.total_q || n64 > 64 * p.words || n64 > len) {
    if (threadIdx.x == 0 && p.ws) report_error(p.ws, RPA_DEVERR_LENGTHS, s);
    return;
  }
  const int32_t n = static_cast<int32_t>(n64);
  for (int32_t i = threadIdx.x; i < n; i += kThreads) {
    int32_t j = __ldg(p.parents + q0 + i);
    if (j < -1 || j >= i) {
      if (p.ws) report_error(p.ws, RPA_DEVERR_LENGTHS, s);
      j = -1;
    }
    parent[i] = static_cast<int16_t>(j);
  }
  __syncthreads();
  const int32_t most = w > 0 ? w : n;  // nodes of a path that its last one sees
  for (int32_t i = threadIdx.x; i < n; i += kThreads) {
    unsigned long long* row = p.mask + static_cast<int64_t>(q0 + i) * p.words;
    for (int32_t k = p.words - 1; k > i >> 6; --k) row[k] = 0;
    int32_t k = i >> 6, depth = 0;
    unsigned long long bits = 0;
    for (int32_t j = i;;) {
      if (depth < most) bits |= 1ull << (j & 63);
      j = parent[j];
      if (j < 0) break;
      ++depth;
      for (; k > j >> 6; --k) {
        row[k] = bits;
        bits = 0;
      }
    }
    row[k] = bits;
    while (--k >= 0) row[k] = 0;
    p.positions[q0 + i] = len - n + depth;
  }
}

constexpr int kMaxPath = 1024;
constexpr int kAtOnce = 8;

struct CommitTreeParams {
  uint4* k_pages;
  uint4* v_pages;
  const int64_t* slots;
  const int32_t* cu;
  const int32_t* path;
  unsigned char* ws;
  int64_t pool_slots;
  int32_t total_q, max_path, row16;  // row16: 16-byte pieces of a row
};

__global__ void __launch_bounds__(kThreads) commit_tree_kernel(const CommitTreeParams p) {
  __shared__ int64_t src[kMaxPath], dst[kMaxPath];
  __shared__ int32_t s_len, s_bad;
  const int32_t s = blockIdx.x;
  if (threadIdx.x == 0) {
    s_len = p.max_path;
    s_bad = 0;
  }
  __syncthreads();
  const int32_t q0 = __ldg(p.cu + s), q1 = __ldg(p.cu + s + 1);
  const bool usable = q0 >= 0 && q1 >= q0 && q1 <= p.total_q;
  const int32_t* path = p.path + static_cast<int64_t>(s) * p.max_path;
  for (int32_t k = threadIdx.x; k < p.max_path; k += kThreads) {
    const int32_t j = __ldg(path + k), before = k > 0 ? __ldg(path + k - 1) : -1;
    if (j < 0) {
      atomicMin(&s_len, k);
      continue;
    }
    // Increasing nodes from 0 on: path[k] >= k.
    int32_t bad = 0;
    if (!usable || j < k || j >= q1 - q0 || (k > 0 && before < 0) || j <= before) {
      bad = RPA_DEVERR_LENGTHS;
    } else {
      src[k] = __ldg(p.slots + q0 + j);
      dst[k] = __ldg(p.slots + q0 + k);
      if (src[k] < 0 || src[k] >= p.pool_slots || dst[k] < 0 || dst[k] >= p.pool_slots) bad = RPA_DEVERR_PAGE_ID;
    }
    if (bad) atomicMax(&s_bad, bad);
  }
  __syncthreads();
  if (s_bad) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && p.ws) report_error(p.ws, s_bad, s);
    return;
  }
  const int32_t n = s_len;
  // Pieces of a K row, then of a V row.
  for (int32_t c = blockIdx.y * kThreads + threadIdx.x; c < 2 * p.row16; c += gridDim.y * kThreads) {
    uint4* pool = c < p.row16 ? p.k_pages : p.v_pages;
    const int32_t at = c < p.row16 ? c : c - p.row16;
    for (int32_t k0 = 0; k0 < n; k0 += kAtOnce) {
      uint4 r[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (k0 + i < n && src[k0 + i] != dst[k0 + i]) r[i] = pool[src[k0 + i] * p.row16 + at];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (k0 + i < n && src[k0 + i] != dst[k0 + i]) pool[dst[k0 + i] * p.row16 + at] = r[i];
    }
  }
}

}  // namespace

int launch_build_tree(const BuildTreeArgs& a, void* stream) {
  if (a.num_seqs == 0) return 0;
  const BuildTreeParams p{a.parents, a.cu_q_lens, a.kv_lens, a.window,
                          reinterpret_cast<unsigned long long*>(a.mask), a.positions, a.workspace,
                          a.total_q, a.words};
  build_tree_kernel<<<a.num_seqs, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  if (cudaError_t e = cudaGetLastError()) return static_cast<int>(e);
  trace_mark(RPA_KERNEL_BUILD_TREE, stream);
  return 0;
}

int launch_commit_tree(const CommitTreeArgs& a, void* stream) {
  if (a.num_seqs == 0 || a.max_path == 0) return 0;
  const int32_t row16 = static_cast<int32_t>(a.row_bytes / 16);
  const CommitTreeParams p{static_cast<uint4*>(a.k_pages), static_cast<uint4*>(a.v_pages), a.slot_map,
                           a.cu_q_lens, a.path, a.workspace, a.pool_slots, a.total_q, a.max_path, row16};
  // A CTA per request and 128 pieces of its rows.
  const dim3 grid(a.num_seqs, std::min((2 * static_cast<int64_t>(row16) + kThreads - 1) / kThreads, int64_t{256}));
  commit_tree_kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  if (cudaError_t e = cudaGetLastError()) return static_cast<int>(e);
  trace_mark(RPA_KERNEL_COMMIT_TREE, stream);
  return 0;
}

}  // namespace rpa
