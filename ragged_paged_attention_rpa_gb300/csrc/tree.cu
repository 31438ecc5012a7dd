// Drafted trees beside their attention: masks and positions from the nodes'
// parents, and the rows of an accepted path moved together in the cache.
//
// build_tree: with depth(i) = 0 for a node that follows the context and
// depth(parent) + 1 otherwise, positions = C + depth, and bit j of row i says
// whether node j is i or an ancestor of it.  A request is one CTA.  Parents come first, so
// its warps take 32 nodes each and find the ancestors among these by doubling (five rounds
// of shuffles), and the first ancestor before them; then the 32s' rows in turn: a row is
// that ancestor's, with those among the 32 set.  The path's nodes have rising numbers, so
// a window's are a row's highest bits.  64 requests of up to 256 nodes take 5.4 us (7.1 with
// one warp that did both for 32 nodes after 32; 41 where a thread walked from its node to
// the root and chains were among them), 128 requests of 8 nodes 2.2.
//
// commit_tree: row k of the path takes the K and V of node path[k] >= k.  A thread
// owns 16 bytes of the row and goes down the path, eight nodes read before eight
// are written: a later node's source lies behind every place written so far, so
// nothing is lost where source and destination rows overlap.  A row is read once and
// written once; the path, its slots and the rows are three dependent reads.  128 paths of
// up to 4 rows of 512 bytes: 2.4 us; 64 of up to 16 rows of 8 KB: 7.2 us (14.7 MB, 2.0 TB/s;
// with the path's eights on threads of their own, all read before one writes, 5% less, and
// 3% more for the small one).
#include <algorithm>

#include "common.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kThreads = 128;
constexpr uint32_t kAll = 0xffffffffu;

struct BuildTreeParams {
  const int32_t* parents;
  const int32_t* cu;
  const int32_t* kv;
  const int32_t* window;
  uint32_t* mask;
  int32_t* positions;
  unsigned char* ws;
  int32_t total_q, words;  // words of 32 bits
};

// Clears the lowest `n` set bits of w, and takes them off n.
__device__ __forceinline__ uint32_t drop_lowest(uint32_t w, int32_t& n) {
  const int32_t c = __popc(w);
  if (n >= c) {
    n -= c;
    return 0;
  }
  for (; n > 0; --n) w &= w - 1;
  return w;
}

__global__ void __launch_bounds__(kThreads) build_tree_kernel(const BuildTreeParams p) {
  extern __shared__ uint32_t smem[];
  const int32_t s = blockIdx.x, lane = threadIdx.x & 31;
  const int32_t q0 = __ldg(p.cu + s), q1 = __ldg(p.cu + s + 1), len = __ldg(p.kv + s);
  const int32_t w = p.window ? __ldg(p.window + s) : 0;
  // (In 64 bits: lengths that cannot be used may be anything.)
  const int64_t n64 = static_cast<int64_t>(q1) - q0;
  if (q0 < 0 || n64 < 0 || q1 > p.total_q || n64 > 32 * p.words || n64 > len) {
    if (threadIdx.x == 0 && p.ws) report_error(p.ws, RPA_DEVERR_LENGTHS, s);
    return;
  }
  const int32_t n = static_cast<int32_t>(n64), W = p.words;
  // Rows [node][W + 1] (the odd length keeps 32 rows' words in different banks), parents,
  // which become each node's first ancestor before its 32, and depths.
  uint32_t* rows = smem;
  int32_t* ups = reinterpret_cast<int32_t*>(smem + 32 * W * (W + 1));
  int32_t* depths = ups + 32 * W;
  for (int32_t i0 = threadIdx.x & ~31; i0 < n; i0 += kThreads) {
    const int32_t i = i0 + lane;
    int32_t up = i < n ? __ldg(p.parents + q0 + i) : -1;
    if (up < -1 || up >= i) {
      if (p.ws) report_error(p.ws, RPA_DEVERR_LENGTHS, s);
      up = -1;
    }
    // Ancestors among the 32 (and the node): after k rounds those within 2^k steps.
    uint32_t mine = 1u << lane;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const bool within = up >= i0;
      if (!__any_sync(kAll, within)) break;
      const int from = within ? up - i0 : lane;
      const uint32_t theirs = __shfl_sync(kAll, mine, from);
      const int32_t further = __shfl_sync(kAll, up, from);
      if (within) {
        mine |= theirs;
        up = further;
      }
    }
    if (i < n) {
      rows[i * (W + 1) + (i0 >> 5)] = mine;
      ups[i] = up;
      depths[i] = __popc(mine) - 1;  // among the 32
    }
  }
  __syncthreads();
  // The words before the 32's own, and the depths, from that ancestor.
  for (int32_t i0 = 32; i0 < n; i0 += 32) {
    const int32_t i = i0 + lane;
    if (i < n) {
      const int32_t up = ups[i];
      for (int32_t k = threadIdx.x >> 5; k < i0 >> 5; k += kThreads / 32)
        rows[i * (W + 1) + k] = k <= up >> 5 ? rows[up * (W + 1) + k] : 0u;
      if (threadIdx.x < 32 && up >= 0) depths[i] += depths[up] + 1;
    }
    __syncthreads();
  }
  for (int32_t i = threadIdx.x; i < n; i += kThreads) p.positions[q0 + i] = len - n + depths[i];
  uint32_t* out = p.mask + static_cast<int64_t>(q0) * W;
  if (w <= 0) {
    for (int32_t u = threadIdx.x; u < n * W; u += kThreads) {
      const int32_t i = u / W, k = u - i * W;
      out[u] = k <= i >> 5 ? rows[i * (W + 1) + k] : 0u;
    }
    return;
  }
  for (int32_t i = threadIdx.x; i < n; i += kThreads) {
    int32_t drop = max(0, depths[i] + 1 - w);  // nodes of the path that lie too far back
    for (int32_t k = 0; k < W; ++k) {
      const uint32_t bits = k <= i >> 5 ? rows[i * (W + 1) + k] : 0u;
      out[i * W + k] = drop > 0 ? drop_lowest(bits, drop) : bits;
    }
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
  // (An empty path has not looked at the lengths.  Asked ahead of the copies it costs 4% of a long path.)
  if (n == 0 && !usable && threadIdx.x == 0 && blockIdx.y == 0 && p.ws) report_error(p.ws, RPA_DEVERR_LENGTHS, s);
}

}  // namespace

int launch_build_tree(const BuildTreeArgs& a, void* stream) {
  if (a.num_seqs == 0) return 0;
  const int32_t W = 2 * a.words;
  const BuildTreeParams p{a.parents, a.cu_q_lens, a.kv_lens, a.window, reinterpret_cast<uint32_t*>(a.mask),
                          a.positions, a.workspace, a.total_q, W};
  const int bytes = 32 * W * (W + 3) * static_cast<int>(sizeof(uint32_t));
  const int most = 64 * kTreeMaxWords * (2 * kTreeMaxWords + 3) * static_cast<int>(sizeof(uint32_t));
  if (bytes > 48 * 1024)
    if (int e = ensure_dynamic_smem(reinterpret_cast<const void*>(build_tree_kernel), most)) return e;
  build_tree_kernel<<<a.num_seqs, kThreads, bytes, static_cast<cudaStream_t>(stream)>>>(p);
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
