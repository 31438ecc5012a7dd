// What the kernels of drafted trees share: a request's list entries, and which
// keys a node sees.
//
// Node i of a request with context C and `nodes` nodes sees key j < C iff pos - j < W
// (or W = 0), and key C + j iff bit j of its mask row is set.
#pragma once

#include "common.cuh"
#include "rpa_internal.h"

namespace rpa {

// A launch's requests (in order of their first nodes).
template <int N>
struct TreeSeqs {
  int32_t n;
  TreeSeq s[N];
};

// Device lengths against the plan's (the plan's are used).
__device__ __forceinline__ void tree_check_lengths(const TreeSeq& s, const int32_t* cu, const int32_t* kv,
                                                   unsigned char* ws) {
  if (__ldg(cu + s.seq) != s.q0 || __ldg(cu + s.seq + 1) != s.q0 + s.nodes || __ldg(kv + s.seq) != s.len)
    report_error(ws, RPA_DEVERR_LENGTHS, s.seq);
}

// First context key that node t sees under the request's window; the position is
// held to the request's.
__device__ __forceinline__ int32_t tree_first_key(const TreeSeq& s, const int32_t* positions, int32_t t,
                                                  unsigned char* ws) {
  if (s.window <= 0) return 0;
  const int32_t pos = __ldg(positions + t), ctx = s.len - s.nodes;
  if (pos < ctx || pos >= s.len) report_error(ws, RPA_DEVERR_LENGTHS, s.seq);
  return max(0, min(max(pos, ctx), s.len - 1) - s.window + 1);
}

// Bits [a, b) of 32, each limit clamped to [0, 32].
__device__ __forceinline__ uint32_t bit_range(int32_t a, int32_t b) {
  a = max(0, min(32, a));
  b = max(0, min(32, b));
  const uint32_t below_b = b == 32 ? ~0u : (1u << b) - 1u, below_a = a == 32 ? ~0u : (1u << a) - 1u;
  return below_b & ~below_a;
}

// Which of keys [key, key + 32) a node sees whose first visible context key is `lo`.
// `row`: its mask words.
__device__ __forceinline__ uint32_t tree_sees32(const TreeSeq& s, const uint64_t* row, int32_t lo, int32_t key) {
  const int32_t ctx = s.len - s.nodes;
  uint32_t bits = bit_range(lo - key, ctx - key);
  const int32_t off = key - ctx;  // node of the first key
  if (off > -32 && off < s.nodes) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
    const int32_t i = off >> 5, last = (s.nodes - 1) >> 5;  // (rounds down)
    const uint32_t low = i >= 0 ? __ldg(w + i) : 0u, high = i < last ? __ldg(w + i + 1) : 0u;
    bits |= __funnelshift_r(low, high, off & 31) & bit_range(0, s.nodes - off);
  }
  return bits;
}

}  // namespace rpa
