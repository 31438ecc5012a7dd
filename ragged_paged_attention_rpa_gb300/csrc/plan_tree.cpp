// The scheduler for drafted trees (rpa_plan_options.tree_words).  Host only.
//
// On tensor cores a request's nodes are row tiles of 128 / G nodes by G heads, and
// a segment is (request, KV head, one or two row tiles) over the 128-key tiles its
// nodes can see.  The segments' key tiles, each segment's followed by a charge for
// its ends, form one line, which is cut into equal ranges, one per CTA.
#include <algorithm>
#include <cstdint>
#include <vector>

#include "rpa_internal.h"

namespace rpa {
namespace {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The line is counted in quarters of a key tile: what a segment's queries, first tile
// and output cost, and the fewest worth a CTA of its own.
constexpr int32_t kTile = 4;
constexpr int32_t kSegCost = 6;
constexpr int32_t kLeast = 4;

rpa_status_t cut_line(Plan& plan, TreeLaunch& l) {
  const int32_t per = kTreeRows / (plan.hq / plan.hkv) * tree_row_tiles(plan.d);  // nodes of a segment
  const int32_t n_seq = l.seq_end - l.seq_begin;
  auto seq = [&](int32_t i) -> const TreeSeq& { return plan.tree_seqs[l.seq_begin + i]; };
  auto tiles = [&](int32_t i) { return (seq(i).len - 1) / kTreeKeys + 1 - tree_first_tile(seq(i)); };
  auto segments = [&](int32_t i) { return ceil_div(seq(i).nodes, per); };  // of a head
  std::vector<int64_t> v0(1, 0);  // the requests' starts on the line
  for (int32_t i = 0; i < n_seq; ++i)
    v0.push_back(v0.back() + (static_cast<int64_t>(tiles(i)) * kTile + kSegCost) * segments(i) * plan.hkv);
  const int64_t total = v0.back();
  const int64_t most = std::min<int64_t>(plan.num_sms, kTreeMaxCtas);
  const int64_t n = std::max<int64_t>(1, std::min(most, total / kLeast));
  // (A range's tiles travel in 31 bits.)
  if (ceil_div(total, n) > 0x3fffffff) return RPA_ERR_UNSUPPORTED;
  l.start_begin = static_cast<int32_t>(plan.tree_starts.size());
  l.n_ctas = static_cast<int32_t>(n);
  l.cut_begin = static_cast<int32_t>(plan.tree_cuts.size());
  int32_t i = 0;
  int64_t done = 0;  // tiles before the current range, charges left out
  std::vector<int64_t> before(1, 0);
  for (int32_t k = 0; k < n_seq; ++k) before.push_back(before.back() + tiles(k) * segments(k) * plan.hkv);
  for (int64_t c = 0; c <= n; ++c) {
    const int64_t x = total * c / n;
    while (i < n_seq && v0[i + 1] <= x) ++i;
    // The boundary as a tile: one inside a charge is the segment's end.
    TreeStart st{i, 0, 0, 0, 0};
    int64_t at = before[i];
    bool inside = false;
    if (i < n_seq) {
      const int64_t cost = static_cast<int64_t>(tiles(i)) * kTile + kSegCost, off = (x - v0[i]) % cost / kTile;
      int64_t sg = (x - v0[i]) / cost;
      at += sg * tiles(i) + std::min<int64_t>(off, tiles(i));
      inside = off > 0 && off < tiles(i);
      if (off >= tiles(i)) ++sg;  // the next segment's first tile
      const int64_t per_head = segments(i);
      if (sg == per_head * plan.hkv) {
        st.i = i + 1;
      } else {
        st.head = static_cast<int32_t>(sg / per_head);
        st.st = static_cast<int32_t>(sg % per_head);
        st.j = inside ? static_cast<int32_t>(off) : 0;
      }
    }
    if (c > 0) plan.tree_starts.back().tiles = static_cast<int32_t>(at - done);
    done = at;
    if (c == n) break;
    plan.tree_starts.push_back(st);
    if (!inside) continue;
    // The segment is cut here: between this CTA and the one before it.
    TreeCut* last = l.n_cut > 0 ? &plan.tree_cuts.back() : nullptr;
    if (last && last->i == st.i && last->head == st.head && last->st == st.st) {
      ++last->nparts;
    } else {
      const TreeStart& prev = plan.tree_starts[plan.tree_starts.size() - 2];
      const int32_t first = prev.i == st.i && prev.head == st.head && prev.st == st.st ? 0 : 1;
      plan.tree_cuts.push_back({st.i, st.head, st.st, static_cast<int32_t>(c - 1), first, 2});
      ++l.n_cut;
    }
  }
  for (int32_t k = 0; k < l.n_cut; ++k)
    plan.max_splits = std::max(plan.max_splits, plan.tree_cuts[l.cut_begin + k].nparts);
  plan.max_splits = std::max(plan.max_splits, 1);
  plan.kv_split = std::max(plan.kv_split, static_cast<int32_t>(std::min<int64_t>(
                                              ceil_div(total, n * kTile) * kTreeKeys, 0x7fffffff)));
  plan.decode_ctas += n;
  plan.tree_slots = std::max(plan.tree_slots, static_cast<int32_t>(2 * n));
  return RPA_OK;
}

}  // namespace

rpa_status_t build_tree_schedule(Plan& plan, const int32_t* cu, const int32_t* kv, const int32_t* win,
                                 const rpa_plan_options& opts) {
  const int32_t group = plan.hq / plan.hkv;
  if (opts.path != RPA_PATH_AUTO && opts.path != RPA_PATH_SIMT && opts.path != RPA_PATH_TC)
    return RPA_ERR_INVALID_ARG;
  if ((opts.kv_dtype != 0 && opts.kv_dtype != plan.dtype) || opts.q_block != 0 || opts.kv_split != 0 ||
      opts.prefill_pairs != 0 || opts.prefill_split != 0 || opts.decode_sms != 0 || opts.decode_kernel != 0 ||
      opts.prefill_dynamic != 0 || opts.prefill_grouping != 0)
    return RPA_ERR_UNSUPPORTED;
  // (A row of the pool is a 31-bit coordinate of its tensor map.)
  const bool tc = plan.dtype == RPA_DTYPE_BF16 && tree_tc_supported(plan.d, plan.p, group) &&
                  static_cast<int64_t>(plan.num_pages) * plan.p <= 0x7fffffff;
  if (opts.path == RPA_PATH_TC && !tc) return RPA_ERR_UNSUPPORTED;
  if (plan.hq > 65535) return RPA_ERR_UNSUPPORTED;  // (the CUDA-core grid's second side)
  plan.tree_words = opts.tree_words;
  plan.path = tc && opts.path != RPA_PATH_SIMT ? RPA_PATH_TC : RPA_PATH_SIMT;
  for (int32_t s = 0; s < plan.num_seqs; ++s) {
    const int32_t n = cu[s + 1] - cu[s];
    if (n > 64 * opts.tree_words) return RPA_ERR_INVALID_ARG;
    if (n > 0) plan.tree_seqs.push_back({s, cu[s], n, kv[s], win ? std::max(win[s], 0) : 0});
  }
  const int32_t total = static_cast<int32_t>(plan.tree_seqs.size());
  plan.num_decode = total;
  for (int32_t i = 0; i < total; i += kTreeSeqsLarge) {
    TreeLaunch l{i, std::min(total, i + kTreeSeqsLarge), 0, 0, 0, 0};
    if (plan.path == RPA_PATH_TC)
      if (rpa_status_t st = cut_line(plan, l)) return st;
    plan.tree_launches.push_back(l);
  }
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  if (!plan.tree_cuts.empty()) {
    const size_t rows = static_cast<size_t>(plan.tree_slots) * kTreeRows * tree_row_tiles(plan.d);
    plan.off_partial_o = take(rows * plan.d * sizeof(float));
    plan.off_partial_lse = take(rows * sizeof(float));
  }
  plan.ws_bytes = off;
  return RPA_OK;
}

}  // namespace rpa
