// The scheduler for drafted trees (rpa_plan_options.tree_words).  Host only.
//
// On tensor cores a request's nodes are row tiles of 128 / G nodes by G heads, and
// a segment is (request, KV head, one or two row tiles) over the 128-key tiles its
// nodes can see.  A request's segments run in passes of `width` segments side by side.
// The passes' key tiles, each pass followed by a charge for its ends, form one line,
// which is cut into equal ranges, one per group of `width` CTAs (or between passes, where
// that costs less than joining their parts): the CTAs of a group read the same keys of a
// head at the same time, so that all but one find them in L2.
#include <algorithm>
#include <cstdint>
#include <numeric>
#include <vector>

#include "rpa_internal.h"

namespace rpa {
namespace {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The line is counted in quarters of a key tile: what a segment's queries, first tile
// and output cost (0 to 12 are within 2% of each other on 128 requests of 8 nodes), and the
// fewest worth a CTA of its own (6 nodes after 700 keys take 8.1 us with 4, 9.0 with 6, 9.3
// with 8, 10.5 with 12, 12.9 with 24).
constexpr int32_t kTile = 4;
constexpr int32_t kSegCost = 6;
constexpr int32_t kLeast = 4;

// What the kernel that joins the parts of segments costs, and its launch: 5 us, about 4 tiles.
// (17 requests of 65 to 195 nodes after up to 150 keys, 16 heads a KV head: 31.6 us cut, 23.8 in
// whole passes; 83 of 2 to 8 nodes under a window of 371: 72 and 56.)
constexpr int32_t kCombine = 16;
// What a key tile that no other CTA reads at the same time costs on top: 64 heads over 40000
// keys of 8 KV heads run at 1391 TFLOP/s with their row tiles one after the other, at 1634
// side by side, where only one CTA in 8 reads HBM; 8 requests of 256 nodes take 239 and 215 us.
constexpr double kAlone = 0.27;
constexpr int32_t kMaxWidth = 32;

rpa_status_t cut_line(Plan& plan, TreeLaunch& l) {
  const int32_t per = kTreeRows / (plan.hq / plan.hkv) * tree_row_tiles(plan.d);  // nodes of a segment
  const int32_t n_seq = l.seq_end - l.seq_begin;
  auto seq = [&](int32_t i) -> const TreeSeq& { return plan.tree_seqs[l.seq_begin + i]; };
  auto tiles = [&](int32_t i) { return (seq(i).len - 1) / kTreeKeys + 1 - tree_first_tile(seq(i)); };
  auto per_head = [&](int32_t i) -> int64_t { return seq(i).per_head; };
  auto segments = [&](int32_t i) { return per_head(i) * plan.hkv; };
  auto cost = [&](int32_t i) { return static_cast<int64_t>(tiles(i)) * kTile + kSegCost; };
  // Requests by their segments of a head: what a pass of each costs, and its tiles.
  struct Kind {
    int64_t cost = 0, tiles = 0;
  };
  std::vector<Kind> kinds(2);
  int64_t work = 0;
  for (int32_t i = 0; i < n_seq; ++i) {
    const int64_t s = ceil_div(seq(i).nodes, per);
    plan.tree_seqs[l.seq_begin + i].per_head = static_cast<uint16_t>(s);
    if (static_cast<int64_t>(kinds.size()) <= s) kinds.resize(s + 1);
    kinds[s].cost += cost(i);
    kinds[s].tiles += tiles(i);
    work += cost(i) * segments(i);
  }
  const int64_t most_heads = static_cast<int64_t>(kinds.size()) - 1;
  const int64_t most = std::min<int64_t>(plan.num_sms, kTreeMaxCtas);
  const int64_t ctas = std::max<int64_t>(1, std::min(most, work / kLeast));
  // The width of least time: the longest lane's tiles, each a little more where its keys
  // are read by it alone.
  int64_t width = 1;
  double least = 0;
  for (int64_t w = 1; w <= std::min<int64_t>({kMaxWidth, ctas, most_heads > 1 ? kMaxWidth : 1}); ++w) {
    int64_t line = 0, reads = 0, all = 0;
    for (int64_t s = 1; s <= most_heads; ++s) {
      if (kinds[s].tiles == 0) continue;
      const int64_t passes = ceil_div(s * plan.hkv, w), step = s / std::gcd(s, w);
      line += passes * kinds[s].cost;
      // Heads that the passes read: one more for each pass that begins inside a head.
      reads += (plan.hkv + passes - 1 - (passes - 1) / step) * kinds[s].tiles;
      all += s * plan.hkv * kinds[s].tiles;
    }
    const double t = static_cast<double>(line) / static_cast<double>(ctas / w) * (1 + kAlone * reads / all);
    if (w > 1 && t >= least) continue;
    least = t;
    width = w;
  }
  int64_t groups = ctas / width;
  auto passes = [&](int32_t i) { return ceil_div(segments(i), width); };
  std::vector<int64_t> v0(1, 0);  // the requests' starts on the line
  for (int32_t i = 0; i < n_seq; ++i) v0.push_back(v0.back() + cost(i) * passes(i));
  const int64_t total = v0.back();
  // The ranges' ends on the line: equal ranges, or whole passes where the longest of such
  // ranges is not much longer.
  std::vector<int64_t> ends;
  auto whole_passes = [&](int64_t most) {
    ends.assign(1, 0);
    for (int32_t i = 0; i < n_seq; ++i) {
      const int64_t c = cost(i);
      if (c > most) return false;
      for (int64_t at = v0[i]; at < v0[i + 1];) {
        const int64_t fit = (ends.back() + most - at) / c;  // passes that the range still takes
        if (fit > 0)
          at = std::min(v0[i + 1], at + fit * c);
        else
          ends.push_back(at);
        if (static_cast<int64_t>(ends.size()) > groups) return false;
      }
    }
    ends.push_back(total);
    return true;
  };
  int64_t least_most = total / groups + kCombine;
  if (groups > 1 && whole_passes(least_most)) {
    for (int64_t low = total / groups; low < least_most;) {
      const int64_t mid = (low + least_most) / 2;
      if (whole_passes(mid))
        least_most = mid;
      else
        low = mid + 1;
    }
    whole_passes(least_most);
    groups = static_cast<int64_t>(ends.size()) - 1;
  } else {
    ends.clear();
    for (int64_t g = 0; g <= groups; ++g) ends.push_back(total * g / groups);
  }
  // (A range's tiles travel in 31 bits.)
  if (ceil_div(total, groups) > 0x3fffffff) return RPA_ERR_UNSUPPORTED;
  l.start_begin = static_cast<int32_t>(plan.tree_starts.size());
  l.n_ctas = static_cast<int32_t>(groups * width);
  l.cut_begin = static_cast<int32_t>(plan.tree_cuts.size());
  l.width = static_cast<int32_t>(width);
  // A lane's segments of request i: lane, lane + width, ...
  auto of_lane = [&](int32_t i, int64_t lane) { return segments(i) <= lane ? 0 : (segments(i) - lane - 1) / width + 1; };
  std::vector<int64_t> before(width, 0);  // the lanes' tiles before request `i`
  std::vector<int64_t> done(width, 0);    // ... before the current range
  std::vector<int32_t> last(width, -1);   // the lanes' last cuts
  int32_t i = 0;
  for (int64_t g = 0; g <= groups; ++g) {
    const int64_t x = ends[g];
    for (; i < n_seq && v0[i + 1] <= x; ++i)
      for (int64_t lane = 0; lane < width; ++lane) before[lane] += of_lane(i, lane) * tiles(i);
    // The boundary as a pass and a tile: one inside a charge is the pass's end.
    int64_t pass = 0, j = 0;
    if (i < n_seq) {
      pass = (x - v0[i]) / cost(i);
      j = (x - v0[i]) % cost(i) / kTile;
      if (j >= tiles(i)) {
        ++pass;
        j = 0;
      }
    }
    for (int64_t lane = 0; lane < width; ++lane) {
      // The lane's first tile from there on.
      TreeStart st{static_cast<uint16_t>(i), 0, 0, static_cast<uint16_t>(lane), 0, 0};
      int64_t at = before[lane], seg = pass * width + lane;
      bool inside = false;
      if (i < n_seq && seg < segments(i)) {
        at += pass * tiles(i) + j;
        inside = j > 0;
        st.j = static_cast<int32_t>(j);
      } else {
        if (i < n_seq) {
          at += of_lane(i, lane) * tiles(i);
          ++st.i;
        }
        while (st.i < n_seq && segments(st.i) <= lane) ++st.i;
        seg = lane;
      }
      if (st.i < n_seq) {
        st.head = static_cast<uint16_t>(seg / per_head(st.i));
        st.st = static_cast<uint16_t>(seg % per_head(st.i));
      }
      TreeStart* prev = g > 0 ? &plan.tree_starts[l.start_begin + (g - 1) * width + lane] : nullptr;
      if (prev) prev->tiles = static_cast<int32_t>(at - done[lane]);
      done[lane] = at;
      if (g == groups) continue;
      plan.tree_starts.push_back(st);
      if (!inside) continue;
      // The segment is cut here: between this CTA and the lane's one before it.
      prev = &plan.tree_starts[l.start_begin + (g - 1) * width + lane];
      TreeCut* cut = last[lane] >= 0 ? &plan.tree_cuts[last[lane]] : nullptr;
      if (cut && cut->i == st.i && cut->head == st.head && cut->st == st.st) {
        ++cut->nparts;
      } else {
        const uint16_t first = prev->i == st.i && prev->head == st.head && prev->st == st.st ? 0 : 1;
        last[lane] = static_cast<int32_t>(plan.tree_cuts.size());
        plan.tree_cuts.push_back({st.i, st.head, st.st, static_cast<uint16_t>((g - 1) * width + lane), first, 2});
        ++l.n_cut;
      }
    }
  }
  for (int32_t k = 0; k < l.n_cut; ++k)
    plan.max_splits = std::max<int32_t>(plan.max_splits, plan.tree_cuts[l.cut_begin + k].nparts);
  plan.max_splits = std::max(plan.max_splits, 1);
  plan.kv_split = std::max(plan.kv_split, static_cast<int32_t>(std::min<int64_t>(
                                              ceil_div(total, groups * kTile) * kTreeKeys, 0x7fffffff)));
  plan.decode_ctas += l.n_ctas;
  plan.tree_slots = std::max(plan.tree_slots, 2 * l.n_ctas);
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
    if (kv[s] > kTreeMaxLen) return RPA_ERR_UNSUPPORTED;
    if (n > 0)
      plan.tree_seqs.push_back({s, cu[s], kv[s], win ? std::max(win[s], 0) : 0, static_cast<uint16_t>(n), 0});
  }
  const int32_t total = static_cast<int32_t>(plan.tree_seqs.size());
  plan.num_decode = total;
  for (int32_t i = 0; i < total; i += kTreeSeqsLarge) {
    TreeLaunch l{i, std::min(total, i + kTreeSeqsLarge), 0, 0, 0, 0, 1};
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
