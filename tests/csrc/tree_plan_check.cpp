// The schedule of drafted trees (plan_tree.cpp): the CTAs' ranges hold every key tile
// of every segment once, in order, and the cut list names the CTAs of each cut segment
// and their slots.  Random batches; prints one line and returns 0 on success.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "rpa_internal.h"

namespace rpa {
bool tree_tc_supported(int32_t, int32_t, int32_t) { return true; }
}  // namespace rpa

#define CHECK(x) \
  if (!(x)) { std::printf("batch %d: %s\n", batch, #x); return 1; }

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  long cuts = 0, parts_seen = 0, widths = 0;
  for (int batch = 0; batch < 3000; ++batch) {
    rpa::Plan p;
    const int dims[] = {64, 128, 256};
    const int group = pick(0, 3) ? pick(1, 16) : pick(1, 128);
    p.d = dims[pick(0, 2)];
    p.hkv = pick(1, 5);
    p.hq = p.hkv * group;
    p.p = 16;
    p.num_sms = pick(0, 2) ? 152 : pick(1, 300);
    p.num_seqs = pick(0, 9) ? pick(0, 40) : pick(1000, 2500);
    std::vector<int32_t> cu(1, 0), kv, win;
    const int most = pick(1, 200), longest = pick(0, 3) ? 4000 : 40000;
    for (int s = 0; s < p.num_seqs; ++s) {
      const int n = pick(0, most);
      cu.push_back(cu.back() + n);
      kv.push_back(n + pick(0, longest));
      win.push_back(pick(0, 1) ? 0 : pick(1, 3000));
    }
    rpa_plan_options o{};
    o.tree_words = 4;
    CHECK(build_tree_schedule(p, cu.data(), kv.data(), win.data(), o) == RPA_OK);
    const int per = 128 / group * rpa::tree_row_tiles(p.d);
    int seqs = 0;
    for (const rpa::TreeLaunch& l : p.tree_launches) {
      CHECK(l.seq_begin == seqs && l.seq_end > l.seq_begin && l.seq_end - l.seq_begin <= rpa::kTreeSeqsLarge);
      seqs = l.seq_end;
      CHECK(l.n_ctas >= 1 && l.n_ctas <= p.num_sms && l.n_ctas <= rpa::kTreeMaxCtas);
      CHECK(l.width >= 1 && l.n_ctas % l.width == 0);
      widths += l.width > 1;
      std::map<std::tuple<int, int, int>, std::vector<std::pair<int, int>>> where;  // (cta, slot) of cut segments' parts
      std::map<std::tuple<int, int, int>, int> seen;                                // tiles of each segment so far
      for (int c = 0; c < l.n_ctas; ++c) {  // (a lane's CTAs come in the order of their keys)
        const rpa::TreeStart& s = p.tree_starts[l.start_begin + c];
        CHECK(s.tiles >= 0);
        int left = s.tiles, ordinal = 0, i = s.i, head = s.head, st = s.st, j = s.j;
        while (left > 0) {
          CHECK(i >= 0 && i < l.seq_end - l.seq_begin && head >= 0 && head < p.hkv && st >= 0);
          const rpa::TreeSeq& q = p.tree_seqs[l.seq_begin + i];
          const int per_head = (q.nodes + per - 1) / per;
          CHECK(st < per_head && (head * per_head + st) % l.width == c % l.width);
          const int nb = (q.len - 1) / 128 + 1 - rpa::tree_first_tile(q), n = std::min(left, nb - j);
          CHECK(n >= 1 && (seen[{i, head, st}] == j));
          seen[{i, head, st}] += n;
          if (n < nb) where[{i, head, st}].push_back({c, 2 * c + (ordinal > 0)});
          ++ordinal;
          ++parts_seen;
          left -= n;
          j += n;
          if (j == nb) {
            j = 0;
            int at = head * per_head + st + l.width;  // the request's segment
            if (at >= per_head * p.hkv) {
              at = c % l.width;
              do ++i;
              while (i < l.seq_end - l.seq_begin &&
                     (p.tree_seqs[l.seq_begin + i].nodes + per - 1) / per * p.hkv <= at);
            }
            if (i < l.seq_end - l.seq_begin) {
              const int next = (p.tree_seqs[l.seq_begin + i].nodes + per - 1) / per;
              head = at / next;
              st = at % next;
            }
          }
        }
      }
      for (int i = 0; i < l.seq_end - l.seq_begin; ++i) {
        const rpa::TreeSeq& q = p.tree_seqs[l.seq_begin + i];
        for (int head = 0; head < p.hkv; ++head)
          for (int st = 0; st * per < q.nodes; ++st)
            CHECK((seen[{i, head, st}] == (q.len - 1) / 128 + 1 - rpa::tree_first_tile(q)));
      }
      CHECK(static_cast<int>(where.size()) == l.n_cut && l.n_cut <= rpa::kTreeMaxCtas);
      for (int k = 0; k < l.n_cut; ++k) {
        const rpa::TreeCut& c = p.tree_cuts[l.cut_begin + k];
        const auto& w = where.at({c.i, c.head, c.st});
        CHECK(static_cast<int>(w.size()) == c.nparts);
        for (int x = 0; x < c.nparts; ++x) {
          const int at = c.cta + x * l.width;
          CHECK(w[x].first == at && w[x].second == 2 * at + (x == 0 ? c.first : 0));
          CHECK(w[x].second < p.tree_slots);
        }
        ++cuts;
      }
    }
    CHECK(seqs == static_cast<int>(p.tree_seqs.size()));
    const size_t rows = static_cast<size_t>(p.tree_slots) * 128 * rpa::tree_row_tiles(p.d);
    CHECK(p.tree_cuts.empty() || p.ws_bytes >= 256 + rows * (p.d + 1) * 4);
  }
  std::printf("tree plans ok: %ld parts, %ld cut segments, %ld launches of several lanes\n", parts_seen, cuts, widths);
  return 0;
}
