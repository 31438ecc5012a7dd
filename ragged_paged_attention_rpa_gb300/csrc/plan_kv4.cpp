// The scheduler for 4-bit pages (RPA_DTYPE_FP4_E2M1).  Host only.
//
// Sequences of few query rows per KV head (q_len x G; single tokens always) run
// on the split-KV kernels, in tiles of 8 or 16 rows (kv4_decode.cu) or of 64
// (kv4_rows.cu) that each widen the keys anew; the others' visible keys are widened to bf16 once
// (kv4_expand.cu) and run on the tensor-core prefill, as a plan of its own
// (Plan::kv4_prefill) over the widened pages.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "rpa_internal.h"

namespace rpa {

int prefill_tokens_per_block(int32_t head_dim, int32_t group);  // prefill_tc.cu

namespace {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which part is faster for a sequence of several rows depends on the batch: the
// prefill does not split a sequence's keys over CTAs, the split-KV kernels widen
// them once a tile (128 sequences of 64 rows over 128-2048 keys of 256: 72 us on
// the prefill, 62 split; 64 of 128 rows over as many: 51 against 61; 8 of 64 rows
// over 16k-30k keys: 459 against 71).  So the row limit is the one of these
// with the smallest modelled time.
constexpr int32_t kRowLimits[] = {16, 32, 64, 128};
// Fewest key blocks (segment charges included) a warp of the split-KV kernel
// gets before the batch is cut over more CTAs.
constexpr int32_t kBlocksPerWarp = 2;

// The split-KV kernel's model, fitted to GB300 timings on 12-152 SMs: 4-bit
// bytes it widens a second on an SM (a single tile of 8 rows, several of them,
// tiles of 16, tiles of 64), bytes from HBM, and its start, merge and combine; and the
// bandwidth of the widening to bf16.
constexpr double kOneTileGBs = 43.0;
constexpr double kTilesGBs = 30.0;
constexpr double kTile16GBs = 26.0;
constexpr double kRows64GBs = 5.8;
constexpr double kHbmGBs = 5700.0;
constexpr double kFixedUs = 18.0;
constexpr double kExpandGBs = 5000.0;
// Beside a prefill an SM of the split-KV kernel runs at this share of its rate.
// Side by side is taken where it promises this much of the time, and with an
// eighth of the SMs at least for either part (512 contexts of 4k-16k beside one
// chunk of 512 on 6 SMs took 378 us for the 322 modelled; 305 one after the
// other).
constexpr double kBesideShare = 0.8;
constexpr double kBesideGain = 0.95;
constexpr int32_t kBesideLeast = 8;
// The prefill's: a 128-key tile and an item's end at 256 dimensions (both scale
// with them), and its start and tail.
constexpr double kPrefillTileUs256 = 1.6;
constexpr double kPrefillItemUs256 = 3.2;
constexpr double kPrefillFixedUs = 20.0;

struct Problem {
  const Plan& plan;
  const int32_t* cu;
  const int32_t* kv;
  const int32_t* win;
  int32_t group, q_block;
  int32_t q_len(int32_t s) const { return cu[s + 1] - cu[s]; }
  // First key the query at position pos of sequence s sees.
  int32_t first_key(int32_t s, int32_t pos) const {
    const int32_t w = win ? win[s] : 0;
    return w > 0 && pos - (w - 1) > 0 ? pos - (w - 1) : 0;
  }
};

// Rows of a split-KV tile.  Up to two tiles of kv4_decode.cu: 8 rows, or 16 where
// a sequence has more than 8 and the kernel's registers hold them (head_dim below
// 256).  Beyond, tiles of 64 (32 sequences of 32 rows of 128 dimensions, 8 heads,
// over 120-4000 keys: 62 us in tiles of 16, 73 in one of 64; 128 sequences of 32
// rows of 256: 73 us on the prefill, 48 in one of 64).
int32_t tile_rows(int32_t head_dim, int32_t rows) {
  if (rows > (head_dim == 256 ? 16 : 32)) return 8 * kKv4RowsTile;
  return rows > 8 && head_dim < 256 ? 16 : 8;
}

// Modelled work of the two parts where sequences of q_len >= min_q are prefill.
struct Work {
  bool dec = false, pre = false;
  double sm_us = 0, hbm_us = 0;  // split-KV part: time on one SM, and of HBM
  double expand_us = 0;
  int64_t tiles = 0, longest = 0, items = 0;  // of the prefill
  double decode_us(double sms) const { return dec ? std::max(sm_us / sms, hbm_us) + kFixedUs : 0.0; }
  double prefill_us(int32_t head_dim, int32_t sms) const {
    if (!pre) return 0.0;
    const double f = head_dim / 256.0;
    return std::max(static_cast<double>(tiles) / sms, static_cast<double>(longest)) * kPrefillTileUs256 * f +
           std::ceil(static_cast<double>(items) / sms) * kPrefillItemUs256 * f + kPrefillFixedUs + expand_us;
  }
};

Work work_of(const Problem& b, int32_t min_q) {
  const Plan& p = b.plan;
  Work k;
  for (int32_t s = 0; s < p.num_seqs; ++s) {
    const int32_t ql = b.q_len(s);
    if (ql < 1) continue;
    const int32_t pos0 = b.kv[s] - ql;
    const double elems = 2.0 * (b.kv[s] - b.first_key(s, pos0)) * p.hkv * p.d, bytes = 0.5625 * elems;
    if (ql < min_q) {
      const int32_t rows = ql * b.group, tile = tile_rows(p.d, rows);
      k.dec = true;
      k.sm_us += bytes * static_cast<double>(ceil_div(rows, tile)) * 1e-3 /
                 (tile > 16 ? kRows64GBs : tile == 16 ? kTile16GBs : rows > 8 ? kTilesGBs : kOneTileGBs);
      k.hbm_us += bytes * 1e-3 / kHbmGBs;
      continue;
    }
    k.pre = true;
    k.expand_us += (bytes + 2.0 * elems) * 1e-3 / kExpandGBs;
    for (int32_t t = 0; t < ql; t += b.q_block) {
      const int32_t last = pos0 + std::min(t + b.q_block, ql) - 1;
      const int64_t n = (last - b.first_key(s, pos0 + t) / kPrefillTileAlign * kPrefillTileAlign) / kPrefillTileKeys + 1;
      k.tiles += n * p.hkv;
      k.longest = std::max(k.longest, n);
      k.items += p.hkv;
    }
  }
  return k;
}

// Row tiles, launches and CTA ranges of the split-KV part.
rpa_status_t plan_split(Plan& plan, const Problem& b, int32_t min_q) {
  for (const int32_t nt : {1, 2, kKv4RowsTile}) {
    const Kv4Grain grain = kv4_grain(plan.d, nt);
    const int32_t first = static_cast<int32_t>(plan.kv4_tiles.size());
    for (int32_t s = 0; s < plan.num_seqs; ++s) {
      const int32_t ql = b.q_len(s), rows = ql * b.group;
      if (ql < 1 || ql >= min_q || tile_rows(plan.d, rows) != 8 * nt) continue;
      ++plan.num_decode;
      const int32_t pos0 = b.kv[s] - ql;
      for (int32_t r0 = 0; r0 < rows; r0 += 8 * nt) {
        const int32_t n = std::min(8 * nt, rows - r0);
        const int32_t fb = b.first_key(s, pos0 + r0 / b.group) / grain.block_keys;
        const int32_t lb = (pos0 + (r0 + n - 1) / b.group) / grain.block_keys;
        plan.kv4_tiles.push_back({s, b.cu[s], r0, n, pos0, b.win ? std::max(b.win[s], 0) : 0, fb, lb - fb + 1});
      }
    }
    const int32_t last = static_cast<int32_t>(plan.kv4_tiles.size());
    for (int32_t t0 = first; t0 < last; t0 += kKv4TilesLarge) {
      const int32_t t1 = std::min(last, t0 + kKv4TilesLarge);
      std::vector<int64_t> v0(1, 0);  // the tiles' starts on the line
      for (int32_t i = t0; i < t1; ++i)
        v0.push_back(v0.back() + static_cast<int64_t>(plan.kv4_tiles[i].nb + kKv4SegCost) * plan.hkv);
      const int64_t total = v0.back();
      const int64_t most =
          std::min<int64_t>(plan.decode_sms > 0 ? plan.decode_sms : plan.num_sms, kKv4MaxCtas);
      // (A range's length travels in 31 bits.)
      const int64_t n = std::max<int64_t>(
          std::max<int64_t>(1, std::min(most, total / (kBlocksPerWarp * grain.warps))),
          std::min(most, ceil_div(total, 0x3fffffff)));
      if (ceil_div(total, n) > 0x7fffffff) return RPA_ERR_UNSUPPORTED;
      Plan::Kv4Launch l{t0, t1, nt, static_cast<int32_t>(plan.kv4_starts.size()), static_cast<int32_t>(n), false};
      // Equal ranges of the line; the boundaries that fall inside a segment cut it.
      int64_t seg = -1, parts = 1;
      for (int64_t c = 0; c < n; ++c) {
        const int64_t x = total * c / n, end = total * (c + 1) / n;
        const size_t i = static_cast<size_t>(std::upper_bound(v0.begin(), v0.end(), x) - v0.begin()) - 1;
        const int32_t nb = plan.kv4_tiles[t0 + static_cast<int32_t>(i)].nb;
        const int64_t cost = nb + kKv4SegCost, off = (x - v0[i]) % cost;
        plan.kv4_starts.push_back({static_cast<int32_t>(i), static_cast<int32_t>((x - v0[i]) / cost),
                                   static_cast<int32_t>(off), static_cast<int32_t>(end - x)});
        if (off == 0 || off >= nb) continue;
        l.cut = true;
        parts = x - off == seg ? parts + 1 : 2;
        seg = x - off;
        plan.max_splits = std::max(plan.max_splits, static_cast<int32_t>(parts));
      }
      if (plan.kv_split == 0)
        plan.kv_split = static_cast<int32_t>(std::min<int64_t>(ceil_div(total, n) * grain.block_keys, 0x7fffffff));
      plan.max_splits = std::max(plan.max_splits, 1);
      plan.decode_ctas += n;
      plan.kv4_part_rows = std::max(plan.kv4_part_rows, 2 * n * nt * 8);
      if (nt != kKv4RowsTile) plan.kv4_piece_rows = std::max(plan.kv4_piece_rows, grain.warps * n * nt * 8);
      plan.kv4_launches.push_back(l);
    }
  }
  return RPA_OK;
}

// The prefill part: the pages to widen, and its plan, which sees the split-KV
// sequences as empty ones and the widened pages as its pool.
rpa_status_t plan_widened(Plan& plan, const Problem& b, int32_t min_q, const rpa_plan_options& opts) {
  std::vector<int32_t> cu(static_cast<size_t>(plan.num_seqs) + 1, 0);
  int64_t pages = 0;
  for (int32_t s = 0; s < plan.num_seqs; ++s) {
    const int32_t ql = b.q_len(s);
    cu[s + 1] = cu[s];
    if (ql < min_q) continue;
    ++plan.num_prefill;
    cu[s + 1] += ql;
    const int32_t lo = b.first_key(s, b.kv[s] - ql), slot0 = lo / plan.p;
    plan.kv4_expand.push_back({s, slot0, static_cast<int32_t>(pages), lo, b.kv[s], b.cu[s], ql});
    pages += ceil_div(b.kv[s], plan.p) - slot0;
    // (The widening counts the rows of all heads in 31 bits.)
    if (pages * plan.p * plan.hkv > 0x7fffffff) return RPA_ERR_UNSUPPORTED;
  }
  plan.kv4_scratch_pages = static_cast<int32_t>(pages);
  if (plan.num_prefill == 0) return RPA_OK;
  if (plan.hkv > kPlanMaxKvHeads) return RPA_ERR_UNSUPPORTED;
  plan.kv4_prefill.reset(new (std::nothrow) Plan());
  if (!plan.kv4_prefill) return RPA_ERR_INVALID_ARG;
  Plan& f = *plan.kv4_prefill;
  f.num_seqs = plan.num_seqs;
  f.hq = plan.hq;
  f.hkv = plan.hkv;
  f.d = plan.d;
  f.p = plan.p;
  f.mpps = plan.mpps;
  f.num_pages = plan.kv4_scratch_pages;
  f.dtype = plan.dtype;
  f.has_window = plan.has_window;
  f.total_q = plan.total_q;
  f.num_sms = plan.prefill_sms > 0 ? plan.prefill_sms : plan.num_sms;
  rpa_plan_options o = opts;
  o.kv_dtype = 0;
  o.decode_sms = 0;
  return build_schedule(f, cu.data(), b.kv, b.win, o);
}

}  // namespace

rpa_status_t build_kv4_schedule(Plan& plan, const int32_t* cu, const int32_t* kv, const int32_t* win,
                                const rpa_plan_options& opts) {
  const int32_t group = plan.hq / plan.hkv;
  if (opts.path != RPA_PATH_AUTO && opts.path != RPA_PATH_SIMT && opts.path != RPA_PATH_TC)
    return RPA_ERR_INVALID_ARG;
  if (plan.dtype != RPA_DTYPE_BF16 || opts.path == RPA_PATH_SIMT || plan.p < 16 ||
      !prefill_tc_supported(plan.d, plan.p, group) || opts.kv_split != 0 || opts.prefill_pairs == 2 ||
      opts.prefill_split > 0 || opts.decode_kernel != 0 ||
      opts.q_block > prefill_tokens_per_block(plan.d, group))
    return RPA_ERR_UNSUPPORTED;
  plan.kv_fp4 = true;
  plan.path = RPA_PATH_TC;
  const Problem b{plan, cu, kv, win, group,
                  opts.q_block > 0 ? opts.q_block : prefill_tokens_per_block(plan.d, group)};

  // The row limit (single tokens stay on the split-KV kernel).
  const int32_t n = plan.num_sms;
  Work best;
  double best_t = 0;
  int32_t min_q = 0;
  for (const int32_t limit : kRowLimits) {
    const int32_t q = std::max(2, limit / group + 1);
    if (q == min_q) continue;
    const Work k = work_of(b, q);
    const double t = k.decode_us(n) + k.prefill_us(plan.d, n);
    if (min_q != 0 && t >= best_t) continue;
    best = k;
    best_t = t;
    min_q = q;
  }
  // A mixed batch's split of the SMs between the two parts, as for 16-bit
  // pages: side by side where the split that evens their modelled times beats
  // one after the other (512 single tokens and 4 chunks of 2048: 189 us at 39 /
  // 113 SMs, 208 us one after the other).
  if (best.dec && best.pre && opts.decode_sms >= 0 && n >= 2) {
    int32_t x = opts.decode_sms > 0 ? std::min(opts.decode_sms, n - 1) : 0;
    best_t *= kBesideGain;
    const int32_t least = std::max(1, n / kBesideLeast);
    for (int32_t i = least; i <= n - least && opts.decode_sms == 0; ++i) {
      const double t = std::max(best.decode_us(i * kBesideShare), best.prefill_us(plan.d, n - i));
      if (t < best_t) {
        best_t = t;
        x = i;
      }
    }
    if (x > 0) {
      plan.overlap = true;
      plan.decode_sms = x;
      plan.prefill_sms = n - x;
      plan.est_decode_us = static_cast<float>(best.decode_us(x * kBesideShare));
      plan.est_prefill_us = static_cast<float>(best.prefill_us(plan.d, n - x));
    }
  }
  if (rpa_status_t st = plan_split(plan, b, min_q)) return st;
  if (rpa_status_t st = plan_widened(plan, b, min_q, opts)) return st;

  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  if (plan.kv4_part_rows > 0) {
    plan.off_partial_o = take(static_cast<size_t>(plan.kv4_part_rows) * plan.d * sizeof(float));
    plan.off_partial_lse = take(static_cast<size_t>(plan.kv4_part_rows) * sizeof(float));
    plan.off_kv4_pieces = take(static_cast<size_t>(plan.kv4_piece_rows) * plan.d * sizeof(float));
  }
  if (plan.num_prefill > 0) {
    const size_t bytes = static_cast<size_t>(plan.kv4_scratch_pages) * plan.p * plan.hkv * plan.d * 2;
    plan.off_kv4_k = take(bytes);
    plan.off_kv4_v = take(bytes);
    plan.off_kv4_table = take(static_cast<size_t>(plan.num_seqs) * plan.mpps * sizeof(int32_t));
  }
  plan.ws_bytes = off;
  return RPA_OK;
}

}  // namespace rpa
