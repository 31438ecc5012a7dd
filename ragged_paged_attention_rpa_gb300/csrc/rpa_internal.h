// Internal declarations shared by the host API, the scheduler and the kernel
// launchers of librpa.  Not part of the public interface (include/rpa.h).
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>
#include <memory>
#include <vector>

#include "rpa.h"

#ifdef __CUDACC__
#define RPA_HD __host__ __device__
#else
#define RPA_HD
#endif

namespace rpa {

// Workspace layout: a 256-byte header (error word first), then the decode
// split partials.  Offsets are multiples of 256 bytes.
constexpr size_t kHeaderBytes = 256;
// Offset in the header of the dynamic prefill item counter (two int32: items
// taken, CTAs finished), zero between launches.
constexpr size_t kPrefillCounterOff = 64;
// Offset in the header of the table kernels' counter (one int32: CTAs
// finished), zero between launches.
constexpr size_t kTablesCounterOff = 128;
// Offset in the header of the 4-bit prompts' words (two int32: whether the
// widening met a NaN in V, CTAs finished), zero between calls.
constexpr size_t kKv4NanOff = 192;
// Most requests, pages and tokens of a table call (its loop indices add a grid's
// threads to them in 31 bits).
constexpr int32_t kTablesMost = 1 << 30;

// Most KV heads of a plan's tensor-core work (its items and segments hold a head
// in eight bits).
constexpr int32_t kPlanMaxKvHeads = 256;

// One prefill work item: query block `qb` (of plan.q_block tokens) of
// sequence `seq`, for KV head `head`.  Ordered longest first in the plan.
struct PrefillItem {
  int32_t seq;
  int32_t qb_head;  // (query block index << 8) | kv head
  // 0: every key tile of the item.  Else one part of an item whose key
  // tiles the plan split across CTAs: (slot << 21) | (first tile << 10) |
  // tile count, as unsigned bits; the part leaves an fp32 partial in `slot`
  // and a combine merges the parts.  seq < 0: padding, skipped.
  int32_t split;
};
constexpr int kSplitMaxSlots = 2048, kSplitMaxFirst = 2048, kSplitMaxTiles = 1023;
RPA_HD constexpr int32_t split_code(int32_t slot, int32_t j0, int32_t n) {
  return static_cast<int32_t>((static_cast<uint32_t>(slot) << 21) |
                              (static_cast<uint32_t>(j0) << 10) | static_cast<uint32_t>(n));
}
RPA_HD constexpr int32_t split_slot(int32_t c) {
  return static_cast<int32_t>(static_cast<uint32_t>(c) >> 21);
}
RPA_HD constexpr int32_t split_first(int32_t c) {
  return static_cast<int32_t>((static_cast<uint32_t>(c) >> 10) & 2047u);
}
RPA_HD constexpr int32_t split_tiles(int32_t c) {
  return static_cast<int32_t>(static_cast<uint32_t>(c) & 1023u);
}

// Most work items one tensor-core prefill launch carries in its parameters;
// longer lists are split over several launches.
constexpr int kMaxItemsPerLaunch = 2048;

// Score tiles of the tensor-core prefill: 128 keys, starting on multiples of
// 64 keys at or below the first visible key.
constexpr int kPrefillTileKeys = 128;
constexpr int kPrefillTileAlign = 64;

// An item split into parts: its partial slots are [slot0, slot0 + nparts).
struct PrefillSplit {
  int32_t seq, qb_head, slot0, nparts;
};
constexpr int kMaxSplitGroupsPerLaunch = 1024;
// Largest persistent prefill grid whose per-CTA item lists the launch
// parameters carry.
constexpr int kMaxPrefillGrid = 256;

// Decode schedule limits: segments one decode launch carries in its
// parameters (two sizes), and segments / pages one decode CTA's range may
// touch (their tables sit in shared memory).
constexpr int kDecodeSegSmall = 256;
constexpr int kDecodeSegLarge = 1024;
constexpr int kMaxCtaSegs = 64;
constexpr int kMaxCtaPages = 512;
// Most CTAs a cost-balanced decode launch lists (their range starts travel in
// the launch parameters), and the charge, in 16-key blocks, for each segment
// a CTA's range touches (its in-CTA merge and output).
constexpr int kMaxDecodeCtas = 1024;
// Largest decode grid the plan's per-CTA range table describes (one wave:
// at most one CTA per SM).
constexpr int kMaxDecodeGrid = 512;
constexpr int kDecodeSegCost = 7;

// Split-KV attention over 4-bit pages (kv4_decode.cu): row tiles one launch
// carries in its parameters (two sizes), CTAs of its grid (whose starts travel
// there too), and the charge, in key blocks, for each segment (its merge and
// output).
constexpr int kKv4TilesSmall = 160;
constexpr int kKv4TilesLarge = 864;
constexpr int kKv4MaxCtas = 256;
constexpr int kKv4SegCost = 3;
constexpr int kKv4RowsTile = 8;  // the tiles of kv4_rows.cu, in rows of 8
// Sequences whose 4-bit pages one expansion launch lists.
constexpr int kKv4ExpandSeqs = 1024;

// Attention of drafted trees (tree_attn.cu, tree_simt.cu).  A request: its row of
// the page table, first node, nodes, keys (nodes included) and window.
// (These lists travel as launch parameters, in few bytes: 128 requests of 8 nodes take 40.6
// us with room for 1024 requests, 37.4 with room for 128.)
struct TreeSeq {
  int32_t seq, q0, len, window;
  uint16_t nodes, per_head;  // per_head: segments of a head (tensor cores)
};
// Row tiles of the tensor-core kernel: 128 rows are 128 / G nodes of G heads; a
// segment is (request, KV head, row_tiles(D) such tiles), its keys in tiles of 128.
// A request's segments, in (head, row tiles) order, run in passes of `width` segments, a
// lane each; the passes' key tiles lie end to end, and a group of `width` CTAs, one per
// lane, takes a contiguous range of them: for a CTA `tiles` tiles of its lane from tile j
// of (request i, head, segment st) on.
struct TreeStart {
  uint16_t i, head, st, lane;
  int32_t j, tiles;
};
// A segment cut across CTAs cta, cta + width, ..., nparts of them: the first holds its
// partial in slot 2 cta + first, each later CTA c in slot 2 c.
struct TreeCut {
  uint16_t i, head, st, cta, first, nparts;
};
struct TreeLaunch {
  int32_t seq_begin, seq_end, start_begin, n_ctas, cut_begin, n_cut, width;
};
constexpr int kTreeMaxWords = 16;
constexpr int32_t kTreeMaxLen = 0x7fffffff - 1023;  // the kernels step past the last key in 32 bits
constexpr int kTreeRows = 128;
constexpr int kTreeKeys = 128;
constexpr int kTreeSeqsSmall = 128;   // requests a launch carries in its parameters
constexpr int kTreeSeqsLarge = 1024;
constexpr int kTreeMaxCtas = 160;
RPA_HD constexpr int32_t tree_row_tiles(int32_t head_dim) { return head_dim == 256 ? 1 : 2; }
// First of the 128-key tiles that a request's nodes can see (a node's position is
// at least that of the first behind the context).
RPA_HD constexpr int32_t tree_first_tile(const TreeSeq& s) {
  const int32_t ctx = s.len - s.nodes;
  return s.window > 0 && ctx - s.window + 1 > 0 ? (ctx - s.window + 1) / kTreeKeys : 0;
}

struct Plan {
  // Problem description (checked against every rpa_forward call).
  int32_t num_seqs = 0, hq = 0, hkv = 0, d = 0, p = 0, mpps = 0, num_pages = 0;
  int32_t dtype = RPA_DTYPE_BF16;
  bool kv_fp8 = false;               // K/V pages are e4m3 bytes (decode only)
  bool kv_fp4 = false;               // K/V pages are 4-bit codes with block scales
  bool has_window = false;
  int64_t total_q = 0;

  int32_t path = RPA_PATH_SIMT;     // path actually used
  bool simt_decode = false;          // decode sequences handled by the SIMT kernel
  bool simt_prefill = false;         // prefill sequences handled by the SIMT kernel
  bool decode_tc = false;            // split-KV decode on the tensor-core kernel
  int32_t num_sms = 152;
  // Mixed batches (decode and tensor-core prefill work in one call): the two
  // persistent grids run side by side on disjoint SMs, decode on
  // decode_sms of them and prefill on prefill_sms (forked onto a second
  // stream and joined back); 0: each grid takes every SM, one after the other.
  bool overlap = false;
  int32_t decode_sms = 0, prefill_sms = 0;
  // The planner's cost estimates (microseconds) behind that choice.
  float est_decode_us = 0.f, est_prefill_us = 0.f;

  // Decode (q_len == 1) on the split-KV kernel.  Segments = (sequence, KV
  // head) pairs in stream order; blocks are 16 keys; each launch cuts its
  // segments' block stream into contiguous ranges, one per CTA: ranges of
  // equal cost (blocks plus a fixed charge per segment touched), listed in
  // dcta_blk0, or, where bpc > 0, ranges of bpc blocks each.
  struct DecodeLaunch {
    int32_t seg_begin, seg_end;  // segments [seg_begin, seg_end)
    int32_t bpc;                 // > 0: blocks per CTA (uniform ranges)
    int32_t n_ctas;
    int32_t slot_base;           // first partial slot (two per CTA)
    int32_t cta_begin;           // bpc == 0: ranges in dcta_blk0[cta_begin ...]
    int32_t cut_begin, n_cut;    // segments cut across CTAs: dcut[cut_begin ...]
  };
  // A segment cut across CTAs ca .. ca + nparts - 1 of its launch: CTA ca
  // holds its partial in slot 2 ca + first (first = 1 when the segment is
  // not the first of ca's range), every later CTA c in slot 2 c.
  struct DecodeCut {
    int32_t ca, first, nparts, q0, g;
  };
  int32_t num_decode = 0;
  int32_t kv_split = 0;   // tokens of the longest CTA range of the first launch
  int32_t max_splits = 0; // most CTAs any segment is cut across
  int64_t decode_ctas = 0;
  std::vector<int32_t> dseg_seqhead;  // (sequence << 8) | kv head
  std::vector<int32_t> dseg_blk0;     // block prefix, size segments + 1
  std::vector<int32_t> dseg_q0, dseg_lo, dseg_len;  // query token, first visible key, length
  std::vector<DecodeLaunch> dlaunch;
  std::vector<int32_t> dcta_blk0;     // per launch: n_ctas + 1 range starts (launch-relative)
  std::vector<DecodeCut> dcut;
  int32_t dec_slots = 0;              // partial slots over all launches

  // 4-bit pages: sequences of few query rows run on the split-KV kernel of
  // kv4_decode.cu as row tiles (rows [r0, r0 + nrows) of the sequence, nb key
  // blocks); the others' visible pages are widened to bf16 in the workspace
  // (kv4_expand.cu) and run as prefill work.
  struct Kv4Tile {
    int32_t seq, q0, r0, nrows, pos0, window, fb, nb;
  };
  // A CTA's range of the line of segments: from block j of (tile, head) on,
  // len blocks and merge charges.  Tiles relative to the launch.
  struct Kv4Start {
    int32_t tile, head, j, len;
  };
  struct Kv4Launch {
    int32_t begin, end;  // tiles [begin, end)
    int32_t nt;          // rows a tile: 8 nt
    int32_t cta_begin, n_ctas;  // kv4_starts[cta_begin ...]
    bool cut;            // some segment is cut across CTAs
  };
  // A sequence's pages from table slot `slot0` on, widened to scratch pages
  // from `page0` on; keys [lo, hi) are converted, hi is its length; its query
  // tokens.
  struct Kv4Expand {
    int32_t seq, slot0, page0, lo, hi, q0, q_len;
  };
  std::vector<Kv4Tile> kv4_tiles;
  std::vector<Kv4Start> kv4_starts;
  std::vector<Kv4Launch> kv4_launches;
  std::vector<Kv4Expand> kv4_expand;
  int64_t kv4_part_rows = 0;      // rows of the split-KV partials (two tiles a CTA)
  int64_t kv4_piece_rows = 0;     // rows of its warps' pieces (one tile a warp)
  int32_t kv4_scratch_pages = 0;
  size_t off_kv4_pieces = 0;
  size_t off_kv4_k = 0, off_kv4_v = 0, off_kv4_table = 0;

  std::unique_ptr<Plan> kv4_prefill;  // the prefill part's plan, over the widened pages

  // Trees of drafted tokens (plan_tree.cpp).
  int32_t tree_words = 0;             // 64-bit words of a mask row (0: not such a plan)
  std::vector<TreeSeq> tree_seqs;     // requests with nodes
  std::vector<TreeLaunch> tree_launches;
  std::vector<TreeStart> tree_starts;
  std::vector<TreeCut> tree_cuts;
  int32_t tree_slots = 0;             // partial slots of the largest launch

  // Prefill (q_len > 1).
  int32_t num_prefill = 0;
  int32_t q_block = 0;
  bool prefill_pairs = false;      // items are pairs of query blocks (SM-pair kernel)
  // Items in longest-first order, each taken by the next CTA to get free
  // (else CTA c runs its own list, pcta0).
  bool prefill_dynamic = false;
  int32_t prefill_groups = 0;         // groups of the dynamic prefill list
  std::vector<PrefillItem> items;  // longest first, or per-CTA lists (pcta0)
  // Per-CTA item lists: CTA c runs items [pcta0[c], pcta0[c + 1]) in order;
  // empty: CTA c runs items c, c + grid, ... (a list too long for one launch).
  std::vector<int32_t> pcta0;
  int32_t prefill_max_tiles = 0;    // key tiles of the busiest CTA
  std::vector<PrefillSplit> psplit; // items split across CTAs (combined afterwards)
  int32_t n_split_items = 0;        // partial slots (parts of split items)
  int32_t prefill_ctas = 0;

  // Workspace.
  size_t off_partial_o = 0, off_partial_lse = 0, ws_bytes = kHeaderBytes;
  size_t off_ppart_o = 0, off_ppart_lse = 0;   // prefill parts: [slot][128 rows][D], [slot][128]
};

// Scheduler (plan.cpp): fills everything but the problem description, which
// the caller has set and validated.
rpa_status_t build_schedule(Plan& plan, const int32_t* cu_q_lens, const int32_t* kv_lens,
                            const int32_t* window, const rpa_plan_options& opts);

// The scheduler for 4-bit pages (plan_kv4.cpp), for a plan as build_schedule's.
rpa_status_t build_kv4_schedule(Plan& plan, const int32_t* cu_q_lens, const int32_t* kv_lens,
                                const int32_t* window, const rpa_plan_options& opts);

// The scheduler for drafted trees (plan_tree.cpp), likewise.
rpa_status_t build_tree_schedule(Plan& plan, const int32_t* cu_q_lens, const int32_t* kv_lens,
                                 const int32_t* window, const rpa_plan_options& opts);

// Host-side checks of the metadata (plan.cpp).
rpa_status_t validate_metadata(const int32_t* cu_q_lens, const int32_t* kv_lens,
                               int32_t num_seqs, int32_t page_size,
                               int32_t max_pages_per_seq);

// Arguments every kernel launcher receives.
struct Args {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  const int32_t* window;
  float sm_scale;
  void* out;
  unsigned char* workspace;
  const float* k_scale = nullptr;  // fp8 pages: per-KV-head scales of K and V
  const float* v_scale = nullptr;
  const uint8_t* k_block_scales = nullptr;  // 4-bit pages: a scale byte per 16 dimensions
  const uint8_t* v_block_scales = nullptr;
  // The prefill over widened 4-bit pages: the 4-bit pages' table and number.
  const int32_t* kv4_page_table = nullptr;
  int32_t kv4_num_pages = 0;
  const uint64_t* tree_mask = nullptr;  // drafted trees
  const int32_t* positions = nullptr;
};

// Kernel launchers; each returns cudaError_t as int (0 = success).
int launch_simt(const Plan& plan, const Args& a, void* stream);
int launch_decode(const Plan& plan, const Args& a, void* stream);
int launch_prefill_tc(const Plan& plan, const Args& a, void* stream);
int launch_prefill_pair(const Plan& plan, const Args& a, void* stream);

// KV-cache write of a step's new tokens (kv_write.cu).
struct KvWriteArgs {
  const void* k_new;
  const void* v_new;
  void* k_pages;
  void* v_pages;
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  unsigned char* workspace;  // error word, or null
  int32_t num_seqs, total_q, hkv, head_dim, elem_bytes, page_size, mpps, num_pages;
};
int launch_kv_write(const KvWriteArgs& a, void* stream);

// The q/k/v prologue (prologue.cu): q/k RMS norm + rotary embedding, v norm,
// q to q_out and k/v into their pages.
struct PrologueArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* q_weight;  // null: no norm
  const float* k_weight;
  const float* v_weight;
  float eps, rope_theta;  // rope_theta <= 0: no rotation
  void* q_out;
  void* k_pages;
  void* v_pages;
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  unsigned char* workspace;  // error word, or null
  int32_t num_seqs, total_q, hq, hkv, head_dim, elem_bytes, page_size, mpps, num_pages;
};
bool prologue_supported(int32_t head_dim);
int launch_prologue(const PrologueArgs& a, void* stream);

// Attention over 4-bit pages: the split-KV kernel over the plan's row tiles
// (kv4_decode.cu), its grain for row tiles of 8 nt rows, and the widening of the
// prefill sequences' visible pages into the workspace, with a page table of
// their own (kv4_expand.cu).
int launch_kv4_decode(const Plan& plan, const Args& a, void* stream);
struct Kv4Grain {
  int32_t warps, block_keys;  // of a CTA (one a SM); keys of a block
};
Kv4Grain kv4_grain(int32_t head_dim, int32_t nt);
Kv4Grain kv4_rows_grain(int32_t head_dim);
int launch_kv4_rows(const Plan& plan, const Args& a, const Plan::Kv4Launch& l, void* stream);
int launch_kv4_expand(const Plan& plan, const Args& a, void* stream);

// The 4-bit cache's write and read (kv4_cache.cu).
struct Kv4CacheArgs {
  const void* k_rows;  // written by a read
  const void* v_rows;
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_scales;
  uint8_t* v_scales;
  const int64_t* slot_map;
  unsigned char* workspace;  // error word, or null
  int32_t tokens, hkv, head_dim, elem_bytes, page_size, num_pages;
  bool read;
};
int launch_kv4_cache(const Kv4CacheArgs& a, void* stream);

// Page tables built and released on the GPU (tables.cu).
struct TableArgs {
  const int32_t* lens;  // build: new tokens; release: finished flags
  const int32_t* kv_lens_prev;
  int32_t* page_table;
  int32_t* free_pages;
  const int32_t* free_count_prev;
  int32_t* cu_q_lens;   // build only, as slot_map and max_tokens
  int32_t* kv_lens;
  int64_t* slot_map;
  int32_t* free_count;
  unsigned char* workspace;
  int32_t num_seqs, page_size, mpps, num_pages, max_tokens;
  enum Kind { kBuild, kRelease, kTrim } kind;
};
int launch_tables(const TableArgs& a, void* stream);

// Attention of drafted trees: on tensor cores (tree_attn.cu) or CUDA cores
// (tree_simt.cu).
bool tree_tc_supported(int32_t head_dim, int32_t page_size, int32_t group);
int launch_tree_attn(const Plan& plan, const Args& a, void* stream);
int launch_tree_simt(const Plan& plan, const Args& a, void* stream);

// Masks and positions of drafted trees, and the rows of an accepted path moved
// (tree.cu).
struct BuildTreeArgs {
  const int32_t* parents;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  const int32_t* window;
  uint64_t* mask;
  int32_t* positions;
  unsigned char* workspace;  // error word, or null
  int32_t num_seqs, total_q, words;
};
int launch_build_tree(const BuildTreeArgs& a, void* stream);
struct CommitTreeArgs {
  void* k_pages;
  void* v_pages;
  const int64_t* slot_map;
  const int32_t* cu_q_lens;
  const int32_t* path;
  unsigned char* workspace;  // error word, or null
  int32_t num_seqs, total_q, max_path;
  int64_t pool_slots, row_bytes;
};
int launch_commit_tree(const CommitTreeArgs& a, void* stream);

// Rotation and cache write at given positions and slots (rope_append.cu).
struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const int64_t* slot_map;
  const float* inv_freq;
  int32_t rotary_dim;
  bool interleaved;
  void* q_out;
  void* k_pages;
  void* v_pages;
  const float* k_scale;  // e4m3 pages, else null
  const float* v_scale;
  unsigned char* workspace;  // error word, or null
  int32_t tokens, hq, hkv, head_dim;
  int64_t pool_slots;
  bool f32;
};
int launch_append_rope(const AppendArgs& a, void* stream);

// Raise a kernel's dynamic shared-memory limit to `bytes` on the current
// device, once per (kernel, device); thread-safe.  Returns a cudaError_t.
int ensure_dynamic_smem(const void* kernel, int bytes);

// Per-thread host staging for a launch's parameter block (large structs that
// are filled, then copied into the launch): one heap copy per thread, freed
// when the thread exits.
template <typename T>
T& thread_staging() {
  static thread_local std::unique_ptr<T> buf;
  if (!buf) buf.reset(new T());
  return *buf;
}

// Tracing hooks (trace.cpp): trace_start before a call's first launch,
// trace_mark after each launch (no-ops unless tracing is on).
void trace_start(void* stream);
void trace_mark(int kernel, void* stream);

// Whether the tensor-core prefill supports this shape (prefill_tc.cu).
bool prefill_tc_supported(int32_t head_dim, int32_t page_size, int32_t group);
// Whether the SM-pair prefill supports this shape (prefill_pair.cu).
bool prefill_pair_supported(int32_t head_dim, int32_t page_size, int32_t group);
// Device address of the fixed no-allocation scratch array on the current
// device (decode.cu); resolved on the first call per device.
int noalloc_scratch(void** ptr);

// Whether the split-KV decode supports this shape (decode.cu).
bool decode_supported(int32_t head_dim, int32_t group, int32_t page_size);
// Whether its tensor-core kernel does (decode_tc.cu), and that kernel's
// launcher (launch_decode hands over to it when plan.decode_tc is set).
bool decode_tc_supported(int32_t head_dim, int32_t group, int32_t page_size, bool kv_fp8);
int launch_decode_tc(const Plan& plan, const Args& a, void* stream);

// TMA tensor maps (tmap.cpp): a 3-D bf16 tensor [outer][mid][d] with a
// 128-byte-swizzled box of (64, box_mid, box_outer) elements.
bool tmap_available();
bool make_tmap_3d(CUtensorMap* m, const void* base, uint64_t d, uint64_t mid, uint64_t outer,
                  uint32_t box_mid, uint32_t box_outer);
// The same tensor as 4-D (64-element chunks outermost): one box brings every
// chunk of box_outer rows, landing as [chunk][row][128 B] (bytes for fp8).
bool make_tmap_4d_chunks(CUtensorMap* m, const void* base, uint64_t d, uint64_t mid,
                         uint64_t outer, uint32_t box_mid, uint32_t box_outer, bool fp8);
// The same over a byte tensor (fp8 pages), box (128, box_mid, box_outer).
bool make_tmap_3d_u8(CUtensorMap* m, const void* base, uint64_t d, uint64_t mid, uint64_t outer,
                     uint32_t box_mid, uint32_t box_outer);

}  // namespace rpa
