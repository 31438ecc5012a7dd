// Attention of drafted trees on tensor cores (tcgen05 + TMA), split over the keys.
//
// A node sees its request's whole context (within its window) and, of the tree, the
// nodes of its mask.  The 128 rows of an MMA are 128 / G nodes by the G query heads
// of one KV head; a segment is (request, KV head, one such row tile, or two where
// head_dim leaves tensor memory for two outputs), its keys come in tiles of 128.
// plan_tree.cpp lays the segments' tiles end to end (where a head has several segments,
// these side by side) and cuts the line into equal ranges, one per CTA, one CTA per SM:
// few rows over long contexts are bound by HBM, and only all SMs together reach it.  A
// CTA's range is a list of parts of segments; a part that is not its whole segment leaves
// fp32 O / l and log2-sum-exps, which tree_combine_kernel joins.
//
// Within a part the score tile S = Q K^T (SMEM x SMEM -> TMEM) runs one ahead of
// O += P V (P from TMEM, written over half of its S; V MN-major from SMEM).  With two
// streams (head_dim 64 and 128) two softmax warpgroups take the score tiles by turns, each with
// an S buffer and an O of its own:
//   two row tiles: a stream per row tile, both fed from the same K and V stages;
//   one row tile: the streams take the key tiles by turns and merge at the part's
//   end (by the maxima and sums that they swap through shared memory).
// At head_dim 256 one O fills half of tensor memory: one stream, two S buffers.
//
// Warps: 0 copies Q, K and V (TMA boxes through the page table, into one ring in the
// order of their use), 2 issues the MMAs, 1 and 3 make V safe (below), 4 on are the
// softmax warpgroups, a thread per row; each writes its rows at the part's end while the
// copies run on into the ring.
//
// Masks are looked up where a tile holds nodes or a window's edge; 128 bits a row.
// A product gives 0 * NaN to the rows that do not see a key, so in those tiles a warp
// goes over V before the MMA reads it: rows of keys that no node sees become zero,
// and of the others each NaN or infinity, which the rows that see it then get back
// from memory after they are written (add_unseen).
//
// Rounding: P to bf16 (2^-8 of itself; the sums take it unrounded), O / l to bf16.
// Every wait is bounded; see prefill_tc.cu for what follows when one gives up.
//
// What bounds it.  Long contexts, HBM: 32 requests of 16 to 48 nodes after 4k to 32k keys
// (32 heads of 128, 8 KV heads) read 2.17 GB in 362 us, 6.0 TB/s.  Many nodes, the tensor
// cores and the softmax between their products: 8 requests of 256 nodes (64 heads of 128)
// take 213 us, 1405 TFLOP/s; segments that need no cut run at 1790, and 10 us are the
// combine's.  128 requests of 8 nodes (8 heads of 256, one KV head) after 120 to 2040 keys:
// 37.4 us for 137 MB: 30 here (HBM's share of 22, the start, ranges that end apart), the
// rest the combine and its launch.
//
// Measured against this: no second MMA warp (one a stream: 326 us where 255 were, the two
// streams' products then wait for each other); no exponentials on the FMA pipe (its slots
// are the softmax's own); the loops' code kept short (a tile written out twice, for the
// raised reference and not: 251 us where 240 were; the instruction caches hold one).
#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "tree.cuh"

namespace rpa {
namespace {

using namespace sm100;

constexpr int kSub = 16384;  // a 64-dimension chunk of 128 keys of K, or 8192 / D keys of V
// A row's weights are 2^(score - reference).  The reference is kAbove over the maximum of the
// first tile that the row sees; when a later tile's maximum passes it, it goes up to kAbove over
// that one.  So the weights need not wait for a tile's maximum: they are worked out under the
// reference while the maximum is taken, and worked out again in the rare case.  Weights stay
// at 1 or below, so O stays in the range of 32 bits (bf16 has the same) while the row's keys
// times the largest value do, as on CUDA cores.  (8 and 16 take the same times.)
constexpr float kAbove = 8.f;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;

// A wait (mbar_wait) of a converged warp, which agrees on the answer; what follows a phase that
// is not complete yet stays out of the way of the caller's code.  kWho: callers that
// differ in their registers have functions of their own.
template <int kWho>
__device__ __noinline__ bool warp_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit_ns));
}
template <int kWho>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
  return warp_wait_slow<kWho>(bar, parity, abort, limit_ns);
}

template <int N>
struct TreeWork {
  TreeSeqs<N> seqs;
  TreeStart start[kTreeMaxCtas];
};

struct TreeParams {
  const int32_t* page_table;
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  const uint64_t* mask;
  const int32_t* positions;
  const __nv_bfloat16* v_pages;
  __nv_bfloat16* out;
  float* part_o;    // [slot][D / 8][row][8]
  float* part_lse;  // [slot][row]
  unsigned char* ws;
  int32_t hq, hkv, group, per_tile;  // nodes a row tile
  int32_t page_size, page_shift, mpps, num_pages, words;
  int32_t box_nodes_q, box_rows_k, box_rows_v, v_4d, out_v8, width;  // width: lanes of a group of CTAs
  float scale_log2;  // sm_scale log2(e)
};

template <int D>
struct Layout {
  static constexpr int kStreams = tree_row_tiles(D);
  static constexpr int kThreads = 128 + 128 * kStreams;
  // Registers a thread with two streams (setmaxnreg), within the launch's 384 x 168; the
  // 256 threads of one stream may have 255 each as they are.
  static constexpr int kRegsCtl = 104, kRegsSoftmax = 200;
  static_assert(kStreams == 1 || 128 * kRegsCtl + 256 * kRegsSoftmax <= 384 * 168, "registers");
  static constexpr int kChunks = D / 64;         // 128-byte pieces of a row; 16 KB pieces of a tile, of K and of V
  static constexpr int kVKeys = 8192 / D;        // keys of such a piece of V
  // One ring for K and V, filled in the order in which the MMAs take them: a slot is a
  // tile of K or of V, or half of one of 256 dimensions.
  static constexpr int kSubs = D == 64 ? 1 : 2, kSlots = kChunks / kSubs, kSlot = kSubs * kSub;
  static constexpr int kDepth = D == 64 ? 12 : 5;
  static constexpr int kQTile = kTreeRows * D * 2;
  static constexpr int kRingOff = kStreams * kQTile;
  static constexpr int kBarOff = kRingOff + kDepth * kSlot;
  static constexpr int kXchOff = kBarOff + 512;  // [stream][row] (maximum, sum)
  static constexpr int kUsed = kXchOff + (kStreams == 2 ? 2 * kTreeRows * 8 : 0);
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;  // one CTA per SM
  static_assert(kUsed <= 227 * 1024, "more shared memory than one CTA may have");
  // Tensor memory: the streams' O, then two S buffers of 128 columns.
  static constexpr int kSCol = kStreams * D;
  static constexpr int kCols = 512;
  static_assert(kSCol + 256 <= kCols, "tensor memory");
};

struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t full[12], empty[12];
  uint64_t s_full[2], p_most[2], p_full[2];
  uint64_t o_done[2];       // one stream: a product of each S buffer; two: [0], the part's products
  uint64_t o_free;          // every row of the part's O has been read
  uint64_t xch;             // the streams' maxima and sums are posted
  uint64_t v_ask[2], v_safe[2];  // by turns: a masked tile's V is on its way / may be read
  uint64_t fin;
  uint32_t tmem_base;
  int abort;
  int32_t poison[2];        // 1 + the part of this parity in which something was taken out of V
};
static_assert(sizeof(Barriers) <= 512, "barrier block");

// A part of a segment.
struct Part {
  TreeSeq s;
  int32_t head, node0, n0, n1;  // first node, nodes of the first and the second row tile
  int32_t key0, n;              // first key, key tiles
  int32_t lo;                   // first key that any node can see
  int32_t masked_below, masked_from;  // tiles that begin below or end behind these are masked
  bool whole;
  __device__ __forceinline__ bool masked(int32_t key) const { return key < masked_below || key + kTreeKeys > masked_from; }
};

// A CTA's parts, in order.
template <int D, int N>
struct Walk {
  int32_t i, head, st, j, left;
  __device__ __forceinline__ explicit Walk(const TreeWork<N>& w) {
    const TreeStart& s = w.start[blockIdx.x];
    i = s.i;
    head = s.head;
    st = s.st;
    j = s.j;
    left = s.tiles;
  }
  __device__ __forceinline__ bool next(const TreeWork<N>& w, const TreeParams& p, Part& a) {
    if (left <= 0) return false;
    a.s = w.seqs.s[i];
    const int32_t per = p.per_tile * Layout<D>::kStreams, first = tree_first_tile(a.s);
    const int32_t nb = (a.s.len - 1) / kTreeKeys + 1 - first;
    a.head = head;
    a.node0 = st * per;
    a.n0 = min(p.per_tile, a.s.nodes - a.node0);
    a.n1 = Layout<D>::kStreams == 2 ? max(0, min(p.per_tile, a.s.nodes - a.node0 - p.per_tile)) : 0;
    a.n = min(left, nb - j);
    a.key0 = (first + j) * kTreeKeys;
    a.whole = a.n == nb;
    const int32_t ctx = a.s.len - a.s.nodes, w0 = a.s.window;
    a.lo = w0 > 0 ? max(0, ctx - w0 + 1) : 0;
    a.masked_below = w0 > 0 ? min(ctx, a.s.len - w0) : 0;
    a.masked_from = ctx;
    left -= a.n;
    j += a.n;
    if (j == nb) {
      j = 0;
      // The lane's next segment; a request begins with a new pass.
      st += p.width;
      while (left > 0 && st >= w.seqs.s[i].per_head) {
        st -= w.seqs.s[i].per_head;
        if (++head == p.hkv) {
          head = 0;
          st = w.start[blockIdx.x].lane;
          ++i;
        }
      }
    }
    return true;
  }
};

// TMA source row of the box of `rows` keys from `key` on (in one page); -rows, which
// is filled with zeros, where no node sees any of them or the page is not one.
__device__ __forceinline__ int32_t box_row(const TreeParams& p, const Part& a, int32_t key, int32_t rows) {
  if (key >= a.s.len || key + rows <= a.lo) return -rows;
  const int32_t page = __ldg(p.page_table + static_cast<int64_t>(a.s.seq) * p.mpps + (key >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    report_error(p.ws, RPA_DEVERR_PAGE_ID, a.s.seq);
    return -rows;
  }
  return page * p.page_size + (key & (p.page_size - 1));
}

// Whether one of two bf16 is NaN or infinite, and the two without such ones.
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// 16 KB of V ([chunk][key][128 B]) of keys from `key` on made safe (whole warp); true
// where a NaN or an infinity of a visible key was taken out.  Mostly there is none: a
// first pass takes the largest magnitude (its bits are in order) of everything.
template <int D>
__device__ __noinline__ bool make_safe(uint8_t* piece, int32_t key, int32_t lo, int32_t len, int lane) {
  constexpr int kVKeys = Layout<D>::kVKeys, kUnits = kSub / 16;
  uint4* at = reinterpret_cast<uint4*>(piece);
  auto row_of = [&](int u) { return (u >> 3) & (kVKeys - 1); };
  const int32_t a = max(0, min(kVKeys, lo - key)), b = max(0, min(kVKeys, len - key));  // rows [a, b) are visible
  uint32_t top = 0;
#pragma unroll 1
  for (int u0 = 0; u0 < kUnits; u0 += 32 * 8) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = at[u0 + 32 * i + lane];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = __vmaxu2(__vmaxu2(__vmaxu2(top, v[i].x & 0x7fff7fffu), v[i].y & 0x7fff7fffu),
                     __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
  }
  const bool any = __any_sync(0xffffffffu, not_finite2(top));
  bool found = false;
  if (any) {
    for (int u = lane; u < kUnits; u += 32) {
      if (row_of(u) < a || row_of(u) >= b) continue;
      const uint4 v = at[u];
      if (not_finite2(v.x) || not_finite2(v.y) || not_finite2(v.z) || not_finite2(v.w)) {
        at[u] = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
        found = true;
      }
    }
    // Rows that nobody sees.
    for (int u = lane; u < kUnits; u += 32)
      if (row_of(u) < a || row_of(u) >= b) at[u] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  return __any_sync(0xffffffffu, found);
}

// The bits of 128 keys (tree_sees32), out of the way of the tiles that need none.
__device__ __noinline__ uint4 tree_sees128(int32_t len, int32_t nodes, const uint64_t* row, int32_t lo, int32_t key) {
  const TreeSeq s{0, 0, len, 0, static_cast<uint16_t>(nodes), 0};
  return make_uint4(tree_sees32(s, row, lo, key), tree_sees32(s, row, lo, key + 32), tree_sees32(s, row, lo, key + 64),
                    tree_sees32(s, row, lo, key + 96));
}

// What make_safe took out of the part's tiles and this row sees, added to what was
// stored of columns [c0, c1) (T: bf16 outputs or fp32 partials; every eight of a row's
// columns lie `step` elements behind the eight before).
template <typename T>
__device__ __noinline__ void add_unseen(const TreeParams& p, const Part a, const uint64_t* mask_row, int32_t first,
                                        int32_t d, int32_t c0, int32_t c1, T* row, int32_t step) {
  for (int32_t k0 = a.key0; k0 < a.key0 + a.n * kTreeKeys; k0 += kTreeKeys) {
    if (!a.masked(k0)) continue;
    for (int32_t k = k0; k < min(k0 + kTreeKeys, a.s.len); k += 32) {
      for (uint32_t bits = tree_sees32(a.s, mask_row, first, k); bits; bits &= bits - 1) {
        const int32_t key = k + __ffs(bits) - 1;
        if (key >= a.s.len) break;
        const int32_t from = box_row(p, a, key, 1);
        if (from < 0) continue;
        const __nv_bfloat16* v = p.v_pages + (static_cast<int64_t>(from) * p.hkv + a.head) * d;
        for (int32_t c = c0; c < c1; ++c) {
          const float x = to_float(v[c]);
          T* at = row + (c >> 3) * step + (c & 7);
          if (!(fabsf(x) < INFINITY)) *at = from_float<T>(to_float(*at) + x);
        }
      }
    }
  }
}

// The largest of N floats (their bits), as a tree of three-input maxima.
template <int N>
__device__ __forceinline__ float max_tree(const uint32_t* v) {
  if constexpr (N == 1) {
    return __uint_as_float(v[0]);
  } else if constexpr (N == 2) {
    return fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
  } else {
    constexpr int M = (N + 2) / 3;
    uint32_t t[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float a = __uint_as_float(v[3 * i]);
      float m = a;
      if (3 * i + 2 < N)
        m = fmax3(a, __uint_as_float(v[3 * i + 1]), __uint_as_float(v[3 * i + 2]));
      else if (3 * i + 1 < N)
        m = fmaxf(a, __uint_as_float(v[3 * i + 1]));
      t[i] = __float_as_uint(m);
    }
    return max_tree<M>(t);
  }
}

// One 32-byte store, or two 16-byte ones.
__device__ __forceinline__ void store32(void* dst, bool whole, const uint32_t (&w)[8]) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The ring's next slot and its phase.
template <int kDepth>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kDepth) {
      slot = 0;
      phase ^= 1;
    }
  }
};

template <int D, int N>
__global__ void __launch_bounds__(Layout<D>::kThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p,
                 const __grid_constant__ TreeWork<N> work) {
  using Lay = Layout<D>;
  constexpr int kChunks = Lay::kChunks, kStreams = Lay::kStreams, kSubs = Lay::kSubs, kSlots = Lay::kSlots;
  constexpr int kDepth = Lay::kDepth;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {
    if (threadIdx.x == 0) report_error(p.ws, RPA_DEVERR_LAUNCH, blockIdx.x);
    return;
  }
  // The combine may be scheduled now; it waits for this grid.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Barriers& B = *reinterpret_cast<Barriers*>(smem + Lay::kBarOff);
  volatile int* abort = &B.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&B.q_full, 1);
    mbar_init(&B.q_empty, 1);
    for (int i = 0; i < kDepth; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_most[i], 4);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.o_done[i], 1);
      mbar_init(&B.v_ask[i], 1);
      mbar_init(&B.v_safe[i], 2);
      B.poison[i] = 0;
    }
    mbar_init(&B.o_free, 4 * kStreams);
    mbar_init(&B.xch, 8);
    mbar_init(&B.fin, 1);
    B.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 2) {
    tmem_alloc(&B.tmem_base, Lay::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // What came before on the stream has ended (this launch may be early: the barriers and
  // tensor memory are set up while it ends).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = B.tmem_base;
  Walk<D, N> walk(work);
  Part a{};
  if (warp < 4) {
  if constexpr (kStreams == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Lay::kRegsCtl));
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait<0>(bar, parity, abort, kWaitNs); };
  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const int rows_k = p.box_rows_k, rows_v = p.box_rows_v;
    const int nk = kTreeKeys / rows_k, nv = Lay::kVKeys / rows_v;  // boxes of 16 KB
    // Q's boxes: 32 rows where these are whole nodes, and those without a node are zeros, for
    // which the tensor cores take less power: run for seconds, 32 long contexts take 382 us
    // at 1780 MHz, 401 at 1660 with rows of the nodes that follow; 128 requests of 8 nodes
    // draw 897 W in place of 978.
    const int q_nodes = p.box_nodes_q, q_rows = p.group * q_nodes;
    int q_used[2] = {kTreeRows / q_rows, kTreeRows / q_rows};  // boxes that are not zeros
    auto boxes_of = [&](int nodes) { return (nodes + q_nodes - 1) / q_nodes; };
    // (Nothing waits for it: nobody reads what becomes of these rows.)
    auto clear_q = [&](int t, int boxes) {
      uint8_t* tile = smem + t * Lay::kQTile;
      const int32_t from = boxes * q_rows * 8, units = (q_used[t] - boxes) * q_rows * 8;  // of 16 bytes
      for (int32_t u = lane; u < units; u += 32)
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          reinterpret_cast<uint4*>(tile + c * (kTreeRows * 128))[from + u] = make_uint4(0u, 0u, 0u, 0u);
      if (units > 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      q_used[t] = boxes;
    };
    auto copy_q = [&](int t, int boxes) {
      for (int x = lane; x < boxes * kChunks; x += 32) {
        const int c = x % kChunks, b = x / kChunks;
        tma_load_3d(smem + t * Lay::kQTile + c * (kTreeRows * 128) + b * q_rows * 128, &tm_q, &B.q_full, c * 64,
                    a.head * p.group, a.s.q0 + a.node0 + t * p.per_tile + b * q_nodes);
      }
    };
    Ring<kDepth> ring;
    uint32_t filled = 0, parts = 0, issued_q = 0;
    bool alive = true;
    // The next slot, empty, with its bytes announced.
    auto take = [&]() -> bool {
      if (lane == 0) alive = mbar_wait(&B.empty[ring.slot], ring.phase ^ 1, abort, kWaitNs);
      alive = __shfl_sync(0xffffffffu, alive, 0);
      if (!alive) return false;
      if (lane == 0) mbar_arrive_expect_tx(&B.full[ring.slot], Lay::kSlot);
      ++filled;
      __syncwarp();
      return true;
    };
    // A tile's source rows, one box a lane: of K, and of each 16 KB of V.
    struct Rows {
      int32_t k, v[kChunks];
    };
    auto rows_of = [&](int j) -> Rows {
      Rows r;
      const int32_t k0 = a.key0 + j * kTreeKeys;
      r.k = lane < nk ? box_row(p, a, k0 + lane * rows_k, rows_k) : 0;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        r.v[c] = lane < nv ? box_row(p, a, k0 + c * Lay::kVKeys + lane * rows_v, rows_v) : 0;
      return r;
    };
    auto copy_k = [&](const Rows& r) -> bool {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c % kSubs == 0 && !take()) return false;
        if (lane < nk)
          tma_load_3d(smem + Lay::kRingOff + ring.slot * Lay::kSlot + (c % kSubs) * kSub + lane * rows_k * 128, &tm_k,
                      &B.full[ring.slot], c * 64, a.head, r.k);
        if (c % kSubs == kSubs - 1) ring.step();
      }
      return true;
    };
    auto copy_v = [&](const Rows& r) -> bool {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c % kSubs == 0 && !take()) return false;
        uint8_t* dst = smem + Lay::kRingOff + ring.slot * Lay::kSlot + (c % kSubs) * kSub + lane * rows_v * 128;
        if (lane < nv) {
          if (p.v_4d) {
            tma_load_4d(dst, &tm_v, &B.full[ring.slot], 0, a.head, r.v[c], 0);
          } else {
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
              tma_load_3d(dst + x * Lay::kVKeys * 128, &tm_v, &B.full[ring.slot], x * 64, a.head, r.v[c]);
          }
        }
        if (c % kSubs == kSubs - 1) ring.step();
      }
      return true;
    };
    for (; alive && walk.next(work, p, a); ++parts) {
      const bool two = a.n1 > 0;
      // (Looked up before they are wanted.)
      Rows now = rows_of(0), next = now;
      if (lane == 0) {
        // (The device's lengths, once a request.)
        if (a.head == 0 && a.node0 == 0 && a.key0 + a.n * kTreeKeys >= a.s.len)
          tree_check_lengths(a.s, p.cu_q_lens, p.kv_lens, p.ws);
        alive = mbar_wait(&B.q_empty, (parts & 1) ^ 1, abort, kWaitNs);
      }
      alive = __shfl_sync(0xffffffffu, alive, 0);
      const int b0 = boxes_of(a.n0), b1 = kStreams == 2 && two ? boxes_of(a.n1) : 0;
      if (alive) {
        if (lane == 0) mbar_arrive_expect_tx(&B.q_full, static_cast<uint32_t>((b0 + b1) * q_rows) * 128u * kChunks);
        __syncwarp();
        copy_q(0, b0);
        if (kStreams == 2 && b1 > 0) copy_q(kStreams - 1, b1);
        ++issued_q;
      }
      // K runs a tile ahead of V where a score tile runs ahead of the product of the
      // tile before; with two row tiles it is the second one's that does.
      if (alive) alive = copy_k(now);
      clear_q(0, b0);
      if (kStreams == 2 && two) clear_q(kStreams - 1, b1);
      for (int j = 0; j < a.n && alive; ++j) {
        if (j + 1 < a.n) next = rows_of(j + 1);
        if (!two && j + 1 < a.n && !copy_k(next)) break;
        if (!copy_v(now)) break;
        if (two && j + 1 < a.n && !copy_k(next)) break;
        now = next;
      }
    }
    if (!alive && lane == 0) {
      // Every copy lands before its shared memory goes.
      report_error(p.ws, RPA_DEVERR_TIMEOUT, blockIdx.x);
      int none = 0;
      for (uint32_t t = filled > kDepth ? filled - kDepth : 0; t < filled; ++t)
        mbar_wait(&B.full[t % kDepth], (t / kDepth) & 1, &none, kDrainNs);
      if (issued_q > 0) mbar_wait(&B.q_full, (issued_q - 1) & 1, &none, kDrainNs);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMAs
    // Between two score tiles and two products this warp has 1024 cycles of the tensor
    // cores (D = 128), and its instructions are fetched anew each time it goes on (the
    // softmax warps' code takes the caches): so few of them, in straight lines, each S
    // buffer with code of its own.
    constexpr uint32_t kIdS = idesc_bf16(kTreeKeys, 0), kIdPV = idesc_bf16(D, 1);
    // Operands differ from these in the start address alone (see prefill_tc.cu).
    const uint64_t q_d0 = smem_desc(smem_addr(smem), 16, 1024);
    const uint64_t k_d0 = smem_desc(smem_addr(smem + Lay::kRingOff), 16, 1024);
    const uint64_t v_d0 = smem_desc(smem_addr(smem + Lay::kRingOff), Lay::kVKeys * 128, 1024);
    Ring<kDepth> ring;
    uint32_t parts = 0, p_ph = 0;  // p_ph: a phase bit per S buffer
    bool alive = true;
    // S into buffer b from the K tile in `slot` (or the next slots) and row tile t.
    auto mma_s = [&](auto bc, int t, int slot) {
      constexpr int b = decltype(bc)::value;
      const uint32_t sc = tmem + Lay::kSCol + b * kTreeKeys;
      const uint64_t qd = q_d0 + static_cast<uint64_t>(t * (Lay::kQTile >> 4));
      const uint64_t kd = k_d0 + static_cast<uint64_t>(slot * (Lay::kSlot >> 4));
      if constexpr (D == 64)
        mma_ss_chunk(sc, qd, kd, kIdS, 0);
      else
        mma_ss_2chunks(sc, qd, kd, kIdS, 0);
    };
    // O += P V, P in buffer b, V in `slot`, the first 96 keys as soon as their part of P is
    // there; `acc` 0: the stream's first in the part.
    auto mma_pv = [&](auto bc, int slot, uint32_t acc) -> bool {
      constexpr int b = decltype(bc)::value;
      const uint32_t o = tmem + b * D, pc = tmem + Lay::kSCol + b * kTreeKeys;
      const uint64_t vd = v_d0 + static_cast<uint64_t>(slot * (Lay::kSlot >> 4));
      if (!wait(&B.p_most[b], p_ph >> b & 1u)) return false;
      tc_fence_after();
      constexpr uint64_t kHalf = D == 64 ? 512 : kSub / 16;  // 64 keys on
      mma_ts_64keys(o, pc, vd, kIdPV, acc);
      mma_ts2(o, pc + 32, pc + 40, vd + kHalf, vd + kHalf + 128, kIdPV, 1);
      if (!wait(&B.p_full[b], p_ph >> b & 1u)) return false;
      p_ph ^= 1u << b;
      tc_fence_after();
      mma_ts2(o, pc + 48, pc + 56, vd + kHalf + 256, vd + kHalf + 384, kIdPV, 1);
      return true;
    };
    // A masked tile's V: announced where the ring's slots of it hold nothing older that
    // has not landed (a tile ahead; for 256 dimensions, where half the ring is one tile, at
    // its own score tile), used once it is safe.
    uint32_t asked = 0, used_safe = 0;
    auto ask = [&]() {
      if (lane == 0) mbar_arrive(&B.v_ask[asked & 1]);
      ++asked;
    };
    auto safe = [&]() -> bool {
      const uint32_t k = used_safe++;
      return wait(&B.v_safe[k & 1], k >> 1 & 1);
    };
    using B0 = std::integral_constant<int, 0>;
    using B1 = std::integral_constant<int, 1>;
    while (alive && walk.next(work, p, a)) {
      if (!(alive = wait(&B.q_full, parts & 1))) break;
      auto masked = [&](int j) { return __builtin_expect(a.masked(a.key0 + j * kTreeKeys), 0); };
      if (kStreams == 2 && masked(0)) ask();
      alive = [&]() -> bool {
        if constexpr (kStreams == 2) {
          if (a.n1 > 0) {
            // Two row tiles: S(0, j), then S(1, j), O_0 += P(0, j) V(j), S(0, j + 1),
            // O_1 += P(1, j) V(j).
            if (!wait(&B.full[ring.slot], ring.phase)) return false;
            tc_fence_after();
            int ks = ring.slot;
            ring.step();
            mma_s(B0{}, 0, ks);
            mma_commit(&B.s_full[0]);
#pragma unroll 1
            for (int j = 0;; ++j) {
              const bool more = j + 1 < a.n;
              if (more && masked(j + 1)) ask();
              mma_s(B1{}, 1, ks);
              mma_commit(&B.s_full[1]);
              mma_commit(&B.empty[ks]);
              if (!more) mma_commit(&B.q_empty);
              if (masked(j) && !safe()) return false;
              if (!wait(&B.full[ring.slot], ring.phase)) return false;
              if (j == 0 && !wait(&B.o_free, (parts & 1) ^ 1)) return false;
              const int vs = ring.slot;
              ring.step();
              if (!mma_pv(B0{}, vs, j > 0)) return false;
              if (more) {
                if (!wait(&B.full[ring.slot], ring.phase)) return false;
                tc_fence_after();
                ks = ring.slot;
                ring.step();
                mma_s(B0{}, 0, ks);
                mma_commit(&B.s_full[0]);
              }
              if (!mma_pv(B1{}, vs, j > 0)) return false;
              mma_commit(&B.empty[vs]);
              if (!more) break;
            }
            mma_commit(&B.o_done[0]);
            return true;
          }
          // One row tile, its key tiles by turns: S(j + 1), O_(j % 2) += P(j) V(j).
          auto score = [&](auto bc) -> bool {
            if (!wait(&B.full[ring.slot], ring.phase)) return false;
            tc_fence_after();
            mma_s(bc, 0, ring.slot);
            mma_commit(&B.s_full[decltype(bc)::value]);
            mma_commit(&B.empty[ring.slot]);
            ring.step();
            return true;
          };
          auto product = [&](auto bc, int j) -> bool {
            if (j + 1 < a.n && masked(j + 1)) ask();
            if (masked(j) && !safe()) return false;
            if (!wait(&B.full[ring.slot], ring.phase)) return false;
            if (j == 0 && !wait(&B.o_free, (parts & 1) ^ 1)) return false;
            if (!mma_pv(bc, ring.slot, j > 1)) return false;
            mma_commit(&B.empty[ring.slot]);
            ring.step();
            return true;
          };
          if (!score(B0{})) return false;
          if (a.n == 1) mma_commit(&B.q_empty);
#pragma unroll 1
          for (int j = 0; j < a.n; j += 2) {
            if (j + 1 < a.n && !score(B1{})) return false;
            if (j + 2 == a.n) mma_commit(&B.q_empty);
            if (!product(B0{}, j)) return false;
            if (j + 1 >= a.n) break;
            if (j + 2 < a.n && !score(B0{})) return false;
            if (j + 3 == a.n) mma_commit(&B.q_empty);
            if (!product(B1{}, j + 1)) return false;
          }
          mma_commit(&B.o_done[0]);
          return true;
        } else {
          // One stream, tiles in halves: S(j + 1) into the other buffer, O += P(j) V(j).
          auto score = [&](int b) -> bool {
#pragma unroll
            for (int h = 0; h < kSlots; ++h) {
              if (!wait(&B.full[ring.slot], ring.phase)) return false;
              tc_fence_after();
              mma_ss_2chunks(tmem + Lay::kSCol + b * kTreeKeys, q_d0 + static_cast<uint64_t>(h * (2 * kSub >> 4)),
                             k_d0 + static_cast<uint64_t>(ring.slot * (Lay::kSlot >> 4)), kIdS, h > 0 ? 1u : 0u);
              mma_commit(&B.empty[ring.slot]);
              ring.step();
            }
            mma_commit(&B.s_full[b]);
            return true;
          };
          auto product = [&](int b, int j) -> bool {
            if (masked(j) && !safe()) return false;
            if (j == 0 && !wait(&B.o_free, (parts & 1) ^ 1)) return false;
#pragma unroll
            for (int h = 0; h < kSlots; ++h) {
              if (!wait(&B.full[ring.slot], ring.phase)) return false;
              if (!wait(h == 0 ? &B.p_most[b] : &B.p_full[b], p_ph >> b & 1u)) return false;
              tc_fence_after();
              mma_ts_2x32keys(tmem, tmem + Lay::kSCol + b * kTreeKeys + 32 * h,
                              v_d0 + static_cast<uint64_t>(ring.slot * (Lay::kSlot >> 4)), kIdPV,
                              j > 0 || h > 0 ? 1u : 0u);
              mma_commit(&B.empty[ring.slot]);
              ring.step();
            }
            p_ph ^= 1u << b;
            mma_commit(&B.o_done[b]);
            return true;
          };
          if (!score(0)) return false;
          if (a.n == 1) mma_commit(&B.q_empty);
#pragma unroll 1
          for (int j = 0; j < a.n; ++j) {
            if (masked(j)) ask();
            if (j + 1 < a.n && !score((j + 1) & 1)) return false;
            if (j + 2 == a.n) mma_commit(&B.q_empty);
            if (!product(j & 1, j)) return false;
          }
          return true;
        }
      }();
      ++parts;
    }
    // Every MMA issued finishes before tensor memory is released.
    mma_commit(&B.fin);
    int none = 0;
    mbar_wait(&B.fin, 0, &none, kDrainNs);
    __syncwarp();
    if (!alive && lane == 0) report_error(p.ws, RPA_DEVERR_TIMEOUT, blockIdx.x);
  } else {
    // ------------------------------------------------------------ V made safe
    // Warps 1 and 3, every second 16 KB each.
    const int half = warp >> 1;
    uint32_t asked = 0, parts = 0;
    uint32_t base = 0;  // slots filled before the part
    bool alive = true;
    for (; alive && walk.next(work, p, a); ++parts) {
      for (int j = 0; j < a.n; ++j) {
        const int32_t k0 = a.key0 + j * kTreeKeys;
        if (!a.masked(k0)) continue;
        if (!(alive = wait(&B.v_ask[asked & 1], asked >> 1 & 1))) break;
        // The tile's place among the part's (see the copies).
        const uint32_t at = base + (a.n1 > 0 || j == a.n - 1 ? 2 * j + 1 : 2 * j + 2) * kSlots;
        bool found = false;
        for (int c = half; c < kChunks && alive; c += 2) {
          const uint32_t n = at + c / kSubs;
          if (!(alive = wait(&B.full[n % kDepth], n / kDepth & 1))) break;
          found |= make_safe<D>(smem + Lay::kRingOff + n % kDepth * Lay::kSlot + (c % kSubs) * kSub,
                                k0 + c * Lay::kVKeys, a.lo, a.s.len, lane);
        }
        if (!alive) break;
        __syncwarp();
        if (lane == 0) {
          if (found) *reinterpret_cast<volatile int32_t*>(&B.poison[parts & 1]) = static_cast<int32_t>(parts) + 1;
          mbar_arrive(&B.v_safe[asked & 1]);
        }
        ++asked;
      }
      base += 2u * a.n * kSlots;
    }
    if (!alive && lane == 0) report_error(p.ws, RPA_DEVERR_TIMEOUT, blockIdx.x);
  }
  } else {
    if constexpr (kStreams == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Lay::kRegsSoftmax));
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait<1>(bar, parity, abort, kWaitNs); };
    // ------------------------------------------------------------ softmax and output
    const int w = kStreams == 2 ? (warp - 4) >> 2 : 0;  // stream
    const int q4 = warp & 3, r = 32 * q4 + lane;        // lane quarter, row
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const int G = p.group, tok = r / G, hd = r - tok * G;
    const float c = p.scale_log2;
    uint32_t used = 0;  // operations seen of each S buffer, modulo 2: a bit each
    uint32_t parts = 0, merges = 0;
    bool alive = true;
    // A warp's arrival, after what its lanes have done.
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (; alive && walk.next(work, p, a); ++parts) {
      const bool two = a.n1 > 0;
      const int tile_w = two ? w : 0;                     // row tile of this warp
      const int nodes = tile_w ? a.n1 : a.n0;
      const bool valid = tok < nodes && tok < p.per_tile;
      const int32_t node = a.s.q0 + a.node0 + tile_w * p.per_tile + tok;
      const uint64_t* mask_row = p.mask + static_cast<int64_t>(valid ? node : a.s.q0) * p.words;
      const int32_t first = valid ? tree_first_key(a.s, p.positions, node, p.ws) : 0;
      const bool some = __any_sync(0xffffffffu, valid);
      // This stream's operations: all, or every second one.
      const int ops = two ? 2 * a.n : a.n, step = kStreams;
      float m_ref = -INFINITY, l = 0.f;
      int mine = 0, last_b = 0;
      for (int op = w; op < ops; op += step, ++mine) {
        const int b = op & 1;
        // (The mask's words come while the scores are awaited.)
        const int32_t key = a.key0 + (two ? op >> 1 : op) * kTreeKeys;
        const bool masked = a.masked(key);
        uint4 bits = make_uint4(0u, 0u, 0u, 0u);
        if (__builtin_expect(masked, 0)) {
          if (valid) bits = tree_sees128(a.s.len, a.s.nodes, mask_row, first, key);
          __syncwarp();
        }
        if (!(alive = wait(&B.s_full[b], used >> b & 1u))) break;
        last_b = b;
        used ^= 1u << b;
        tc_fence_after();
        if (__builtin_expect(!some, 0)) {  // no row of this warp is one: its P may be anything
          tc_fence_before();
          arrive(&B.p_most[b]);
          arrive(&B.p_full[b]);
          continue;
        }
        const uint32_t s_col = lane_addr + Lay::kSCol + b * kTreeKeys;
        uint32_t sr[4][32], pk[2][16];
        const uint64_t c2 = f2_pack(c, c);
        uint64_t acc, nm2;
        // P over the first half of its scores, three quarters of it first: the product
        // starts on these while the others are exponentiated.
        auto weights = [&](const uint32_t (&x)[32], uint32_t (&w16)[16]) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t x2 =
                f2_fma(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, nm2);
            float x0, x1;
            f2_unpack(x2, x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            acc = f2_add(acc, f2_pack(p0, p1));
            w16[k] = pack_bf16x2(p0, p1);
          }
        };
#pragma unroll 1
        for (;;) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_col + 32 * i, sr[i]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_loaded(sr[i]);
          if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t seen = i == 0 ? bits.x : i == 1 ? bits.y : i == 2 ? bits.z : bits.w;
#pragma unroll
              for (int x = 0; x < 32; ++x) sr[i][x] = seen & 1u << x ? sr[i][x] : 0xff800000u;  // -inf
            }
          }
          float mx = max_tree<128>(&sr[0][0]);
          mx = mx == -INFINITY ? -INFINITY : mx * c;
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          acc = f2_pack(0.f, 0.f);
          nm2 = f2_pack(-m_use, -m_use);
          weights(sr[0], pk[0]);
          weights(sr[1], pk[1]);
          const bool grow = mx > m_ref;  // also for the first visible key
          if (__builtin_expect(!__any_sync(0xffffffffu, grow), 1)) break;
          // The reference goes up over the tile's maximum, and the tile is gone over again; O,
          // which holds earlier tiles, is scaled after the last of their products (with
          // two streams that was issued before this score tile, and ended with it).
          const float up = mx + kAbove, f = grow && m_ref != -INFINITY ? fast_exp2(m_ref - up) : 1.f;
          if (mine > 0) {
            if (kStreams == 1 && !(alive = wait(&B.o_done[b ^ 1], (used >> (b ^ 1) & 1u) ^ 1u))) break;
            tc_fence_after();
            const uint32_t o_col = lane_addr + (kStreams == 2 ? w * D : 0);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(o_col + c0, o);
              tmem_wait_ld();
              tmem_loaded(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st16(o_col + c0, o);
            }
            tmem_wait_st();
          }
          l *= f;
          if (grow) m_ref = up;
        }
        if (!alive) break;
        tmem_st16(s_col, pk[0]);
        tmem_st16(s_col + 16, pk[1]);
        weights(sr[2], pk[0]);
        tmem_st16(s_col + 32, pk[0]);
        tmem_wait_st();
        tc_fence_before();
        arrive(&B.p_most[b]);
        weights(sr[3], pk[1]);
        tmem_st16(s_col + 48, pk[1]);
        float a0, a1;
        f2_unpack(acc, a0, a1);
        l += a0 + a1;
        tmem_wait_st();
        tc_fence_before();
        arrive(&B.p_full[b]);
      }
      if (!alive) break;
      // The part's rows: this stream's, or half the columns of both streams' sum.
      if constexpr (kStreams == 2)
        alive = wait(&B.o_done[0], parts & 1);
      else
        alive = wait(&B.o_done[last_b], (used >> last_b & 1u) ^ 1u);
      if (!alive) break;
      tc_fence_after();
      const bool merge = kStreams == 2 && !two;
      float f0 = 1.f, f1 = 0.f, m = m_ref, sum = l;  // O = f0 O_0 + f1 O_1
      if (merge) {
        // (This part's products have ended, so the last part's values have been read.)
        float2* x = reinterpret_cast<float2*>(smem + Lay::kXchOff);
        if (mine > 0) x[w * kTreeRows + r] = make_float2(m_ref, l);
        tc_fence_before();
        arrive(&B.xch);
        if (!(alive = wait(&B.xch, merges & 1))) break;
        ++merges;
        tc_fence_after();
        const float2 e0 = x[r], e1 = ops > 1 ? x[kTreeRows + r] : make_float2(-INFINITY, 0.f);
        m = fmaxf(e0.x, e1.x);
        f0 = e0.y == 0.f ? 0.f : e0.x == m ? 1.f : fast_exp2(e0.x - m);
        f1 = e1.y == 0.f ? 0.f : e1.x == m ? 1.f : fast_exp2(e1.x - m);
        sum = f0 * e0.y + f1 * e1.y;
      }
      if (some) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        f0 *= inv;
        f1 *= inv;
        const int c0 = merge ? w * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
        const bool both = merge && ops > 1;  // (else the second O holds nothing of this part)
        const uint32_t o_col = lane_addr + (kStreams == 2 && !merge ? w * D : 0);
        __nv_bfloat16* out = p.out + (static_cast<int64_t>(node) * p.hq + a.head * G + hd) * D;
        // A partial's rows lie next to each other in pieces of eight columns: the warp's
        // stores, and the combine's loads, are whole lines.
        constexpr int kRows = kTreeRows * kStreams;
        const int64_t slot = 2ll * blockIdx.x + (parts > 0 ? 1 : 0);
        const int32_t row = tile_w * kTreeRows + r;
        float* part = p.part_o + slot * (kRows * D) + row * 8;
        // 32 columns of the row, as they come from tensor memory.
        auto store = [&](const uint32_t (&o)[32], int col) {
          if (!valid) return;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t t[8];
            if (a.whole) {
              if (i & 1) continue;
#pragma unroll
              for (int x = 0; x < 8; ++x)
                t[x] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * x]), __uint_as_float(o[8 * i + 2 * x + 1]));
              store32(out + col + 8 * i, p.out_v8, t);
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x) t[x] = o[8 * i + x];
              store32(part + (col / 8 + i) * (kRows * 8), true, t);
            }
          }
        };
        if constexpr (kStreams == 2) {
#pragma unroll 1
          for (int col = c0; col < c1; col += 32) {
            uint32_t o[32], o1[32];
            tmem_ld32(o_col + col, o);
            if (both) tmem_ld32(o_col + D + col, o1);
            tmem_wait_ld();
            tmem_loaded(o);
            if (both) {
              tmem_loaded(o1);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(fmaf(__uint_as_float(o[i]), f0, __uint_as_float(o1[i]) * f1));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
            }
            store(o, col);
          }
        } else {
          // The next columns load while these are stored.
          uint32_t o[32], o1[32];
          auto scale = [&](uint32_t (&x)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
          };
          tmem_ld32(o_col, o);
#pragma unroll 1
          for (int col = 0; col < D; col += 64) {
            tmem_wait_ld();
            tmem_loaded(o);
            tmem_ld32(o_col + col + 32, o1);
            scale(o);
            store(o, col);
            tmem_wait_ld();
            tmem_loaded(o1);
            if (col + 64 < D) tmem_ld32(o_col + col + 64, o);
            scale(o1);
            store(o1, col + 32);
          }
        }
        if (valid && !a.whole && (!merge || w == 0))
          p.part_lse[slot * kRows + row] = sum == 0.f ? -INFINITY : m + __log2f(sum);
        if (valid && *reinterpret_cast<volatile int32_t*>(&B.poison[parts & 1]) == static_cast<int32_t>(parts) + 1) {
          if (a.whole)
            add_unseen(p, a, mask_row, first, D, c0, c1, out, 8);
          else
            add_unseen(p, a, mask_row, first, D, c0, c1, part, kRows * 8);
        }
        __syncwarp();
      }
      tc_fence_before();
      arrive(&B.o_free);
    }
    if (!alive && lane == 0) report_error(p.ws, RPA_DEVERR_TIMEOUT, blockIdx.x);
  }
  // Every MMA is finished before tensor memory is released.
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, Lay::kCols);
  }
}

template <int N>
struct CutList {
  int32_t n;
  TreeCut cut[kTreeMaxCtas];
  TreeSeqs<N> seqs;
};

// The parts of each cut segment joined: out = sum_k 2^(lse_k - M) O_k / sum_k
// 2^(lse_k - M), M the largest lse_k.  A thread has 16 columns of a row, a warp those of
// 32 rows.  Many parts are shared out to several warps, which add up in shared memory (6
// parts of one request: 8.24 us in all, 8.57 by one warp).
// 38 MB of partials (8 requests of 256 nodes) take 10 us, the few rows of 128 requests of 8
// nodes 4.5, a launch and its reads.  Joined in the attention kernel by the last CTA of a
// segment to end, these two took 253 us in place of 241 and 42.9 in place of 37.6: a CTA
// has too few loads in flight.
constexpr int kCombineThreads = 256;
__host__ __device__ constexpr int combine_warps(int nparts) { return nparts <= 4 ? 1 : nparts <= 16 ? 4 : 8; }
template <int D, int N, bool kShared>
__global__ void __launch_bounds__(kCombineThreads, 4)
tree_combine_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CutList<N> list) {
  constexpr int kRows = kTreeRows * tree_row_tiles(D), kAtOnce = 2;
  const TreeCut& g = list.cut[blockIdx.x];
  const TreeSeq& s = list.seqs.s[g.i];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = kShared ? combine_warps(g.nparts) : 1, share = warp & (W - 1);
  const int unit = (blockIdx.y * 8 + warp) / W, rows32 = unit / (D / 16), col = unit % (D / 16) * 16;
  const int row = rows32 * 32 + lane, tile = row / kTreeRows, r = row % kTreeRows, tok = r / p.group;
  const int32_t node = (g.st * tree_row_tiles(D) + tile) * p.per_tile + tok;
  const bool valid = row < kRows && tok < p.per_tile && node < s.nodes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto slot = [&](int k) -> int64_t { return (2ll * (g.cta + k * p.width) + (k == 0 ? g.first : 0)) * kRows; };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float acc[16], sum = 0.f, M = -INFINITY;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  if (valid) {
    // Two parts at a time, by a running maximum; the loads of both come first.
    for (int k0 = share; k0 < g.nparts; k0 += kAtOnce * W) {
      float4 v[kAtOnce][4];
      float lse[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int k = k0 + q * W;
        lse[q] = -INFINITY;
        if (k >= g.nparts) continue;
        lse[q] = p.part_lse[slot(k) + row];
        const float* src = p.part_o + slot(k) * D + col * kRows + row * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[q][i] = *reinterpret_cast<const float4*>(src + (i >> 1) * (kRows * 8) + (i & 1) * 4);
      }
      float top = M;
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) top = fmaxf(top, lse[q]);
      if (top != M) {
        const float f = M == -INFINITY ? 0.f : fast_exp2(M - top);
        M = top;
        sum *= f;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] *= f;
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        if (lse[q] == -INFINITY) continue;
        const float w = lse[q] == M ? 1.f : fast_exp2(lse[q] - M);
        sum += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[4 * i] = fmaf(w, v[q][i].x, acc[4 * i]);
          acc[4 * i + 1] = fmaf(w, v[q][i].y, acc[4 * i + 1]);
          acc[4 * i + 2] = fmaf(w, v[q][i].z, acc[4 * i + 2]);
          acc[4 * i + 3] = fmaf(w, v[q][i].w, acc[4 * i + 3]);
        }
      }
    }
  }
  if (kShared && W > 1) {
    __shared__ float sums[kShared ? 8 : 1][17][32];
    // The shares' maxima, then their sums under the largest.
    sums[warp][16][lane] = M;
    __syncthreads();
    const int w0 = warp - share;
    float top = -INFINITY;
    for (int q = 0; q < W; ++q) top = fmaxf(top, sums[w0 + q][16][lane]);
    const float f = M == top ? 1.f : M == -INFINITY ? 0.f : fast_exp2(M - top);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[warp][i][lane] = acc[i] * f;
    sums[warp][16][lane] = sum * f;
    __syncthreads();
    if (share != 0) return;
    for (int q = 1; q < W; ++q) {
      if (q == 1) {
        sum = sums[w0][16][lane];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = sums[w0][i][lane];
      }
      sum += sums[w0 + q][16][lane];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] += sums[w0 + q][i][lane];
    }
  }
  if (!valid) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  store32(p.out + (static_cast<int64_t>(s.q0 + node) * p.hq + g.head * p.group + (r - tok * p.group)) * D + col,
          p.out_v8, t);
}

template <int D, int N>
int launch_one(const Plan& plan, const TreeLaunch& l, const CUtensorMap& tq, const CUtensorMap& tk,
               const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  using Lay = Layout<D>;
  if (int e = ensure_dynamic_smem(reinterpret_cast<const void*>(tree_attn_kernel<D, N>), Lay::kBytes)) return e;
  TreeWork<N>& w = thread_staging<TreeWork<N>>();
  w.seqs.n = l.seq_end - l.seq_begin;
  std::copy(plan.tree_seqs.begin() + l.seq_begin, plan.tree_seqs.begin() + l.seq_end, w.seqs.s);
  std::copy_n(plan.tree_starts.begin() + l.start_begin, l.n_ctas, w.start);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(l.n_ctas);
  cfg.blockDim = dim3(Lay::kThreads);
  cfg.dynamicSmemBytes = Lay::kBytes;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, N>, tq, tk, tv, p, w)) return static_cast<int>(e);
  trace_mark(RPA_KERNEL_TREE_ATTN, stream);
  if (l.n_cut == 0) return 0;
  CutList<N>& c = thread_staging<CutList<N>>();
  std::copy_n(plan.tree_cuts.begin() + l.cut_begin, l.n_cut, c.cut);
  std::copy_n(w.seqs.s, w.seqs.n, c.seqs.s);
  // Warps of the segment that wants most: 32 rows and 16 columns each, times the shares
  // of its parts.
  int64_t warps = 0;
  bool shared = false;
  for (int i = 0; i < l.n_cut; ++i) {
    shared |= combine_warps(c.cut[i].nparts) > 1;
    const int32_t nodes = std::min<int32_t>(w.seqs.s[c.cut[i].i].nodes - c.cut[i].st * p.per_tile * Lay::kStreams,
                                   p.per_tile * Lay::kStreams);
    const int32_t rows = nodes > p.per_tile ? kTreeRows + (nodes - p.per_tile) * p.group : nodes * p.group;
    warps = std::max<int64_t>(warps, static_cast<int64_t>((rows + 31) / 32) * (D / 16) * combine_warps(c.cut[i].nparts));
  }
  cfg.gridDim = dim3(l.n_cut, static_cast<unsigned>((warps + 7) / 8));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.dynamicSmemBytes = 0;
  if (cudaError_t e = shared ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, N, true>, p, c)
                             : cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, N, false>, p, c))
    return static_cast<int>(e);
  trace_mark(RPA_KERNEL_TREE_COMBINE, stream);
  return 0;
}

template <int D>
int launch_d(const Plan& plan, const Args& a, cudaStream_t stream) {
  using Lay = Layout<D>;
  const int G = plan.hq / plan.hkv;
  TreeParams p;
  p.page_table = a.page_table;
  p.cu_q_lens = a.cu_q_lens;
  p.kv_lens = a.kv_lens;
  p.mask = a.tree_mask;
  p.positions = a.positions;
  p.v_pages = static_cast<const __nv_bfloat16*>(a.v_pages);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.part_o = reinterpret_cast<float*>(a.workspace + plan.off_partial_o);
  p.part_lse = reinterpret_cast<float*>(a.workspace + plan.off_partial_lse);
  p.ws = a.workspace;
  p.hq = plan.hq;
  p.hkv = plan.hkv;
  p.group = G;
  p.per_tile = kTreeRows / G;
  p.page_size = plan.p;
  p.page_shift = 0;
  while ((1 << p.page_shift) < plan.p) ++p.page_shift;
  p.mpps = plan.mpps;
  p.num_pages = plan.num_pages;
  p.words = plan.tree_words;
  // A quarter of a row tile a box of Q where a quarter's rows are whole nodes (else the tile:
  // its last rows then hold what follows in q, and nobody reads what becomes of them).
  p.box_nodes_q = p.per_tile * G == kTreeRows && p.per_tile % 4 == 0 ? p.per_tile / 4 : p.per_tile;
  // Boxes never cross a page (32 contexts of 4k to 32k keys: 489 us with pages of 16, 375 with
  // 32, 362 with 64).
  p.box_rows_k = std::min(plan.p, 64);  // (the last tile's second half often lies behind the keys)
  p.box_rows_v = std::min(plan.p, Lay::kVKeys);
  // A V stage in one page takes all its 64-dimension chunks in one box (128 requests of 8
  // nodes: 38.1 us, 38.6 with a box a chunk).
  p.v_4d = Lay::kChunks > 1 && p.box_rows_v == Lay::kVKeys ? 1 : 0;
  p.out_v8 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 ? 1 : 0;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  CUtensorMap tq, tk, tv;
  const uint64_t pool_rows = static_cast<uint64_t>(plan.num_pages) * plan.p;
  if (!make_tmap_3d(&tq, a.q, D, plan.hq, static_cast<uint64_t>(plan.total_q), G, p.box_nodes_q) ||
      !make_tmap_3d(&tk, a.k_pages, D, plan.hkv, pool_rows, 1, p.box_rows_k) ||
      !(p.v_4d ? make_tmap_4d_chunks(&tv, a.v_pages, D, plan.hkv, pool_rows, 1, p.box_rows_v, false)
               : make_tmap_3d(&tv, a.v_pages, D, plan.hkv, pool_rows, 1, p.box_rows_v)))
    return static_cast<int>(cudaErrorInvalidValue);
  for (const TreeLaunch& l : plan.tree_launches) {
    p.width = l.width;
    const int e = l.seq_end - l.seq_begin <= kTreeSeqsSmall
                      ? launch_one<D, kTreeSeqsSmall>(plan, l, tq, tk, tv, p, stream)
                      : launch_one<D, kTreeSeqsLarge>(plan, l, tq, tk, tv, p, stream);
    if (e) return e;
  }
  return 0;
}

}  // namespace

bool tree_tc_supported(int32_t head_dim, int32_t page_size, int32_t group) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) && page_size >= 16 && group >= 1 &&
         group <= kTreeRows;
}

int launch_tree_attn(const Plan& plan, const Args& a, void* stream) {
  // (The maxima are taken before the scale, so it must not turn them round; and the infinity of
  // a masked score times zero would be NaN.)
  if (!(a.sm_scale * 1.4426950408889634f >= FLT_MIN)) return launch_tree_simt(plan, a, stream);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (plan.d) {
    case 64: return launch_d<64>(plan, a, s);
    case 128: return launch_d<128>(plan, a, s);
    case 256: return launch_d<256>(plan, a, s);
    default: return static_cast<int>(cudaErrorInvalidValue);
  }
}

}  // namespace rpa
