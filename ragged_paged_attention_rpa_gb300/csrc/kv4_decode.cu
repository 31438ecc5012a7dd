// Attention over 4-bit pages for sequences with few query rows (one decoded
// token, or a handful of drafted ones): split-KV, codes widened in registers.
//
// Work.  The query rows of a sequence that share a KV head (token-major, G
// heads a token) are cut into tiles of 8 or 16 rows; every (row tile, KV head)
// is a segment of blocks of 16 to 64 keys over the keys any of its rows sees.  The
// segments are laid end to end, each followed by a fixed charge for its merge,
// and the line is cut into equal ranges, one per CTA, one wave.
//
// CTA.  A warp takes a contiguous share of the CTA's range and meets the others
// once, at the range's end.  Per 16 keys it runs
//     S^T[16 keys x rows] = K . Q^T        (mma.m16n8k16, f16 -> fp32)
//     O^T[D x rows]     += V^T . P^T
// with an online softmax whose reference is 10 below the largest score when it
// is raised, which is when a score passes it by 15 (kv4_split.cuh: the
// probabilities stay at or below 2^15).
//
// Layout.  A product's order of terms is free, so which dimension a fragment's
// k index means is chosen such that a lane needs a contiguous run of bytes: of
// K rows g and g + 8 its quarter of the row (Q is fetched with the same
// permutation), of V its eighth of the rows of its four keys.  Every warp copies
// its own blocks with cp.async, a few ahead, into a ring of its own.
// Of V, two keys' codes are interleaved with two bit selects per eight codes
// before they are widened, which gives the register pairs along the keys that
// the second product wants without a transpose.
//
// Numbers.  Codes widen to f16 exactly, and times their scale they are still
// exact.  Q is bf16 made f16 after a power of two for the row (its largest
// element in [1, 2)): what rounds is below 2^-25 of the row's largest element.
// P is rounded to f16 for the second product: at most 2^-11 of itself down to
// 2^-24 of the score that the reference was raised for, 2^-35 of that below.
// Scores, maxima, sums and O are fp32.
//
// A key no row of the tile sees has its V scale set to zero (its bytes may be
// anything, a NaN scale included) and its scores replaced by -inf; a NaN at a key
// that only some rows see reaches those alone (kv4_split.cuh).  A bad page id
// sets the error word; its keys count as not seen.
//
// What bounds it: 0.5625 bytes an element come from HBM, and each element
// costs about one issue slot in 32 (widen, scale, multiply).  Long contexts run
// at HBM's rate: 32 tokens over 4096-32768 keys of 8 heads of 128 (727 MB)
// 125.6 us, 5.8 TB/s, with the schedulers 65% busy and no pipe above 50%; 152
// contexts of 16k keys of 256 dimensions 113.4 us, 6.3 TB/s; at 64 dimensions,
// where a row's scale and address work is shared by fewer elements, issue is the
// limit: 32 contexts of 8 heads 71.0 us, 5.1 TB/s.  Short ones are latency: 128
// tokens over 128-2048 keys of 256 (37.6 MB) take 20.2 us, of which 6 until the
// first data, 5-7 for the range, 4-6 for the merge and the combine (17.8 us where
// the pages are in L2); one token over 700 keys of 64 takes 7.0 us.  (Calls
// replayed from a graph, the inputs rotated past L2.)
#include <algorithm>
#include <type_traits>

#include "kv4_split.cuh"

namespace rpa {
namespace {

// What a warp holds of a segment it shares: blocks [j0, j1) of segment (e, g);
// e < 0: nothing.
struct Piece {
  int32_t e, g, j0, j1;
};

// Scale byte `i` (0 or 1) of s, whose upper half is zero, as f16 in both
// halves; and of two such words, in the low and the high half.
__device__ __forceinline__ uint32_t scale_dup(uint32_t s, int i) {
  return __byte_perm(s, 0, i == 0 ? 0x3030 : 0x3131) << 7;
}
__device__ __forceinline__ uint32_t scale_pair_of(uint32_t lo, uint32_t hi, int i) {
  return __byte_perm(lo, hi, i == 0 ? 0x3430 : 0x3531) << 7;
}

// Where 16 keys' rows of D / 2 bytes sit in shared memory: in order, as lines of
// 128 bytes, the eight 16-byte chunks of line n permuted by XOR with swz(n).  A
// copy instruction then fills four whole lines from 512 contiguous bytes, and
// the reads below meet every bank once.  (Each lane copying just what it reads
// itself costs a wavefront a lane instead of one for eight: 263 of them a
// 256-wide block of 16 keys, as long as all the rest of the block.)
template <int D>
struct RowLayout {
  static __device__ __forceinline__ uint32_t swz(uint32_t line) {
    return D == 256 ? line & 7 : D == 128 ? 2 * (line & 3) : 2 * (line & 1);
  }
  // Byte of the lane's chunk in the first copy instruction, and in the i-th.
  static __device__ __forceinline__ uint32_t copy_at(uint32_t lane) {
    return (lane >> 3) * 128 + ((lane & 7) ^ swz(lane >> 3)) * 16;
  }
  static __device__ __forceinline__ uint32_t copy_step(uint32_t at, int i) {
    return i * 512 + (D == 256 && (i & 1) ? at ^ 64 : at);  // lines 4 on: swz of 256-wide rows + 4
  }
  // Byte `at` (a multiple of what is read) of row r.
  static __device__ __forceinline__ uint32_t byte(uint32_t r, uint32_t at) {
    const uint32_t b = r * (D / 2) + at, line = b >> 7;
    return line * 128 + (((b >> 4 & 7) ^ swz(line)) * 16) + (b & 15);
  }
};

// Shapes of an instance: D, NT tiles of 8 rows, W warps a CTA, SUB 16-key parts
// a block, S blocks in flight a warp.  One CTA a SM: of two or three, the SM
// serves the oldest first (with equal shares of the 32 long contexts the first
// CTAs of the SMs ended after 112 us, the second after 130 us), while the warps
// of one CTA end together.  O takes D NT / 4 registers of a thread and Q D NT / 8;
// blocks of 32 keys halve the cost of the loop around the products and give a
// warp two independent chains of them.  Measured (warps x keys a block, each
// with the registers it leaves): 256 dimensions 8 x 32 6.35 TB/s of 4-bit pages
// over 152 contexts of 16k, 12 x 16 6.02, 16 x 16 6.16 with spills, 12 x 32
// spills; 128 dimensions 12 x 32 5.80 over 32 long contexts, 16 x 32 5.75,
// 16 x 16 5.29; 64 dimensions 16 x 64 4.60 over 32 long contexts, 16 x 32 4.22;
// 10 or 14 warps, which the four schedulers cannot share evenly,
// 5 to 11% below their neighbours.
// Two blocks in flight a warp are enough: more only make the first ones wait
// (the 32 long contexts took 132.4 us with three, 129.7 us with two).
template <int D_, int NT_>
struct Kv4Shape {
  static constexpr int D = D_, NT = NT_;
  static constexpr int W = D == 256 ? 8 : D == 128 ? 12 : 16;
  static constexpr int SUB = D * NT == 64 ? 4 : D == 128 && NT == 2 ? 1 : 2;
  static constexpr int S = 2;
  static constexpr int kBlk = 16 * SUB;
  static constexpr int kRows = 8 * NT;
  static constexpr int KC = D == 256 ? 2 : 1;   // chunks of a K row a lane
  static constexpr int KG = D / 8 / KC;         // bytes of such a chunk
  static constexpr int KW = KG / 4;             // words
  static constexpr int VG = D / 16;             // bytes of a V row a lane
  static constexpr int VW = VG / 4;
  static constexpr int MT = D / 16;             // 16-dimension tiles of O^T
  // A part of a stage: K, V, K scales, V scales of 16 keys.
  static constexpr int kVOff = 8 * D, kSOff = 16 * D, kPart = 18 * D;
  static constexpr int kStage = SUB * kPart;
  static constexpr int kRing = W * S * kStage;
  static constexpr int kMerge = W * MT * NT * 512;  // the merge meets in the ring
  static constexpr int kBytes = kRing > kMerge ? kRing : kMerge;
  static_assert(kBytes + 2 * W * (16 * kRows + 16) + 1024 <= 228 * 1024, "shared memory of an SM");
  static_assert((2 * W * kRows) % 32 == 0 && 2 * W <= 32 && SUB * S <= 32, "merge and flags");
};

template <typename Sh, int NSEG>
__global__ void __launch_bounds__(Sh::W * 32, 1)
kv4_decode_kernel(const Kv4Params p, const __grid_constant__ Kv4Sched<NSEG> sc) {
  constexpr int D = Sh::D, NT = Sh::NT, W = Sh::W, S = Sh::S, MT = Sh::MT, SUB = Sh::SUB;
  constexpr int KC = Sh::KC, KG = Sh::KG, KW = Sh::KW, VG = Sh::VG, VW = Sh::VW;
  using Lay = RowLayout<D>;
  constexpr int kBlk = Sh::kBlk;
  extern __shared__ __align__(128) uint8_t smem[];
  // Per warp up to two pieces of segments it shares with others: one that ends
  // in its range (its state goes to the workspace) and the one it ends in
  // (kept in registers); their references and sums per row.
  __shared__ Piece s_piece[2 * W];
  __shared__ float wm[2 * W][Sh::kRows], wl[2 * W][Sh::kRows];
  __shared__ __align__(8) float s_share[2 * W][Sh::kRows];
  __shared__ float s_lse[2 * W][Sh::kRows];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  const Kv4Start start = sc.cta[blockIdx.x];
  if (start.len <= 0) return;
  Place cs{start.tile, start.head, start.j, start.len, sc.tile[start.tile].nb};
  {
    // This warp's share: an equal, contiguous part of the CTA's range.
    const int32_t w0 = static_cast<int32_t>(static_cast<int64_t>(start.len) * warp / W);
    const int32_t w1 = static_cast<int32_t>(static_cast<int64_t>(start.len) * (warp + 1) / W);
    place_skip(sc, p, cs, w0);
    cs.rem = w1 - w0;
    if (lane < 2) s_piece[2 * warp + lane].e = -1;
  }
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S * Sh::kStage;
  float4* mbuf = reinterpret_cast<float4*>(smem);

  // ---- The copies' side.  This warp's blocks of the range, in order, come in
  // batches of up to 32 of one segment: lane i holds the page ids of the
  // batch's block i, read a batch ahead of their use.
  struct Batch {
    int32_t n, blk;        // blocks; the first one
    int32_t g, seq, lo, hi;  // KV head, sequence, keys the tile sees
    int32_t page[SUB];     // (lane) pages of the block's parts
  };
  Place bs = cs;          // where the next batch comes from
  int32_t bj = bs.j;
  auto next_batch = [&](Batch& b) {
    int32_t j1 = 0;
    for (;; place_next(sc, p, bs), bj = bs.j) {
      if (bs.rem <= 0) {
        b.n = 0;
        return;
      }
      j1 = min(bs.nb, bs.j + bs.rem);
      if (bj < j1) break;
    }
    const Kv4Tile& t = sc.tile[bs.e];
    b.n = min(32, j1 - bj);
    b.blk = t.fb + bj;
    b.g = bs.g;
    b.seq = t.seq;
    b.lo = first_visible(t.pos0 + t.r0 / p.group, t.window);
    b.hi = t.pos0 + (t.r0 + t.nrows - 1) / p.group;
    if (lane < b.n) {
      const int32_t key = (b.blk + lane) * kBlk;
      const int32_t* row = p.page_table + static_cast<int64_t>(t.seq) * p.mpps;
      // One page holds the block, or each part is looked up for itself; then
      // those that no row of the tile sees are not (-2).
#pragma unroll
      for (int h = 0; h < SUB; ++h) {
        const int32_t k0 = key + 16 * h;
        const bool one_page = (1 << p.page_shift) >= kBlk;
        if (h > 0 && one_page) {
          b.page[h] = b.page[0];
        } else if (!one_page && (k0 > b.hi || k0 + 15 < b.lo)) {
          b.page[h] = -2;
        } else {
          const int32_t slot = k0 >> p.page_shift;
          b.page[h] = slot < p.mpps ? __ldg(row + slot) : p.num_pages;
        }
      }
    }
    bj += 32;
  };
  Batch cur, nxt;
  next_batch(cur);
  next_batch(nxt);
  int32_t bi = 0;          // next block of `cur`
  uint32_t bad_parts = 0;  // bit st * SUB + h: that part has no good page
  const uint8_t* const k_lane = p.k + lane * 16;
  const uint8_t* const v_lane = p.v + lane * 16;
  const uint32_t copy_at = Lay::copy_at(lane);
  constexpr int H = D / 16;  // 16-byte pieces of 16 keys' K (or V) scales
  const uint8_t* const s_lane = (lane < H ? p.ks : p.vs) + (lane & (H - 1)) * 16;
  // Parts [h0, h0 + N) of the block into stage st, from page `page` on.
  auto copy_parts = [&](int st, int32_t key, int32_t page, int h0, auto parts) {
    constexpr int N = decltype(parts)::value;
    const bool ok = page >= 0 && page < p.num_pages;
    const uint32_t bits = ((1u << N) - 1u) << (st * SUB + h0);
    bad_parts = ok ? bad_parts & ~bits : bad_parts | bits;
    if (!ok && page != -2 && lane == 0)
      report_error(p.ws, (key >> p.page_shift) < p.mpps ? RPA_DEVERR_PAGE_ID : RPA_DEVERR_LENGTHS, cur.seq);
    // The first row in the pool (rows of one head in a page are contiguous);
    // without a page the bytes arrive as zeros.
    const int64_t row = ok ? ((static_cast<int64_t>(page) * p.hkv + cur.g) << p.page_shift) +
                                 (key & ((1 << p.page_shift) - 1))
                           : 0;
    const uint32_t bytes = ok ? 16 : 0;
    const uint32_t d = ring + st * Sh::kStage + h0 * Sh::kPart;
    const uint8_t* kp = k_lane + row * (D / 2);
    const uint8_t* vp = v_lane + row * (D / 2);
    const uint8_t* sp = s_lane + row * (D / 16);
#pragma unroll
    for (int h = 0; h < N; ++h) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {  // 512 bytes of K and of V each
        copy_async(d + h * Sh::kPart + Lay::copy_step(copy_at, i), kp + (h * 8 * D + i * 512), bytes);
        copy_async(d + h * Sh::kPart + Sh::kVOff + Lay::copy_step(copy_at, i), vp + (h * 8 * D + i * 512), bytes);
      }
      if (lane < 2 * H) copy_async(d + h * Sh::kPart + Sh::kSOff + lane * 16, sp + h * D, bytes);
    }
  };
  auto issue = [&](int st) {
    if (bi < cur.n) {
      const int32_t key = (cur.blk + bi) * kBlk;
      if ((1 << p.page_shift) >= kBlk) {
        copy_parts(st, key, __shfl_sync(0xffffffffu, cur.page[0], bi), 0, std::integral_constant<int, SUB>());
      } else {
#pragma unroll
        for (int h = 0; h < SUB; ++h)
          copy_parts(st, key + 16 * h, __shfl_sync(0xffffffffu, cur.page[h], bi), h, std::integral_constant<int, 1>());
      }
      if (++bi == cur.n) {
        cur = nxt;
        bi = 0;
        if (cur.n > 0) next_batch(nxt);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int st = 0; st < S; ++st) issue(st);
  if (const int t = blockIdx.x + gridDim.x * tid; t < sc.n_tiles)
    check_lengths(sc.tile, t, sc.n_tiles, sc.cu_q_lens, sc.kv_lens, sc.num_seqs, sc.total_q, p.ws);


  // What this lane reads: of K rows g and g + 8 its quarter (KC chunks), of V
  // its eighth of keys 2c, 2c + 1 and those eight on.
  uint32_t k_at[KC], v_at[2];
#pragma unroll
  for (int j = 0; j < KC; ++j) k_at[j] = Lay::byte(g, (KC * c + j) * KG);
#pragma unroll
  for (int b = 0; b < 2; ++b) v_at[b] = Lay::byte(2 * c + b, g * VG);

  int st = 0;
  float o[MT][NT][4];
  // Columns' reference (a finite stand-in for -inf until the first score) and
  // this lane's sums.
  float m0[NT], m1[NT], l0[NT], l1[NT];
  bool held = false;  // o, m and l are the piece kept for the merge
  // By column (16 bits each): the blocks of dimensions into which a NaN of V at
  // an uneven key goes, once the segment's O is in memory, where the loop need not
  // be unrolled.
  uint32_t nan_hit[NT];
  auto nan_to_state = [&](float4* state) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nan_hit[nt] != 0)
#pragma unroll 1
        for (int t = 0; t < MT; ++t) {
          float* const f = reinterpret_cast<float*>(state + (t * NT + nt) * 32);
          const uint32_t hit = nan_hit[nt] >> ((g * (D / 8) + 2 * t) / 16);  // dimensions g (D / 8) + 2 t, + 1
          if (hit & 1u) f[0] = f[2] = quiet_nan();
          if (hit & 0x10000u) f[1] = f[3] = quiet_nan();
        }
  };
  for (; cs.rem > 0; place_next(sc, p, cs)) {
    const int32_t j1 = min(cs.nb, cs.j + cs.rem);
    if (cs.j >= j1) continue;  // only the segment's charge lies in this range
    const Kv4Tile& tl = sc.tile[cs.e];
    const int G = p.group;
    // ---- The tile's queries as B fragments: lane (g, c) holds row g (+ 8 nt)
    // and the dimensions of its chunks, word by word.
    constexpr int QW = KC * KW;
    uint32_t qf[QW][NT][4];
    float sc0[NT], sc1[NT];   // logit scales of this lane's columns 2c, 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = g + 8 * nt;
      const int r = tl.r0 + n;
      const bool has = n < tl.nrows;
      const int64_t off = (static_cast<int64_t>(tl.q0 + r / G) * p.hq + cs.g * G + r % G) * D;
      uint4 u[QW];
      uint32_t top = 0;  // the row's largest magnitude, as bf16 bits
#pragma unroll
      for (int w = 0; w < QW; ++w) {
        u[w] = make_uint4(0, 0, 0, 0);
        if (has) u[w] = __ldg(reinterpret_cast<const uint4*>(p.q + off + (KC * c) * (2 * KG) + 8 * w));
      }
#pragma unroll
      for (int w = 0; w < QW; ++w) {
        top = __vmaxu2(top, u[w].x & 0x7fff7fffu);
        top = __vmaxu2(top, u[w].y & 0x7fff7fffu);
        top = __vmaxu2(top, u[w].z & 0x7fff7fffu);
        top = __vmaxu2(top, u[w].w & 0x7fff7fffu);
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^ex: the power of two at or below it.
      uint32_t ex = top >> 7;
      if (ex == 0 || ex == 255) ex = 127;
      ex = min(ex, 253u);
      const float down = __uint_as_float((254u - ex) << 23), up = __uint_as_float(ex << 23);
      auto half = [&](uint32_t v) {
        return pack_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xffff0000u) * down);
      };
#pragma unroll
      for (int w = 0; w < QW; ++w) {
        qf[w][nt][0] = half(u[w].x);
        qf[w][nt][1] = half(u[w].y);
        qf[w][nt][2] = half(u[w].z);
        qf[w][nt][3] = half(u[w].w);
      }
      sc0[nt] = p.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * c);
      sc1[nt] = p.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * c + 4);
    }
    const int32_t seg_hi = tl.pos0 + (tl.r0 + tl.nrows - 1) / G;
    // Keys every row sees.
    const int32_t all_lo = first_visible(seg_hi, tl.window), all_hi = tl.pos0 + tl.r0 / G;
    uint32_t nan_seen = 0;  // scales of NaN taken out (kv4_split.cuh)

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m0[nt] = m1[nt] = kNoScore;
      l0[nt] = l1[nt] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.f;
    }

    for (int32_t j = cs.j; j < j1; ++j) {
      copy_wait<S - 1>();
      __syncwarp();  // the scales are other lanes' copies
      const uint32_t src = ring + st * Sh::kStage;
      const int32_t key0 = (tl.fb + j) * kBlk;
      const uint32_t bad = (bad_parts >> (st * SUB)) & ((1u << SUB) - 1);
      const bool edge = bad != 0 || key0 < all_lo || key0 + kBlk - 1 > all_hi;
      // ---- S^T = K Q^T
      float x[SUB][NT][4];
#pragma unroll
      for (int h = 0; h < SUB; ++h) {
        const uint32_t part = src + h * Sh::kPart;
        // One chain of products per part and row tile; a block of one part and
        // one tile takes two, so that the products need not wait for one another.
        constexpr int CH = SUB * NT == 1 ? 2 : 1;
        float acc[CH][NT][4];
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.f;
#pragma unroll
        for (int jc = 0; jc < KC; ++jc) {
          uint32_t ka[KW], kb[KW];
          lds<KW>(part + k_at[jc], ka);
          lds<KW>(part + k_at[jc] + 4 * D, kb);  // eight rows on
          // Scale bytes of the chunk's 16-dimension blocks (two, or one of
          // 64-dimension rows) in rows g and g + 8.
          uint32_t sa, sb;
          if constexpr (KW == 4) {
            sa = lds_u16(part + Sh::kSOff + g * (D / 16) + (KC * c + jc) * 2);
            sb = lds_u16(part + Sh::kSOff + (g + 8) * (D / 16) + (KC * c + jc) * 2);
          } else {
            sa = lds_u8(part + Sh::kSOff + g * (D / 16) + c);
            sb = lds_u8(part + Sh::kSOff + (g + 8) * (D / 16) + c);
          }
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const uint32_t ha = scale_dup(sa, w >> 1), hb = scale_dup(sb, w >> 1);
            uint32_t a[4], b[4];
            kv4::decode8(ka[w], a);
            kv4::decode8(kb[w], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = kv4::hmul2(a[i], ha);
              b[i] = kv4::hmul2(b[i], hb);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t (&q)[4] = qf[jc * KW + w][nt];
              mma_f16(acc[0][nt], a[0], b[0], a[1], b[1], q[0], q[1]);
              mma_f16(acc[CH - 1][nt], a[2], b[2], a[3], b[3], q[2], q[3]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[h][nt][i] = CH == 2 ? acc[0][nt][i] + acc[CH - 1][nt][i] : acc[0][nt][i];
      }
      // ---- Online softmax: exponents against the columns' references; where
      // one passes kRaiseAt, the references are raised first.
      float y[SUB][NT][4];
      auto exponents = [&]() {
#pragma unroll
        for (int h = 0; h < SUB; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            y[h][nt][0] = fmaf(x[h][nt][0], sc0[nt], -m0[nt]);
            y[h][nt][1] = fmaf(x[h][nt][1], sc1[nt], -m1[nt]);
            y[h][nt][2] = fmaf(x[h][nt][2], sc0[nt], -m0[nt]);
            y[h][nt][3] = fmaf(x[h][nt][3], sc1[nt], -m1[nt]);
          }
        if (edge) {
          // Blocks at a row's edges, or without a page.  Rows past the tile's
          // last take its last row's keys; they are not written.
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int32_t last = tl.r0 + tl.nrows - 1, n = tl.r0 + 8 * nt + 2 * c;
            const int32_t hi0 = tl.pos0 + min(n, last) / G, hi1 = tl.pos0 + min(n + 1, last) / G;
            const int32_t lo0 = first_visible(hi0, tl.window), lo1 = first_visible(hi1, tl.window);
#pragma unroll
            for (int h = 0; h < SUB; ++h) {
              const int32_t ka = key0 + 16 * h + g, kb = ka + 8;
              const bool no = (bad >> h) & 1u;
              if (no || ka < lo0 || ka > hi0) y[h][nt][0] = -INFINITY;
              if (no || ka < lo1 || ka > hi1) y[h][nt][1] = -INFINITY;
              if (no || kb < lo0 || kb > hi0) y[h][nt][2] = -INFINITY;
              if (no || kb < lo1 || kb > hi1) y[h][nt][3] = -INFINITY;
            }
          }
        }
      };
      exponents();
      float top = -INFINITY;
#pragma unroll
      for (int h = 0; h < SUB; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          top = fmaxf(fmaxf(top, fmaxf(y[h][nt][0], y[h][nt][1])), fmaxf(y[h][nt][2], y[h][nt][3]));
      if (__any_sync(0xffffffffu, top > kRaiseAt)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // The columns' largest exponents, relative to the references.
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int h = 0; h < SUB; ++h) {
            t0 = fmaxf(t0, fmaxf(y[h][nt][0], y[h][nt][2]));
            t1 = fmaxf(t1, fmaxf(y[h][nt][1], y[h][nt][3]));
          }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, off));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, off));
          }
          // Raised from the stand-in, the reference comes from the score itself
          // (the difference to the stand-in has lost its low bits).
          const bool new0 = m0[nt] == kNoScore, new1 = m1[nt] == kNoScore;
          t0 = fmaxf(t0 - kBelowTop, 0.f);
          t1 = fmaxf(t1 - kBelowTop, 0.f);
          float n0 = m0[nt] + t0, n1 = m1[nt] + t1;
          // (For the whole warp: with a window, columns get their first score in
          // different blocks, and the shuffles take every lane.)
          if (__any_sync(0xffffffffu, new0 || new1)) {
            float s0 = -INFINITY, s1 = -INFINITY;
#pragma unroll
            for (int h = 0; h < SUB; ++h) {
              if (y[h][nt][0] > -INFINITY) s0 = fmaxf(s0, x[h][nt][0] * sc0[nt]);
              if (y[h][nt][2] > -INFINITY) s0 = fmaxf(s0, x[h][nt][2] * sc0[nt]);
              if (y[h][nt][1] > -INFINITY) s1 = fmaxf(s1, x[h][nt][1] * sc1[nt]);
              if (y[h][nt][3] > -INFINITY) s1 = fmaxf(s1, x[h][nt][3] * sc1[nt]);
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              s0 = fmaxf(s0, __shfl_xor_sync(0xffffffffu, s0, off));
              s1 = fmaxf(s1, __shfl_xor_sync(0xffffffffu, s1, off));
            }
            if (new0) n0 = s0 == -INFINITY ? kNoScore : s0 - kBelowTop;
            if (new1) n1 = s1 == -INFINITY ? kNoScore : s1 - kBelowTop;
          }
          const float f0 = new0 ? 1.f : fast_exp2(m0[nt] - n0), f1 = new1 ? 1.f : fast_exp2(m1[nt] - n1);
          m0[nt] = n0;
          m1[nt] = n1;
          l0[nt] *= f0;
          l1[nt] *= f1;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[t][nt][0] *= f0;
            o[t][nt][1] *= f1;
            o[t][nt][2] *= f0;
            o[t][nt][3] *= f1;
          }
        }
        exponents();
#pragma unroll
        for (int h = 0; h < SUB; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[h][nt][i] = raised(y[h][nt][i]);
      }
      uint32_t pb[SUB][NT][2];
#pragma unroll
      for (int h = 0; h < SUB; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float p0 = fast_exp2(y[h][nt][0]), p1 = fast_exp2(y[h][nt][1]);
          const float p2 = fast_exp2(y[h][nt][2]), p3 = fast_exp2(y[h][nt][3]);
          l0[nt] += p0 + p2;
          l1[nt] += p1 + p3;
          pb[h][nt][0] = transpose8x8(pack_f16x2(p0, p1));
          pb[h][nt][1] = transpose8x8(pack_f16x2(p2, p3));
        }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int h = 0; h < SUB; ++h) {
        const uint32_t part = src + h * Sh::kPart;
        uint32_t vw[4][VW];
        uint32_t sv[4];  // scale bytes of this lane's dimensions in its four keys
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 2 * c + (i & 1) + 8 * (i >> 1);
          lds<VW>(part + Sh::kVOff + v_at[i & 1] + (i >> 1) * 4 * D, vw[i]);
          if constexpr (D == 256)
            sv[i] = lds_u16(part + Sh::kSOff + D + kk * (D / 16) + 2 * g);
          else
            sv[i] = lds_u8(part + Sh::kSOff + D + kk * (D / 16) + (D == 128 ? g : g >> 1));
        }
        if (edge) {
          // Keys no row sees: whatever their bytes, their values are zeros.  A NaN
          // of a key that some do not see is put into the others' rows at the end.
          const int32_t seg_lo = first_visible(all_hi, tl.window);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t key = key0 + 16 * h + 2 * c + (i & 1) + 8 * (i >> 1);
            if (((bad >> h) & 1u) || key < seg_lo || key > seg_hi) sv[i] = 0;
            const uint32_t nan = key < all_lo || key > all_hi ? kv4::nan_bytes(sv[i]) : 0u;
            sv[i] = kv4::without_nan(sv[i], nan);
            nan_seen |= nan;
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t s01 = scale_pair_of(sv[0], sv[1], D == 256 ? w >> 1 : 0);
          const uint32_t s23 = scale_pair_of(sv[2], sv[3], D == 256 ? w >> 1 : 0);
          constexpr uint32_t kLow = 0x0f0f0f0fu;
          uint32_t e01[4], d01[4], e23[4], d23[4];  // even and odd dimensions, key pairs
          kv4::decode8(bit_select(kLow, vw[0][w], vw[1][w] << 4), e01);
          kv4::decode8(bit_select(kLow, vw[0][w] >> 4, vw[1][w]), d01);
          kv4::decode8(bit_select(kLow, vw[2][w], vw[3][w] << 4), e23);
          kv4::decode8(bit_select(kLow, vw[2][w] >> 4, vw[3][w]), d23);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t a0 = kv4::hmul2(e01[t], s01), a1 = kv4::hmul2(d01[t], s01);
            const uint32_t a2 = kv4::hmul2(e23[t], s23), a3 = kv4::hmul2(d23[t], s23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[4 * w + t][nt], a0, a1, a2, a3, pb[h][nt][0], pb[h][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the scales: the stage may be refilled
      issue(st);
      if (++st == S) st = 0;
    }

    // ---- The segment's end in this warp's range.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) nan_hit[nt] = 0;
    if (__any_sync(0xffffffffu, nan_seen != 0)) {
      each_uneven_nan<D>(p, tl.seq, cs.g, max((tl.fb + cs.j) * kBlk, first_visible(all_hi, tl.window)),
                         min((tl.fb + j1) * kBlk - 1, seg_hi), all_lo, all_hi, [&](int32_t key, uint32_t blocks) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int32_t hi = tl.pos0 + min(tl.r0 + 8 * nt + 2 * c + i, tl.r0 + tl.nrows - 1) / G;
            if (key <= hi && key >= first_visible(hi, tl.window)) nan_hit[nt] |= blocks << (16 * i);
          }
      });
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0[nt] += __shfl_xor_sync(0xffffffffu, l0[nt], off);
        l1[nt] += __shfl_xor_sync(0xffffffffu, l1[nt], off);
      }
    if (cs.j == 0 && j1 == cs.nb) {
      // All of it: normalise and store, 16 bytes (8 dimensions) at a time.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float l = h ? l1[nt] : l0[nt];
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int n = 8 * nt + 2 * c + h, r = tl.r0 + n;
          if (n < tl.nrows) {
            __nv_bfloat16* dst =
                p.out + (static_cast<int64_t>(tl.q0 + r / G) * p.hq + cs.g * G + r % G) * D + g * (D / 8);
#pragma unroll
            for (int w = 0; w < MT / 4; ++w) {
              uint32_t v[4];
#pragma unroll
              for (int t = 0; t < 4; ++t)
                v[t] = pack_bf16x2(o[4 * w + t][nt][h] * inv, o[4 * w + t][nt][2 + h] * inv);
              reinterpret_cast<uint4*>(dst)[w] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            if (const uint32_t blocks = nan_hit[nt] >> (16 * h) & 0xffffu)
#pragma unroll 1
              for (int t = 0; t < MT; ++t)
                if (blocks >> ((g * (D / 8) + 2 * t) / 16) & 1u) reinterpret_cast<uint32_t*>(dst)[t] = 0x7fff7fffu;
          }
        }
      continue;
    }
    held = cs.rem <= cs.nb + kKv4SegCost - cs.j;  // nothing follows in this range
    const int piece = 2 * warp + (held ? 1 : 0);
    if (lane == 0) s_piece[piece] = Piece{cs.e, cs.g, cs.j, j1};
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        wm[piece][8 * nt + 2 * c] = m0[nt];
        wm[piece][8 * nt + 2 * c + 1] = m1[nt];
        wl[piece][8 * nt + 2 * c] = l0[nt];
        wl[piece][8 * nt + 2 * c + 1] = l1[nt];
      }
    }
    if (held) break;
    float4* dst = p.piece_o + (static_cast<int64_t>(blockIdx.x) * W + warp) * (MT * NT * 32) + lane;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        dst[(t * NT + nt) * 32] = make_float4(o[t][nt][0], o[t][nt][1], o[t][nt][2], o[t][nt][3]);
    nan_to_state(dst);
  }
  // ---- Merge the CTA's pieces, once.  Those of one segment follow one another:
  // the kept ones of warps in order (one without blocks has a zero share), then
  // (of the warp it ends in) one from the workspace.  Their sum, each times its
  // share of the normalised result, is taken in that order.  The states meet in the ring, which
  // is free by now.  (Rolled loops: this code runs once a launch, and fetching
  // it, fully unrolled, took longer than running it.)
  copy_wait<0>();
  // The combine may be scheduled now (it waits for this grid's end).  From the
  // start on, its waiting CTAs would keep registers that a prefill grid beside
  // this one needs.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mbuf[(warp * MT * NT + t * NT + nt) * 32 + lane] =
          held ? make_float4(o[t][nt][0], o[t][nt][1], o[t][nt][2], o[t][nt][3]) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (held) nan_to_state(mbuf + warp * MT * NT * 32 + lane);
  // Lane k looks at piece k: which others are its segment's.
  const int my_e = lane < 2 * W ? s_piece[lane].e : -1;
  const uint32_t my_members =
      __match_any_sync(0xffffffffu, my_e < 0 ? -1ll : (static_cast<int64_t>(my_e) << 32) + s_piece[lane].g);
  const uint32_t heads = __ballot_sync(0xffffffffu, my_e >= 0 && __ffs(my_members) - 1 == lane);
  // Thread (i, n): piece i's share of row n, 2^(m_i - M) / sum_k 2^(m_k - M) l_k.
#pragma unroll 1
  for (int it = tid; it < 2 * W * Sh::kRows; it += W * 32) {
    const int pi = it / Sh::kRows, pn = it % Sh::kRows;
    const uint32_t members =
        __shfl_sync(0xffffffffu, my_members, pi) & (__shfl_sync(0xffffffffu, my_e, pi) < 0 ? 0u : ~0u);
    float M = kNoScore, L = 0.f;
#pragma unroll 8
    for (int k = 0; k < 2 * W; ++k) {
      const float m = wm[k][pn];
      M = fmaxf(M, (members >> k) & 1u ? m : kNoScore);
    }
#pragma unroll 8
    for (int k = 0; k < 2 * W; ++k) {
      const float f = fast_exp2(wm[k][pn] - M) * wl[k][pn];
      L += (members >> k) & 1u ? f : 0.f;
    }
    // (A segment without a score has L = 0; a NaN stays.)
    s_share[pi][pn] = members == 0 || L == 0.f ? 0.f : fast_exp2(wm[pi][pn] - M) / L;
    s_lse[pi][pn] = L == 0.f ? -INFINITY : M + __log2f(L);
  }
  __syncthreads();
  constexpr int kItems = MT * NT * 32;  // float4 of a state: a multiple of the warp
  const int total = __popc(heads) * kItems;
#pragma unroll 1
  for (int idx = tid; idx < total; idx += W * 32) {
    uint32_t head_bits = heads;  // (the same for the whole warp)
    for (int q = idx / kItems; q > 0; --q) head_bits &= head_bits - 1;
    const int k0 = __ffs(head_bits) - 1;
    const int k1 = 31 - __clz(__shfl_sync(0xffffffffu, my_members, k0));
    const int i = idx % kItems;
    // Loads from far first.
    float4 far = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((k1 & 1) == 0) far = p.piece_o[(static_cast<int64_t>(blockIdx.x) * W + (k1 >> 1)) * kItems + i];
    const Piece head = s_piece[k0];
    const Kv4Tile tl = sc.tile[head.e];
    const int mt = (i >> 5) / NT, nt = (i >> 5) % NT;
    // Lane (g, c) holds columns 2c, 2c + 1 of dimensions d, d + 1.
    const int d = g * (D / 8) + 2 * mt, n = 8 * nt + 2 * c;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, const float4& b) {
      const float2 f = *reinterpret_cast<const float2*>(&s_share[k][n]);
      a.x = fmaf(b.x, f.x, a.x);
      a.y = fmaf(b.y, f.y, a.y);
      a.z = fmaf(b.z, f.x, a.z);
      a.w = fmaf(b.w, f.y, a.w);
    };
#pragma unroll 4
    for (int k = k0 | 1; k <= k1; k += 2) add(k, mbuf[(k >> 1) * kItems + i]);
    if ((k1 & 1) == 0) add(k1, far);
    if (head.j0 == 0 && s_piece[k1].j1 == tl.nb) {
      const int r = tl.r0 + n;
      __nv_bfloat16* const col = p.out + static_cast<int64_t>(head.g * p.group) * D + d;
      auto row = [&](int r) {
        return (static_cast<int64_t>(tl.q0 + r / p.group) * p.hq + r % p.group) * D;
      };
      if (n < tl.nrows) *reinterpret_cast<uint32_t*>(col + row(r)) = pack_bf16x2(a.x, a.z);
      if (n + 1 < tl.nrows) *reinterpret_cast<uint32_t*>(col + row(r + 1)) = pack_bf16x2(a.y, a.w);
    } else {
      // Cut across CTAs: the normalised part goes out with its log2-sum-exp.
      const int64_t slot = 2 * blockIdx.x + (head.e == start.tile && head.g == start.head ? 0 : 1);
      float* const dst = p.part_o + (slot * Sh::kRows + n) * D + d;
      *reinterpret_cast<float2*>(dst) = make_float2(a.x, a.z);
      *reinterpret_cast<float2*>(dst + D) = make_float2(a.y, a.w);
      if (mt == 0 && g == 0)
        *reinterpret_cast<float2*>(&p.part_lse[slot * Sh::kRows + n]) = make_float2(s_lse[k0][n], s_lse[k0][n + 1]);
    }
  }
}

template <int D, int NT, int NSEG>
int launch_t(const Plan& plan, const Args& a, const Kv4Params& p, const Plan::Kv4Launch& l, cudaStream_t stream) {
  using Sh = Kv4Shape<D, NT>;
  return launch_split<D, Sh::kRows, NSEG>(plan, a, p, l, Sh::W * 32, Sh::kBytes, kv4_decode_kernel<Sh, NSEG>, stream);
}

template <int D, int NT>
int launch_n(const Plan& plan, const Args& a, const Kv4Params& p, const Plan::Kv4Launch& l, cudaStream_t stream) {
  // Two sizes of launch parameters: 9 KB and 32 KB.
  return l.end - l.begin <= kKv4TilesSmall ? launch_t<D, NT, kKv4TilesSmall>(plan, a, p, l, stream)
                                           : launch_t<D, NT, kKv4TilesLarge>(plan, a, p, l, stream);
}

}  // namespace

Kv4Grain kv4_grain(int32_t head_dim, int32_t nt) {
  if (nt == kKv4RowsTile) return kv4_rows_grain(head_dim);
  switch (head_dim * 8 + nt) {
    case 64 * 8 + 1: return {Kv4Shape<64, 1>::W, Kv4Shape<64, 1>::kBlk};
    case 64 * 8 + 2: return {Kv4Shape<64, 2>::W, Kv4Shape<64, 2>::kBlk};
    case 128 * 8 + 1: return {Kv4Shape<128, 1>::W, Kv4Shape<128, 1>::kBlk};
    case 128 * 8 + 2: return {Kv4Shape<128, 2>::W, Kv4Shape<128, 2>::kBlk};
    default: return {Kv4Shape<256, 1>::W, Kv4Shape<256, 1>::kBlk};
  }
}

int launch_kv4_decode(const Plan& plan, const Args& a, void* stream) {
  const Kv4Params p = kv4_params(plan, a);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (const Plan::Kv4Launch& l : plan.kv4_launches) {
    int e = static_cast<int>(cudaErrorInvalidValue);
    if (l.nt == kKv4RowsTile) {
      if ((e = launch_kv4_rows(plan, a, l, stream)) != 0) return e;
      continue;
    }
    switch (plan.d * 8 + l.nt) {
      case 64 * 8 + 1: e = launch_n<64, 1>(plan, a, p, l, s); break;
      case 64 * 8 + 2: e = launch_n<64, 2>(plan, a, p, l, s); break;
      case 128 * 8 + 1: e = launch_n<128, 1>(plan, a, p, l, s); break;
      case 128 * 8 + 2: e = launch_n<128, 2>(plan, a, p, l, s); break;
      case 256 * 8 + 1: e = launch_n<256, 1>(plan, a, p, l, s); break;
    }
    if (e) return e;
  }
  return 0;
}

}  // namespace rpa
