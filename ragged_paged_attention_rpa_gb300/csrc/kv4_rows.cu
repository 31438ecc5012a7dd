// Attention over 4-bit pages for sequences with some tens of query rows (drafted
// tokens, short chunks): split-KV, a block's codes widened once for 64 rows.
//
// The kernel of kv4_decode.cu widens a segment's keys in registers, once a tile
// of 8 or 16 rows; past two tiles the widening is most of its work.  Here a CTA
// takes tiles of up to 64 rows and widens each block to f16 in shared memory,
// where its warps share it.  Segments, ranges, charges and the combine are that
// kernel's (kv4_split.cuh); a range belongs to the whole CTA.
//
// CTA.  8 warps, blocks of 8192 / D keys.  Per block a warp
//   - widens an eighth of it, 2048 elements of K or of V, which it copied itself
//     (cp.async, four blocks in flight; the codes need no barrier);
//   - after a barrier of the four warps that share its half of the block's keys
//     (the f16 blocks are double-buffered) takes 16 rows of the tile: S = Q K^T,
//     an online softmax, and O += P V (mma.m16n8k16, f16 -> fp32).
// The two halves of the keys meet at the segment's end.
//
// Layout.  A row of f16 is lines of 128 bytes whose 16-byte chunks are permuted
// by XOR with the key and the line, such that eight lanes' stores (64 dimensions
// a lane) and the eight rows of an ldmatrix meet every bank once.
//
// Numbers, unseen keys and bad pages: as in kv4_decode.cu.
//
// What bounds it: instructions.  A warp runs some 500 a block (64 products, 32
// ldmatrix, the widening, the softmax, the next copies) at about four cycles
// each, two warps a scheduler: O and Q of 16 rows take 192 registers at 256
// dimensions.  128 sequences of 64 rows over 128-2048 keys of 256 dimensions take
// 63.6 us (61.6 with the 47 MB of pages in L2); 32 rows of each 48.5 us.  While it
// took 59 of those 61.6 (the looks for NaN in V and at the lengths are the rest):
// widening to bf16 pages and the prefill kernel 72.7 us, tiles of 8 rows 77 us; one
// barrier for both halves as fast (at 128 dimensions 32 sequences of 64 rows over
// 120-4000 keys of 8 heads 96 us, 92 so); the next block's widening between this
// one's products 61 us; 16 warps of 128 registers, each with a quarter of the keys
// for S and of the dimensions for O, 69 us (the copies' and the softmax's
// instructions then run in twice as many warps).
#include "kv4_split.cuh"

namespace rpa {
namespace {

template <int D_>
struct RowsShape {
  static constexpr int D = D_, W = 8, kRows = 64;
  static constexpr int S = 4;             // blocks of codes in flight
  static constexpr int kBlk = 8192 / D;   // keys a block
  static constexpr int kWarpKeys = kBlk / 4;
  static constexpr int SUB = kBlk / 32;   // 16-key parts of half a block
  static constexpr int NP = kWarpKeys > 16 ? 2 : 1;  // pages a warp's keys may lie in
  static constexpr int KT = D / 16;       // 16-dimension steps
  static constexpr int kStage = 8 * 1024 + 8 * 128;
  static constexpr int kHalf = 16384;     // f16 K (or V) of a block
  static constexpr int kMerge = D * 256;  // O of half the keys
  static constexpr int kBytes = 4 * kHalf + S * kStage + kMerge;
};

__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// A barrier of the four warps of a half.
__device__ __forceinline__ void half_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <typename Sh, int NSEG>
__global__ void __launch_bounds__(Sh::W * 32, 1)
kv4_rows_kernel(const Kv4Params p, const __grid_constant__ Kv4Sched<NSEG> sc) {
  constexpr int D = Sh::D, S = Sh::S, SUB = Sh::SUB, NP = Sh::NP, KT = Sh::KT, kBlk = Sh::kBlk;
  constexpr int kLineSwz = D == 256 ? 1 : 2;  // line u of a row: chunks XORed with u << this
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint8_t s_bad[2][2 * SUB];       // (block parity) 16-key parts without a good page
  __shared__ float s_m[Sh::kRows], s_l[Sh::kRows];
  __shared__ int32_t s_nan;                   // last segment with a NaN taken out of V (kv4_split.cuh)
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  // Warps 0-3 and 4-7 take a half of each block's keys each, and widen just
  // that: they need not keep in step, so that one half's products run beside
  // the other's widening.  A scheduler has a warp of either; of a tile of 32 rows
  // it has one that multiplies.
  const int ks = warp >> 2, rg = (warp & 3) ^ (2 * ks);  // half of the keys; 16 rows
  const int quarter = 2 * ks + (warp & 1);               // of K or V, that the warp widens
  const bool is_k = (warp & 3) < 2;
  const Kv4Start start = sc.cta[blockIdx.x];
  if (start.len <= 0) return;
  if (tid == 0) s_nan = -1;
  __syncthreads();
  const uint32_t half0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t ring = half0 + 4 * Sh::kHalf;

  // The place `s` moved on past merge charges, to a block or the range's end.
  auto to_block = [&](Place& s) {
    while (s.rem > 0 && s.j >= s.nb) place_next(sc, p, s);
  };
  Place cs{start.tile, start.head, start.j, start.len, sc.tile[start.tile].nb};
  to_block(cs);

  // ---- The copies' side: a warp copies what it widens.
  Place cp = cs;
  int32_t page[NP];        // of the next block to copy
  // By stage: whether this lane's key is one that a row sees, and whether the 16
  // keys around it have a page.
  uint32_t seen = 0, paged = 0;
  const uint8_t* const codes = (is_k ? p.k : p.v) + lane * 16;
  const uint8_t* const scales = (is_k ? p.ks : p.vs) + (NP == 2 ? lane & 15 : lane) * 4;
  const int wkey = quarter * Sh::kWarpKeys + lane / (D / 64), wline = lane & (D / 64 - 1);  // of a block
  // Its first key, the keys that its tile's rows see, and their row of the page
  // table (worked out once a segment: of the divisions alone, a block would run
  // a hundred instructions).
  int32_t c_key = 0, c_lo = 0, c_hi = 0;
  const int32_t* c_row = nullptr;
  auto enter = [&]() {
    to_block(cp);
    if (cp.rem <= 0) return;
    const Kv4Tile& t = sc.tile[cp.e];
    c_key = (t.fb + cp.j) * kBlk;
    c_lo = first_visible(t.pos0 + t.r0 / p.group, t.window);
    c_hi = t.pos0 + (t.r0 + t.nrows - 1) / p.group;
    c_row = p.page_table + static_cast<int64_t>(t.seq) * p.mpps;
  };
  auto find_pages = [&]() {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int32_t k0 = (c_key + quarter * Sh::kWarpKeys + 16 * i) & ~15, slot = k0 >> p.page_shift;
      if (k0 > c_hi || k0 + 15 < c_lo)
        page[i] = -2;      // no row of the tile sees these 16
      else
        page[i] = slot < p.mpps ? __ldg(c_row + slot) : p.num_pages;
    }
  };
  auto issue = [&](int st) {
    if (cp.rem > 0) {
      const uint32_t dst = ring + st * Sh::kStage;
      const int32_t key = c_key + wkey;
      int64_t row[NP];
      bool ok[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int32_t k0 = c_key + quarter * Sh::kWarpKeys + 16 * i;
        ok[i] = page[i] >= 0 && page[i] < p.num_pages;
        if (!ok[i] && page[i] != -2 && lane == 0)
          report_error(p.ws, (k0 >> p.page_shift) < p.mpps ? RPA_DEVERR_PAGE_ID : RPA_DEVERR_LENGTHS,
                       sc.tile[cp.e].seq);
        row[i] = ok[i] ? ((static_cast<int64_t>(page[i]) * p.hkv + cp.g) << p.page_shift) +
                             (k0 & ((1 << p.page_shift) - 1))
                       : 0;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int q = NP == 2 ? i : 0;  // (two groups of 16 keys are 512 bytes each)
        copy_async(dst + warp * 1024 + i * 512 + (lane ^ (lane >> 3 & 1)) * 16,
                   codes + row[q] * (D / 2) + (NP == 2 ? 0 : i * 512),
                   ok[q] ? 16 : 0);
      }
      const bool upper = NP == 2 && lane >= 16, mine = upper ? ok[NP - 1] : ok[0];
      copy_async4(dst + 8192 + warp * 128 + lane * 4, scales + (upper ? row[NP - 1] : row[0]) * (D / 16),
                  mine ? 4 : 0);
      const bool visible = mine && key >= c_lo && key <= c_hi;
      seen = (seen & ~(1u << st)) | (static_cast<uint32_t>(visible) << st);
      paged = (paged & ~(1u << st)) | (static_cast<uint32_t>(mine) << st);
      ++cp.j;
      --cp.rem;
      c_key += kBlk;
      if (cp.rem <= 0 || cp.j >= cp.nb) enter();
      if (cp.rem > 0) find_pages();
    }
    copy_commit();
  };
  enter();
  if (cp.rem > 0) find_pages();
#pragma unroll
  for (int st = 0; st < S; ++st) issue(st);
  if (const int t = blockIdx.x + gridDim.x * tid; t < sc.n_tiles)
    check_lengths(sc.tile, t, sc.n_tiles, sc.cu_q_lens, sc.kv_lens, sc.num_seqs, sc.total_q, p.ws);


  // ---- Widening: 64 dimensions of one key a lane, in four pieces of 16.
  const uint32_t wdst = half0 + (is_k ? 0 : Sh::kHalf) + wkey * 2 * D + wline * 128;
  const uint32_t wswz = ((wkey & 7) ^ (wline << kLineSwz)) << 4;
  int st = 0, par = 0;     // the next block's stage; its half of the f16 buffer
  uint32_t wscale = 0;
  auto widen_begin = [&](int to) {
    copy_wait<S - 1>();
    __syncwarp();  // the codes are other lanes' copies
    uint32_t w[1];
    lds<1>(ring + st * Sh::kStage + 8192 + warp * 128 + lane * 4, w);
    wscale = (seen >> st) & 1u ? w[0] : 0u;  // keys no row sees: whatever their bytes, zeros
    if (is_k && (lane & 15) == 0) s_bad[to][wkey >> 4] = !((paged >> st) & 1u);
  };
  auto widen = [&](int to, int b) {
    uint32_t w[2], h[8];
    // (Every other four lanes' codes lie with their 16-byte halves swapped.)
    lds<2>(ring + st * Sh::kStage + warp * 1024 + lane * 32 + (((b >> 1) ^ (lane >> 2 & 1)) * 16 + (b & 1) * 8), w);
    kv4::decode_block(make_uint2(w[0], w[1]), (wscale >> (8 * b)) & 0xffu, h);
    const uint32_t dst = wdst + to * 2 * Sh::kHalf;
    sts128(dst + (((2 * b) << 4) ^ wswz), h[0], h[1], h[2], h[3]);
    sts128(dst + (((2 * b + 1) << 4) ^ wswz), h[4], h[5], h[6], h[7]);
  };
  auto widen_end = [&]() {
    __syncwarp();  // every lane has read the codes: the stage may be refilled
    issue(st);
    if (++st == S) st = 0;
  };

  // (A quarter of a line has its two chunks at one of four places: quarter q of
  // line u at at[q ^ u], of two lines at at[q ^ 2 u].)
  uint32_t at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    at[q] = half0 + (ks * (kBlk / 2) + (lane & 15)) * 2 * D + (((2 * q) ^ (lane & 7) ^ (lane >> 4)) << 4);

  auto at_flip = [&]() {  // to the other f16 block
    const uint32_t by = par ? 2 * Sh::kHalf : 0u - 2 * Sh::kHalf;
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] += by;
  };
  float4* const mbuf = reinterpret_cast<float4*>(smem + 4 * Sh::kHalf + S * Sh::kStage) + rg * (D / 8) * 32 + lane;
  while (cs.rem > 0) {
    const Kv4Tile& tl = sc.tile[cs.e];
    const int32_t seg = cs.e * p.hkv + cs.g;
    const int G = p.group, head = cs.g;  // (`cs` moves on before the output is written)
    const int32_t j1 = min(cs.nb, cs.j + cs.rem);
    const bool active = rg * 16 < tl.nrows;
    const int last = tl.r0 + tl.nrows - 1;
    const int ra = tl.r0 + rg * 16 + g, rb = ra + 8;  // this lane's rows
    auto row_at = [&](int r) { return (static_cast<int64_t>(tl.q0 + r / G) * p.hq + head * G + r % G) * D; };
    // Keys each row sees (rows past the tile's last take its last row's; they
    // are not written), and every row does.
    const int32_t hi_a = tl.pos0 + min(ra, last) / G, hi_b = tl.pos0 + min(rb, last) / G;
    const int32_t lo_a = first_visible(hi_a, tl.window), lo_b = first_visible(hi_b, tl.window);
    const int32_t all_hi = tl.pos0 + tl.r0 / G;
    const int32_t all_lo = first_visible(tl.pos0 + last / G, tl.window);
    // ---- Q: f16 after a power of two for the row, as A fragments.
    uint32_t qf[KT][4];
    float sca = 0.f, scb = 0.f;
    if (active) {
      const uint32_t* const qa = reinterpret_cast<const uint32_t*>(p.q + row_at(min(ra, last))) + c;
      const uint32_t* const qb = reinterpret_cast<const uint32_t*>(p.q + row_at(min(rb, last))) + c;
      uint32_t ta = 0, tb = 0;
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        qf[k][0] = __ldg(qa + 8 * k);
        qf[k][1] = __ldg(qb + 8 * k);
        qf[k][2] = __ldg(qa + 8 * k + 4);
        qf[k][3] = __ldg(qb + 8 * k + 4);
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        ta = __vmaxu2(__vmaxu2(ta, qf[k][0] & 0x7fff7fffu), qf[k][2] & 0x7fff7fffu);
        tb = __vmaxu2(__vmaxu2(tb, qf[k][1] & 0x7fff7fffu), qf[k][3] & 0x7fff7fffu);
      }
      // The row's power of two, 1 where it has none (zeros, NaN, infinity).
      auto power = [](uint32_t t) {
        t = max(t & 0xffffu, t >> 16);
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        uint32_t ex = t >> 7;
        if (ex == 0 || ex == 255) ex = 127;
        return min(ex, 253u);
      };
      const uint32_t ea = power(ta), eb = power(tb);
      const float da = __uint_as_float((254u - ea) << 23), db = __uint_as_float((254u - eb) << 23);
      sca = p.scale_log2 * __uint_as_float(ea << 23);
      scb = p.scale_log2 * __uint_as_float(eb << 23);
      auto half = [](uint32_t v, float f) {
        return pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
      };
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        qf[k][0] = half(qf[k][0], da);
        qf[k][1] = half(qf[k][1], db);
        qf[k][2] = half(qf[k][2], da);
        qf[k][3] = half(qf[k][3], db);
      }
    }
    float o[D / 8][4];
    float m_a = kNoScore, m_b = kNoScore, l_a = 0.f, l_b = 0.f;
#pragma unroll
    for (int t = 0; t < D / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    for (int32_t j = cs.j; j < j1; ++j) {
      const int32_t key0 = (tl.fb + j) * kBlk;
      bool edge = key0 < all_lo || key0 + kBlk - 1 > all_hi;
      widen_begin(par);
#pragma unroll
      for (int b = 0; b < 4; ++b) widen(par, b);
      if (edge && !is_k && (key0 + wkey < all_lo || key0 + wkey > all_hi)) {
        // A NaN of V at a key that not every row sees: once more without it.
        if (const uint32_t nan = kv4::nan_bytes(wscale)) {
          wscale = kv4::without_nan(wscale, nan);
          s_nan = seg;
#pragma unroll 1
          for (int b = 0; b < 4; ++b) widen(par, b);
        }
      }
      widen_end();
      half_sync(1 + ks);  // the half is widened, and its warps done with the one before
      if (active) {
        // The products' B fragments in order, K's steps and then V's, each read
        // two steps before its use.
        constexpr int kSteps = SUB * KT, kAhead = 2;
        uint32_t b[kAhead + 1][4];
        auto fetch = [&](int i) {
          uint32_t(&r)[4] = b[i % (kAhead + 1)];
          const int t = i % KT, h = i % kSteps / KT, u = t >> 2;
          const uint32_t from = at[(t & 3) ^ (D == 256 ? u : 2 * u)] + h * 32 * D + u * 128;
          if (i < kSteps) ldmatrix4(from, r);
          else ldmatrix4_trans(from + Sh::kHalf, r);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
        // ---- S = Q K^T
        float x[SUB][2][4];
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
          constexpr int CH = SUB == 1 ? 2 : 1;  // independent chains of products
          float acc[CH][2][4];
#pragma unroll
          for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const int i = h * KT + k;
            fetch(i + kAhead);
            const uint32_t(&r)[4] = b[i % (kAhead + 1)];  // keys 0-7, 8-15 of dimensions 0-7; of 8-15
            mma_f16(acc[k % CH][0], qf[k][0], qf[k][1], qf[k][2], qf[k][3], r[0], r[2]);
            mma_f16(acc[k % CH][1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], r[1], r[3]);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h][n][i] = CH == 2 ? acc[0][n][i] + acc[CH - 1][n][i] : acc[0][n][i];
        }
        // ---- Online softmax, the references raised where a score passes them by kRaiseAt.
        const int32_t mykey0 = key0 + ks * (kBlk / 2);
        uint32_t bad = 0;
#pragma unroll
        for (int h = 0; h < SUB; ++h) bad |= static_cast<uint32_t>(s_bad[par][ks * SUB + h]) << h;
        edge = edge || bad != 0;
        float y[SUB][2][4];
        auto exponents = [&]() {
#pragma unroll
          for (int h = 0; h < SUB; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                y[h][n][i] = fmaf(x[h][n][i], sca, -m_a);
                y[h][n][2 + i] = fmaf(x[h][n][2 + i], scb, -m_b);
              }
          if (edge) {
#pragma unroll
            for (int h = 0; h < SUB; ++h)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int32_t key = mykey0 + 16 * h + 8 * n + 2 * c + i;
                  const bool no = (bad >> h) & 1u;
                  if (no || key < lo_a || key > hi_a) y[h][n][i] = -INFINITY;
                  if (no || key < lo_b || key > hi_b) y[h][n][2 + i] = -INFINITY;
                }
          }
        };
        exponents();
        float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
        for (int h = 0; h < SUB; ++h)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            ta = fmaxf(ta, fmaxf(y[h][n][0], y[h][n][1]));
            tb = fmaxf(tb, fmaxf(y[h][n][2], y[h][n][3]));
          }
        if (__any_sync(0xffffffffu, fmaxf(ta, tb) > kRaiseAt)) {
          // (From the scores: a difference to the stand-in has lost its low bits.)
          float sa = -INFINITY, sb = -INFINITY;
#pragma unroll
          for (int h = 0; h < SUB; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (y[h][n][i] > -INFINITY) sa = fmaxf(sa, x[h][n][i] * sca);
                if (y[h][n][2 + i] > -INFINITY) sb = fmaxf(sb, x[h][n][2 + i] * scb);
              }
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) {
            sa = fmaxf(sa, __shfl_xor_sync(0xffffffffu, sa, off));
            sb = fmaxf(sb, __shfl_xor_sync(0xffffffffu, sb, off));
          }
          const float na = fmaxf(m_a, sa - kBelowTop), nb = fmaxf(m_b, sb - kBelowTop);
          const float fa = fast_exp2(m_a - na), fb = fast_exp2(m_b - nb);
          m_a = na;
          m_b = nb;
          l_a *= fa;
          l_b *= fb;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            o[t][0] *= fa;
            o[t][1] *= fa;
            o[t][2] *= fb;
            o[t][3] *= fb;
          }
          exponents();
#pragma unroll
          for (int h = 0; h < SUB; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) y[h][n][i] = raised(y[h][n][i]);
        }
        uint32_t pa[SUB][4];
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = fast_exp2(y[h][n][0]), p1 = fast_exp2(y[h][n][1]);
            const float p2 = fast_exp2(y[h][n][2]), p3 = fast_exp2(y[h][n][3]);
            l_a += p0 + p1;
            l_b += p2 + p3;
            pa[h][2 * n] = pack_f16x2(p0, p1);
            pa[h][2 * n + 1] = pack_f16x2(p2, p3);
          }
        }
        // ---- O += P V
#pragma unroll
        for (int h = 0; h < SUB; ++h)
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const int i = kSteps + h * KT + t;
            if (i + kAhead < 2 * kSteps) fetch(i + kAhead);
            const uint32_t(&r)[4] = b[i % (kAhead + 1)];
            mma_f16(o[2 * t], pa[h][0], pa[h][1], pa[h][2], pa[h][3], r[0], r[1]);
            mma_f16(o[2 * t + 1], pa[h][0], pa[h][1], pa[h][2], pa[h][3], r[2], r[3]);
          }
      }
      par ^= 1;
      at_flip();
    }

    // ---- The segment's end in this range: the halves of the keys meet.
    const bool whole = cs.j == 0 && j1 == cs.nb;
    const int32_t key_from = (tl.fb + cs.j) * kBlk, key_to = (tl.fb + j1) * kBlk - 1;
    const int32_t slot = 2 * blockIdx.x + (cs.e == start.tile && cs.g == start.head ? 0 : 1);
    cs.rem -= j1 - cs.j;
    cs.j = j1;
    to_block(cs);
    // The combine may be scheduled now (it waits for this grid's end).
    if (cs.rem <= 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      l_a += __shfl_xor_sync(0xffffffffu, l_a, off);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, off);
    }
    if (ks == 1 && active) {
#pragma unroll
      for (int t = 0; t < D / 8; ++t) mbuf[t * 32] = make_float4(o[t][0], o[t][1], o[t][2], o[t][3]);
      if (c == 0) {
        s_m[rg * 16 + g] = m_a;
        s_m[rg * 16 + g + 8] = m_b;
        s_l[rg * 16 + g] = l_a;
        s_l[rg * 16 + g + 8] = l_b;
      }
    }
    __syncthreads();
    if (ks == 0 && active) {
      if (s_nan == seg)
        each_uneven_nan<D>(p, tl.seq, head, max(key_from, first_visible(all_hi, tl.window)),
                           min(key_to, tl.pos0 + last / G), all_lo, all_hi, [&](int32_t key, uint32_t blocks) {
          const uint32_t in_a = key >= lo_a && key <= hi_a ? blocks : 0u, in_b = key >= lo_b && key <= hi_b ? blocks : 0u;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            if (in_a >> (t >> 1) & 1u) o[t][0] = o[t][1] = quiet_nan();
            if (in_b >> (t >> 1) & 1u) o[t][2] = o[t][3] = quiet_nan();
          }
        });
      const float ma2 = s_m[rg * 16 + g], mb2 = s_m[rg * 16 + g + 8];
      const float Ma = fmaxf(m_a, ma2), Mb = fmaxf(m_b, mb2);
      float fa = fast_exp2(m_a - Ma), fa2 = fast_exp2(ma2 - Ma);
      float fb = fast_exp2(m_b - Mb), fb2 = fast_exp2(mb2 - Mb);
      const float La = fa * l_a + fa2 * s_l[rg * 16 + g], Lb = fb * l_b + fb2 * s_l[rg * 16 + g + 8];
      // (A row without a score has L = 0; a NaN stays.)
      const float ia = La == 0.f ? 0.f : 1.f / La, ib = Lb == 0.f ? 0.f : 1.f / Lb;
      fa *= ia;
      fa2 *= ia;
      fb *= ib;
      fb2 *= ib;
      const bool has_a = ra <= last, has_b = rb <= last;
      const int na = rg * 16 + g, nb = na + 8;
      __nv_bfloat16* const oa = p.out + row_at(min(ra, last)) + 2 * c;
      __nv_bfloat16* const ob = p.out + row_at(min(rb, last)) + 2 * c;
      float* const pa = p.part_o + (static_cast<int64_t>(slot) * Sh::kRows + na) * D + 2 * c;
      float* const pb = p.part_o + (static_cast<int64_t>(slot) * Sh::kRows + nb) * D + 2 * c;
#pragma unroll
      for (int t = 0; t < D / 8; ++t) {
        const float4 u = mbuf[t * 32];
        const float a0 = fa * o[t][0] + fa2 * u.x, a1 = fa * o[t][1] + fa2 * u.y;
        const float b0 = fb * o[t][2] + fb2 * u.z, b1 = fb * o[t][3] + fb2 * u.w;
        if (whole) {
          if (has_a) *reinterpret_cast<uint32_t*>(oa + 8 * t) = pack_bf16x2(a0, a1);
          if (has_b) *reinterpret_cast<uint32_t*>(ob + 8 * t) = pack_bf16x2(b0, b1);
        } else {
          if (has_a) *reinterpret_cast<float2*>(pa + 8 * t) = make_float2(a0, a1);
          if (has_b) *reinterpret_cast<float2*>(pb + 8 * t) = make_float2(b0, b1);
        }
      }
      if (!whole && c == 0) {
        if (has_a) p.part_lse[static_cast<int64_t>(slot) * Sh::kRows + na] = La == 0.f ? -INFINITY : Ma + __log2f(La);
        if (has_b) p.part_lse[static_cast<int64_t>(slot) * Sh::kRows + nb] = Lb == 0.f ? -INFINITY : Mb + __log2f(Lb);
      }
    }
    __syncthreads();  // read: the next segment's may come
  }
  copy_wait<0>();
}

template <int D, int NSEG>
int launch_rows_t(const Plan& plan, const Args& a, const Kv4Params& p, const Plan::Kv4Launch& l, cudaStream_t stream) {
  using Sh = RowsShape<D>;
  return launch_split<D, Sh::kRows, NSEG>(plan, a, p, l, Sh::W * 32, Sh::kBytes, kv4_rows_kernel<Sh, NSEG>, stream);
}
template <int D>
int launch_rows_n(const Plan& plan, const Args& a, const Kv4Params& p, const Plan::Kv4Launch& l, cudaStream_t stream) {
  return l.end - l.begin <= kKv4TilesSmall ? launch_rows_t<D, kKv4TilesSmall>(plan, a, p, l, stream)
                                           : launch_rows_t<D, kKv4TilesLarge>(plan, a, p, l, stream);
}

}  // namespace

Kv4Grain kv4_rows_grain(int32_t head_dim) { return {1, 8192 / head_dim}; }

int launch_kv4_rows(const Plan& plan, const Args& a, const Plan::Kv4Launch& l, void* stream) {
  const Kv4Params p = kv4_params(plan, a);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (plan.d) {
    case 64: return launch_rows_n<64>(plan, a, p, l, s);
    case 128: return launch_rows_n<128>(plan, a, p, l, s);
    default: return launch_rows_n<256>(plan, a, p, l, s);
  }
}

}  // namespace rpa
