// What the split-KV kernels over 4-bit pages share: their parameters, the line
// of segments and its cut into the CTAs' ranges, the combine of the segments cut
// across CTAs, and the launch.
#pragma once

#include "common.cuh"
#include "kv4.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

struct Kv4Params {
  const __nv_bfloat16* q;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  const int32_t* page_table;
  __nv_bfloat16* out;
  unsigned char* ws;
  float* part_o;    // [2 * CTAs][rows][D]
  float* part_lse;  // [2 * CTAs][rows]
  float4* piece_o;  // [CTAs * warps][accumulator tiles][32 lanes]
  int32_t hq, hkv, group, page_shift, mpps, num_pages;
  float scale_log2;
};

// One launch's row tiles: tile e covers rows [r0, r0 + nrows) of sequence seq,
// whose first query token is q0, at position pos0.  Its segments (one per KV
// head) have nb blocks from block fb on.  The CTAs' ranges of the line, by
// where they start: block j of segment (tile, head), and their length
// (blocks and merge charges); computed by the plan, since a search for it
// would cost a CTA several misses of the constant cache before its first copy.
struct Kv4Tile {
  int32_t seq, q0, r0, nrows, pos0, window, fb, nb;
};
struct Kv4Start {
  int32_t tile, head, j, len;
};
template <int NSEG>
struct Kv4Sched {
  Kv4Start cta[kKv4MaxCtas];
  Kv4Tile tile[NSEG];
  // What check_lengths compares with the tiles.  (Here, not in Kv4Params: with
  // the arrays above 24 bytes further on in the parameters a sequence of 128 rows
  // took 26.1 us instead of 22.9.)
  const int32_t* cu_q_lens;
  const int32_t* kv_lens;
  int32_t n_tiles, num_seqs, total_q;
};

// Whether the device's lengths are the plan's, by which the tiles were cut: each
// CTA looks at its share of the tiles, while its first copies are on their way.
// (Out of line: inlined, it took up to 27 registers from the kernels' loops.)
__device__ __noinline__ void check_lengths(const Kv4Tile* tiles, int t, int n_tiles, const int32_t* cu_q_lens,
                                           const int32_t* kv_lens, int32_t num_seqs, int32_t total_q,
                                           unsigned char* ws) {
  for (; t < n_tiles; t += gridDim.x * blockDim.x) {
    const Kv4Tile& tl = tiles[t];
    const int32_t* cu = cu_q_lens + tl.seq;
    const int32_t q0 = __ldg(cu), q1 = __ldg(cu + 1), kv = __ldg(kv_lens + tl.seq), total = __ldg(cu_q_lens + num_seqs);
    if (q0 != tl.q0 || kv - (q1 - q0) != tl.pos0 || total != total_q) report_error(ws, RPA_DEVERR_LENGTHS, tl.seq);
  }
}

// A place on the line: segment (e, g) entered at block j, rem units of the
// range left from there.
struct Place {
  int32_t e, g, j, rem;
  int32_t nb;
};
template <int NSEG>
__device__ __forceinline__ void place_next(const Kv4Sched<NSEG>& sc, const Kv4Params& p, Place& s) {
  s.rem -= s.nb + kKv4SegCost - s.j;
  s.j = 0;
  if (++s.g == p.hkv) {
    s.g = 0;
    ++s.e;
  }
  if (s.rem > 0) s.nb = sc.tile[s.e].nb;
}
// The place `off` units further on (0 <= off <= rem).
template <int NSEG>
__device__ __forceinline__ void place_skip(const Kv4Sched<NSEG>& sc, const Kv4Params& p, Place& s, int32_t off) {
  while (off > 0 && off >= s.nb + kKv4SegCost - s.j) {
    off -= s.nb + kKv4SegCost - s.j;
    place_next(sc, p, s);
  }
  s.j += off;
  s.rem -= off;
}

// 16 bytes from global to shared memory; zeros where src_bytes is 0.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int WORDS>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (WORDS == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t bit_select(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xca;" : "=r"(r) : "r"(m), "r"(a), "r"(b));
  return r;
}

// NaN in V at keys that some rows of a tile see and others do not.  In the
// product it would reach every row (0 times NaN), so such scales are zeroed as
// the block is widened, and a segment that had one looks its uneven keys'
// scales up again at its end and puts the NaN into the rows that see them.

// The 16-dimension blocks of `key`'s row of V that read as NaN, a bit each.
template <int D>
__device__ __forceinline__ uint32_t nan_blocks(const Kv4Params& p, int32_t seq, int32_t head, int32_t key) {
  const int32_t slot = key >> p.page_shift;
  if (slot >= p.mpps) return 0;
  const int32_t page = __ldg(p.page_table + static_cast<int64_t>(seq) * p.mpps + slot);
  if (page < 0 || page >= p.num_pages) return 0;
  const int64_t row = ((static_cast<int64_t>(page) * p.hkv + head) << p.page_shift) +
                      (key & ((1 << p.page_shift) - 1));
  return kv4::nan_blocks<D>(p.vs + row * (D / 16));
}

// Calls f(key, blocks) for the keys in [first, last] with such blocks that not
// every row sees (every row sees [all_lo, all_hi]).
template <int D, typename F>
__device__ __forceinline__ void each_uneven_nan(const Kv4Params& p, int32_t seq, int32_t head, int32_t first,
                                                int32_t last, int32_t all_lo, int32_t all_hi, F&& f) {
#pragma unroll 1
  for (int32_t key = first; key <= last; ++key) {
    if (key >= all_lo && key <= all_hi) {
      key = all_hi;
      continue;
    }
    if (const uint32_t blocks = nan_blocks<D>(p, seq, head, key)) f(key, blocks);
  }
}
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7fffffffu); }

// The column reference before any score: below every scaled score that is not
// -inf itself, and small enough that a score minus it is still finite.
constexpr float kNoScore = -1e38f;
// A column's reference is this much below its largest score when it is raised,
// which is where a score passes it by kRaiseAt: probabilities up to 2^15 fit f16,
// and those down to 2^-24 of the score that raised it keep all their bits (with
// the reference at the score itself down to 2^-14: what 200 keys of 2^-20.4 of the
// largest add up to came out 4% off).
constexpr float kBelowTop = 10.f, kRaiseAt = 15.f;
// An exponent against a raised reference: of scores beyond 2^26, whose steps are
// 8 and more, the difference may round past what f16 holds.
__device__ __forceinline__ float raised(float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kRaiseAt));
  return r;
}

// The segments cut across CTAs: out = sum_c 2^(lse_c - M) O_c / sum_c 2^(lse_c - M)
// over the CTAs that hold a part.  One CTA per boundary between two ranges;
// the first boundary inside a segment takes it, one warp per row.
template <int D, int ROWS, int NSEG>
__global__ void __launch_bounds__(256)
kv4_combine_kernel(const Kv4Params p, const __grid_constant__ Kv4Sched<NSEG> sc) {
  constexpr int E = D / 32;
  const int b = blockIdx.x + 1;
  const Kv4Start s = sc.cta[b], before = sc.cta[b - 1];
  const Kv4Tile& tl = sc.tile[s.tile];
  const bool same = before.tile == s.tile && before.head == s.head;
  const bool mine = s.j > 0 && s.j < tl.nb && !(same && before.j > 0);
  int parts = 2;
  if (mine)
    while (b - 1 + parts <= static_cast<int>(gridDim.x) && sc.cta[b - 1 + parts].tile == s.tile &&
           sc.cta[b - 1 + parts].head == s.head && sc.cta[b - 1 + parts].j < tl.nb)
      ++parts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const int lane = threadIdx.x & 31;
  for (int n = blockIdx.y * 8 + (threadIdx.x >> 5); n < tl.nrows; n += 8 * gridDim.y) {
    // The first part is its CTA's first segment only if the range starts with it.
    auto slot = [&](int k) {
      return static_cast<int64_t>(2 * (b - 1 + k) + (k == 0 && !same ? 1 : 0)) * ROWS + n;
    };
    // The first parts' rows are on their way while the log-sum-exps come.
    constexpr int kAhead = 4;
    float2 first[kAhead][E / 2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int e = 0; e < E; e += 2)
        first[k][e / 2] = k < parts ? *reinterpret_cast<const float2*>(p.part_o + slot(k) * D + lane * E + e)
                                    : make_float2(0.f, 0.f);
    const float lse0 = lane < parts ? p.part_lse[slot(lane)] : -INFINITY;
    float M = lse0;
    for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, p.part_lse[slot(k)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float acc[E], wsum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < parts; k0 += 32) {
      const int nk = min(32, parts - k0);
      const float lse = k0 == 0 ? lse0 : lane < nk ? p.part_lse[slot(k0 + lane)] : -INFINITY;
      const float w_l = lse == -INFINITY ? 0.f : fast_exp2(lse - M);
      auto add = [&](int k, const float2* row) {
        const float w = __shfl_sync(0xffffffffu, w_l, k);
        wsum += w;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          acc[e] = fmaf(w, row[e / 2].x, acc[e]);
          acc[e + 1] = fmaf(w, row[e / 2].y, acc[e + 1]);
        }
      };
      if (k0 == 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (k < nk) add(k, first[k]);
      }
      for (int k = k0 == 0 ? kAhead : 0; k < nk; ++k) {
        float2 row[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2)
          row[e / 2] = *reinterpret_cast<const float2*>(p.part_o + slot(k0 + k) * D + lane * E + e);
        add(k, row);
      }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    const int r = tl.r0 + n;
    __nv_bfloat16* dst = p.out +
        (static_cast<int64_t>(tl.q0 + r / p.group) * p.hq + s.head * p.group + r % p.group) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

inline Kv4Params kv4_params(const Plan& plan, const Args& a) {
  Kv4Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k_pages);
  p.v = static_cast<const uint8_t*>(a.v_pages);
  p.ks = a.k_block_scales;
  p.vs = a.v_block_scales;
  p.page_table = a.page_table;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ws = a.workspace;
  p.part_o = reinterpret_cast<float*>(a.workspace + plan.off_partial_o);
  p.part_lse = reinterpret_cast<float*>(a.workspace + plan.off_partial_lse);
  p.piece_o = reinterpret_cast<float4*>(a.workspace + plan.off_kv4_pieces);
  p.hq = plan.hq;
  p.hkv = plan.hkv;
  p.group = plan.hq / plan.hkv;
  int shift = 0;
  while ((1 << shift) < plan.p) ++shift;
  p.page_shift = shift;
  p.mpps = plan.mpps;
  p.num_pages = plan.num_pages;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  return p;
}

// The launch of a split-KV kernel over one launch's tiles, and of the combine.
template <int D, int ROWS, int NSEG>
int launch_split(const Plan& plan, const Args& a, const Kv4Params& p, const Plan::Kv4Launch& l, int threads, int smem,
                 void (*kernel)(const Kv4Params, const Kv4Sched<NSEG>), cudaStream_t stream) {
  if (int e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return e;
  Kv4Sched<NSEG>& sc = thread_staging<Kv4Sched<NSEG>>();  // copied into the launch parameters
  for (int i = l.begin; i < l.end; ++i) {
    const Plan::Kv4Tile& t = plan.kv4_tiles[i];
    sc.tile[i - l.begin] = Kv4Tile{t.seq, t.q0, t.r0, t.nrows, t.pos0, t.window, t.fb, t.nb};
  }
  sc.cu_q_lens = a.cu_q_lens;
  sc.kv_lens = a.kv_lens;
  sc.n_tiles = l.end - l.begin;
  sc.num_seqs = plan.num_seqs;
  sc.total_q = static_cast<int32_t>(plan.total_q);
  for (int i = 0; i < l.n_ctas; ++i) {
    const Plan::Kv4Start& c = plan.kv4_starts[l.cta_begin + i];
    sc.cta[i] = Kv4Start{c.tile, c.head, c.j, c.len};
  }
  kernel<<<l.n_ctas, threads, smem, stream>>>(p, sc);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  trace_mark(RPA_KERNEL_KV4_DECODE, stream);
  if (!l.cut) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.n_ctas - 1, ROWS > 16 ? ROWS / 8 : 1);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, ROWS, NSEG>, p, sc);
  if (e != cudaSuccess) return static_cast<int>(e);
  trace_mark(RPA_KERNEL_KV4_COMBINE, stream);
  return 0;
}

}  // namespace
}  // namespace rpa
