// Page tables, slot maps and lengths of a serving step, built on the GPU.
//
// The pages no request holds form a stack: free_pages[0 .. count), the last
// one taken first.  A step that appends new_lens[s] tokens to every request s
// (kv_lens_prev[s] of them cached) takes
//   need_s = ceil((prev_s + new_s) / P) - ceil(prev_s / P)
// pages for it; the k-th page of the step, counted over the requests in order,
// is free_pages[count - 1 - k].  A token's slot is its page times P plus its
// position in the page.  Releasing requests pushes their pages back in
// (request, slot) order, and cutting requests short pushes the pages behind their
// new lengths.  All or nothing: a step that the stack or the slot map cannot hold
// changes nothing and sets the error word.  (A trim of 512 requests takes 4.3 us, of 2048
// requests that drop up to 256 tokens 4.6.)
//
// Integer work on a few kilobytes: what bounds it is latency, so every CTA
// scans all the requests' lengths for itself (L2 reads, two block scans) and
// the CTAs never wait on one another; they then share out the step's tokens
// and pages.  Where an output replaces its input (lengths or the stack's
// height advanced in place) the last CTA to finish, by a counter in the
// workspace header, writes it after all the others have read it.  512 decoding
// requests take 4.9 us, 192 prompts with a slot map of 262144 5.7 us, a release
// among 2048 requests 4.6 us (replayed from a graph): the launch, two dependent
// reads and two scans.
#include <algorithm>

#include "common.cuh"
#include "rpa_internal.h"

namespace rpa {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;                      // requests a thread scans at once
constexpr int kChunk = kThreads * kPer;      // requests scanned at once
constexpr int kWarps = kThreads / 32;

struct TableParams {
  const int32_t* lens;       // build: new_lens; release: the finished flags; trim: drop_lens
  const int32_t* kv_prev;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* count_prev;
  int32_t* cu;
  int32_t* kv;
  int64_t* slots;
  int32_t* count;
  unsigned char* ws;
  int32_t num_seqs, mpps, num_pages, page_size, page_shift, max_tokens;
};

using Kind = TableArgs::Kind;

struct Totals {
  int64_t tokens, pages;
  int32_t bad;
};

// Shared memory of a CTA: one chunk of requests.
struct Chunk {
  int32_t cu[kChunk + 1];    // tokens before each request (build)
  int32_t base[kChunk + 1];  // pages before each request
  int32_t prev[kChunk];      // tokens held (trim: tokens left)
  uint32_t warp_sum[2][kWarps];
  long long tot[2];
  int32_t bad;
};

__device__ __forceinline__ int32_t pages_of(const TableParams& p, int32_t n) {
  return static_cast<int32_t>((static_cast<uint32_t>(n) + (p.page_size - 1)) >> p.page_shift);
}

// Tokens and pages of request s, and whether its lengths are unusable.
template <Kind kKind>
__device__ __forceinline__ void request(const TableParams& p, int32_t s, int32_t& prev,
                                        int32_t& tok, int32_t& pg, bool& bad) {
  prev = p.kv_prev[s];
  const int32_t n = p.lens[s];
  tok = pg = 0;
  if constexpr (kKind == Kind::kRelease) {
    if (n == 0) return;
    bad = prev < 0 || pages_of(p, prev) > p.mpps;
    if (!bad) pg = pages_of(p, prev);
  } else if constexpr (kKind == Kind::kTrim) {
    bad = n < 0 || n > prev || pages_of(p, prev) > p.mpps;
    if (!bad) {
      pg = pages_of(p, prev) - pages_of(p, prev - n);
      prev -= n;
    }
  } else {
    const int64_t sum = static_cast<int64_t>(prev) + n;
    bad = prev < 0 || n < 0 || sum > 0x7fffffff - p.page_size ||
          pages_of(p, static_cast<int32_t>(sum)) > p.mpps;
    if (!bad) {
      tok = n;
      pg = pages_of(p, static_cast<int32_t>(sum)) - pages_of(p, prev);
    }
  }
}

// Exclusive prefix sums of the chunk of requests from c0 on into shared
// memory, continuing from (tok0, pg0); the chunk's sums are added to the
// totals.  Every thread of the CTA takes part; ends with a barrier.
template <Kind kKind>
__device__ __forceinline__ void scan_chunk(const TableParams& p, Chunk& ch, int32_t c0, uint32_t tok0,
                           uint32_t pg0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t t[kPer], g[kPer];
  uint32_t st = 0, sg = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int32_t l = tid * kPer + i, s = c0 + l;
    int32_t prev = 0, tok = 0, pg = 0;
    bool bad = false;
    if (s < p.num_seqs) request<kKind>(p, s, prev, tok, pg, bad);
    ch.prev[l] = prev;
    t[i] = st;
    g[i] = sg;
    st += static_cast<uint32_t>(tok);
    sg += static_cast<uint32_t>(pg);
  }
  uint32_t xt = st, xg = sg;  // inclusive over the warp
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, xt, off);
    const uint32_t b = __shfl_up_sync(0xffffffffu, xg, off);
    if (lane >= off) {
      xt += a;
      xg += b;
    }
  }
  if (lane == 31) {
    ch.warp_sum[0][warp] = xt;
    ch.warp_sum[1][warp] = xg;
  }
  __syncthreads();
  uint32_t bt = tok0, bg = pg0;
  for (int w = 0; w < warp; ++w) {
    bt += ch.warp_sum[0][w];
    bg += ch.warp_sum[1][w];
  }
  bt += xt - st;
  bg += xg - sg;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    ch.cu[tid * kPer + i] = static_cast<int32_t>(bt + t[i]);
    ch.base[tid * kPer + i] = static_cast<int32_t>(bg + g[i]);
  }
  if (tid == kThreads - 1) {
    ch.cu[kChunk] = static_cast<int32_t>(bt + st);
    ch.base[kChunk] = static_cast<int32_t>(bg + sg);
  }
  __syncthreads();
}

// The step's totals, in 64 bits (every thread of the CTA returns them).
template <Kind kKind>
__device__ __forceinline__ Totals totals(const TableParams& p, Chunk& ch) {
  if (threadIdx.x == 0) {
    ch.tot[0] = ch.tot[1] = 0;
    ch.bad = 0;
  }
  __syncthreads();
  long long tok_sum = 0, pg_sum = 0;
  bool any_bad = false;
  for (int32_t s = threadIdx.x; s < p.num_seqs; s += kThreads) {
    int32_t prev, tok, pg;
    bool bad = false;
    request<kKind>(p, s, prev, tok, pg, bad);
    tok_sum += tok;
    pg_sum += pg;
    any_bad |= bad;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    tok_sum += __shfl_xor_sync(0xffffffffu, tok_sum, off);
    pg_sum += __shfl_xor_sync(0xffffffffu, pg_sum, off);
  }
  any_bad = __any_sync(0xffffffffu, any_bad);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&ch.tot[0]), static_cast<unsigned long long>(tok_sum));
    atomicAdd(reinterpret_cast<unsigned long long*>(&ch.tot[1]), static_cast<unsigned long long>(pg_sum));
    if (any_bad) ch.bad = 1;
  }
  __syncthreads();
  return Totals{ch.tot[0], ch.tot[1], ch.bad};
}

// Largest i in [0, kChunk) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int owner(const int32_t* a, int32_t x) {
  int lo = 0, hi = kChunk - 1;
#pragma unroll
  for (int k = 0; k < 11; ++k) {  // 2^11 = kChunk
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
static_assert(kChunk == 1 << 11, "search depth");

// Page k of the step, or -1 (and the error word) where the stack holds no page id.
__device__ __forceinline__ int32_t take_page(const TableParams& p, int32_t count, int32_t k) {
  const int32_t page = __ldg(p.free_pages + (count - 1 - k));
  if (page < 0 || page >= p.num_pages) {
    report_error(p.ws, RPA_DEVERR_PAGE_ID, k);
    return -1;
  }
  return page;
}

// The last CTA of the grid to arrive (the counter goes back to zero); every
// thread of the CTA gets the answer.
__device__ __forceinline__ bool last_cta(unsigned char* ws) {
  __shared__ int32_t s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    int32_t* ctr = reinterpret_cast<int32_t*>(ws + kTablesCounterOff);
    __threadfence();
    s_last = atomicAdd(ctr, 1) == static_cast<int32_t>(gridDim.x) - 1;
    if (s_last) atomicExch(ctr, 0);
  }
  __syncthreads();
  return s_last != 0;
}

// New lengths and stack height.  In place (kv == kv_prev, count == count_prev)
// the last CTA writes them, else the CTAs between them as they go.
template <Kind kKind>
__device__ __forceinline__ void write_state(const TableParams& p, bool ok, int32_t count_new) {
  const bool kv_in_place = p.kv == p.kv_prev, count_in_place = p.count == p.count_prev;
  auto lengths = [&](int32_t first, int32_t step) {
    for (int32_t s = first; s < p.num_seqs; s += step) {
      const int32_t prev = p.kv_prev[s], n = p.lens[s];
      if (!ok)
        p.kv[s] = prev;
      else if (kKind == Kind::kRelease)
        p.kv[s] = n != 0 ? 0 : prev;
      else
        p.kv[s] = kKind == Kind::kTrim ? prev - n : prev + n;
    }
  };
  if (!kv_in_place) lengths(blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
  if (!count_in_place && blockIdx.x == 0 && threadIdx.x == 0) *p.count = count_new;
  if (!kv_in_place && !count_in_place) return;
  if (gridDim.x > 1 && !last_cta(p.ws)) return;
  if (gridDim.x == 1) __syncthreads();
  if (kv_in_place) lengths(threadIdx.x, kThreads);
  if (count_in_place && threadIdx.x == 0) *p.count = count_new;
}

__global__ void __launch_bounds__(kThreads) build_tables_kernel(const TableParams p) {
  __shared__ Chunk ch;
  const int32_t gtid = blockIdx.x * kThreads + threadIdx.x, gstep = gridDim.x * kThreads;
  const int32_t count = *p.count_prev;
  const Totals tot = totals<Kind::kBuild>(p, ch);
  const bool ok = !tot.bad && tot.tokens <= p.max_tokens && count >= 0 && count <= p.num_pages &&
                  tot.pages <= count;
  if (!ok && gtid == 0)
    report_error(p.ws, tot.bad || tot.tokens > p.max_tokens ? RPA_DEVERR_LENGTHS : RPA_DEVERR_PAGES,
                 0);
  const int32_t total = ok ? static_cast<int32_t>(tot.tokens) : 0;
  for (int32_t t = total + gtid; t < p.max_tokens; t += gstep) p.slots[t] = -1;
  if (!ok) {
    for (int32_t s = gtid; s <= p.num_seqs; s += gstep) p.cu[s] = 0;
    write_state<Kind::kBuild>(p, false, count);
    return;
  }
  uint32_t tok0 = 0, pg0 = 0;
  for (int32_t c0 = 0; c0 < p.num_seqs; c0 += kChunk) {
    scan_chunk<Kind::kBuild>(p, ch, c0, tok0, pg0);
    const int32_t tok1 = ch.cu[kChunk], pg1 = ch.base[kChunk];
    const int32_t n = min(kChunk, p.num_seqs - c0);
    for (int32_t l = gtid; l < n; l += gstep) p.cu[c0 + l] = ch.cu[l];
    for (int32_t t = static_cast<int32_t>(tok0) + gtid; t < tok1; t += gstep) {
      const int l = owner(ch.cu, t);
      const int32_t prev = ch.prev[l];
      const int32_t pos = prev + (t - ch.cu[l]);
      const int32_t j = pos >> p.page_shift, held = pages_of(p, prev);
      int32_t page;
      if (j < held) {
        page = __ldg(p.table + static_cast<int64_t>(c0 + l) * p.mpps + j);
        if (page < 0 || page >= p.num_pages) {
          report_error(p.ws, RPA_DEVERR_PAGE_ID, c0 + l);
          page = -1;
        }
      } else {
        page = take_page(p, count, ch.base[l] + (j - held));
      }
      p.slots[t] = page < 0 ? -1
                            : (static_cast<int64_t>(page) << p.page_shift) +
                                  (pos & (p.page_size - 1));
    }
    for (int32_t k = static_cast<int32_t>(pg0) + gtid; k < pg1; k += gstep) {
      const int l = owner(ch.base, k);
      p.table[static_cast<int64_t>(c0 + l) * p.mpps + pages_of(p, ch.prev[l]) + (k - ch.base[l])] =
          take_page(p, count, k);
    }
    tok0 = static_cast<uint32_t>(tok1);
    pg0 = static_cast<uint32_t>(pg1);
    __syncthreads();  // the next chunk overwrites this one
  }
  if (gtid == 0) p.cu[p.num_seqs] = total;
  write_state<Kind::kBuild>(p, true, count - static_cast<int32_t>(tot.pages));
}

// Pages pushed back: those of finished requests (kRelease), or those behind the new
// lengths (kTrim).
template <Kind kKind>
__global__ void __launch_bounds__(kThreads) release_tables_kernel(const TableParams p) {
  __shared__ Chunk ch;
  const int32_t gtid = blockIdx.x * kThreads + threadIdx.x, gstep = gridDim.x * kThreads;
  const int32_t count = *p.count_prev;
  const Totals tot = totals<kKind>(p, ch);
  const bool ok = !tot.bad && count >= 0 && count + tot.pages <= p.num_pages;
  if (!ok) {
    if (gtid == 0) report_error(p.ws, tot.bad ? RPA_DEVERR_LENGTHS : RPA_DEVERR_PAGES, 0);
    write_state<kKind>(p, false, count);
    return;
  }
  uint32_t pg0 = 0;
  for (int32_t c0 = 0; c0 < p.num_seqs; c0 += kChunk) {
    scan_chunk<kKind>(p, ch, c0, 0, pg0);
    const int32_t pg1 = ch.base[kChunk];
    for (int32_t k = static_cast<int32_t>(pg0) + gtid; k < pg1; k += gstep) {
      const int l = owner(ch.base, k);
      const int32_t first = kKind == Kind::kTrim ? pages_of(p, ch.prev[l]) : 0;
      int32_t page = __ldg(p.table + static_cast<int64_t>(c0 + l) * p.mpps + first + (k - ch.base[l]));
      if (page < 0 || page >= p.num_pages) {
        report_error(p.ws, RPA_DEVERR_PAGE_ID, c0 + l);
        page = -1;
      }
      p.free_pages[count + k] = page;
    }
    pg0 = static_cast<uint32_t>(pg1);
    __syncthreads();
  }
  write_state<kKind>(p, true, count + static_cast<int32_t>(tot.pages));
}

}  // namespace

int launch_tables(const TableArgs& a, void* stream) {
  TableParams p;
  p.lens = a.lens;
  p.kv_prev = a.kv_lens_prev;
  p.table = a.page_table;
  p.free_pages = a.free_pages;
  p.count_prev = a.free_count_prev;
  p.cu = a.cu_q_lens;
  p.kv = a.kv_lens;
  p.slots = a.slot_map;
  p.count = a.free_count;
  p.ws = a.workspace;
  p.num_seqs = a.num_seqs;
  p.mpps = a.mpps;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  int shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  p.page_shift = shift;
  p.max_tokens = a.max_tokens;
  // One CTA per 512 tokens (build) or pages (release, trim: at most the pool's) of
  // the step, one wave at most.
  const int64_t items = a.kind == Kind::kBuild
                            ? a.max_tokens
                            : std::min<int64_t>(static_cast<int64_t>(a.num_seqs) * a.mpps, a.num_pages);
  const int64_t most = std::max<int64_t>(items, a.num_seqs);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((most + kThreads - 1) / kThreads, 152)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int mark = RPA_KERNEL_BUILD_TABLES;
  if (a.kind == Kind::kBuild) {
    build_tables_kernel<<<grid, kThreads, 0, s>>>(p);
  } else if (a.kind == Kind::kRelease) {
    release_tables_kernel<Kind::kRelease><<<grid, kThreads, 0, s>>>(p);
    mark = RPA_KERNEL_RELEASE_TABLES;
  } else {
    release_tables_kernel<Kind::kTrim><<<grid, kThreads, 0, s>>>(p);
    mark = RPA_KERNEL_TRIM_TABLES;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  trace_mark(mark, stream);
  return 0;
}

}  // namespace rpa
