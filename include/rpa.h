/*
 * librpa: ragged paged attention on one NVIDIA GB300 (sm_103a).
 *
 * What the library computes (sources named by page title and section):
 *
 *  - "TPU Deep Dive" slides, chapter 8, "Continuous batching with static
 *    shapes": a serving step flattens every query token of every sequence into
 *    one array, and per-sequence metadata carries the ragged structure.  Here
 *    that is q[total_q, Hq, D] with cu_q_lens[num_seqs + 1] (prefix sums of the
 *    per-sequence query counts) and kv_lens[num_seqs].
 *  - Same deck, chapter 8, "KV cache layout", and "Pallas kernel / vLLM on TPU
 *    ... 19,511 tokens per second", section "Strategy 3": the KV cache is
 *    paged in fixed-size blocks (128 tokens there); each sequence reaches its
 *    blocks through a page table.  Here k_pages / v_pages are
 *    [num_pages, page_size, Hkv, D] and page_table is
 *    [num_seqs, max_pages_per_seq] int32 holding physical page ids.
 *  - "Chasing speed of light on TPU v6e", section "Attention" and footnote 5:
 *    the result is exact softmax attention over every key a query may see;
 *    sliding-window layers let a key be seen by the W queries that follow it
 *    (itself included).  Footnote 6: softmax accumulators are fp32.
 *  - "Pallas kernel / vLLM on TPU ...", section "Strategy 3": several query
 *    heads share one KV head (GQA/MQA); query head h reads KV head
 *    h / (Hq / Hkv).
 *
 * For sequence s with q_len = cu_q_lens[s+1] - cu_q_lens[s] and L = kv_lens[s],
 * query i (token t = cu_q_lens[s] + i) sits at position pos = L - q_len + i: the
 * new tokens are the last q_len entries of the cache, already written there
 * (by the caller, or first by rpa_forward_kv / rpa_forward_qkv, the fused KV
 * write of "TPU Deep Dive" chapter 8).  Key j is visible iff j <= pos and,
 * when window[s] > 0,
 * pos - j < window[s].  For every query head h:
 *     out[t][h] = sum_j softmax_j(sm_scale * q[t][h] . k_j) v_j
 * accumulated in fp32 and stored in the output dtype (bf16: round to nearest
 * even).
 *
 * Ownership and threading.  The caller owns every device buffer (q, pages,
 * metadata, out, workspace) and the CUDA stream.  rpa_forward allocates no
 * device memory, never synchronises, and enqueues its work on `stream` only.
 * A plan is a host object owned by the library between rpa_plan and
 * rpa_plan_destroy; it is read-only after creation, so one plan may serve many
 * rpa_forward calls (for instance every layer of a model step).  Two calls
 * that share a workspace must not overlap on the GPU.  Several host threads
 * may call at once, each with the stream's device current (see rpa_forward).
 * The calls enqueue kernels only, so they can be captured into CUDA graphs.
 *
 * Errors.  Every entry point returns an rpa_status_t.  Shapes, dtypes,
 * pointer alignment and the plan/argument match are checked on the host before
 * anything is enqueued; a failed check enqueues nothing.  Problems only the GPU
 * can see (a page id outside [0, num_pages), lengths that disagree with the
 * plan) are never trapped: the kernel skips the bad access, writes a code into
 * the workspace error word and carries on; rpa_get_device_error reads it.
 */
#ifndef RPA_H_
#define RPA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so that this header needs no CUDA
 * header.  NULL means the legacy default stream. */
typedef struct CUstream_st* rpa_stream_t;

typedef int32_t rpa_status_t;
enum {
  RPA_OK = 0,
  RPA_ERR_INVALID_ARG = -1,          /* null pointer, bad shape or metadata   */
  RPA_ERR_UNSUPPORTED = -2,          /* head_dim / page_size / dtype / ratio  */
  RPA_ERR_WORKSPACE_TOO_SMALL = -3,  /* workspace_bytes below the plan's need */
  RPA_ERR_CUDA = -4,                 /* a CUDA runtime call failed            */
  RPA_ERR_DEVICE = -5,               /* the device error word is set          */
  RPA_ERR_PLAN_MISMATCH = -6         /* forward arguments differ from plan's  */
};

/* Element types of q, k_pages, v_pages and out (all four share one). */
enum { RPA_DTYPE_BF16 = 0, RPA_DTYPE_F32 = 1,
       RPA_DTYPE_FP8_E4M3 = 2 /* K/V pages only: OCP e4m3 bytes (bias 7, 3-bit
                                 mantissa, max 448), a float scale per KV head */,
       RPA_DTYPE_FP4_E2M1 = 3 /* K/V pages only: 4-bit codes with a scale byte
                                 per 16 dimensions (see rpa_write_kv4)         */ };

/* Codes written into the workspace error word by the kernels. */
enum {
  RPA_DEVERR_NONE = 0,
  RPA_DEVERR_PAGE_ID = 1,    /* a page-table entry outside [0, num_pages)       */
  RPA_DEVERR_LENGTHS = 2,    /* device lengths disagree with the plan's copies  */
  RPA_DEVERR_PLAN = 3,       /* the work list in the workspace is not this plan */
  RPA_DEVERR_TIMEOUT = 4,    /* a bounded wait inside a kernel gave up          */
  RPA_DEVERR_LAUNCH = 5,     /* a kernel found its launch unusable (shared
                                memory base not 1024-byte aligned) and did
                                nothing                                        */
  RPA_DEVERR_PAGES = 6       /* the stack of free pages is too short for a
                                step's tokens, or too full for a release (see
                                rpa_build_tables): nothing was changed         */
};

/* Kernel paths a plan may use. */
enum {
  RPA_PATH_AUTO = 0,   /* tensor-core prefill + split-KV decode where supported */
  RPA_PATH_SIMT = 1,   /* plain fp32 CUDA-core kernel for every sequence        */
  RPA_PATH_TC = 2      /* tensor-core paths; RPA_ERR_UNSUPPORTED if impossible  */
};

/* Split-KV decode kernels (rpa_plan_options.decode_kernel). */
enum {
  RPA_DECODE_KERNEL_AUTO = 0, /* the planner's choice                            */
  RPA_DECODE_KERNEL_MMA = 1,  /* CUDA-core warp MMAs (mma.sync): every decode
                                 shape of the tensor-core path, fp8 pages too   */
  RPA_DECODE_KERNEL_TC = 2    /* tensor cores (tcgen05.mma, accumulators in
                                 tensor memory): bf16 pages, head_dim 128 or
                                 256, G <= 8, page_size >= 16; else
                                 RPA_ERR_UNSUPPORTED                            */
};

/* Optional knobs for rpa_plan.  Zero-initialise and set struct_size. */
typedef struct rpa_plan_options {
  int32_t struct_size;      /* sizeof(rpa_plan_options)                         */
  int32_t path;             /* RPA_PATH_*                                       */
  int32_t q_block;          /* prefill query block, tokens (0: choose).  At most
                               one 128-row tile per CTA: 128 / G tokens (G =
                               num_q_heads / num_kv_heads); twice that runs on
                               SM pairs (as prefill_pairs = 2, half the block
                               per SM, head_dim 128 or 256); larger blocks are
                               refused with RPA_ERR_UNSUPPORTED             */
  int32_t kv_split;         /* decode split length, tokens (0: choose)          */
  int32_t num_sms;          /* SMs to plan for (0: ask the current device, else 152) */
  int32_t prefill_pairs;    /* tensor-core prefill on SM pairs (one M = 256 MMA
                               over two adjacent query blocks): 0 or 1 not
                               used (single-SM kernel), 2 required (else
                               RPA_ERR_UNSUPPORTED; head_dim 128 or 256)        */
  int32_t kv_dtype;         /* dtype of the K/V pages: 0 or `dtype` (the same),
                               or RPA_DTYPE_FP8_E4M3 with dtype BF16: decode
                               batches only (every q_len <= 1), head_dim 128 or
                               256, run through rpa_forward_fp8kv; or
                               RPA_DTYPE_FP4_E2M1 with dtype BF16, any q_len,
                               page_size >= 16, num_q_heads / num_kv_heads <=
                               128 (and at most 256 KV heads where a sequence
                               runs on the prefill), run through
                               rpa_forward_kv4 (of the other
                               options it takes path AUTO or TC, q_block of one
                               tile, num_sms, decode_sms, prefill_dynamic and
                               prefill_grouping; the rest must be 0, else
                               RPA_ERR_UNSUPPORTED)                             */
  int32_t prefill_split;    /* 0 or -1: whole prefill work items; n > 0: lay
                               the items' key tiles (128 keys each) end to end
                               and cut them into ranges of n tiles, one per
                               CTA; items crossing a range boundary run as
                               parts whose fp32 partials a combine kernel
                               merges                                           */
  int32_t decode_sms;       /* batches with both decode and tensor-core prefill
                               work: 0 let the planner split the SMs between
                               the two persistent grids (HBM-bound decode,
                               tensor-bound prefill) and run them side by side,
                               or not when its cost model says one after the
                               other is faster; n > 0: decode on n SMs,
                               prefill on the rest; -1: one after the other,
                               each on every SM                                 */
  int32_t decode_kernel;    /* RPA_DECODE_KERNEL_* for the split-KV decode      */
  int32_t prefill_dynamic;  /* tensor-core prefill (single-SM kernel, whole
                               items): 0 items taken longest first by whichever
                               CTA gets free (a work counter in the workspace
                               header), -1 each CTA runs the list the planner
                               gave it (longest processing time first)         */
  int32_t prefill_grouping; /* dynamic prefill list: 0 group the (sequence, KV
                               head) pairs so that items sharing keys run
                               together when every prefill sequence sees its
                               whole prefix and their K and V outgrow L2
                               (DRAM reads near the algorithmic bytes, ~1%
                               longer on the causal 8k prefill), -1 longest
                               first over the whole batch                      */
  int32_t tree_words;       /* 0: none of the below.  1..16: a plan for
                               rpa_forward_tree, whose masks have that many
                               64-bit words a row (every q_len at most 64 times
                               as many); of the other options it takes path and
                               num_sms, the rest must be 0, and every kv_len
                               is at most 2^31 - 1024, else
                               RPA_ERR_UNSUPPORTED                              */
} rpa_plan_options;

/* What a plan chose; filled by rpa_plan_get_info. */
typedef struct rpa_plan_info {
  int32_t path;             /* RPA_PATH_SIMT or RPA_PATH_TC                     */
  int32_t num_decode_seqs;  /* sequences with q_len == 1 (4-bit pages: those of
                               few query rows, on the split-KV kernel; trees:
                               requests with nodes)                             */
  int32_t num_prefill_seqs; /* sequences with q_len > 1 (4-bit pages: the
                               others, on the tensor-core prefill)              */
  int32_t q_block;          /* prefill query block in tokens (query tokens of
                               one work item; on SM pairs, of both CTAs)     */
  int32_t kv_split;         /* decode split length in tokens (trees: keys of the
                               longest CTA range)                               */
  int32_t max_splits;       /* largest split count of any decode sequence (trees:
                               of any segment)                                  */
  int32_t num_prefill_items;/* (sequence, query block, kv head) work items      */
  int32_t prefill_ctas;     /* persistent prefill CTAs launched                 */
  int64_t workspace_bytes;  /* bytes rpa_forward needs                          */
  int32_t prefill_pairs;    /* 1: prefill runs on SM pairs, items are pairs of
                               query blocks                                     */
  int32_t kv_dtype;         /* dtype of the K/V pages (RPA_DTYPE_*)              */
  int32_t prefill_split_items; /* prefill items split across CTAs              */
  int32_t prefill_split_parts; /* parts those items became                     */
  int32_t prefill_max_tiles;   /* key tiles of the busiest prefill CTA        */
  int32_t decode_sms;          /* mixed batch run side by side: SMs of the
                                  decode grid (0: not side by side)          */
  int32_t prefill_sms;         /* ... and of the prefill grid                 */
  int32_t decode_kernel;       /* RPA_DECODE_KERNEL_MMA or _TC for the
                                  split-KV decode (0: no such decode)         */
  int32_t prefill_dynamic;     /* 1: prefill CTAs take items as they get free */
  int32_t prefill_groups;      /* dynamic prefill list: groups of (sequence,
                                  KV head) pairs run one after the other so
                                  that items sharing keys find them in L2
                                  (1: one group, longest first throughout)    */
} rpa_plan_info;

typedef struct rpa_plan rpa_plan_t;

/*
 * Build a plan from HOST copies of the ragged metadata (the scheduler).
 *
 * It classifies each sequence as decode (q_len == 1) or prefill (q_len > 1;
 * q_len == 0 contributes nothing), picks the decode split length and the
 * prefill query block, orders the prefill work items longest first over a
 * persistent grid, and sizes the workspace.  Host only: it launches nothing
 * and touches no device memory.
 *
 *   cu_q_lens_host [num_seqs+1], kv_lens_host [num_seqs]: host int32 arrays
 *       (cu_q_lens_host[0] == 0, non-decreasing; q_len <= kv_len).
 *   window_host: host int32 [num_seqs] (<= 0: full causal), or NULL (all
 *       full causal).  It must match what is later passed to rpa_forward.
 *   num_q_heads % num_kv_heads == 0 (the tensor-core paths take at most 256
 *       KV heads; more run on the CUDA-core one).  head_dim in {64, 128, 256};
 *       page_size a power of two in [1, 256] (the tensor-core prefill needs >= 16);
 *       dtype RPA_DTYPE_BF16 or RPA_DTYPE_F32 (F32 always takes the SIMT path,
 *       the fp32 debug build).
 *   max_pages_per_seq: row length of the page table; every sequence needs
 *       ceil(kv_len / page_size) <= max_pages_per_seq.
 *   num_pages: pages in the pool (page ids must lie in [0, num_pages)).
 *   opts: NULL for defaults.
 *   *plan receives a new plan (free with rpa_plan_destroy); *workspace_bytes
 *       (may be NULL) the device workspace rpa_forward needs.
 * Returns RPA_OK, RPA_ERR_INVALID_ARG or RPA_ERR_UNSUPPORTED; on error *plan
 * is set to NULL.
 * RPA_LOG=1 in the environment makes every rpa_plan print one line about
 * the plan it built (paths, CTAs, ranges, items, workspace) to stderr.
 */
rpa_status_t rpa_plan(rpa_plan_t** plan, const int32_t* cu_q_lens_host,
                      const int32_t* kv_lens_host, const int32_t* window_host,
                      int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t page_size, int32_t max_pages_per_seq,
                      int32_t num_pages, int32_t dtype, const rpa_plan_options* opts,
                      size_t* workspace_bytes);

/* Free a plan (NULL is a no-op).  Must not race with rpa_forward on it. */
rpa_status_t rpa_plan_destroy(rpa_plan_t* plan);

/* Copy out what the plan chose. */
rpa_status_t rpa_plan_get_info(const rpa_plan_t* plan, rpa_plan_info* info);

/*
 * Ragged paged attention for the batch the plan was built for.
 *
 * Device pointers (all on the current device, contiguous, row-major):
 *   q        [total_q, num_q_heads, head_dim]            dtype, 16-B aligned
 *   k_pages, v_pages [num_pages, page_size, num_kv_heads, head_dim]
 *                                                       dtype, 128-B aligned
 *   page_table [num_seqs, max_pages_per_seq] int32; entries past a sequence's
 *            last page are never read
 *   cu_q_lens [num_seqs+1] int32, kv_lens [num_seqs] int32: the same values
 *            the plan was built from
 *   window   [num_seqs] int32 (<= 0: full causal) or NULL (all full causal);
 *            NULL-ness and values must match the plan's window_host
 *   out      [total_q, num_q_heads, head_dim]            dtype, 16-B aligned
 *   workspace: at least the plan's workspace_bytes, 256-B aligned, and
 *            zero-filled before its first use (its error word must start at
 *            zero; the rest is scratch the call overwrites).
 *            Scratch owned by the call while it runs; the error word lives at
 *            its start and is sticky until rpa_get_device_error clears it.
 *   Pages: only the slots of keys some query of the batch sees are used;
 *            every other slot (the free slots of a sequence's last page past
 *            its kv_len, keys before every query's window, pages no sequence
 *            owns) may hold anything, NaN and infinities included.  The
 *            kernels load some of them along with the visible keys (whole
 *            boxes of a page) but zero them before any product uses them.
 *            A NaN in K makes NaN the rows that see its key; a NaN or an
 *            infinity in V those, and in a prefill it may also reach rows of the
 *            same sequence that do not see the key (0 times NaN).
 * The scalar arguments must equal the plan's, else RPA_ERR_PLAN_MISMATCH.
 * sm_scale multiplies q.k before the softmax (1/sqrt(head_dim) is usual); with
 * sequences on the tensor-core prefill, which scales after its maxima, it must
 * be positive.
 * Enqueues on `stream` the split-KV decode kernel and, where a sequence is
 * cut across its CTAs, the log-sum-exp combine kernel (a programmatic
 * dependent launch), then the tensor-core prefill and the CUDA-core path, as
 * the batch needs, and returns without waiting for them.
 * Threads: calls from several host threads may run at once (launch
 * parameters are staged per thread); each calling thread must have the
 * stream's device current (cudaSetDevice, torch.cuda.set_device), else the
 * call fails with RPA_ERR_CUDA (rpa_last_cuda_error gives the cudaError_t),
 * and calls that share a workspace must be ordered on the GPU.
 * CUDA graphs: the call only enqueues kernel launches (no allocation, copy
 * or synchronisation), so it may be captured into a CUDA graph on `stream`;
 * every replay reruns the attention on the same buffers with the schedule
 * the plan held at capture (kernel parameters are baked into the graph), so
 * a new plan needs a new capture.
 */
rpa_status_t rpa_forward(const void* q, const void* k_pages, const void* v_pages,
                         const int32_t* page_table, const int32_t* cu_q_lens,
                         const int32_t* kv_lens, int32_t num_seqs, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                         const int32_t* window, float sm_scale, void* out,
                         rpa_stream_t stream, const rpa_plan_t* plan, void* workspace,
                         size_t workspace_bytes);

/*
 * KV-cache write of a step's new tokens ("TPU Deep Dive" slides, chapter 8,
 * "Continuous batching with static shapes": ragged paged attention writes
 * the KV cache of the step's tokens itself).
 *
 * For every sequence s and each of its q_len = cu_q_lens[s+1] - cu_q_lens[s]
 * new tokens t = cu_q_lens[s] + i, at position pos = kv_lens[s] - q_len + i
 * (the query positions rpa_forward attends from), and every KV head g:
 *   k_pages[page_table[s][pos / page_size]][pos % page_size][g][:] = k_new[t][g][:]
 * and V alike.  Nothing else in the pool changes.
 *
 * Device pointers: k_new, v_new [total_q, num_kv_heads, head_dim] of `dtype`,
 * 16-B aligned; k_pages, v_pages, page_table, cu_q_lens, kv_lens as for
 * rpa_forward (kv_lens include the new tokens).  head_dim * element size must
 * be a multiple of 16 bytes; page_size a power of two.  `workspace` may be
 * NULL; otherwise its error word records a page id outside [0, num_pages)
 * or a position outside the page table (that row is skipped, never trapped).
 * Enqueues one kernel on `stream`; does not synchronise.
 */
rpa_status_t rpa_write_kv(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                          const int32_t* page_table, const int32_t* cu_q_lens,
                          const int32_t* kv_lens, int32_t num_seqs, int32_t total_q,
                          int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                          int32_t max_pages_per_seq, int32_t num_pages, int32_t dtype,
                          void* workspace, rpa_stream_t stream);

/*
 * q/k/v prologue: the step right before attention ("Chasing speed of light on
 * TPU v6e", section "The Long Tail": the q/k/v RMS norms and the rotary
 * embedding run in the kernel before attention, which takes q, k and v as
 * three arrays), fused with the KV-cache write.
 *
 * For every new token t = cu_q_lens[s] + i of sequence s, at position
 * pos = kv_lens[s] - q_len_s + i, and page = page_table[s][pos / page_size]:
 *   q_out[t][h][:]                        = rope(norm(q[t][h][:], q_weight), pos)
 *   k_pages[page][pos % page_size][g][:]  = rope(norm(k[t][g][:], k_weight), pos)
 *   v_pages[page][pos % page_size][g][:]  = norm(v[t][g][:], v_weight)
 * norm(x, w)_d = x_d / sqrt(mean_d(x_d^2) + eps) * w_d, or x itself when w is
 * NULL (a model whose norm scales by 1 + w passes 1 + w).
 * rope (halves convention): for i < D/2, with a = pos * rope_theta^(-2i/D),
 *   out_i = y_i cos a - y_{i+D/2} sin a,  out_{i+D/2} = y_{i+D/2} cos a + y_i sin a;
 * rope_theta <= 0: no rotation.  fp32 arithmetic; the angle is reduced
 * modulo 2 pi in extended precision (accurate for pos * frequency < 2^21).
 *
 * Device pointers: q, q_out [total_q, num_q_heads, head_dim]; k, v
 * [total_q, num_kv_heads, head_dim]; all of `dtype` (BF16 or F32), 16-B
 * aligned; q_out may equal q.  Weights: [head_dim] float32.  Pages, page
 * table and lengths as for rpa_write_kv (kv_lens include the new tokens).
 * head_dim in {64, 128, 256} (else RPA_ERR_UNSUPPORTED); page_size a power
 * of two.  `workspace` may be NULL; otherwise its error word records a page
 * id or position outside the table (that row is skipped, never trapped).
 * Enqueues one kernel on `stream`; does not synchronise.
 */
typedef struct rpa_qkv_norm {
  const float* q_weight; /* [head_dim] or NULL: q not normalised */
  const float* k_weight; /* [head_dim] or NULL: k not normalised */
  const float* v_weight; /* [head_dim] or NULL: v stored as given */
  float eps;             /* added to the mean square */
  float rope_theta;      /* rotary base (> 0), or <= 0 for none */
} rpa_qkv_norm;

rpa_status_t rpa_qkv_prologue(const void* q, const void* k, const void* v,
                              const rpa_qkv_norm* norm, void* q_out, void* k_pages,
                              void* v_pages, const int32_t* page_table,
                              const int32_t* cu_q_lens, const int32_t* kv_lens,
                              int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                              int32_t max_pages_per_seq, int32_t num_pages, int32_t dtype,
                              void* workspace, rpa_stream_t stream);

/*
 * The prologue, then the attention on its output, on one stream: the step
 * from the projection's q, k, v to the attention output.  q_buf receives
 * the normalised, rotated q (rpa_qkv_prologue's q_out) and is the attention's
 * query; the other arguments as rpa_qkv_prologue and rpa_forward (pool size
 * and page-table width are the plan's).
 */
rpa_status_t rpa_forward_qkv(const void* q, const void* k, const void* v,
                             const rpa_qkv_norm* norm, void* q_buf, void* k_pages,
                             void* v_pages, const int32_t* page_table,
                             const int32_t* cu_q_lens, const int32_t* kv_lens,
                             int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size, const int32_t* window,
                             float sm_scale, void* out, rpa_stream_t stream,
                             const rpa_plan_t* plan, void* workspace, size_t workspace_bytes);

/*
 * Decode over fp8 (e4m3) K/V pages with a float scale per KV head
 * ("TPU Deep Dive" slides, chapter 8, "KV cache layout": 8-bit KV packs four
 * per 32-bit word; halving the KV bytes halves decode's dominant traffic).
 * The stored keys and values are k_pages[...][g][:] * k_scale[g] and
 * v_pages[...][g][:] * v_scale[g]; otherwise exactly rpa_forward.  The plan
 * must have kv_dtype RPA_DTYPE_FP8_E4M3 (decode batch, bf16 q and out).
 * k_pages, v_pages: [num_pages, page_size, num_kv_heads, head_dim] bytes,
 * 128-B aligned; k_scale, v_scale: [num_kv_heads] float32 on the device.
 * The products run as f16 (e4m3 is exact in f16; q is converted bf16 -> f16
 * once per sequence), accumulation and softmax in fp32.
 */
rpa_status_t rpa_forward_fp8kv(const void* q, const void* k_pages, const void* v_pages,
                               const float* k_scale, const float* v_scale,
                               const int32_t* page_table, const int32_t* cu_q_lens,
                               const int32_t* kv_lens, int32_t num_seqs, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               const int32_t* window, float sm_scale, void* out,
                               rpa_stream_t stream, const rpa_plan_t* plan, void* workspace,
                               size_t workspace_bytes);

/*
 * rpa_write_kv of k_new / v_new, then rpa_forward over the updated cache, in
 * order on `stream`: the step's cache update and its attention in one call.
 * Arguments as rpa_forward plus k_new, v_new (as rpa_write_kv); the pool
 * size and page-table width are the plan's.
 */
rpa_status_t rpa_forward_kv(const void* q, const void* k_new, const void* v_new, void* k_pages,
                            void* v_pages, const int32_t* page_table, const int32_t* cu_q_lens,
                            const int32_t* kv_lens, int32_t num_seqs, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                            const int32_t* window, float sm_scale, void* out,
                            rpa_stream_t stream, const rpa_plan_t* plan, void* workspace,
                            size_t workspace_bytes);

/*
 * The KV cache in 4 bits: rows of K and V written into 4-bit pages.
 *
 * Format.  A row of head_dim dimensions is blocks of 16.  Each dimension is an
 * e2m1 code (bit 3 sign; magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 for the low three
 * bits), two to a byte, the even dimension in the low half.  Each block has one
 * scale byte without a sign: e = byte >> 3, m = byte & 7, scale = (1 + m / 8) *
 * 2^(e - 15), or m * 2^-17 where e == 0, up to byte 226 (10240); byte 255 is NaN;
 * 227 to 254 are not valid in a visible slot (the kernels read a scale as the
 * f16 of its bits, where some of them overflow).  A stored value is its code's
 * magnitude times the scale.  The format is this library's: its scales are
 * neither the signed e4m3 ones with a second scale per tensor nor the powers of
 * two per 32 elements that other 4-bit formats have.  Pages are arrays
 *   k_pages,  v_pages  [num_pages, num_kv_heads, page_size, head_dim / 2] bytes
 *   k_scales, v_scales [num_pages, num_kv_heads, page_size, head_dim / 16] bytes
 * (a head's rows of a page are contiguous, unlike the 8- and 16-bit pools).
 * 0.5625 bytes an element.
 *
 * Writing.  With a = the largest magnitude of a block, its scale is a / 6
 * rounded to the nearest scale (ties to even) and at most 10240; each code is
 * x / scale rounded to the nearest magnitude (ties to the even code, at most 6).
 * A block of magnitudes below 6 * 2^-18 is stored as zeros; one that holds a NaN
 * or an infinity reads back as NaN in all its 16 places.
 *
 * k_new, v_new [total_q, num_kv_heads, head_dim] of `dtype` (BF16 or F32), 16-B
 * aligned; slot_map [total_q] int64: token t goes to slot slot_map[t] %
 * page_size of page slot_map[t] / page_size (rpa_build_tables makes such a
 * map); a negative entry leaves the token out.  The slots of a call are
 * distinct: where two tokens name one, what it holds afterwards may be one's
 * codes under the other's scales.
 * k_pages, v_pages, k_scales and v_scales 16-B aligned.  head_dim 64, 128 or
 * 256, page_size a power of two in [16, 256] and total_q * num_kv_heads below
 * 2^31, else RPA_ERR_UNSUPPORTED.
 * `workspace` may be NULL; otherwise its error word records a slot outside the
 * pool (that token is left out, never trapped).  Enqueues one kernel on
 * `stream`; does not synchronise.
 */
rpa_status_t rpa_write_kv4(const void* k_new, const void* v_new, uint8_t* k_pages,
                           uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales,
                           const int64_t* slot_map, int32_t total_q, int32_t num_kv_heads,
                           int32_t head_dim, int32_t page_size, int32_t num_pages, int32_t dtype,
                           void* workspace, rpa_stream_t stream);

/*
 * The reverse: rows taken back as values.  k_out, v_out [total_q, num_kv_heads,
 * head_dim] of `dtype` (BF16 or F32; both hold every stored value exactly) get
 * the rows of slots slot_map[t]; rows of negative entries, or of slots outside
 * the pool, are left as they were.  Slots may repeat.  Otherwise as
 * rpa_write_kv4.
 */
rpa_status_t rpa_read_kv4(const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_scales,
                          const uint8_t* v_scales, const int64_t* slot_map, void* k_out,
                          void* v_out, int32_t total_q, int32_t num_kv_heads, int32_t head_dim,
                          int32_t page_size, int32_t num_pages, int32_t dtype, void* workspace,
                          rpa_stream_t stream);

/*
 * Ragged paged attention over 4-bit pages: rpa_forward's definition with the
 * keys and values the pages stand for (rpa_write_kv4), for any mix of single
 * tokens, a few tokens and prompts.  The plan must have kv_dtype
 * RPA_DTYPE_FP4_E2M1; q and out are bf16.  Sequences of few query rows (q_len
 * times num_q_heads / num_kv_heads) run on a split-KV kernel that widens the
 * codes in registers (or, for tens of rows, in shared memory); the others'
 * visible keys are first widened to bf16 in the workspace: 4 * head_dim *
 * num_kv_heads bytes a key (3.6 times the pages' own), for the whole visible
 * prefix of each such sequence and anew at every call, so a chunk of a prompt
 * after 128k keys of 8 heads of 128 takes 537 MB.  A plan whose widened keys
 * times heads pass 2^31 is refused with RPA_ERR_UNSUPPORTED.
 * A block of K that reads as NaN makes NaN the rows that see its key, a block of
 * V its 16 dimensions of them; no other row, on whichever kernel.  sm_scale may
 * be any number.  Device lengths that differ from the plan's (those of a step that
 * rpa_build_tables refused, for one) set RPA_DEVERR_LENGTHS; the rows of such a
 * sequence are then not to be used.  Let the calls of a step share a workspace:
 * one read of its error word then tells of all of them.
 * Pages as rpa_write_kv4's; the other arguments, the error word, unused slots,
 * threads and CUDA graphs as rpa_forward.
 */
rpa_status_t rpa_forward_kv4(const void* q, const uint8_t* k_pages, const uint8_t* v_pages,
                             const uint8_t* k_scales, const uint8_t* v_scales,
                             const int32_t* page_table, const int32_t* cu_q_lens,
                             const int32_t* kv_lens, int32_t num_seqs, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                             const int32_t* window, float sm_scale, void* out,
                             rpa_stream_t stream, const rpa_plan_t* plan, void* workspace,
                             size_t workspace_bytes);

/*
 * A step's page table, slot map and lengths from its requests' lengths, on the
 * GPU.  Works with every kind of page.
 *
 * The pages no request holds are a stack: free_pages[0 .. *free_count_prev),
 * distinct ids, the last one taken first.  Request s has kv_lens_prev[s] tokens
 * in the cache, its page-table row holds their ceil(kv_lens_prev[s] /
 * page_size) pages, and it appends new_lens[s] >= 0 tokens.  The call takes the
 * pages it still needs from the stack, requests in order (the k-th page of the
 * step is free_pages[*free_count_prev - 1 - k]), and writes
 *   page_table  those pages, behind the row's others (nothing else changes);
 *   cu_q_lens   [num_seqs + 1] the prefix sums of new_lens;
 *   kv_lens     [num_seqs] kv_lens_prev + new_lens;
 *   slot_map    [max_tokens] of each new token, requests in order, its page
 *               times page_size plus its place in the page; -1 behind the last;
 *   free_count  [1] the pages left (free_pages itself is only read).
 * kv_lens may be kv_lens_prev, and free_count free_count_prev: the step then
 * advances them in place (a captured call does so at every replay).  Otherwise
 * the outputs do not overlap the inputs (RPA_ERR_INVALID_ARG for those two).
 *
 * All or nothing: a negative length, a request longer than max_pages_per_seq
 * pages or more than max_tokens new tokens sets RPA_DEVERR_LENGTHS, a stack too
 * short RPA_DEVERR_PAGES; then the lengths and the stack's height stay as they
 * were, cu_q_lens is all 0 and slot_map all -1.  A page id outside the pool, in
 * the stack or in a row, sets RPA_DEVERR_PAGE_ID and becomes slot -1.
 *
 * Device pointers, contiguous, 4-byte (slot_map 8-byte) aligned; page_table
 * [num_seqs, max_pages_per_seq], free_pages [num_pages].  page_size a power of
 * two; num_seqs, num_pages and max_tokens at most 2^30, else
 * RPA_ERR_UNSUPPORTED.  `workspace`: 256 bytes or more, 256-B aligned, zero-filled before its
 * first use (any plan's workspace serves); calls that share one do not overlap
 * on the GPU.  Enqueues one kernel on `stream`; does not synchronise.
 */
rpa_status_t rpa_build_tables(const int32_t* new_lens, const int32_t* kv_lens_prev,
                              int32_t* page_table, const int32_t* free_pages,
                              const int32_t* free_count_prev, int32_t* cu_q_lens,
                              int32_t* kv_lens, int64_t* slot_map, int32_t* free_count,
                              int32_t num_seqs, int32_t max_tokens, int32_t page_size,
                              int32_t max_pages_per_seq, int32_t num_pages, void* workspace,
                              rpa_stream_t stream);

/*
 * Finished requests' pages go back to the stack: for every s with finished[s]
 * != 0, its ceil(kv_lens_prev[s] / page_size) pages are pushed in (request,
 * slot) order, free_pages[*free_count_prev ...], and kv_lens[s] becomes 0
 * (kv_lens_prev[s] for the others); free_count is the stack's new height.  The
 * page table is only read.  In place, device pointers and workspace as
 * rpa_build_tables.  All or nothing: a negative length or one beyond the table
 * sets RPA_DEVERR_LENGTHS, more pages than the pool's RPA_DEVERR_PAGES; a page
 * id outside the pool sets RPA_DEVERR_PAGE_ID and pushes -1 (which
 * rpa_build_tables reports when it takes it).
 */
rpa_status_t rpa_release_tables(const int32_t* finished, const int32_t* kv_lens_prev,
                                const int32_t* page_table, int32_t* free_pages,
                                const int32_t* free_count_prev, int32_t* kv_lens,
                                int32_t* free_count, int32_t num_seqs, int32_t page_size,
                                int32_t max_pages_per_seq, int32_t num_pages, void* workspace,
                                rpa_stream_t stream);

/*
 * The steps below are a speculative one whose drafted tokens form a tree: request
 * s verifies its q_len new tokens (nodes) at once, node i following node
 * parents[i] (or the cached context), so that several nodes may hold the same
 * position.  A step is rpa_build_tables (pages and slots for the nodes),
 * rpa_build_tree (masks and positions), for each layer rpa_append_rope and
 * rpa_forward_tree, then the caller's choice of a path, for each layer
 * rpa_commit_tree and at last rpa_trim_tables.  C = kv_lens[s] - q_len is a
 * request's context; node i's row lies at place C + i of its cache until the path
 * is committed.
 */

/*
 * Masks and positions of the nodes from their parents, on the GPU.
 *
 * parents [total_q] int32: for node i of its request an earlier node j of the same
 * request (0 <= j < i), or -1 where it follows the context.  depth(i) is 0 there
 * and depth(j) + 1 otherwise.  Writes
 *   tree_mask [total_q, mask_words] 64-bit words: bit j % 64 of word j / 64 of row
 *             cu_q_lens[s] + i is set iff node j is node i or one of its ancestors
 *             (and, where window[s] > 0, depth(i) - depth(j) < window[s]);
 *   positions [total_q] int32: kv_lens[s] - q_len + depth(i).
 * window [num_seqs] int32 (<= 0: none) or NULL.  Rows behind the last request are
 * left as they were.
 *
 * A parent outside [-1, i) sets RPA_DEVERR_LENGTHS and counts as -1.  A request
 * whose lengths cannot be used (decreasing, more than 64 * mask_words nodes, more
 * nodes than keys, rows behind total_q) sets it too, and its rows are left as they
 * were.  mask_words 1..16.  Device pointers 4-byte (tree_mask 8-byte) aligned;
 * `workspace` may be NULL, otherwise its error word records these.  Enqueues one
 * kernel on `stream`; does not synchronise.
 */
rpa_status_t rpa_build_tree(const int32_t* parents, const int32_t* cu_q_lens,
                            const int32_t* kv_lens, const int32_t* window, uint64_t* tree_mask,
                            int32_t* positions, int32_t num_seqs, int32_t total_q,
                            int32_t mask_words, void* workspace, rpa_stream_t stream);

/*
 * Rows of q and k rotated by given positions, and the rows of k and v written into
 * their pages.  (rpa_qkv_prologue derives consecutive positions and slots from the
 * lengths; here both are given, as a tree of tokens needs them.)
 *
 * With a = positions[t] * inv_freq[i] for i < rotary_dim / 2, dimensions x and y
 * of every q and k row become x cos a - y sin a and y cos a + x sin a, where (x, y)
 * are (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when `interleaved` is nonzero;
 * dimensions from rotary_dim on, and v, stay as they are.  fp32 arithmetic; the
 * angle is reduced in fixed point, its error at most 2^-47 |a| + 2^-28.  Any int32
 * is a position, and a frequency may have either sign (-f turns back); one that is
 * NaN or infinite makes its pairs NaN.
 */
typedef struct rpa_rope {
  const float* inv_freq; /* device, [rotary_dim / 2]; NULL with rotary_dim 0   */
  int32_t rotary_dim;    /* a multiple of 16 in [0, head_dim]; 0: no rotation  */
  int32_t interleaved;   /* 0: the two halves turn together; else neighbours   */
} rpa_rope;

/*
 * q [total_q, num_q_heads, head_dim], k, v [total_q, num_kv_heads, head_dim] of
 * `dtype` (BF16 or F32), a token's heads contiguous and tokens q_stride, k_stride
 * and v_stride elements apart (slices of one projection's output, for instance;
 * strides at least a token's heads and a multiple of 16 bytes).  q_out [total_q,
 * num_q_heads, head_dim] contiguous; it may be q.  With num_q_heads 0, q and q_out
 * are not used (NULL).  slot_map [total_q] int64: token t goes to slot slot_map[t]
 * of the pool (slot_map[t] / page_size is its page); of a token with a negative
 * entry only q is written.  The slots of a call are distinct.  A row of k or v may
 * be the slot that it goes to (the cache turned further); otherwise the rows, q_out
 * and the pages lie apart.
 *
 * kv_dtype is `dtype`, or RPA_DTYPE_FP8_E4M3: k_pages, v_pages [num_pages,
 * page_size, num_kv_heads, head_dim] of it.  e4m3 pages hold row / k_scale[head]
 * (v_scale for v; device float32 [num_kv_heads], positive) rounded to the nearest
 * (ties to even) and at most 448, NaN as NaN: what rpa_forward_fp8kv reads.
 * Otherwise k_scale and v_scale are NULL.
 *
 * head_dim 64, 128 or 256 and a page_size that is a power of two, else
 * RPA_ERR_UNSUPPORTED.  Pointers to rows and pages 16-byte aligned.  `workspace` may
 * be NULL; otherwise its error word records a slot outside the pool
 * (RPA_DEVERR_PAGE_ID; of that token, too, only q is written).  Enqueues one
 * kernel on `stream`; does not synchronise.
 */
rpa_status_t rpa_append_rope(const void* q, const void* k, const void* v, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const int32_t* positions,
                             const int64_t* slot_map, const rpa_rope* rope, void* q_out,
                             void* k_pages, void* v_pages, const float* k_scale,
                             const float* v_scale, int32_t total_q, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                             int32_t num_pages, int32_t dtype, int32_t kv_dtype, void* workspace,
                             rpa_stream_t stream);

/*
 * Attention of the nodes over their context and their tree: rpa_forward with
 * another mask.  Node i of request s, at row t = cu_q_lens[s] + i, sees
 *   key j < C          iff window[s] <= 0 or positions[t] - j < window[s];
 *   key C + j, j < q_len, iff bit j % 64 of tree_mask[t][j / 64] is set.
 * Any mask will do (a node need not see itself, and may see a later one).  A row
 * that sees no key, or whose visible scores are all -infinity, is written as zeros.
 * `sm_scale` is any number up to 2^120 in magnitude, else RPA_ERR_INVALID_ARG.
 *
 * The plan must have tree_words > 0; tree_mask [total_q, tree_words] 64-bit words,
 * 8-byte aligned.  positions [total_q] int32 are read where there is a window (with
 * NULL window they may be NULL): those of rpa_build_tree, or any in [C, kv_lens[s]);
 * one outside sets RPA_DEVERR_LENGTHS and counts as the nearest of these.  kv_lens
 * includes the nodes, whose rows are in their pages already.
 *
 * bf16 q, pages and out run on tensor cores (page_size at least 16 and num_q_heads
 * / num_kv_heads at most 128, sm_scale at least 2^-126), fp32 and the rest on CUDA
 * cores, which take far longer.  Scores and sums are 32-bit: a row's output is finite
 * while its scaled scores are, and the keys it sees times the largest |V| among them
 * stay below 2^128.  A NaN or an
 * infinity in K or V reaches the rows that see its key, and no other.  Device
 * lengths that differ from the plan's set RPA_DEVERR_LENGTHS; the call goes by the
 * plan's.  The other arguments, the error word, unused slots, threads and CUDA
 * graphs as rpa_forward.
 */
rpa_status_t rpa_forward_tree(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* page_table, const int32_t* cu_q_lens,
                              const int32_t* kv_lens, const uint64_t* tree_mask,
                              const int32_t* positions, int32_t num_seqs, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                              const int32_t* window, float sm_scale, void* out,
                              rpa_stream_t stream, const rpa_plan_t* plan, void* workspace,
                              size_t workspace_bytes);

/*
 * The accepted path's rows moved together: for every request s and k with
 * path[s][k] >= 0 the rows of K and V of node path[s][k] are copied to node k's
 * slot, as if all were read before any is written.
 *
 * path [num_seqs, max_path] int32: increasing nodes of the request, then -1.
 * slot_map [total_q] int64 as for rpa_append_rope (node i of request s has entry
 * cu_q_lens[s] + i), its slots distinct.  Nothing else in the pool changes.
 * k_pages, v_pages [num_pages, page_size, num_kv_heads, head_dim] of `dtype` (BF16,
 * F32 or FP8_E4M3), 16-byte aligned; head_dim times the element size a multiple
 * of 16 bytes, max_path at most 1024, else RPA_ERR_UNSUPPORTED.
 *
 * A path that does not increase, has a node behind its request's, or one after a
 * -1 sets RPA_DEVERR_LENGTHS (as do lengths that cannot be used), a slot outside
 * the pool RPA_DEVERR_PAGE_ID; that request's rows then stay as they were.
 * `workspace` may be NULL.  Enqueues one kernel on `stream`; does not synchronise.
 */
rpa_status_t rpa_commit_tree(void* k_pages, void* v_pages, const int64_t* slot_map,
                             const int32_t* cu_q_lens, const int32_t* path, int32_t num_seqs,
                             int32_t total_q, int32_t max_path, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size, int32_t num_pages,
                             int32_t dtype, void* workspace, rpa_stream_t stream);

/*
 * Requests cut short: drop_lens[s] >= 0 tokens leave the end of request s, whose
 * pages behind its new length go back to the stack: kv_lens[s] = kv_lens_prev[s] -
 * drop_lens[s], and the pages at slots ceil(kv_lens[s] / page_size) up to
 * ceil(kv_lens_prev[s] / page_size) of its row are pushed in (request, slot) order,
 * free_pages[*free_count_prev ...]; free_count is the stack's new height.  The
 * page table is only read.  In place, device pointers and workspace as
 * rpa_build_tables, all or nothing and its errors as rpa_release_tables (a request
 * that drops more than it has sets RPA_DEVERR_LENGTHS).
 */
rpa_status_t rpa_trim_tables(const int32_t* drop_lens, const int32_t* kv_lens_prev,
                             const int32_t* page_table, int32_t* free_pages,
                             const int32_t* free_count_prev, int32_t* kv_lens,
                             int32_t* free_count, int32_t num_seqs, int32_t page_size,
                             int32_t max_pages_per_seq, int32_t num_pages, void* workspace,
                             rpa_stream_t stream);

/*
 * Read the device error word at the start of `workspace` after everything
 * enqueued on `stream` so far (this call synchronises `stream`), store it in
 * *err (an RPA_DEVERR_* code) and reset it to RPA_DEVERR_NONE.
 * workspace == NULL selects the fixed scratch of rpa_forward_decode_noalloc on
 * the current device (its error word, sticky in the same way).
 */
rpa_status_t rpa_get_device_error(void* workspace, rpa_stream_t stream, int32_t* err);

/* Zero the workspace error word (enqueued on `stream`, no synchronisation);
 * workspace == NULL: that of rpa_forward_decode_noalloc's fixed scratch. */
rpa_status_t rpa_clear_device_error(void* workspace, rpa_stream_t stream);

/*
 * Decode without a caller-supplied workspace: rpa_forward_decode_noalloc.
 *
 * For callers that cannot allocate device memory when they run attention:
 * code that executes inside a framework whose device memory is entirely owned
 * by another allocator, embedded or real-time serving loops that must not
 * call cudaMalloc (it can synchronise the device), and plug-ins that receive
 * only the tensors they work on.  The paper has no counterpart; this is a
 * deployment convenience.
 *
 * Same arguments as rpa_forward without the workspace.  The plan must hold
 * decode sequences only (q_len <= 1) on the split-KV decode kernel, else
 * RPA_ERR_UNSUPPORTED; a plan whose workspace_bytes exceeds
 * RPA_NOALLOC_SCRATCH_BYTES is rejected with RPA_ERR_WORKSPACE_TOO_SMALL.
 * The scratch is one fixed array inside the library (every GPU that loads the
 * library holds it until the process exits), shared by every call and keeping
 * the last call's contents; calls that overlap on the GPU (for example on two
 * streams) race on it.  Only its error word must start at zero: it does (the
 * array is zero when the library loads) and, like a workspace's, it is sticky:
 * a kernel that meets a bad page id or a length that disagrees with the plan
 * sets it and skips the access, and rpa_get_device_error(NULL, stream, &err)
 * reads and clears it.  The split partials are written before they are read
 * within a call.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress, once per device, thread-safe) with that
 * device current; make that first call before any stream capture.  No device
 * memory is allocated or freed.  The call returns RPA_OK once its work is
 * enqueued (RPA_ERR_CUDA with rpa_last_cuda_error set if a CUDA call fails).
 */
#define RPA_NOALLOC_SCRATCH_BYTES (32u << 20) /* 32 MiB */

rpa_status_t rpa_forward_decode_noalloc(const void* q, const void* k_pages,
                                        const void* v_pages, const int32_t* page_table,
                                        const int32_t* cu_q_lens, const int32_t* kv_lens,
                                        int32_t num_seqs, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t page_size, const int32_t* window,
                                        float sm_scale, void* out, rpa_stream_t stream,
                                        const rpa_plan_t* plan);

/*
 * Kernel tracing (off by default).  Between rpa_trace_begin and rpa_trace_end,
 * every rpa_forward call records a CUDA event on its stream before its first
 * kernel and after each kernel it launches, so that the device time of each
 * launch can be read back.  Tracing state is process-wide and not thread-safe;
 * tracing adds one event record per launch to the stream.  A call captured
 * into a CUDA graph while tracing records its marks as event-record nodes of
 * the graph; rpa_trace_end then reads the times of the last replay.
 *
 * rpa_trace_begin: start recording up to `capacity` launches (1..65536).
 * rpa_trace_end: synchronise on the recorded events, write up to *count
 *     records (kernel id, device milliseconds) to `records`, set *count to the
 *     number written, and stop tracing.  Launches beyond `capacity` are not
 *     recorded.
 */
enum {
  RPA_KERNEL_DECODE_SPLIT = 0,   /* split-KV decode                    */
  RPA_KERNEL_DECODE_COMBINE = 1, /* log-sum-exp combine of cut sequences */
  RPA_KERNEL_PREFILL_TC = 2,     /* tensor-core prefill               */
  RPA_KERNEL_SIMT = 3,           /* CUDA-core (fp32) path             */
  RPA_KERNEL_KV_WRITE = 4,       /* KV-cache write of new tokens      */
  RPA_KERNEL_PROLOGUE = 5,       /* q/k/v norm + rotary + KV write    */
  RPA_KERNEL_PREFILL_COMBINE = 6, /* combine of split prefill items   */
  RPA_KERNEL_KV4_DECODE = 7,     /* split-KV attention, 4-bit pages   */
  RPA_KERNEL_KV4_COMBINE = 8,    /* combine of its cut segments       */
  RPA_KERNEL_KV4_EXPAND = 9,     /* 4-bit pages widened for prefill   */
  RPA_KERNEL_KV4_WRITE = 10,     /* 4-bit cache write                 */
  RPA_KERNEL_KV4_READ = 11,      /* 4-bit cache read                  */
  RPA_KERNEL_BUILD_TABLES = 12,  /* page tables and slot maps built   */
  RPA_KERNEL_RELEASE_TABLES = 13, /* finished requests' pages returned */
  RPA_KERNEL_BUILD_TREE = 14,    /* masks and positions of drafted trees */
  RPA_KERNEL_APPEND_ROPE = 15,   /* rotation and cache write          */
  RPA_KERNEL_TREE_ATTN = 16,     /* attention of drafted trees        */
  RPA_KERNEL_TREE_COMBINE = 17,  /* combine of its cut segments       */
  RPA_KERNEL_COMMIT_TREE = 18,   /* an accepted path's rows moved     */
  RPA_KERNEL_TRIM_TABLES = 19    /* requests cut short                */
};
typedef struct rpa_trace_record {
  int32_t kernel; /* RPA_KERNEL_* */
  float ms;       /* device time from the previous mark of the same call */
} rpa_trace_record;

rpa_status_t rpa_trace_begin(int32_t capacity);
rpa_status_t rpa_trace_end(rpa_trace_record* records, int32_t* count);

/* A static, human-readable name for a status code. */
const char* rpa_status_string(rpa_status_t status);

/* The cudaError_t behind the calling thread's last RPA_ERR_CUDA returned by
 * any entry point (0 if none): for diagnostics. */
int32_t rpa_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* RPA_H_ */
