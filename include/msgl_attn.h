/*
 * libmsgl_attn — paged-KV grouped-query attention for GB300 (sm_103a).
 *
 * The attention step a Mini-SGLang-style serving engine runs every forward:
 * new K/V rows are scattered into a unified, paged KV pool, then prefill
 * chunks ("extend") and single-token decode rows attend over each request's
 * pages.  The pages describing the engine define the pieces this ABI takes:
 *
 *   - one unified KV pool, allocated in pages of a configurable size
 *     ("Mini-SGLang 实战指南", §6.2 "Page Size"; §6.5 "Radix Cache";
 *     "不懂SGLang？从miniSGLang开始", §1.2 "调度引擎", item 3);
 *   - attention reads the pool's history plus the newly computed K/V, and
 *     locates each request's data through the page table and positions
 *     ("不懂SGLang？从miniSGLang开始", §1.3 "前向运算", items 1 and 3);
 *   - prefill runs in chunks over a cached (radix-shared) prefix
 *     ("Mini-SGLang 实战指南", §6.1 "Chunked Prefill", §6.5);
 *   - prefill and decode are separate attention calls
 *     ("Mini-SGLang 实战指南", §6.3).
 *
 * Definitions used by every call (the pages fix no formula; this is the
 * plain reading of causal softmax attention with grouped heads):
 *   G        = num_q_heads / num_kv_heads (1..64); q head h reads kv head h / G
 *   slot(j)  = page_table[b][j / page_size] * page_size + j % page_size
 *   a query row at absolute position p attends keys j = 0..p:
 *   s_j = scale * <q, K[slot(j)][h/G]>,  o = sum_j softmax(s)_j V[slot(j)][h/G],
 *   lse = ln(sum_j exp(s_j))   (natural log, fp32)
 *
 * Conventions
 *   - Every pointer named "device" is CUDA device memory owned by the
 *     caller; the library allocates nothing, keeps no state between calls
 *     and never frees caller memory.  All calls are asynchronous on
 *     `stream` (NULL = the legacy default stream) except msgl_read_status.
 *   - bf16 tensors are row-major, contiguous, 16-byte aligned.
 *   - Host-side validation failures return before anything is launched.
 *   - Device-side index errors never trap: the kernel ORs a bit into the
 *     caller's status word (when `status` is non-NULL), skips the bad
 *     access and writes that output row as o = 0, lse = -inf.
 *   - Waits inside kernels are bounded; a wait that gives up sets
 *     MSGL_DEVERR_TIMEOUT and the kernel returns.
 */
#ifndef MSGL_ATTN_H
#define MSGL_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSGL_ABI_VERSION 1

#if defined(__GNUC__)
#define MSGL_API __attribute__((visibility("default")))
#else
#define MSGL_API
#endif

/* A cudaStream_t (the runtime and driver stream handle types are the same pointer). */
typedef struct CUstream_st *msgl_stream_t;

typedef enum msgl_status {
    MSGL_OK = 0,
    MSGL_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size or scalar */
    MSGL_ERR_UNSUPPORTED = 2,   /* valid but not implemented (head_dim != 128, G > 64, ...) */
    MSGL_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed (launch, copy) */
    MSGL_ERR_OUT_OF_RANGE = 4,  /* reported by msgl_read_status: device index error */
    MSGL_ERR_TIMEOUT = 5,       /* reported by msgl_read_status: a bounded wait gave up */
    MSGL_ERR_WORKSPACE = 6      /* workspace missing or smaller than the size query */
} msgl_status;

/* Bits of the device status word (uint32, caller-owned device memory). */
#define MSGL_DEVERR_SLOT_RANGE 0x1u  /* out_loc entry outside [0, num_slots) */
#define MSGL_DEVERR_PAGE_RANGE 0x2u  /* page index >= width, or page id outside the pool */
#define MSGL_DEVERR_LENGTH 0x4u      /* decode seq_len < 1, or lengths inconsistent with cu_ext */
#define MSGL_DEVERR_POSITION 0x8u    /* positions[t] != prefix_len + i for chunk row i */
#define MSGL_DEVERR_TIMEOUT 0x10u    /* a bounded in-kernel wait gave up */
#define MSGL_DEVERR_APPEND_SLOT 0x20u /* decode_append: new_loc[b] is not the slot of key seq_lens[b]-1 */
#define MSGL_DEVERR_GROUP 0x40u      /* group_start / shared_lens do not describe a group (decode_shared) */
#define MSGL_DEVERR_NO_PAGES 0x80u   /* step_tables, fork: the free pages do not reach this far */
#define MSGL_DEVERR_ROW 0x100u       /* fork, free, compact: a row outside the table, or one that forks collide on */
#define MSGL_DEVERR_TOKEN 0x200u     /* verify_drafts: a drafted token outside the vocabulary */
#define MSGL_DEVERR_PROBS 0x400u     /* verify_drafts: a row without a positive finite sum */

/*
 * The unified KV pool of one layer.  k_pool and v_pool are device bf16
 * [num_slots, num_kv_heads, head_dim], slot-major (the row of one slot is
 * num_kv_heads*head_dim contiguous elements).  num_slots must be a multiple
 * of page_size; page_size is a power of two in [1, 256]; head_dim must be 128.
 */
typedef struct msgl_kv_pool {
    void *k_pool;
    void *v_pool;
    int64_t num_slots;
    int32_t page_size;
    int32_t num_kv_heads;
    int32_t head_dim;
} msgl_kv_pool;

/*
 * Per-request page table: device int32 [num_reqs, stride]; row b lists the
 * page ids of request b in sequence order.  Only the first `width` entries
 * of a row may be read; a key whose page index reaches `width`, or whose
 * page id lies outside [0, num_slots/page_size), is a device index error.
 */
typedef struct msgl_page_table {
    const int32_t *page_ids;
    int32_t stride;
    int32_t width;
} msgl_page_table;

/*
 * Store step: write the new K/V rows of this forward into the pool
 * ("不懂SGLang？从miniSGLang开始", §1.3 item 1: the KV an attention call
 * reads is the pool's history plus the newly computed KV; every request
 * allocates from the one pool, §1.2 item 3).
 *
 *   k, v     device bf16 [n_tokens, num_kv_heads, head_dim]
 *   out_loc  device int32 [n_tokens]; row t goes to slot out_loc[t]
 *   status   device uint32 or NULL
 * Pool rows not named in out_loc are untouched.  Duplicate slots in out_loc are
 * undefined (what ends there may be of either row, or of both).  An out-of-range slot sets
 * MSGL_DEVERR_SLOT_RANGE and that row is skipped.  The copy is bit-exact.
 */
MSGL_API msgl_status msgl_store_kv(const msgl_kv_pool *pool, const void *k, const void *v,
                          const int32_t *out_loc, int32_t n_tokens, uint32_t *status,
                          msgl_stream_t stream);

/*
 * Extend (chunked prefill) step: request b has prefix_lens[b] tokens already
 * cached in its pages (a radix-cache hit or earlier chunks) and ext_lens[b]
 * new tokens whose K/V have already been stored in the pool by
 * msgl_store_kv.  Chunk row i of request b sits at absolute position
 * prefix_lens[b] + i and attends keys 0..prefix_lens[b]+i
 * ("Mini-SGLang 实战指南", §6.1 "Chunked Prefill", §6.5 "Radix Cache";
 * "不懂SGLang？从miniSGLang开始", §1.3).
 *
 *   q            device bf16 [total_tokens, num_q_heads, head_dim],
 *                request-major: request b owns rows cu_ext[b]..cu_ext[b+1]-1
 *   prefix_lens, ext_lens   device int32 [num_reqs]
 *   cu_ext       device int32 [num_reqs+1], cu_ext[0] = 0, prefix sums of ext_lens
 *   positions    device int32 [total_tokens] or NULL; when given, each row's
 *                entry must equal prefix_lens[b] + i (checked, else
 *                MSGL_DEVERR_POSITION; the mask always comes from the lengths)
 *   max_ext_len, max_seq_len   host upper bounds of ext_lens[b] and
 *                prefix_lens[b]+ext_lens[b]; they size the grid (a value
 *                that is too small is a device length error, never a wild read)
 *   scale        softmax scale (> 0, finite), normally 1/sqrt(head_dim)
 *   o            device bf16 [total_tokens, num_q_heads, head_dim] (output)
 *   lse          device fp32 [total_tokens, num_q_heads] (output), natural log
 *   workspace    device scratch of msgl_extend_workspace_size() bytes (may be
 *                NULL when that size is 0)
 */
MSGL_API size_t msgl_extend_workspace_size(int32_t num_reqs, int32_t total_tokens, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len);

MSGL_API msgl_status msgl_attn_extend(const msgl_kv_pool *pool, const msgl_page_table *pages,
                             const void *q, int32_t num_q_heads, const int32_t *prefix_lens,
                             const int32_t *ext_lens, const int32_t *cu_ext,
                             const int32_t *positions, int32_t num_reqs, int32_t total_tokens,
                             int32_t max_ext_len, int32_t max_seq_len, float scale, void *o,
                             float *lse, void *workspace, size_t workspace_bytes,
                             uint32_t *status, msgl_stream_t stream);

/*
 * Decode step: one query row per request at position seq_lens[b]-1; it
 * attends all seq_lens[b] keys, the current token's included (stored by
 * msgl_store_kv first) ("Mini-SGLang 实战指南", §6.3 and §6.4: the decode
 * kernel is separate from prefill and is replayed under CUDA graphs, so the
 * grid depends only on the host scalars num_reqs and max_seq_len).
 * The keys are split into chunks processed in parallel, and the partial
 * results are merged by their log-sum-exp in a second kernel.
 *
 *   q          device bf16 [num_reqs, num_q_heads, head_dim]
 *   seq_lens   device int32 [num_reqs], each >= 1 and <= max_seq_len
 *   o, lse     device bf16 [num_reqs, num_q_heads, head_dim], fp32 [num_reqs, num_q_heads]
 *   workspace  device scratch of at least msgl_decode_workspace_size() bytes,
 *              256-byte aligned; it holds the split partials (fp32) and is
 *              fully rewritten by every call
 */
MSGL_API size_t msgl_decode_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t max_seq_len);

MSGL_API msgl_status msgl_attn_decode(const msgl_kv_pool *pool, const msgl_page_table *pages,
                             const void *q, int32_t num_q_heads, const int32_t *seq_lens,
                             int32_t num_reqs, int32_t max_seq_len, float scale, void *o,
                             float *lse, void *workspace, size_t workspace_bytes,
                             uint32_t *status, msgl_stream_t stream);

/*
 * Decode with the current token appended in the same launch: msgl_store_kv of
 * each request's new K/V row followed by msgl_attn_decode, fused.  The K/V an
 * attention call reads is the pool's history plus the newly computed K/V
 * ("不懂SGLang？从miniSGLang开始", §1.3 item 1), and decode runs once per
 * forward for every running request ("Mini-SGLang 实战指南", §6.3, §6.4).
 *
 *   k_new, v_new  device bf16 [num_reqs, num_kv_heads, head_dim]: the K/V of
 *                 each request's current token (key seq_lens[b]-1)
 *   new_loc       device int32 [num_reqs]: its pool slot, which must be the
 *                 page-table slot of key seq_lens[b]-1 (else
 *                 MSGL_DEVERR_APPEND_SLOT; an out-of-range slot sets
 *                 MSGL_DEVERR_SLOT_RANGE and nothing is written)
 * Every other argument, the outputs, the workspace and the status bits are
 * those of msgl_attn_decode.  Key seq_lens[b]-1 is attended from k_new/v_new
 * directly (it is not read back from the pool), and the row is written to
 * the pool bit-exact during the same launch.
 */
MSGL_API msgl_status msgl_attn_decode_append(const msgl_kv_pool *pool, const msgl_page_table *pages,
                                    const void *q, int32_t num_q_heads, const void *k_new,
                                    const void *v_new, const int32_t *new_loc,
                                    const int32_t *seq_lens, int32_t num_reqs, int32_t max_seq_len,
                                    float scale, void *o, float *lse, void *workspace,
                                    size_t workspace_bytes, uint32_t *status, msgl_stream_t stream);

/*
 * One batch of chunked-prefill rows or of decode rows, as the mixed step
 * below takes them.  Each field has the meaning, layout and ownership of
 * the msgl_attn_extend / msgl_attn_decode argument of the same name.  An
 * empty batch (num_reqs = 0) is allowed and launches nothing.
 */
typedef struct msgl_extend_batch {
    msgl_page_table pages;
    const void *q;                 /* device bf16 [total_tokens, num_q_heads, head_dim] */
    const int32_t *prefix_lens;    /* device int32 [num_reqs] */
    const int32_t *ext_lens;       /* device int32 [num_reqs] */
    const int32_t *cu_ext;         /* device int32 [num_reqs + 1] */
    const int32_t *positions;      /* device int32 [total_tokens] or NULL */
    int32_t num_reqs, total_tokens, max_ext_len, max_seq_len;
    void *o;                       /* device bf16 [total_tokens, num_q_heads, head_dim] (output) */
    float *lse;                    /* device fp32 [total_tokens, num_q_heads] (output) */
} msgl_extend_batch;

typedef struct msgl_decode_batch {
    msgl_page_table pages;
    const void *q;                 /* device bf16 [num_reqs, num_q_heads, head_dim] */
    const int32_t *seq_lens;       /* device int32 [num_reqs] */
    int32_t num_reqs, max_seq_len;
    void *o;                       /* device bf16 [num_reqs, num_q_heads, head_dim] (output) */
    float *lse;                    /* device fp32 [num_reqs, num_q_heads] (output) */
} msgl_decode_batch;

/*
 * Mixed step: the chunked-prefill batch and the decode batch of one forward
 * in a single call.  Under chunked prefill a forward carries prefill chunks
 * and decode rows together ("Mini-SGLang 实战指南", §6.1 "Chunked
 * Prefill"), and the engine works to keep the GPU from idling between the
 * pieces of a step (§6.6 "Overlap Scheduling").  The results are those of
 * msgl_attn_extend(ext) and msgl_attn_decode(dec) on the same inputs, bit
 * for bit; only the schedule differs.  The decode's key-range kernel runs
 * first; the extend is launched behind it with programmatic dependent
 * launch, so its CTAs take each SM as soon as that SM's decode range is
 * done instead of waiting for the slowest range; the decode's LSE merge
 * runs last.  Every launch shape depends on host scalars only, so the call
 * can be captured in a CUDA graph.
 *
 *   workspace   device scratch of at least
 *               msgl_decode_workspace_size(dec->num_reqs, ...) +
 *               msgl_extend_workspace_size(...) bytes, 256-byte aligned
 *               (NULL when that total is 0); fully rewritten by every call
 * Host validation and device status bits are those of the two calls.  On a
 * validation failure of either batch nothing is launched.
 */
MSGL_API msgl_status msgl_attn_mixed(const msgl_kv_pool *pool, const msgl_extend_batch *ext,
                                     const msgl_decode_batch *dec, int32_t num_q_heads, float scale,
                                     void *workspace, size_t workspace_bytes, uint32_t *status,
                                     msgl_stream_t stream);

/*
 * Decode for callers that cannot allocate device memory.  It has no
 * counterpart on the pages describing the engine: it is msgl_attn_decode
 * with its split scratch taken from a fixed array inside the library
 * instead of a caller workspace.  Meant for callers whose device memory is
 * all owned by a host pool planned up front, plugin-style interfaces that
 * receive only input and output pointers, and loops that cannot afford
 * cudaMalloc's implicit device synchronisation.
 *
 * Arguments, layouts, outputs and device status bits are those of
 * msgl_attn_decode, minus the workspace.  It allocates nothing: the scratch
 * is a static device array of MSGL_DECODE_NOALLOC_SCRATCH_BYTES that every
 * GPU loading the library holds until the process exits.  A call whose
 * msgl_decode_workspace_size() exceeds that size returns
 * MSGL_ERR_WORKSPACE (msgl_last_error() gives both sizes) without launching.
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and caches it.  Under
 * CUDA's lazy module loading that first call is also what loads the module
 * and places the 32 MiB on the device, an implicit allocation with its
 * possible synchronisation: make it once at start-up, before capturing any
 * stream and outside latency-critical loops.  The cached address assumes
 * one CUDA context per device for the life of the process; after a device
 * reset, or under a different driver-API context, use a fresh process.
 * All calls on a device share the array, which keeps the last call's
 * contents (no call relies on them); calls whose kernels overlap on the GPU
 * race on it, so order them.
 */
#define MSGL_DECODE_NOALLOC_SCRATCH_BYTES (32u << 20)

MSGL_API msgl_status msgl_attn_decode_noalloc(const msgl_kv_pool *pool, const msgl_page_table *pages,
                                     const void *q, int32_t num_q_heads, const int32_t *seq_lens,
                                     int32_t num_reqs, int32_t max_seq_len, float scale, void *o,
                                     float *lse, uint32_t *status, msgl_stream_t stream);

/*
 * Block tables and slot maps of one step, built on the GPU from the request
 * lengths, so that admitting and extending requests costs no host loop over
 * tokens and no table upload: every request's pages come from one allocator
 * ("不懂SGLang？从miniSGLang开始", §1.2 item 3; "Mini-SGLang 实战指南", §6.2),
 * and the page table and positions locate each token ("不懂SGLang？从miniSGLang
 * 开始", §1.3 item 3).  Request b holds cached_lens[b] tokens and gets
 * new_lens[b] more.  With P(x) = ceil(x / page_size), s_b = cached + new,
 * need_b = P(s_b) - P(cached_b), off_b = sum of need_i and cu_b = sum of new_i
 * over i < b:
 *   page p of request b = req_table[row_b][p]                for p < P(cached_b),
 *                         free_pages[off_b + p - P(cached_b)] up to P(s_b)
 *   out->page_ids[b][p]                = page p, p < P(s_b) (later entries are left as they were)
 *   req_table[row_b][p]                = page p, P(cached_b) <= p < P(s_b)
 *   out->seq_lens[b] = s_b,  out->cu_ext[b] = cu_b (and cu_ext[num_reqs] = the sum)
 *   out->positions[cu_b + i] = cached_b + i
 *   out->out_loc[cu_b + i]   = the slot of that position: page id * page_size + offset
 *   out->pages_taken[0]      = sum of need_b: how many of free_pages are now in use
 * These are the arguments of msgl_store_kv, msgl_attn_extend (prefix_lens =
 * cached_lens, ext_lens = new_lens) and msgl_attn_decode (new_lens = 1).
 *
 *   req_table    device int32 [num_rows, table_stride]: the page ids of every running
 *                request, table_width valid columns (in and out)
 *   req_rows     device int32 [num_reqs] or NULL (row_b = b): distinct rows; a row named
 *                twice ends with either one's new pages
 *   cached_lens  device int32 [num_reqs];  new_lens device int32 [num_reqs] or NULL (1 each)
 *   free_pages   device int32 [num_free]: page ids in the order they are handed out
 *   out          total_tokens entries of positions and out_loc; when the step has fewer tokens
 *                (a captured step padded to a bucket) the entries behind them are
 *                positions = 0, out_loc = -1, so that a store skips them
 * No array that the step writes may overlap another of its arrays (MSGL_ERR_INVALID_ARG): a loop that
 * passes the last step's seq_lens on as cached_lens alternates between two sets of outputs.  One
 * exception: out->page_ids may be req_table itself, at the same stride and without req_rows.
 * A request is refused when its
 * length is negative or needs more columns than either table has, or its row is
 * outside the table (MSGL_DEVERR_LENGTH), when its tokens pass total_tokens
 * (MSGL_DEVERR_LENGTH), or when free_pages does not reach its last new page
 * (MSGL_DEVERR_NO_PAGES; its place in the order is kept, so every later request
 * that needs a page is refused too, and pages_taken counts up to the last one
 * served).  A refused request gets seq_lens = 0 (the attention calls then
 * write its row as zero), out_loc = -1 and positions = 0 for its tokens, and its table
 * rows are left as they were.  A token on a page whose id is outside
 * [0, num_slots / page_size) gets out_loc = -1 and MSGL_DEVERR_PAGE_RANGE.
 * num_slots may not pass 2^31 (out_loc is int32).  The launch shape depends on
 * host scalars only.
 */
typedef struct msgl_step_out {
    int32_t *page_ids;             /* device int32 [num_reqs, stride] */
    int32_t stride, width;         /* row pitch and valid columns of page_ids */
    int32_t *seq_lens;             /* device int32 [num_reqs] */
    int32_t *cu_ext;               /* device int32 [num_reqs + 1] */
    int32_t *positions;            /* device int32 [total_tokens] */
    int32_t *out_loc;              /* device int32 [total_tokens] */
    int32_t *pages_taken;          /* device int32 [1] */
    int32_t total_tokens;
} msgl_step_out;

MSGL_API msgl_status msgl_step_tables(int64_t num_slots, int32_t page_size, int32_t *req_table, int32_t num_rows,
                                      int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                                      const int32_t *cached_lens, const int32_t *new_lens, int32_t num_reqs,
                                      const int32_t *free_pages, int32_t num_free, const msgl_step_out *out,
                                      uint32_t *status, msgl_stream_t stream);

/*
 * Store step with the rotation in it: q and k of the new tokens turned by their
 * positions, q written to q_out, k and v to the pool ("不懂SGLang？从miniSGLang开始",
 * §1.3 items 1 and 3: the positions are an input of the forward, the new K/V
 * become part of the pool).  Pair j of a head, (x_j, y_j), turns by
 *   angle_j = positions[axis_j][t] * f_j:
 *   x' = factor * (x cos - y sin),  y' = factor * (y cos + x sin)
 * with x_j, y_j = dims j and j + num_pairs, or (adjacent) 2j and 2j + 1; dims from
 * 2 * num_pairs on stay as they are.  With q_norm / k_norm a head is first
 * replaced by x * w / sqrt(mean(x^2) + eps).  All of it is computed in 32 bits (the
 * angle modulo a turn in 64, then rounded) and rounded to bf16 once; v is copied.
 *
 *   turns        device uint64 [num_pairs]: f_j / (2 pi) * 2^64 modulo 2^64
 *   axes         host uint8 [num_pairs]: axis_j < num_axes, or NULL (all 0)
 *   num_pairs    8, 16, .. 64;  num_axes 1..4
 *   q, k, v      device bf16 [n_tokens, heads, head_dim], token t at t * stride elements
 *                (strides: multiples of 8, at least heads * head_dim), so that they may
 *                be columns of one projection's output
 *   q_out        the same for the turned q; may be q itself (same stride), and may not
 *                otherwise overlap an input
 *                (nor may the pools overlap an input, q_out or each other: k and v of one
 *                token are stored while another's are read)
 *   positions    device int32, axis a of token t at a * axis_stride + t; any int32 value.
 *                axis_stride: at least n_tokens, or 0 (the same positions on every axis)
 *   out_loc      device int32 [n_tokens]: the token's pool slot.  -1: not a token (the
 *                padding of msgl_step_tables, and the tokens of a request that it
 *                refused): nothing is written for it, its row of q_out stays as it
 *                was.  Its rows of q, k and v and its positions may be read, so they
 *                have to be memory like the others'; what they hold does not matter.
 *                Another slot out of range sets MSGL_DEVERR_SLOT_RANGE: q is turned,
 *                nothing stored.
 *   q_norm, k_norm  device bf16 [head_dim] or NULL
 * Duplicate slots are undefined (what ends there may be of either row, or of both).
 */
typedef struct msgl_rope {
    const uint64_t *turns;         /* device */
    const uint8_t *axes;           /* host, or NULL */
    int32_t num_pairs, num_axes;
    int32_t adjacent;
    float factor;                  /* normally 1 */
} msgl_rope;

typedef struct msgl_new_tokens {
    const void *q, *k, *v;         /* device bf16 */
    void *q_out;
    int64_t q_stride, k_stride, v_stride, out_stride;   /* elements */
    const int32_t *positions;      /* device int32 [num_axes, n_tokens], rows axis_stride apart */
    int64_t axis_stride;
    const int32_t *out_loc;        /* device int32 [n_tokens] */
    int32_t n_tokens, num_q_heads;
} msgl_new_tokens;

MSGL_API msgl_status msgl_rope_store_kv(const msgl_kv_pool *pool, const msgl_new_tokens *tokens, const msgl_rope *rope,
                                        const void *q_norm, const void *k_norm, float eps, uint32_t *status,
                                        msgl_stream_t stream);

/*
 * Drafted tokens accepted or replaced by the target's probabilities, from given
 * random numbers, without the host (a decode step is a graph replay: "Mini-SGLang
 * 实战指南", §6.4).  A step fed request b's last token and its drafts, so rows
 * first = cu_ext[b] .. cu_ext[b+1]-1 of the step are its: tokens[first] the token
 * before the drafts, tokens[first + i + 1] draft i, and row first + i of the
 * target's probabilities is the distribution that draft i is held against (the
 * last row: that of the token behind all drafts).  Draft i stands when
 *   accept_u[first + i] * q(x) < p(x),   x = tokens[first + i + 1],
 * p and q rows first + i of target and draft.  With a the number of drafts in
 * front of the first one that does not stand, and r = first + a:
 *   w = max(p_r - q_r, 0) when a draft was refused, p_r when none was or when
 *       that has no positive finite sum (it is zero everywhere, or q_r no probabilities);
 *   the new token = the first v with w_0 + .. + w_v > sample_u[b] * sum(w)
 *       (the last one with w > 0 when there is none, as for sample_u >= 1)
 *   accepted[b] = a;  kv_lens[b] = cached_lens[b] + a + 1
 *   out_tokens[first + i] = draft i for i < a, the new token at i = a, -1 behind it
 * kv_lens counts the tokens whose K/V of this step are kept: the cached_lens of the
 * next msgl_step_tables (the new token's K/V are stored by that step).
 * Weights are taken in 32 bits, sums in pairs of 32-bit numbers (about 46 bits).  What is
 * not a number weighs nothing.
 *
 *   target, draft  device fp32 or bf16 (both the same) [total_tokens, vocab], rows
 *                  stride elements apart; they need not sum to 1.  draft NULL: the
 *                  drafts were not drawn at random, q(x) = 1 for each draft x itself
 *   tokens         device int32 [total_tokens];  cu_ext device int32 [num_reqs + 1]
 *   accept_u       device fp32 [total_tokens] (a request's last entry is not used)
 *   sample_u       device fp32 [num_reqs], in [0, 1)
 *   cached_lens    device int32 [num_reqs] or NULL (0)
 *   accepted, kv_lens  device int32 [num_reqs];  out_tokens device int32 [total_tokens]
 * The outputs may overlap neither an input nor each other (kv_lens may be
 * cached_lens itself).  Rows outside all requests are not touched.  A request without rows
 * gets accepted = 0 and kv_lens = cached_lens; so does one whose cu_ext
 * entries are out of order or range (MSGL_DEVERR_LENGTH).  A draft outside
 * [0, vocab) does not stand (MSGL_DEVERR_TOKEN).  Where w has no positive
 * finite sum the new token is -1 (MSGL_DEVERR_PROBS).  vocab is at most 2^30.
 */
typedef struct msgl_draft_batch {
    const void *target, *draft;
    int64_t target_stride, draft_stride;
    int32_t vocab, is_bf16;
    const int32_t *tokens, *cu_ext;
    const float *accept_u, *sample_u;
    const int32_t *cached_lens;
    int32_t num_reqs, total_tokens;
    int32_t *accepted, *out_tokens, *kv_lens;
} msgl_draft_batch;

MSGL_API msgl_status msgl_verify_drafts(const msgl_draft_batch *batch, uint32_t *status, msgl_stream_t stream);

/*
 * Requests that continue other requests on the same pages (parallel samples of a
 * prompt, beams): fork i gives row child_rows[i] of req_table the first lens[i]
 * tokens of row parent_rows[i].  Whole pages are shared ("Mini-SGLang 实战指南", §6.5:
 * requests hold the same prefix pages); a partly filled last page would be written by
 * both, so the child gets a page of its own for it:
 *   F = lens[i] / page_size, tail = lens[i] % page_size
 *   req_table[child][p] = req_table[parent][p]             for p < F
 *   tail > 0: req_table[child][F] = free_pages[k], k the number of earlier forks with a tail
 *             whose rows and length are in range (refused for something else or not);
 *             copy_src[i] = req_table[parent][F], copy_dst[i] = that page, copy_tokens[i] = tail
 *   else      copy_src[i] = copy_dst[i] = -1, copy_tokens[i] = 0
 *   pages_taken[0] = the number of all such forks, at most num_free: free_pages from there
 *             on are as free as before (so are those in front that a refused fork left)
 * The copies are the arguments of msgl_copy_pages.  Later columns of the child's row stay
 * as they are.  lens[i] counts tokens that the parent keeps: a page that it will write
 * again (under drafts that may yet be refused) is not to be shared.
 *   req_table    device int32 [num_rows, table_stride], table_width valid columns (in and out)
 *   parent_rows, child_rows, lens   device int32 [num_forks]; both rows -1: no fork (padding)
 * Refused are a fork whose rows are outside the table, or whose child is also a parent
 * or another fork's child (MSGL_DEVERR_ROW); one whose length is negative or passes
 * table_width (MSGL_DEVERR_LENGTH); one that free_pages does not reach
 * (MSGL_DEVERR_NO_PAGES); and one whose new page or partly filled page is
 * outside [0, num_slots / page_size) (MSGL_DEVERR_PAGE_RANGE).  A refused fork's
 * row is left as it was and nothing is copied for it.  Its place among the free
 * pages stays unused, so that the others' places do not depend on it; a fork whose
 * rows are outside the table or whose length cannot be has no place.  The outputs
 * may overlap neither an input nor each other.
 */
typedef struct msgl_fork_out {
    int32_t *copy_src, *copy_dst, *copy_tokens;   /* device int32 [num_forks] */
    int32_t *pages_taken;                         /* device int32 [1] */
} msgl_fork_out;

MSGL_API msgl_status msgl_fork_requests(int64_t num_slots, int32_t page_size, int32_t *req_table, int32_t num_rows,
                                        int32_t table_stride, int32_t table_width, const int32_t *parent_rows,
                                        const int32_t *child_rows, const int32_t *lens, int32_t num_forks,
                                        const int32_t *free_pages, int32_t num_free, const msgl_fork_out *out,
                                        uint32_t *status, msgl_stream_t stream);

/*
 * Copies pages within the pools of several layers (one page table serves all layers:
 * "Mini-SGLang 实战指南", §6.2): in every pool, the first tokens[i] slots of page src[i], K
 * and V, go to page dst[i], bit for bit.
 *   pools        host array [num_pools] of the same num_slots, page_size and heads, at most
 *                2^15 of them
 *   src, dst     device int32 [num_pairs]; both -1: no copy (padding)
 *   tokens       device int32 [num_pairs], 0..page_size, or NULL (whole pages)
 *   count        device int32 [1] or NULL: only the first count[0] pairs
 * A page id outside the pool (MSGL_DEVERR_PAGE_RANGE) or a count of tokens out of
 * range (MSGL_DEVERR_LENGTH) skips the pair.  A page that is written and
 * is also another pair's src or dst is undefined (parts of either may end there).
 */
MSGL_API msgl_status msgl_copy_pages(const msgl_kv_pool *pools, int32_t num_pools, const int32_t *src,
                                     const int32_t *dst, const int32_t *tokens, int32_t num_pairs,
                                     const int32_t *count, uint32_t *status, msgl_stream_t stream);

/*
 * The pages that no running request holds, in ascending order: the free_pages of the next
 * msgl_step_tables or msgl_fork_requests.  Request b holds the first
 * ceil(lens[b] / page_size) entries of its row, so pages come back by what the
 * tables no longer say: a finished request is left out, a request whose drafts
 * were refused comes with its shorter length, a page that forks share is free
 * when none of them holds it.
 *   req_table    device int32 [num_rows, table_stride], table_width valid columns
 *   req_rows     device int32 [num_reqs] or NULL (row b); -1: no request (padding)
 *   lens         device int32 [num_reqs], at most 2^24 of them
 *   held         device uint8 [num_slots / page_size] or NULL: not 0 for a page that something
 *                else holds (a radix cache's pages, a request that waits).  The caller keeps
 *                these: include/msgl_radix.h hands page ids out and does not list them
 *   pages        device int32 [num_slots / page_size] (output): the free pages' ids, -1 behind them
 *   num_free     device int32 [1] (output): how many there are
 * A row outside the table (MSGL_DEVERR_ROW) holds nothing; a request whose length is
 * negative or passes table_width (MSGL_DEVERR_LENGTH) holds all of its row, so that none
 * of its pages is given away; an id outside the pool (MSGL_DEVERR_PAGE_RANGE) is
 * skipped.  The outputs may overlap neither an input nor each other.
 *   workspace    device scratch of at least msgl_page_map_workspace_size() bytes, 256-byte
 *                aligned; what it held does not matter.  It may overlap neither an input nor
 *                an output, and two calls (or captured graphs) that may run at once need
 *                one each
 */
MSGL_API size_t msgl_page_map_workspace_size(int64_t num_slots, int32_t page_size);

MSGL_API msgl_status msgl_free_pages(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                                     int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                                     const int32_t *lens, int32_t num_reqs, const uint8_t *held, int32_t *pages,
                                     int32_t *num_free, void *workspace, size_t workspace_bytes, uint32_t *status,
                                     msgl_stream_t stream);

/*
 * The pages in use moved to the front of the pool, so that the pool may shrink
 * or grow, or pages be handed out as long runs.  With U the number of pages that
 * requests hold (as above) or `held` names: the pages that requests hold and
 * `held` does not, with ids from U on, in ascending order, move to the first free
 * ids below U, in ascending order.
 *   out->src, out->dst      the moves (the arguments of msgl_copy_pages, with
 *                           count = out->num_moves), -1 behind them
 *   out->remap[p]           page p's id from now on (p itself when it stays), -1 when it is free
 *   out->page_ids           the rows of the requests with the new ids in their pages' columns;
 *                           may be req_table itself at the same stride.  An id outside the
 *                           pool stays; other columns and rows are left as they were
 *   out->num_used[0]        U
 * A page that `held` names stays where it is (ids from U on may then be in use).
 * The pages have to be copied before they are read or written again.
 * Requests, errors, overlaps and the workspace are those of msgl_free_pages (a request
 * that holds all of its row gets new ids in all of it); a row may be named twice.
 */
typedef struct msgl_compact_out {
    int32_t *page_ids;             /* device int32 [num_rows, stride] */
    int32_t stride;
    int32_t *remap;                /* device int32 [num_slots / page_size] */
    int32_t *src, *dst;            /* device int32 [num_slots / page_size / 2] */
    int32_t *num_moves, *num_used; /* device int32 [1] */
} msgl_compact_out;

MSGL_API msgl_status msgl_compact_pages(int64_t num_slots, int32_t page_size, const int32_t *req_table,
                                        int32_t num_rows, int32_t table_stride, int32_t table_width,
                                        const int32_t *req_rows, const int32_t *lens, int32_t num_reqs,
                                        const uint8_t *held, const msgl_compact_out *out, void *workspace,
                                        size_t workspace_bytes, uint32_t *status, msgl_stream_t stream);

/*
 * Groups of neighbouring requests whose page tables begin with the same pages:
 * the input of msgl_attn_decode_shared.  A radix-cache hit gives requests the
 * same prefix pages ("Mini-SGLang 实战指南", §6.5 "Radix Cache"), so the tables
 * tell which requests share without the tree.  With d_b the number of leading
 * columns on which rows b-1 and b agree (within both requests' pages) and
 * m_b = min(d_b * page_size, seq_lens[b-1], seq_lens[b]):
 *   b joins the group of b-1 when m_b >= min_shared
 *   group_start[b] = the first row of b's group
 *   shared_lens[b] = min of m over the group's joined rows (0 for a group of one)
 * One level of sharing: a batch sorted by prefix gets the most out of it, and
 * min_shared (at least 1) chooses between few groups with a short prefix in
 * common and more groups with longer ones.
 *
 *   seq_lens     device int32 [num_reqs]; a request whose length is outside
 *                [1, max_seq_len] (MSGL_DEVERR_LENGTH) or passes the table's width
 *                (MSGL_DEVERR_PAGE_RANGE) is a group of one; max_seq_len is at most 2^30
 *   group_start, shared_lens   device int32 [num_reqs] (output); they may overlap neither each
 *                other nor an input (MSGL_ERR_INVALID_ARG)
 */
MSGL_API msgl_status msgl_shared_prefixes(const msgl_page_table *pages, const int32_t *seq_lens, int32_t num_reqs,
                                          int32_t page_size, int32_t max_seq_len, int32_t min_shared,
                                          int32_t *group_start, int32_t *shared_lens, uint32_t *status,
                                          msgl_stream_t stream);

/*
 * Decode for a batch in which groups of requests share a prefix: the result of
 * msgl_attn_decode, with the keys that a group shares read once for all of its
 * requests (a shared system prompt or document held once in the pool by the
 * radix cache: "Mini-SGLang 实战指南", §6.5 "Radix Cache", §6.3).
 * The requests of a group are neighbours in the batch.  Row b attends keys
 * 0..shared_lens[b]-1 at the slots of row group_start[b]'s page table, and keys
 * shared_lens[b]..seq_lens[b]-1 at the slots of its own.  Where it pays, a
 * group's query rows go through the tensor cores together against its shared
 * keys, every row's own keys take the decode's path, and the two are joined by
 * their log-sum-exp; elsewhere the decode's path reads a shared key once for
 * each request, out of L2 after the first.
 *
 *   group_start  device int32 [num_reqs]: the first row of b's group, so
 *                group_start[b] is b or group_start[b-1]
 *   shared_lens  device int32 [num_reqs]: 0 <= shared_lens[b] <= seq_lens[b],
 *                the same for all rows of a group (of a group of one it is
 *                not used: all keys are its own)
 *   sharing      MSGL_SHARE_AUTO: by the batch's lengths and groups, found on the
 *                device; MSGL_SHARE_ALWAYS / MSGL_SHARE_NEVER: one or the other, whatever
 *                the batch.  None of them makes a row's bits independent of the rest of the
 *                batch: where a row's keys are cut into pieces follows from the sums over
 *                all rows, and each piece rounds its weights against a maximum of its own.
 *                The same arguments give the same bits.
 *   workspace    device scratch of at least msgl_decode_shared_workspace_size()
 *                bytes, 256-byte aligned, fully rewritten by every call; two calls
 *                (or captured graphs) that may overlap need one each
 * Every other argument, the outputs and the status bits are those of
 * msgl_attn_decode.  A row whose group entries break these rules sets
 * MSGL_DEVERR_GROUP and is written as o = 0, lse = -inf, and so may be the rows
 * of its group behind it; a bad page among the shared keys does that to every
 * row of the group (MSGL_DEVERR_PAGE_RANGE).
 * At most 65535 requests, max_seq_len at most 2^30.  A CTA that would work on one
 * group's shared keys for more than about 2 s (some 170 million keys) gives up with
 * MSGL_DEVERR_TIMEOUT.  The launch shapes depend on host scalars only.
 */
#define MSGL_SHARE_AUTO 0
#define MSGL_SHARE_ALWAYS 1
#define MSGL_SHARE_NEVER 2

MSGL_API size_t msgl_decode_shared_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                  int32_t head_dim, int32_t max_seq_len);

MSGL_API msgl_status msgl_attn_decode_shared(const msgl_kv_pool *pool, const msgl_page_table *pages, const void *q,
                                             int32_t num_q_heads, const int32_t *group_start,
                                             const int32_t *shared_lens, const int32_t *seq_lens,
                                             int32_t num_reqs, int32_t max_seq_len, int32_t sharing,
                                             float scale, void *o, float *lse, void *workspace,
                                             size_t workspace_bytes, uint32_t *status, msgl_stream_t stream);

/*
 * Synchronises `stream`, reads the device status word into *flags (may be
 * NULL) and maps it to a status: MSGL_OK when it is zero, MSGL_ERR_TIMEOUT
 * when the timeout bit is set, else MSGL_ERR_OUT_OF_RANGE.  For tests and
 * debugging; not meant for the hot path.
 */
MSGL_API msgl_status msgl_read_status(const uint32_t *status, uint32_t *flags, msgl_stream_t stream);

/*
 * Self-test of the bounded wait every kernel uses (no counterpart on the
 * pages).  Launches one thread that waits on an mbarrier that nothing arrives
 * at, with a budget of budget_cycles SM clocks (0 < budget <= 4e9; ~1e7 is
 * about 5 ms).  The wait gives up, MSGL_DEVERR_TIMEOUT is ORed into *status,
 * and the kernel returns normally.  Use it to check that a lost arrival turns
 * into a status bit and the context stays usable.
 */
MSGL_API msgl_status msgl_selftest_wait_timeout(uint32_t *status, int64_t budget_cycles,
                                                msgl_stream_t stream);

/*
 * Host-side checks of one step's metadata, for tests and debugging.  They
 * read HOST copies of the arrays (copy the device arrays back first), launch
 * nothing, need no GPU and allocate no device memory.  The kernels check the same
 * conditions on the device and report them through the status word; these
 * calls name the first offending entry in msgl_last_error().  Each returns
 * MSGL_OK, MSGL_ERR_INVALID_ARG (NULL array, bad scalar, inconsistent
 * lengths, wrong position, duplicate slot) or MSGL_ERR_OUT_OF_RANGE (a slot,
 * page index or page id outside the pool or the table).  The store's and the
 * step's keep what they have seen in host memory; where that runs out they
 * return MSGL_ERR_UNSUPPORTED.
 *
 * msgl_check_store_meta:  every out_loc[t] lies in [0, num_slots) and no
 *   slot is named twice (the store's result would depend on which row wins).
 * msgl_check_extend_meta:  prefix_lens[b] >= 0, ext_lens[b] >= 0,
 *   cu_ext[0] = 0, cu_ext[b+1] - cu_ext[b] = ext_lens[b], cu_ext[num_reqs] =
 *   total_tokens, ext_lens[b] <= max_ext_len, prefix_lens[b] + ext_lens[b]
 *   <= max_seq_len, positions[cu_ext[b] + i] = prefix_lens[b] + i (when
 *   positions is non-NULL), and every page that keys 0..prefix_lens[b] +
 *   ext_lens[b] - 1 fall on has an index below width and an id in
 *   [0, num_slots / page_size).
 * msgl_check_decode_meta:  1 <= seq_lens[b] <= max_seq_len and the pages of
 *   keys 0..seq_lens[b] - 1 are in range as above.
 *
 * page_ids is host int32 [num_reqs, stride]; only the first width entries of
 * a row are read.  The pages ("不懂SGLang？从miniSGLang开始", §1.3 item 3;
 * "Mini-SGLang 实战指南", §6.1, §6.2) define what the metadata means; these
 * checks have no counterpart there.
 */
MSGL_API msgl_status msgl_check_store_meta(int64_t num_slots, const int32_t *out_loc, int32_t n_tokens);

MSGL_API msgl_status msgl_check_extend_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids,
                                            int32_t stride, int32_t width, const int32_t *prefix_lens,
                                            const int32_t *ext_lens, const int32_t *cu_ext,
                                            const int32_t *positions, int32_t num_reqs, int32_t total_tokens,
                                            int32_t max_ext_len, int32_t max_seq_len);

MSGL_API msgl_status msgl_check_decode_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids,
                                            int32_t stride, int32_t width, const int32_t *seq_lens,
                                            int32_t num_reqs, int32_t max_seq_len);

/*
 * The same for the arguments of msgl_step_tables and msgl_attn_decode_shared
 * (host copies of the arrays, nothing launched):
 *
 * msgl_check_step_meta:  rows in range and none twice, lengths >= 0, every
 *   request within the table's width, the pages of its cached tokens in the
 *   pool, total_tokens and num_free large enough, and every free page that the
 *   step takes in the pool and not in use by a request of the step.
 * msgl_check_groups_meta:  the rules of group_start and shared_lens, 1 <=
 *   seq_lens[b] <= max_seq_len, and the pages of the keys as they are read
 *   (shared ones through the group's first row) in range.
 */
MSGL_API msgl_status msgl_check_step_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table,
                                          int32_t num_rows, int32_t table_stride, int32_t table_width,
                                          const int32_t *req_rows, const int32_t *cached_lens,
                                          const int32_t *new_lens, int32_t num_reqs, const int32_t *free_pages,
                                          int32_t num_free, int32_t total_tokens);

MSGL_API msgl_status msgl_check_groups_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids,
                                            int32_t stride, int32_t width, const int32_t *group_start,
                                            const int32_t *shared_lens, const int32_t *seq_lens, int32_t num_reqs,
                                            int32_t max_seq_len);

/*
 * The same for the arguments of msgl_fork_requests, msgl_copy_pages, msgl_free_pages and
 * msgl_compact_pages, and msgl_verify_drafts (host copies of the arrays, nothing
 * launched; padding entries of -1 are passed over):
 *
 * msgl_check_fork_meta:  rows in range, no child a parent or another fork's child,
 *   0 <= lens[i] and within the table's width, the parents' pages in the pool,
 *   num_free large enough, and every free page that the forks take in the pool, taken
 *   once and not a page of a parent.
 * msgl_check_copy_meta:  pages in range, 0 <= tokens[i] <= page_size, and no page that is
 *   written is another pair's src or dst.
 * msgl_check_held_meta:  (free, compact) rows in range, lengths within the table's
 *   width, and the requests' pages in the pool.
 * msgl_check_draft_meta:  cu_ext in order and within total_tokens, drafted tokens in
 *   [0, vocab), accept_u and sample_u in [0, 1) where they are used.
 */
MSGL_API msgl_status msgl_check_fork_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table,
                                          int32_t num_rows, int32_t table_stride, int32_t table_width,
                                          const int32_t *parent_rows, const int32_t *child_rows, const int32_t *lens,
                                          int32_t num_forks, const int32_t *free_pages, int32_t num_free);

MSGL_API msgl_status msgl_check_copy_meta(int64_t num_slots, int32_t page_size, const int32_t *src, const int32_t *dst,
                                          const int32_t *tokens, int32_t num_pairs);

MSGL_API msgl_status msgl_check_held_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table,
                                          int32_t num_rows, int32_t table_stride, int32_t table_width,
                                          const int32_t *req_rows, const int32_t *lens, int32_t num_reqs);

MSGL_API msgl_status msgl_check_draft_meta(int32_t vocab, const int32_t *tokens, const int32_t *cu_ext,
                                           const float *accept_u, const float *sample_u, int32_t num_reqs,
                                           int32_t total_tokens);

/* Static description of a status code. */
MSGL_API const char *msgl_status_string(msgl_status s);

/* Thread-local text of the last failure in this thread (empty if none). */
MSGL_API const char *msgl_last_error(void);

/* MSGL_ABI_VERSION of the built library. */
MSGL_API int32_t msgl_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MSGL_ATTN_H */
