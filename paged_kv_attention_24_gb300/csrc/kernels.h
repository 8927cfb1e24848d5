// Launchers shared between the C-ABI layer (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace msgl {

// ---------------------------------------------------------------- store
cudaError_t launch_store_kv(const PoolView &pool, __nv_bfloat16 *k_pool, __nv_bfloat16 *v_pool,
                            const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                            const int32_t *out_loc, int32_t n_tokens, uint32_t *status,
                            cudaStream_t stream);

// --------------------------------------------------------------- decode
struct DecodePlan {
    size_t o_bytes;       // bytes of the fp32 partial outputs (start of the workspace)
    size_t workspace;     // total bytes: partial outputs, then partial LSEs
};
DecodePlan plan_decode(int32_t num_reqs, int32_t hq, int32_t hkv, int32_t max_seq_len);

struct DecodeArgs {
    PoolView pool;
    PageView pages;
    const __nv_bfloat16 *q;
    const int32_t *seq_lens;
    int32_t num_reqs, hq, max_seq_len;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;      // [num_reqs + max CTAs, hq, 128] segment partials
    float *part_lse;    // [num_reqs + max CTAs, hq]
    uint32_t *status;
    const __nv_bfloat16 *k_new = nullptr, *v_new = nullptr;   // append mode (see msgl_attn_decode_append)
    const int32_t *new_loc = nullptr;
    // groups over shared prefixes (see msgl_attn_decode_shared): shared keys are read through the
    // group's first row, or, where that pays, left to the shared-prefix kernel behind which the
    // split is then launched (split phase only, share.sms > 0)
    const int32_t *group_start = nullptr, *shared_lens = nullptr;
    int32_t pair_rows = 0;      // rows of a pair of its Q tiles
    ShareModel share{};
};
// Which kernels of a decode call to launch: the split (partials per key range), the
// merge (LSE fold of the partials, launched with programmatic dependent launch), or both.
enum class DecodePhase { kSplit, kMerge, kBoth };
// The split kernel's grid and speed for these heads and pages (sms and always are not set).
ShareModel decode_split_model(int32_t hq, const PoolView &pool);
cudaError_t launch_decode(const DecodeArgs &a, const DecodePlan &plan, cudaStream_t stream,
                          DecodePhase phase = DecodePhase::kBoth);

// --------------------------------------------------------------- extend
size_t extend_workspace_bytes(int32_t num_reqs, int32_t total_tokens, int32_t hq, int32_t hkv,
                              int32_t max_seq_len);

struct ExtendArgs {
    PoolView pool;
    PageView pages;
    const __nv_bfloat16 *q;
    const int32_t *prefix_lens, *ext_lens, *cu_ext, *positions;
    int32_t num_reqs, total_tokens, hq, max_ext_len, max_seq_len;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    void *workspace;
    uint32_t *status;
    // launch with programmatic dependent launch: CTAs may start while the previous
    // kernel on the stream still runs (the grid's last CTA waits for that kernel, so the
    // grid does not complete before it)
    bool pdl = false;
};
cudaError_t launch_extend(const ExtendArgs &a, cudaStream_t stream);

// ------------------------------------------------- step tables, prefix groups
constexpr int64_t kMaxStepItems = 65535ll * 2048;   // tokens of a step, columns of a table (grid.y)

struct StepTablesArgs {
    int32_t *req_table;
    const int32_t *req_rows, *cached_lens, *new_lens, *free_pages;
    int32_t num_rows, table_stride, num_reqs, num_free, num_pages, log2_ps;
    int32_t max_pages;    // columns that both tables have
    int32_t *page_ids, *seq_lens, *cu_ext, *positions, *out_loc, *pages_taken;
    int32_t stride, total_tokens;
    uint32_t *status;
};
cudaError_t launch_step_tables(const StepTablesArgs &a, cudaStream_t stream);

struct SharedPrefixesArgs {
    PageView pages;
    const int32_t *seq_lens;
    int32_t num_reqs, log2_ps, max_seq_len, min_shared;
    int32_t *group_start, *shared_lens;
    uint32_t *status;
};
cudaError_t launch_shared_prefixes(const SharedPrefixesArgs &a, cudaStream_t stream);

// ------------------------------------------- around the step: rotary store, drafts, pages
struct RopeStoreArgs {
    PoolView pool;
    __nv_bfloat16 *k_pool, *v_pool;
    const __nv_bfloat16 *q, *k, *v, *q_norm, *k_norm;
    __nv_bfloat16 *q_out;
    int64_t q_stride, k_stride, v_stride, out_stride;   // elements from token to token
    const int32_t *positions, *out_loc;
    int64_t axis_stride;
    const uint64_t *turns;                // a pair's frequency: turns per position * 2^64, modulo 2^64
    uint32_t axis_bits[kHeadDim / 32];    // a pair's axis, two bits each
    int32_t pairs, adjacent, n_tokens, hq;
    float factor, eps;
    uint32_t *status;
};
cudaError_t launch_rope_store(const RopeStoreArgs &a, cudaStream_t stream);

constexpr int kMaxDraftReqs = 1 << 24;    // a cluster of up to 8 blocks each (grid.x)

struct VerifyArgs {
    const void *target, *draft;           // [total_tokens, vocab] float or bf16; draft may be NULL
    int64_t target_stride, draft_stride;
    const int32_t *tokens, *cu_ext, *cached_lens;
    const float *accept_u, *sample_u;
    int32_t num_reqs, total_tokens, vocab, bf16;
    int32_t *accepted, *out_tokens, *kv_lens;
    uint32_t *status;
};
cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream);

struct ForkArgs {
    int32_t *req_table;
    const int32_t *parent_rows, *child_rows, *lens, *free_pages;
    int32_t num_rows, table_stride, table_width, num_forks, num_free, num_pages, log2_ps;
    int32_t *copy_src, *copy_dst, *copy_tokens, *pages_taken;
    uint32_t *status;
};
cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream);

constexpr int kMaxCopyPools = 128;        // pools of one copy launch (their addresses are kernel arguments)

struct CopyPagesArgs {
    const int32_t *src, *dst, *tokens, *count;
    int64_t page_vecs;                    // 16-byte vectors of a page and of a slot's row
    int32_t row_vecs, page_size, num_pages, num_pairs, num_buffers;
    int32_t pieces, group, span, turns;   // set by the launcher
    uint32_t *status;
};
// buffers: K and V of each pool, a.num_buffers (at most 2 * kMaxCopyPools) in all
cudaError_t launch_copy_pages(CopyPagesArgs a, void *const *buffers, cudaStream_t stream);

struct PageMapArgs {
    const int32_t *table, *req_rows, *lens;
    const uint8_t *held;
    int32_t num_rows, table_stride, table_width, num_reqs, num_pages, log2_ps;
    int32_t *pages_out;                   // [num_pages]: the free pages; compact: each page's new id
    int32_t *count_out;                   // [1]: free pages; compact: pages that move
    int32_t *table_out, *src, *dst, *used_out;   // compact
    int32_t out_stride;
    uint32_t *used_bits, *stay_bits;      // in the workspace (set by the launchers): by words of 32 pages
    uint2 *moves;                         // compact: which pages of a word move, and how many before them
    uint32_t *status;
};
size_t page_map_workspace_bytes(int32_t num_pages);
cudaError_t launch_free_pages(PageMapArgs a, void *workspace, cudaStream_t stream);
cudaError_t launch_compact_pages(PageMapArgs a, void *workspace, cudaStream_t stream);

// -------------------------------------------------------- shared-prefix decode
size_t decode_shared_workspace_bytes(int32_t num_reqs, int32_t hq, int32_t hkv);

struct DecodeSharedArgs {
    DecodeArgs dec;     // group_start and shared_lens among them
    int32_t sharing;    // MSGL_SHARE_*
    void *workspace;
};
// One launch for short requests (decode_short.cu); the groups' shared keys are read through the
// first row.
cudaError_t launch_decode_short(const DecodeArgs &a, cudaStream_t stream);
cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream);

// The tensor maps of an attention kernel with GQA-packed 128-row Q tiles of `rows` tokens and
// 128-key K/V tiles: q[tokens, hq, 128], four-row gathers from the pools, and (page_size >= 16)
// boxes of whole page runs.
struct AttnMaps {
    CUtensorMap q, k, v, kt, vt;
    int32_t q_box_rows;   // tokens of one Q box
    int32_t box_rows;     // slots of one K/V box (0: gathers or 16-byte copies only)
    int32_t v_blocks;     // V boxes land in blocks of 16 keys
    int32_t oob_row;      // a gather row past the pool (reads as zeros)
};
cudaError_t encode_attn_maps(const PoolView &pool, const __nv_bfloat16 *q, int32_t hq, int32_t tokens, int32_t rows,
                             AttnMaps &m);

// cuTensorMapEncodeTiled from the driver (NULL if unavailable); looked up once.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// SM count of the current device, queried once per device and cached (0..63;
// other ordinals are queried on every call).
int sm_count();

// Sets the text msgl_last_error() returns on this thread.
void set_last_error(const char *msg);

}  // namespace msgl
