// The C ABI of libmsgl_attn: argument checks, launch planning and status
// reporting.  Every compute step runs in the kernels of the other files.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "kernels.h"

namespace {

thread_local char g_last_error[512];

msgl_status fail(msgl_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
msgl_status fail(msgl_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return s;
}

msgl_status cuda_fail(cudaError_t e, const char *what) {
    return fail(MSGL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int log2_exact(int32_t x) {
    if (x <= 0 || (x & (x - 1)) != 0) return -1;
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// Checks shared by every call on the pool; fills the kernels' view of it.
msgl_status check_pool(const msgl_kv_pool *pool, msgl::PoolView &view) {
    if (!pool) return fail(MSGL_ERR_INVALID_ARG, "pool is NULL");
    if (!pool->k_pool || !pool->v_pool) return fail(MSGL_ERR_INVALID_ARG, "pool buffers are NULL");
    if (!aligned16(pool->k_pool) || !aligned16(pool->v_pool))
        return fail(MSGL_ERR_INVALID_ARG, "pool buffers must be 16-byte aligned");
    if (pool->head_dim != msgl::kHeadDim)
        return fail(MSGL_ERR_UNSUPPORTED, "head_dim %d is not supported (only 128)", pool->head_dim);
    if (pool->num_kv_heads <= 0) return fail(MSGL_ERR_INVALID_ARG, "num_kv_heads must be > 0");
    if (pool->num_kv_heads > 64) return fail(MSGL_ERR_UNSUPPORTED, "num_kv_heads > 64");
    const int l2 = log2_exact(pool->page_size);
    if (l2 < 0 || pool->page_size > 256)
        return fail(MSGL_ERR_UNSUPPORTED, "page_size %d is not a power of two in [1, 256]", pool->page_size);
    if (pool->num_slots < 0 || pool->num_slots % pool->page_size != 0)
        return fail(MSGL_ERR_INVALID_ARG, "num_slots must be a non-negative multiple of page_size");
    if (pool->num_slots / pool->page_size > INT32_MAX)
        return fail(MSGL_ERR_UNSUPPORTED, "more than 2^31-1 pages");
    view.k = static_cast<const __nv_bfloat16 *>(pool->k_pool);
    view.v = static_cast<const __nv_bfloat16 *>(pool->v_pool);
    view.num_slots = pool->num_slots;
    view.num_pages = (int32_t)(pool->num_slots / pool->page_size);
    view.log2_ps = l2;
    view.hkv = pool->num_kv_heads;
    return MSGL_OK;
}

msgl_status check_page_size(int32_t page_size, int32_t &log2_ps) {
    log2_ps = log2_exact(page_size);
    if (log2_ps < 0 || page_size > 256)
        return fail(MSGL_ERR_UNSUPPORTED, "page_size %d is not a power of two in [1, 256]", page_size);
    return MSGL_OK;
}

msgl_status check_pages(const msgl_page_table *pages, int32_t num_reqs, msgl::PageView &view) {
    if (!pages) return fail(MSGL_ERR_INVALID_ARG, "page table is NULL");
    if (num_reqs > 0 && !pages->page_ids) return fail(MSGL_ERR_INVALID_ARG, "page_ids is NULL");
    if (pages->width < 0 || pages->stride < pages->width)
        return fail(MSGL_ERR_INVALID_ARG, "page table needs 0 <= width <= stride");
    view.ids = pages->page_ids;
    view.stride = pages->stride;
    view.width = pages->width;
    return MSGL_OK;
}

msgl_status check_heads(int32_t hq, int32_t hkv) {
    if (hq <= 0 || hq % hkv != 0)
        return fail(MSGL_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of num_kv_heads %d", hq, hkv);
    if (hq / hkv > msgl::kMaxGroup)
        return fail(MSGL_ERR_UNSUPPORTED, "more than %d q heads per kv head", msgl::kMaxGroup);
    return MSGL_OK;
}

msgl_status check_scale(float scale) {
    if (!(scale > 0.f) || !isfinite(scale)) return fail(MSGL_ERR_INVALID_ARG, "scale must be finite and > 0");
    return MSGL_OK;
}

// int32 entries in device memory: `rows` rows of `width`, `pitch` apart.
struct Span {
    const int32_t *at;
    int64_t rows, width, pitch;
    const char *name;
};

Span flat(const int32_t *at, int64_t n, const char *name) { return Span{at, 1, n, n, name}; }

// Do two arrays have an entry in common?  Exact, so that two tables may be columns of one allocation.
bool overlap(const Span &a, const Span &b) {
    if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const int64_t size = sizeof(int32_t), a0 = (int64_t)(uintptr_t)a.at, b0 = (int64_t)(uintptr_t)b.at;
    if (a0 + ((a.rows - 1) * a.pitch + a.width) * size <= b0 || b0 + ((b.rows - 1) * b.pitch + b.width) * size <= a0)
        return false;
    if (b.rows > a.rows) return overlap(b, a);
    if (a.pitch == b.pitch) {
        // rows i of a and j of b meet where d - a.width < (i - j) pitch < d + b.width, d their bases' distance: the
        // first such i - j says it for all (columns of one projection of 8000 tokens: the loop below takes 30 us)
        const int64_t pitch = a.pitch * size, over = b0 - a0 - a.width * size;
        int64_t steps = over >= 0 ? over / pitch + 1 : -((-over - 1) / pitch);
        if (steps < 1 - b.rows) steps = 1 - b.rows;
        return steps < a.rows && steps * pitch < b0 - a0 + b.width * size;
    }
    // the last row of a that begins in front of the end of b's row r is the only one that can reach it
    for (int64_t r = 0; r < b.rows; ++r) {
        const int64_t from = b0 + r * b.pitch * size, to = from + b.width * size;
        if (to <= a0) continue;
        const int64_t row = a.rows == 1 ? 0 : (to - 1 - a0) / (a.pitch * size);
        const int64_t last = row < a.rows ? row : a.rows - 1;
        if (a0 + (last * a.pitch + a.width) * size > from) return true;
    }
    return false;
}

// Do n rows, `stride` elements apart, reach further than any memory (so that offsets stay within 64 bits)?
bool too_far(int64_t n, int64_t stride) { return stride > (1ll << 50) / (n > 0 ? n : 1); }

// A byte array as the 32-bit words that it touches.
Span bytes_span(const uint8_t *at, int64_t n, const char *name) {
    const uintptr_t from = (uintptr_t)at & ~(uintptr_t)3;
    return flat(reinterpret_cast<const int32_t *>(from), ((int64_t)((uintptr_t)at - from) + n + 3) / 4, name);
}

// No output over an input or another output.
msgl_status check_overlaps(const Span *outs, int n_outs, const Span *ins, int n_ins) {
    for (int i = 0; i < n_outs; ++i) {
        for (int j = 0; j < n_ins; ++j)
            if (overlap(outs[i], ins[j])) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[j].name, outs[i].name);
    }
    return MSGL_OK;
}

msgl_status check_page_count(int64_t num_slots, int32_t page_size, int32_t &log2_ps, int32_t &num_pages) {
    msgl_status s = check_page_size(page_size, log2_ps);
    if (s) return s;
    if (num_slots < 0 || num_slots % page_size != 0)
        return fail(MSGL_ERR_INVALID_ARG, "num_slots must be a non-negative multiple of page_size");
    if (num_slots / page_size > INT32_MAX) return fail(MSGL_ERR_UNSUPPORTED, "more than 2^31-1 pages");
    num_pages = (int32_t)(num_slots / page_size);
    return MSGL_OK;
}

msgl_status check_req_table(const int32_t *table, int32_t rows, int32_t stride, int32_t width) {
    if (rows < 0) return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (width < 0 || stride < width) return fail(MSGL_ERR_INVALID_ARG, "req_table needs 0 <= table_width <= table_stride");
    if (rows > 0 && width > 0 && !table) return fail(MSGL_ERR_INVALID_ARG, "req_table is NULL");
    return MSGL_OK;
}

msgl_status check_map_workspace(const void *workspace, size_t bytes, int32_t num_pages) {
    const size_t need = msgl::page_map_workspace_bytes(num_pages);
    if (need && (!workspace || bytes < need))
        return fail(MSGL_ERR_WORKSPACE, "needs %zu workspace bytes, got %zu", need, workspace ? bytes : (size_t)0);
    if ((uintptr_t)workspace % 256) return fail(MSGL_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return MSGL_OK;
}

// The part of a page-map workspace that a call writes.
Span map_span(void *workspace, int32_t num_pages) {
    return flat(static_cast<const int32_t *>(workspace), (int64_t)(msgl::page_map_workspace_bytes(num_pages) / 4), "workspace");
}

// The arguments that msgl_free_pages and msgl_compact_pages share.
msgl_status prepare_page_map(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                             int32_t table_stride, int32_t table_width, const int32_t *req_rows, const int32_t *lens,
                             int32_t num_reqs, const uint8_t *held, uint32_t *status, msgl::PageMapArgs &a) {
    msgl_status s = check_page_count(num_slots, page_size, a.log2_ps, a.num_pages);
    if (s) return s;
    if ((s = check_req_table(req_table, num_rows, table_stride, table_width))) return s;
    if (num_reqs < 0) return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_reqs > 0 && !lens) return fail(MSGL_ERR_INVALID_ARG, "lens is NULL");
    if (num_reqs > 1 << 24) return fail(MSGL_ERR_UNSUPPORTED, "more than 2^24 requests");
    if (table_width > msgl::kMaxStepItems)
        return fail(MSGL_ERR_UNSUPPORTED, "more than %lld columns", (long long)msgl::kMaxStepItems);
    a.table = req_table;
    a.req_rows = req_rows;
    a.lens = lens;
    a.held = held;
    a.num_rows = num_rows;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.num_reqs = num_reqs;
    a.status = status;
    return MSGL_OK;
}

}  // namespace

namespace msgl {
// Lets other translation units of the library set this thread's error text.
void set_last_error(const char *msg) { snprintf(g_last_error, sizeof g_last_error, "%s", msg); }

int sm_count() {
    static int cached[64];   // per device; racing first calls store the same value
    int dev = 0;
    cudaGetDevice(&dev);
    int sms = (dev >= 0 && dev < 64) ? cached[dev] : 0;
    if (sms == 0) {
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (sms <= 0) sms = 1;
        if (dev >= 0 && dev < 64) cached[dev] = sms;
    }
    return sms;
}
}  // namespace msgl

// Validates a decode call and fills its kernel arguments (a.num_reqs = 0: nothing to launch).
static msgl_status prepare_decode(const msgl_kv_pool *pool, const msgl_page_table *pages, const void *q,
                                  int32_t num_q_heads, const void *k_new, const void *v_new,
                                  const int32_t *new_loc, const int32_t *seq_lens, int32_t num_reqs,
                                  int32_t max_seq_len, float scale, void *o, float *lse, void *workspace,
                                  size_t workspace_bytes, uint32_t *status, msgl::DecodeArgs &a,
                                  msgl::DecodePlan &plan) {
    msgl::PoolView pv;
    msgl::PageView pg;
    msgl_status s = check_pool(pool, pv);
    if (s) return s;
    if ((s = check_heads(num_q_heads, pool->num_kv_heads))) return s;
    if ((s = check_scale(scale))) return s;
    if (num_reqs < 0) return fail(MSGL_ERR_INVALID_ARG, "num_reqs < 0");
    a = msgl::DecodeArgs{};
    a.num_reqs = num_reqs;
    if (num_reqs == 0) return MSGL_OK;
    if ((s = check_pages(pages, num_reqs, pg))) return s;
    if (max_seq_len <= 0) return fail(MSGL_ERR_INVALID_ARG, "max_seq_len must be > 0");
    if (!q || !seq_lens || !o || !lse) return fail(MSGL_ERR_INVALID_ARG, "q, seq_lens, o and lse must be non-NULL");
    if (!aligned16(q) || !aligned16(o)) return fail(MSGL_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
    plan = msgl::plan_decode(num_reqs, num_q_heads, pool->num_kv_heads, max_seq_len);
    if (!workspace || workspace_bytes < plan.workspace)
        return fail(MSGL_ERR_WORKSPACE, "decode needs %zu workspace bytes, got %zu", plan.workspace,
                    workspace ? workspace_bytes : (size_t)0);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(MSGL_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    a.pool = pv;
    a.pages = pg;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.seq_lens = seq_lens;
    a.hq = num_q_heads;
    a.max_seq_len = max_seq_len;
    a.scale = scale;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.part_o = static_cast<float *>(workspace);
    a.part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.o_bytes);
    a.status = status;
    a.k_new = static_cast<const __nv_bfloat16 *>(k_new);
    a.v_new = static_cast<const __nv_bfloat16 *>(v_new);
    a.new_loc = new_loc;
    return MSGL_OK;
}

static msgl_status decode_impl(const msgl_kv_pool *pool, const msgl_page_table *pages, const void *q,
                               int32_t num_q_heads, const void *k_new, const void *v_new,
                               const int32_t *new_loc, const int32_t *seq_lens, int32_t num_reqs,
                               int32_t max_seq_len, float scale, void *o, float *lse, void *workspace,
                               size_t workspace_bytes, uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    msgl::DecodeArgs a;
    msgl::DecodePlan plan{};
    msgl_status s = prepare_decode(pool, pages, q, num_q_heads, k_new, v_new, new_loc, seq_lens, num_reqs,
                                   max_seq_len, scale, o, lse, workspace, workspace_bytes, status, a, plan);
    if (s || num_reqs == 0) return s;
    cudaError_t e = msgl::launch_decode(a, plan, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "decode launch");
}

// Validates an extend call and fills its kernel arguments (a.num_reqs = 0: nothing to launch).
static msgl_status prepare_extend(const msgl_kv_pool *pool, const msgl_page_table *pages, const void *q,
                                  int32_t num_q_heads, const int32_t *prefix_lens, const int32_t *ext_lens,
                                  const int32_t *cu_ext, const int32_t *positions, int32_t num_reqs,
                                  int32_t total_tokens, int32_t max_ext_len, int32_t max_seq_len, float scale,
                                  void *o, float *lse, void *workspace, size_t workspace_bytes,
                                  uint32_t *status, msgl::ExtendArgs &a) {
    msgl::PoolView pv;
    msgl::PageView pg;
    msgl_status s = check_pool(pool, pv);
    if (s) return s;
    if ((s = check_heads(num_q_heads, pool->num_kv_heads))) return s;
    if ((s = check_scale(scale))) return s;
    if (num_reqs < 0 || total_tokens < 0 || max_ext_len < 0 || max_seq_len < 0)
        return fail(MSGL_ERR_INVALID_ARG, "negative size");
    a = msgl::ExtendArgs{};
    if (num_reqs == 0 || total_tokens == 0) return MSGL_OK;
    if ((s = check_pages(pages, num_reqs, pg))) return s;
    if (max_ext_len == 0 || max_seq_len < max_ext_len)
        return fail(MSGL_ERR_INVALID_ARG, "need 0 < max_ext_len <= max_seq_len");
    if (!q || !prefix_lens || !ext_lens || !cu_ext || !o || !lse)
        return fail(MSGL_ERR_INVALID_ARG, "q, prefix_lens, ext_lens, cu_ext, o and lse must be non-NULL");
    if (!aligned16(q) || !aligned16(o)) return fail(MSGL_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
    const size_t need = msgl::extend_workspace_bytes(num_reqs, total_tokens, num_q_heads,
                                                     pool->num_kv_heads, max_seq_len);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(MSGL_ERR_WORKSPACE, "extend needs %zu workspace bytes", need);
    a.pool = pv;
    a.pages = pg;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.prefix_lens = prefix_lens;
    a.ext_lens = ext_lens;
    a.cu_ext = cu_ext;
    a.positions = positions;
    a.num_reqs = num_reqs;
    a.total_tokens = total_tokens;
    a.hq = num_q_heads;
    a.max_ext_len = max_ext_len;
    a.max_seq_len = max_seq_len;
    a.scale = scale;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.workspace = workspace;
    a.status = status;
    return MSGL_OK;
}

extern "C" {

int32_t msgl_abi_version(void) { return MSGL_ABI_VERSION; }

const char *msgl_last_error(void) { return g_last_error; }

const char *msgl_status_string(msgl_status s) {
    switch (s) {
        case MSGL_OK: return "ok";
        case MSGL_ERR_INVALID_ARG: return "invalid argument";
        case MSGL_ERR_UNSUPPORTED: return "unsupported argument";
        case MSGL_ERR_CUDA: return "CUDA error";
        case MSGL_ERR_OUT_OF_RANGE: return "device index out of range";
        case MSGL_ERR_TIMEOUT: return "in-kernel wait timed out";
        case MSGL_ERR_WORKSPACE: return "workspace missing or too small";
    }
    return "unknown status";
}

msgl_status msgl_store_kv(const msgl_kv_pool *pool, const void *k, const void *v,
                          const int32_t *out_loc, int32_t n_tokens, uint32_t *status,
                          msgl_stream_t stream) {
    g_last_error[0] = 0;
    msgl::PoolView pv;
    msgl_status s = check_pool(pool, pv);
    if (s) return s;
    if (n_tokens < 0) return fail(MSGL_ERR_INVALID_ARG, "n_tokens < 0");
    if (n_tokens == 0) return MSGL_OK;
    if (!k || !v || !out_loc) return fail(MSGL_ERR_INVALID_ARG, "k, v and out_loc must be non-NULL");
    if (!aligned16(k) || !aligned16(v)) return fail(MSGL_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    cudaError_t e = msgl::launch_store_kv(pv, static_cast<__nv_bfloat16 *>(pool->k_pool),
                                          static_cast<__nv_bfloat16 *>(pool->v_pool),
                                          static_cast<const __nv_bfloat16 *>(k),
                                          static_cast<const __nv_bfloat16 *>(v), out_loc, n_tokens,
                                          status, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "store_kv launch");
}

size_t msgl_decode_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t max_seq_len) {
    if (num_reqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim != msgl::kHeadDim ||
        max_seq_len <= 0)
        return 0;
    return msgl::plan_decode(num_reqs, num_q_heads, num_kv_heads, max_seq_len).workspace;
}

msgl_status msgl_attn_decode(const msgl_kv_pool *pool, const msgl_page_table *pages,
                             const void *q, int32_t num_q_heads, const int32_t *seq_lens,
                             int32_t num_reqs, int32_t max_seq_len, float scale, void *o,
                             float *lse, void *workspace, size_t workspace_bytes,
                             uint32_t *status, msgl_stream_t stream) {
    return decode_impl(pool, pages, q, num_q_heads, nullptr, nullptr, nullptr, seq_lens, num_reqs,
                       max_seq_len, scale, o, lse, workspace, workspace_bytes, status, stream);
}

msgl_status msgl_attn_decode_append(const msgl_kv_pool *pool, const msgl_page_table *pages,
                                    const void *q, int32_t num_q_heads, const void *k_new,
                                    const void *v_new, const int32_t *new_loc,
                                    const int32_t *seq_lens, int32_t num_reqs, int32_t max_seq_len,
                                    float scale, void *o, float *lse, void *workspace,
                                    size_t workspace_bytes, uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (num_reqs > 0) {
        if (!k_new || !v_new || !new_loc)
            return fail(MSGL_ERR_INVALID_ARG, "k_new, v_new and new_loc must be non-NULL");
        if (!aligned16(k_new) || !aligned16(v_new))
            return fail(MSGL_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    }
    return decode_impl(pool, pages, q, num_q_heads, k_new, v_new, new_loc, seq_lens, num_reqs,
                       max_seq_len, scale, o, lse, workspace, workspace_bytes, status, stream);
}

size_t msgl_extend_workspace_size(int32_t num_reqs, int32_t total_tokens, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len) {
    if (num_reqs <= 0 || total_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        head_dim != msgl::kHeadDim)
        return 0;
    return msgl::extend_workspace_bytes(num_reqs, total_tokens, num_q_heads, num_kv_heads, max_seq_len);
}

msgl_status msgl_attn_extend(const msgl_kv_pool *pool, const msgl_page_table *pages,
                             const void *q, int32_t num_q_heads, const int32_t *prefix_lens,
                             const int32_t *ext_lens, const int32_t *cu_ext,
                             const int32_t *positions, int32_t num_reqs, int32_t total_tokens,
                             int32_t max_ext_len, int32_t max_seq_len, float scale, void *o,
                             float *lse, void *workspace, size_t workspace_bytes,
                             uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    msgl::ExtendArgs a;
    msgl_status s = prepare_extend(pool, pages, q, num_q_heads, prefix_lens, ext_lens, cu_ext, positions,
                                   num_reqs, total_tokens, max_ext_len, max_seq_len, scale, o, lse, workspace,
                                   workspace_bytes, status, a);
    if (s || a.num_reqs == 0) return s;
    cudaError_t e = msgl::launch_extend(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "extend launch");
}

msgl_status msgl_attn_mixed(const msgl_kv_pool *pool, const msgl_extend_batch *ext, const msgl_decode_batch *dec,
                            int32_t num_q_heads, float scale, void *workspace, size_t workspace_bytes,
                            uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!ext || !dec) return fail(MSGL_ERR_INVALID_ARG, "ext and dec must be non-NULL");
    // the decode partials take the front of the workspace, the extend's share follows
    msgl::DecodeArgs da;
    msgl::DecodePlan plan{};
    msgl_status s = prepare_decode(pool, &dec->pages, dec->q, num_q_heads, nullptr, nullptr, nullptr,
                                   dec->seq_lens, dec->num_reqs, dec->max_seq_len, scale, dec->o, dec->lse,
                                   workspace, workspace_bytes, status, da, plan);
    if (s) return s;
    const size_t dec_bytes = dec->num_reqs > 0 ? (plan.workspace + 255) / 256 * 256 : 0;
    msgl::ExtendArgs ea;
    void *ext_ws = workspace && workspace_bytes > dec_bytes ? static_cast<char *>(workspace) + dec_bytes : nullptr;
    s = prepare_extend(pool, &ext->pages, ext->q, num_q_heads, ext->prefix_lens, ext->ext_lens, ext->cu_ext,
                       ext->positions, ext->num_reqs, ext->total_tokens, ext->max_ext_len, ext->max_seq_len,
                       scale, ext->o, ext->lse, ext_ws, ext_ws ? workspace_bytes - dec_bytes : 0, status, ea);
    if (s) return s;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (da.num_reqs > 0 && ea.num_reqs > 0) {
        // split first; the extend's CTAs fill SMs as the split's ranges finish; merge last
        e = msgl::launch_decode(da, plan, st, msgl::DecodePhase::kSplit);
        if (e == cudaSuccess) {
            ea.pdl = true;
            e = msgl::launch_extend(ea, st);
        }
        if (e == cudaSuccess) e = msgl::launch_decode(da, plan, st, msgl::DecodePhase::kMerge);
    } else if (da.num_reqs > 0) {
        e = msgl::launch_decode(da, plan, st);
    } else if (ea.num_reqs > 0) {
        e = msgl::launch_extend(ea, st);
    }
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "mixed step launch");
}

msgl_status msgl_step_tables(int64_t num_slots, int32_t page_size, int32_t *req_table, int32_t num_rows,
                             int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                             const int32_t *cached_lens, const int32_t *new_lens, int32_t num_reqs,
                             const int32_t *free_pages, int32_t num_free, const msgl_step_out *out,
                             uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!out) return fail(MSGL_ERR_INVALID_ARG, "out is NULL");
    msgl::StepTablesArgs a{};
    msgl_status s = check_page_size(page_size, a.log2_ps);
    if (s) return s;
    if (num_slots < 0 || num_slots % page_size != 0)
        return fail(MSGL_ERR_INVALID_ARG, "num_slots must be a non-negative multiple of page_size");
    if (num_slots > (int64_t)INT32_MAX + 1)
        return fail(MSGL_ERR_UNSUPPORTED, "out_loc is int32: num_slots may not pass 2^31");
    if (num_reqs < 0 || num_free < 0 || num_rows < 0 || out->total_tokens < 0)
        return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_reqs == INT32_MAX) return fail(MSGL_ERR_UNSUPPORTED, "num_reqs + 1 passes int32");
    if (table_width < 0 || table_stride < table_width)
        return fail(MSGL_ERR_INVALID_ARG, "req_table needs 0 <= table_width <= table_stride");
    if (out->width < 0 || out->stride < out->width)
        return fail(MSGL_ERR_INVALID_ARG, "out needs 0 <= width <= stride");
    if (!out->cu_ext || !out->pages_taken)
        return fail(MSGL_ERR_INVALID_ARG, "out->cu_ext and out->pages_taken must be non-NULL");
    if (out->total_tokens > 0 && (!out->positions || !out->out_loc))
        return fail(MSGL_ERR_INVALID_ARG, "out->positions and out->out_loc must be non-NULL");
    if (num_reqs > 0 && (!cached_lens || !out->seq_lens))
        return fail(MSGL_ERR_INVALID_ARG, "cached_lens and out->seq_lens must be non-NULL");
    a.max_pages = table_width < out->width ? table_width : out->width;
    if (num_reqs > 0 && num_rows > 0 && a.max_pages > 0 && (!req_table || !out->page_ids))
        return fail(MSGL_ERR_INVALID_ARG, "req_table and out->page_ids must be non-NULL");
    if (num_free > 0 && !free_pages) return fail(MSGL_ERR_INVALID_ARG, "free_pages is NULL");
    if (out->total_tokens > msgl::kMaxStepItems || a.max_pages > msgl::kMaxStepItems)
        return fail(MSGL_ERR_UNSUPPORTED, "more than %lld tokens or columns", (long long)msgl::kMaxStepItems);
    // Every block takes the sums over the lengths before its own while others write, so an output over an
    // input would race with them.
    const Span outs[] = {{out->page_ids, num_reqs, a.max_pages, out->stride, "out->page_ids"},
                         {req_table, num_rows, a.max_pages, table_stride, "req_table"},
                         flat(out->seq_lens, num_reqs, "out->seq_lens"),
                         flat(out->cu_ext, (int64_t)num_reqs + 1, "out->cu_ext"),
                         flat(out->positions, out->total_tokens, "out->positions"),
                         flat(out->out_loc, out->total_tokens, "out->out_loc"),
                         flat(out->pages_taken, 1, "out->pages_taken")};
    const Span ins[] = {flat(cached_lens, num_reqs, "cached_lens"), flat(new_lens, num_reqs, "new_lens"),
                        flat(req_rows, num_reqs, "req_rows"), flat(free_pages, num_free, "free_pages")};
    const bool in_place = out->page_ids == req_table && out->stride == table_stride && !req_rows;
    constexpr int kOuts = sizeof outs / sizeof outs[0];
    for (int i = 0; i < kOuts; ++i) {
        for (const Span &in : ins)
            if (overlap(outs[i], in)) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, in.name);
        for (int j = 0; j < i; ++j)
            if (!(j == 0 && i == 1 && in_place) && overlap(outs[i], outs[j]))
                return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[j].name, outs[i].name);
    }
    a.req_table = req_table;
    a.req_rows = req_rows;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.free_pages = free_pages;
    a.num_rows = num_rows;
    a.table_stride = table_stride;
    a.num_reqs = num_reqs;
    a.num_free = num_free;
    a.num_pages = (int32_t)(num_slots / page_size < INT32_MAX ? num_slots / page_size : INT32_MAX);
    a.page_ids = out->page_ids;
    a.seq_lens = out->seq_lens;
    a.cu_ext = out->cu_ext;
    a.positions = out->positions;
    a.out_loc = out->out_loc;
    a.pages_taken = out->pages_taken;
    a.stride = out->stride;
    a.total_tokens = out->total_tokens;
    a.status = status;
    cudaError_t e = msgl::launch_step_tables(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "step_tables launch");
}

msgl_status msgl_shared_prefixes(const msgl_page_table *pages, const int32_t *seq_lens, int32_t num_reqs,
                                 int32_t page_size, int32_t max_seq_len, int32_t min_shared,
                                 int32_t *group_start, int32_t *shared_lens, uint32_t *status,
                                 msgl_stream_t stream) {
    g_last_error[0] = 0;
    msgl::SharedPrefixesArgs a{};
    msgl_status s = check_page_size(page_size, a.log2_ps);
    if (s) return s;
    if (num_reqs < 0) return fail(MSGL_ERR_INVALID_ARG, "num_reqs < 0");
    if (num_reqs == 0) return MSGL_OK;
    if ((s = check_pages(pages, num_reqs, a.pages))) return s;
    if (max_seq_len <= 0) return fail(MSGL_ERR_INVALID_ARG, "max_seq_len must be > 0");
    if (max_seq_len > (1 << 30)) return fail(MSGL_ERR_UNSUPPORTED, "max_seq_len may not pass 2^30");
    if (min_shared <= 0) return fail(MSGL_ERR_INVALID_ARG, "min_shared must be > 0");
    if (!seq_lens || !group_start || !shared_lens)
        return fail(MSGL_ERR_INVALID_ARG, "seq_lens, group_start and shared_lens must be non-NULL");
    // (the common lengths travel in shared_lens while other blocks still read the inputs)
    const Span ins[] = {flat(seq_lens, num_reqs, "seq_lens"),
                        {a.pages.ids, num_reqs, a.pages.width, a.pages.stride, "page_ids"}};
    const Span outs[] = {flat(group_start, num_reqs, "group_start"), flat(shared_lens, num_reqs, "shared_lens")};
    for (const Span &out : outs)
        for (const Span &in : ins)
            if (overlap(out, in)) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
    if (overlap(outs[0], outs[1])) return fail(MSGL_ERR_INVALID_ARG, "group_start overlaps shared_lens");
    a.seq_lens = seq_lens;
    a.num_reqs = num_reqs;
    a.max_seq_len = max_seq_len;
    a.min_shared = min_shared;
    a.group_start = group_start;
    a.shared_lens = shared_lens;
    a.status = status;
    cudaError_t e = msgl::launch_shared_prefixes(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "shared_prefixes launch");
}

size_t msgl_decode_shared_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t max_seq_len) {
    if (num_reqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim != msgl::kHeadDim || max_seq_len <= 0)
        return 0;
    return msgl::decode_shared_workspace_bytes(num_reqs, num_q_heads, num_kv_heads);
}

msgl_status msgl_attn_decode_shared(const msgl_kv_pool *pool, const msgl_page_table *pages, const void *q,
                                    int32_t num_q_heads, const int32_t *group_start, const int32_t *shared_lens,
                                    const int32_t *seq_lens, int32_t num_reqs, int32_t max_seq_len, int32_t sharing,
                                    float scale, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                    uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (sharing < MSGL_SHARE_AUTO || sharing > MSGL_SHARE_NEVER)
        return fail(MSGL_ERR_INVALID_ARG, "sharing %d is not one of MSGL_SHARE_*", sharing);
    if (num_reqs > 0 && (!group_start || !shared_lens))
        return fail(MSGL_ERR_INVALID_ARG, "group_start and shared_lens must be non-NULL");
    if (num_reqs > 65535) return fail(MSGL_ERR_UNSUPPORTED, "more than 65535 requests");
    if (max_seq_len > (1 << 30)) return fail(MSGL_ERR_UNSUPPORTED, "max_seq_len may not pass 2^30");
    msgl::DecodeSharedArgs a;
    msgl::DecodePlan plan{};
    msgl_status s = prepare_decode(pool, pages, q, num_q_heads, nullptr, nullptr, nullptr, seq_lens, num_reqs,
                                   max_seq_len, scale, o, lse, workspace, workspace_bytes, status, a.dec, plan);
    if (num_reqs > 0 && (!s || s == MSGL_ERR_WORKSPACE)) {
        // (a decode's workspace is part of it)
        const size_t need = msgl::decode_shared_workspace_bytes(num_reqs, num_q_heads, pool->num_kv_heads);
        if (!workspace || workspace_bytes < need)
            return fail(MSGL_ERR_WORKSPACE, "decode_shared needs %zu workspace bytes, got %zu", need,
                        workspace ? workspace_bytes : (size_t)0);
    }
    if (s || num_reqs == 0) return s;
    a.dec.group_start = group_start;
    a.dec.shared_lens = shared_lens;
    a.sharing = sharing;
    a.workspace = workspace;
    cudaError_t e = msgl::launch_decode_shared(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "decode_shared launch");
}

msgl_status msgl_rope_store_kv(const msgl_kv_pool *pool, const msgl_new_tokens *tokens, const msgl_rope *rope,
                               const void *q_norm, const void *k_norm, float eps, uint32_t *status,
                               msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!tokens || !rope) return fail(MSGL_ERR_INVALID_ARG, "tokens and rope must be non-NULL");
    const msgl_new_tokens &n = *tokens;
    msgl::RopeStoreArgs a{};
    msgl_status s = check_pool(pool, a.pool);
    if (s) return s;
    if ((s = check_heads(n.num_q_heads, a.pool.hkv))) return s;
    if (!rope->turns) return fail(MSGL_ERR_INVALID_ARG, "rope->turns is NULL");
    if (rope->num_pairs <= 0 || rope->num_pairs > msgl::kHeadDim / 2)
        return fail(MSGL_ERR_INVALID_ARG, "num_pairs %d is outside [1, %d]", rope->num_pairs, msgl::kHeadDim / 2);
    if (rope->num_pairs % 8) return fail(MSGL_ERR_UNSUPPORTED, "num_pairs %d is not a multiple of 8", rope->num_pairs);
    if (rope->num_axes < 1 || rope->num_axes > 4)
        return fail(MSGL_ERR_INVALID_ARG, "num_axes %d is outside [1, 4]", rope->num_axes);
    if (!isfinite(rope->factor)) return fail(MSGL_ERR_INVALID_ARG, "factor must be finite");
    if ((q_norm || k_norm) && !(eps >= 0.f && isfinite(eps)))
        return fail(MSGL_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (n.n_tokens < 0) return fail(MSGL_ERR_INVALID_ARG, "n_tokens < 0");
    for (int j = 0; j < rope->num_pairs; ++j) {
        const uint32_t axis = rope->axes ? rope->axes[j] : 0;
        if (axis >= (uint32_t)rope->num_axes)
            return fail(MSGL_ERR_INVALID_ARG, "axes[%d] = %u but num_axes = %d", j, axis, rope->num_axes);
        a.axis_bits[j / 16] |= axis << (2 * (j % 16));
    }
    if (n.n_tokens == 0) return MSGL_OK;
    if (!n.q || !n.k || !n.v || !n.q_out || !n.positions || !n.out_loc)
        return fail(MSGL_ERR_INVALID_ARG, "q, k, v, q_out, positions and out_loc must be non-NULL");
    if (!aligned16(n.q) || !aligned16(n.k) || !aligned16(n.v) || !aligned16(n.q_out) || !aligned16(q_norm) ||
        !aligned16(k_norm))
        return fail(MSGL_ERR_INVALID_ARG, "q, k, v, q_out and the norms must be 16-byte aligned");
    if ((uintptr_t)rope->turns % 8) return fail(MSGL_ERR_INVALID_ARG, "rope->turns must be 8-byte aligned");
    const int64_t q_row = (int64_t)n.num_q_heads * msgl::kHeadDim, kv_row = (int64_t)a.pool.hkv * msgl::kHeadDim;
    const struct {
        int64_t stride, row;
        const char *name;
    } strides[] = {{n.q_stride, q_row, "q_stride"}, {n.k_stride, kv_row, "k_stride"}, {n.v_stride, kv_row, "v_stride"},
                   {n.out_stride, q_row, "out_stride"}};
    for (const auto &x : strides)
        if (x.stride % 8 || x.stride < x.row || too_far(n.n_tokens, x.stride))
            return fail(MSGL_ERR_INVALID_ARG, "%s %lld is not a multiple of 8 from %lld on that memory can hold", x.name,
                        (long long)x.stride, (long long)x.row);
    if (rope->num_axes > 1 && n.axis_stride != 0 && (n.axis_stride < n.n_tokens || too_far(rope->num_axes, n.axis_stride)))
        return fail(MSGL_ERR_INVALID_ARG, "axis_stride %lld is neither 0 nor n_tokens %d or more (or past all memory)",
                    (long long)n.axis_stride, n.n_tokens);
    const bool one_axis = rope->num_axes == 1 || n.axis_stride == 0;
    // (two bf16 an entry; tokens are turned by blocks of their own, in any order)
    auto span = [&](const void *p, int64_t row, int64_t stride, const char *name) {
        return Span{static_cast<const int32_t *>(p), n.n_tokens, row / 2, stride / 2, name};
    };
    const Span out = span(n.q_out, q_row, n.out_stride, "q_out");
    const Span ins[] = {span(n.q, q_row, n.q_stride, "q"), span(n.k, kv_row, n.k_stride, "k"),
                        span(n.v, kv_row, n.v_stride, "v"),
                        flat(static_cast<const int32_t *>(q_norm), msgl::kHeadDim / 2, "q_norm"),
                        flat(static_cast<const int32_t *>(k_norm), msgl::kHeadDim / 2, "k_norm"),
                        {n.positions, one_axis ? 1 : rope->num_axes, n.n_tokens, one_axis ? n.n_tokens : n.axis_stride, "positions"},
                        flat(n.out_loc, n.n_tokens, "out_loc"),
                        flat(reinterpret_cast<const int32_t *>(rope->turns), 2 * rope->num_pairs, "rope->turns")};
    const int64_t pool_words = pool->num_slots * (kv_row / 2);
    const Span pools[] = {flat(static_cast<const int32_t *>(pool->k_pool), pool_words, "the K pool"),
                          flat(static_cast<const int32_t *>(pool->v_pool), pool_words, "the V pool")};
    const bool in_place = n.q_out == n.q && n.out_stride == n.q_stride;
    for (const Span &in : ins) {
        if (&in == &ins[0] && in_place) continue;   // (q alone: k or v may begin where it does and be turned while they are read)
        if (overlap(out, in)) return fail(MSGL_ERR_INVALID_ARG, "q_out overlaps %s", in.name);
    }
    for (const Span &rows : pools)
        if (overlap(out, rows)) return fail(MSGL_ERR_INVALID_ARG, "q_out overlaps %s", rows.name);
    // (the pools are outputs too)
    if ((s = check_overlaps(pools, 2, ins, 8))) return s;
    a.k_pool = static_cast<__nv_bfloat16 *>(pool->k_pool);
    a.v_pool = static_cast<__nv_bfloat16 *>(pool->v_pool);
    a.q = static_cast<const __nv_bfloat16 *>(n.q);
    a.k = static_cast<const __nv_bfloat16 *>(n.k);
    a.v = static_cast<const __nv_bfloat16 *>(n.v);
    a.q_norm = static_cast<const __nv_bfloat16 *>(q_norm);
    a.k_norm = static_cast<const __nv_bfloat16 *>(k_norm);
    a.q_out = static_cast<__nv_bfloat16 *>(n.q_out);
    a.q_stride = n.q_stride;
    a.k_stride = n.k_stride;
    a.v_stride = n.v_stride;
    a.out_stride = n.out_stride;
    a.turns = rope->turns;
    a.positions = n.positions;
    a.out_loc = n.out_loc;
    a.axis_stride = one_axis ? 0 : n.axis_stride;
    a.pairs = rope->num_pairs;
    a.adjacent = rope->adjacent != 0;
    a.n_tokens = n.n_tokens;
    a.hq = n.num_q_heads;
    a.factor = rope->factor;
    a.eps = eps;
    a.status = status;
    cudaError_t e = msgl::launch_rope_store(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "rope_store launch");
}

msgl_status msgl_verify_drafts(const msgl_draft_batch *batch, uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!batch) return fail(MSGL_ERR_INVALID_ARG, "batch is NULL");
    const msgl_draft_batch &d = *batch;
    if (d.num_reqs < 0 || d.total_tokens < 0) return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (d.vocab <= 0) return fail(MSGL_ERR_INVALID_ARG, "vocab must be > 0");
    if (d.vocab > (1 << 30)) return fail(MSGL_ERR_UNSUPPORTED, "vocab may not pass 2^30");
    if (d.num_reqs > msgl::kMaxDraftReqs) return fail(MSGL_ERR_UNSUPPORTED, "more than %d requests", msgl::kMaxDraftReqs);
    if (d.num_reqs == 0) return MSGL_OK;
    if (!d.cu_ext || !d.sample_u || !d.accepted || !d.kv_lens)
        return fail(MSGL_ERR_INVALID_ARG, "cu_ext, sample_u, accepted and kv_lens must be non-NULL");
    if (d.total_tokens > 0 && (!d.target || !d.tokens || !d.accept_u || !d.out_tokens))
        return fail(MSGL_ERR_INVALID_ARG, "target, tokens, accept_u and out_tokens must be non-NULL");
    if (d.target_stride < d.vocab || too_far(d.total_tokens, d.target_stride))
        return fail(MSGL_ERR_INVALID_ARG, "target_stride %lld is below vocab %d (or past all memory)",
                    (long long)d.target_stride, d.vocab);
    if (d.draft && (d.draft_stride < d.vocab || too_far(d.total_tokens, d.draft_stride)))
        return fail(MSGL_ERR_INVALID_ARG, "draft_stride %lld is below vocab %d (or past all memory)",
                    (long long)d.draft_stride, d.vocab);
    const uintptr_t size = d.is_bf16 ? 2 : 4;
    if ((uintptr_t)d.target % size || (uintptr_t)d.draft % size)
        return fail(MSGL_ERR_INVALID_ARG, "target and draft must be aligned to their type");
    // (every block of a request reads its inputs while another writes its outputs)
    const Span outs[] = {flat(d.accepted, d.num_reqs, "accepted"), flat(d.kv_lens, d.num_reqs, "kv_lens"),
                         flat(d.out_tokens, d.total_tokens, "out_tokens")};
    auto probs = [&](const void *p, int64_t stride, const char *name) {
        const int64_t bytes = p && d.total_tokens > 0 ? ((d.total_tokens - 1) * stride + d.vocab) * (int64_t)size : 0;
        const uintptr_t at = (uintptr_t)p & ~(uintptr_t)3;
        return flat(reinterpret_cast<const int32_t *>(at), ((int64_t)((uintptr_t)p - at) + bytes + 3) / 4, name);
    };
    const Span ins[] = {flat(d.tokens, d.total_tokens, "tokens"), flat(d.cu_ext, (int64_t)d.num_reqs + 1, "cu_ext"),
                        flat(reinterpret_cast<const int32_t *>(d.accept_u), d.total_tokens, "accept_u"),
                        flat(reinterpret_cast<const int32_t *>(d.sample_u), d.num_reqs, "sample_u"),
                        flat(d.cached_lens, d.num_reqs, "cached_lens"), probs(d.target, d.target_stride, "target"),
                        probs(d.draft, d.draft_stride, "draft")};
    for (int i = 0; i < 3; ++i) {
        for (const Span &in : ins) {
            if (&outs[i] == &outs[1] && &in == &ins[4] && d.kv_lens == d.cached_lens) continue;   // in place: one thread reads, then writes
            if (overlap(outs[i], in)) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, in.name);
        }
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return fail(MSGL_ERR_INVALID_ARG, "%s overlaps %s", outs[j].name, outs[i].name);
    }
    msgl::VerifyArgs a{};
    a.target = d.target;
    a.draft = d.draft;
    a.target_stride = d.target_stride;
    a.draft_stride = d.draft_stride;
    a.tokens = d.tokens;
    a.cu_ext = d.cu_ext;
    a.cached_lens = d.cached_lens;
    a.accept_u = d.accept_u;
    a.sample_u = d.sample_u;
    a.num_reqs = d.num_reqs;
    a.total_tokens = d.total_tokens;
    a.vocab = d.vocab;
    a.bf16 = d.is_bf16 != 0;
    a.accepted = d.accepted;
    a.out_tokens = d.out_tokens;
    a.kv_lens = d.kv_lens;
    a.status = status;
    cudaError_t e = msgl::launch_verify_drafts(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "verify_drafts launch");
}

msgl_status msgl_fork_requests(int64_t num_slots, int32_t page_size, int32_t *req_table, int32_t num_rows,
                               int32_t table_stride, int32_t table_width, const int32_t *parent_rows,
                               const int32_t *child_rows, const int32_t *lens, int32_t num_forks,
                               const int32_t *free_pages, int32_t num_free, const msgl_fork_out *out,
                               uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!out) return fail(MSGL_ERR_INVALID_ARG, "out is NULL");
    msgl::ForkArgs a{};
    msgl_status s = check_page_count(num_slots, page_size, a.log2_ps, a.num_pages);
    if (s) return s;
    if ((s = check_req_table(req_table, num_rows, table_stride, table_width))) return s;
    if (num_forks < 0 || num_free < 0) return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_forks == INT32_MAX) return fail(MSGL_ERR_UNSUPPORTED, "num_forks + 1 passes int32");
    if (table_width > msgl::kMaxStepItems)
        return fail(MSGL_ERR_UNSUPPORTED, "more than %lld columns", (long long)msgl::kMaxStepItems);
    if (!out->pages_taken) return fail(MSGL_ERR_INVALID_ARG, "out->pages_taken must be non-NULL");
    if (num_forks > 0 && (!parent_rows || !child_rows || !lens || !out->copy_src || !out->copy_dst || !out->copy_tokens))
        return fail(MSGL_ERR_INVALID_ARG, "parent_rows, child_rows, lens and the copies must be non-NULL");
    if (num_free > 0 && !free_pages) return fail(MSGL_ERR_INVALID_ARG, "free_pages is NULL");
    const Span outs[] = {{req_table, num_rows, table_width, table_stride, "req_table"},
                         flat(out->copy_src, num_forks, "out->copy_src"),
                         flat(out->copy_dst, num_forks, "out->copy_dst"),
                         flat(out->copy_tokens, num_forks, "out->copy_tokens"),
                         flat(out->pages_taken, 1, "out->pages_taken")};
    const Span ins[] = {flat(parent_rows, num_forks, "parent_rows"), flat(child_rows, num_forks, "child_rows"),
                        flat(lens, num_forks, "lens"), flat(free_pages, num_free, "free_pages")};
    if ((s = check_overlaps(outs, 5, ins, 4))) return s;
    a.req_table = req_table;
    a.parent_rows = parent_rows;
    a.child_rows = child_rows;
    a.lens = lens;
    a.free_pages = free_pages;
    a.num_rows = num_rows;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.num_forks = num_forks;
    a.num_free = num_free;
    a.copy_src = out->copy_src;
    a.copy_dst = out->copy_dst;
    a.copy_tokens = out->copy_tokens;
    a.pages_taken = out->pages_taken;
    a.status = status;
    cudaError_t e = msgl::launch_fork(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "fork_requests launch");
}

msgl_status msgl_copy_pages(const msgl_kv_pool *pools, int32_t num_pools, const int32_t *src, const int32_t *dst,
                            const int32_t *tokens, int32_t num_pairs, const int32_t *count, uint32_t *status,
                            msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (num_pools < 0 || num_pairs < 0) return fail(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_pools > 1 << 15) return fail(MSGL_ERR_UNSUPPORTED, "more than 2^15 pools");
    if (num_pools > 0 && !pools) return fail(MSGL_ERR_INVALID_ARG, "pools is NULL");
    msgl::PoolView view{};
    for (int i = 0; i < num_pools; ++i) {
        msgl_status s = check_pool(pools + i, view);
        if (s) return s;
        if (pools[i].num_slots != pools[0].num_slots || pools[i].page_size != pools[0].page_size ||
            pools[i].num_kv_heads != pools[0].num_kv_heads)
            return fail(MSGL_ERR_INVALID_ARG, "pool %d has another num_slots, page_size or num_kv_heads than pool 0", i);
    }
    if (num_pools == 0 || num_pairs == 0) return MSGL_OK;
    if (!src || !dst) return fail(MSGL_ERR_INVALID_ARG, "src and dst must be non-NULL");
    msgl::CopyPagesArgs a{};
    void *buffers[2 * msgl::kMaxCopyPools];
    a.src = src;
    a.dst = dst;
    a.tokens = tokens;
    a.count = count;
    a.row_vecs = view.hkv * msgl::kHeadDim * 2 / 16;
    a.page_size = pools[0].page_size;
    a.page_vecs = (int64_t)a.row_vecs * a.page_size;
    a.num_pages = view.num_pages;
    a.num_pairs = num_pairs;
    a.status = status;
    for (int i0 = 0; i0 < num_pools; i0 += msgl::kMaxCopyPools) {
        const int n = num_pools - i0 < msgl::kMaxCopyPools ? num_pools - i0 : msgl::kMaxCopyPools;
        for (int i = 0; i < n; ++i) {
            buffers[2 * i] = pools[i0 + i].k_pool;
            buffers[2 * i + 1] = pools[i0 + i].v_pool;
        }
        a.num_buffers = 2 * n;
        cudaError_t e = msgl::launch_copy_pages(a, buffers, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_fail(e, "copy_pages launch");
    }
    return MSGL_OK;
}

size_t msgl_page_map_workspace_size(int64_t num_slots, int32_t page_size) {
    if (page_size <= 0 || num_slots < 0 || num_slots / page_size > INT32_MAX) return 0;
    return msgl::page_map_workspace_bytes((int32_t)(num_slots / page_size));
}

msgl_status msgl_free_pages(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                            int32_t table_stride, int32_t table_width, const int32_t *req_rows, const int32_t *lens,
                            int32_t num_reqs, const uint8_t *held, int32_t *pages, int32_t *num_free,
                            void *workspace, size_t workspace_bytes, uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    msgl::PageMapArgs a{};
    msgl_status s = prepare_page_map(num_slots, page_size, req_table, num_rows, table_stride, table_width, req_rows, lens,
                                     num_reqs, held, status, a);
    if (s) return s;
    if (!num_free || (a.num_pages > 0 && !pages))
        return fail(MSGL_ERR_INVALID_ARG, "pages and num_free must be non-NULL");
    const Span outs[] = {flat(pages, a.num_pages, "pages"), flat(num_free, 1, "num_free"), map_span(workspace, a.num_pages)};
    const Span ins[] = {{req_table, num_rows, table_width, table_stride, "req_table"}, flat(req_rows, num_reqs, "req_rows"),
                        flat(lens, num_reqs, "lens"), bytes_span(held, a.num_pages, "held")};
    if ((s = check_overlaps(outs, 3, ins, 4))) return s;
    if ((s = check_map_workspace(workspace, workspace_bytes, a.num_pages))) return s;
    a.pages_out = pages;
    a.count_out = num_free;
    cudaError_t e = msgl::launch_free_pages(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "free_pages launch");
}

msgl_status msgl_compact_pages(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                               int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                               const int32_t *lens, int32_t num_reqs, const uint8_t *held,
                               const msgl_compact_out *out, void *workspace, size_t workspace_bytes,
                               uint32_t *status, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!out) return fail(MSGL_ERR_INVALID_ARG, "out is NULL");
    msgl::PageMapArgs a{};
    msgl_status s = prepare_page_map(num_slots, page_size, req_table, num_rows, table_stride, table_width, req_rows, lens,
                                     num_reqs, held, status, a);
    if (s) return s;
    if (!out->num_moves || !out->num_used || (a.num_pages > 0 && !out->remap) ||
        (a.num_pages > 1 && (!out->src || !out->dst)) || (num_rows > 0 && table_width > 0 && !out->page_ids))
        return fail(MSGL_ERR_INVALID_ARG, "out's arrays must be non-NULL");
    if (out->stride < table_width) return fail(MSGL_ERR_INVALID_ARG, "out needs stride >= table_width");
    const bool in_place = out->page_ids == req_table;
    if (in_place && out->stride != table_stride)
        return fail(MSGL_ERR_INVALID_ARG, "out->page_ids overlaps req_table at another stride");
    const Span outs[] = {flat(out->remap, a.num_pages, "out->remap"), flat(out->src, a.num_pages / 2, "out->src"),
                         flat(out->dst, a.num_pages / 2, "out->dst"), flat(out->num_moves, 1, "out->num_moves"),
                         flat(out->num_used, 1, "out->num_used"),
                         {out->page_ids, num_rows, table_width, out->stride, "out->page_ids"},
                         map_span(workspace, a.num_pages)};
    const Span ins[] = {flat(req_rows, num_reqs, "req_rows"), flat(lens, num_reqs, "lens"),
                        bytes_span(held, a.num_pages, "held"),
                        {in_place ? nullptr : req_table, num_rows, table_width, table_stride, "req_table"}};
    if ((s = check_overlaps(outs, 7, ins, 4))) return s;
    if ((s = check_map_workspace(workspace, workspace_bytes, a.num_pages))) return s;
    a.pages_out = out->remap;
    a.count_out = out->num_moves;
    a.used_out = out->num_used;
    a.src = out->src;
    a.dst = out->dst;
    a.table_out = out->page_ids;
    a.out_stride = out->stride;
    cudaError_t e = msgl::launch_compact_pages(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? MSGL_OK : cuda_fail(e, "compact_pages launch");
}

msgl_status msgl_read_status(const uint32_t *status, uint32_t *flags, msgl_stream_t stream) {
    g_last_error[0] = 0;
    if (!status) return fail(MSGL_ERR_INVALID_ARG, "status is NULL");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
    uint32_t h = 0;
    e = cudaMemcpy(&h, status, sizeof h, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "status copy");
    if (flags) *flags = h;
    if (h == 0) return MSGL_OK;
    if (h & MSGL_DEVERR_TIMEOUT) return MSGL_ERR_TIMEOUT;
    return MSGL_ERR_OUT_OF_RANGE;
}

}  // extern "C"
