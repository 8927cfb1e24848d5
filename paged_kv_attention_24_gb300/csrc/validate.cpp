// Host-side metadata checks (msgl_check_*_meta): the conditions the kernels
// check on the device, evaluated on host copies of the arrays so that a test
// or a debugging session learns which entry is wrong.  Nothing here touches
// the GPU.  What the metadata means: "不懂SGLang？从miniSGLang开始", §1.3
// item 3 (page table and positions locate each request's KV in the pool);
// "Mini-SGLang 实战指南", §6.1 (a chunk sits after its cached prefix) and
// §6.2 (the page is the pool's allocation unit).
#include <stdarg.h>
#include <stdio.h>

#include <exception>
#include <initializer_list>
#include <unordered_set>

#include "../../include/msgl_attn.h"

namespace msgl {
void set_last_error(const char *msg);
}

namespace {

msgl_status bad(msgl_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
msgl_status bad(msgl_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    msgl::set_last_error(buf);
    return s;
}

bool pow2(int32_t x) { return x > 0 && (x & (x - 1)) == 0; }

// Pages of keys 0..n_keys-1 of request b, which are row `row` of the table: index below width, id
// inside the pool.
msgl_status check_pages(int64_t num_pages, int32_t page_size, const int32_t *page_ids, int32_t stride,
                        int32_t width, int32_t b, int32_t row, int64_t n_keys, const char *who = "request") {
    const int64_t n_pages = (n_keys + page_size - 1) / page_size;
    if (n_pages > width)
        return bad(MSGL_ERR_OUT_OF_RANGE, "%s %d: %lld keys need %lld pages but the table width is %d", who, b,
                   (long long)n_keys, (long long)n_pages, width);
    for (int64_t p = 0; p < n_pages; ++p) {
        const int32_t id = page_ids[(int64_t)row * stride + p];
        if (id < 0 || id >= num_pages)
            return bad(MSGL_ERR_OUT_OF_RANGE, "%s %d: page_ids[%lld] = %d is outside [0, %lld)", who, b,
                       (long long)p, id, (long long)num_pages);
    }
    return MSGL_OK;
}

msgl_status check_pool_scalars(int64_t num_slots, int32_t page_size, const int32_t *page_ids, int32_t stride,
                               int32_t width) {
    if (num_slots < 0) return bad(MSGL_ERR_INVALID_ARG, "num_slots must be >= 0");
    if (!pow2(page_size) || page_size > 256)
        return bad(MSGL_ERR_INVALID_ARG, "page_size %d is not a power of two in [1, 256]", page_size);
    if (num_slots % page_size) return bad(MSGL_ERR_INVALID_ARG, "num_slots is not a multiple of page_size");
    if (width < 0 || stride < width) return bad(MSGL_ERR_INVALID_ARG, "page table needs 0 <= width <= stride");
    if (!page_ids && width > 0) return bad(MSGL_ERR_INVALID_ARG, "page_ids is NULL");
    return MSGL_OK;
}

// The sets of slots, rows and pages seen are the only thing here that can throw.
msgl_status no_memory() { return bad(MSGL_ERR_UNSUPPORTED, "out of host memory for the check"); }

}  // namespace

extern "C" {

msgl_status msgl_check_store_meta(int64_t num_slots, const int32_t *out_loc, int32_t n_tokens) try {
    msgl::set_last_error("");
    if (n_tokens < 0 || num_slots < 0) return bad(MSGL_ERR_INVALID_ARG, "n_tokens and num_slots must be >= 0");
    if (n_tokens > 0 && !out_loc) return bad(MSGL_ERR_INVALID_ARG, "out_loc is NULL");
    std::unordered_set<int32_t> seen;
    seen.reserve((size_t)n_tokens);
    for (int32_t t = 0; t < n_tokens; ++t) {
        const int32_t s = out_loc[t];
        if (s < 0 || s >= num_slots)
            return bad(MSGL_ERR_OUT_OF_RANGE, "out_loc[%d] = %d is outside [0, %lld)", t, s, (long long)num_slots);
        if (!seen.insert(s).second)
            return bad(MSGL_ERR_INVALID_ARG, "out_loc[%d] = %d names a slot an earlier row already writes", t, s);
    }
    return MSGL_OK;
} catch (const std::exception &) {
    return no_memory();
}

msgl_status msgl_check_extend_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids, int32_t stride,
                                   int32_t width, const int32_t *prefix_lens, const int32_t *ext_lens,
                                   const int32_t *cu_ext, const int32_t *positions, int32_t num_reqs,
                                   int32_t total_tokens, int32_t max_ext_len, int32_t max_seq_len) {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, page_ids, stride, width);
    if (rc) return rc;
    if (num_reqs < 0 || total_tokens < 0) return bad(MSGL_ERR_INVALID_ARG, "num_reqs and total_tokens must be >= 0");
    if (num_reqs > 0 && (!prefix_lens || !ext_lens || !cu_ext))
        return bad(MSGL_ERR_INVALID_ARG, "prefix_lens, ext_lens and cu_ext must be non-NULL");
    if (num_reqs == 0) {
        if (total_tokens != 0) return bad(MSGL_ERR_INVALID_ARG, "no requests but total_tokens = %d", total_tokens);
        return MSGL_OK;
    }
    if (cu_ext[0] != 0) return bad(MSGL_ERR_INVALID_ARG, "cu_ext[0] = %d, expected 0", cu_ext[0]);
    const int64_t num_pages = num_slots / page_size;
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t pre = prefix_lens[b], ext = ext_lens[b];
        if (pre < 0 || ext < 0)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: prefix_len %d and ext_len %d must be >= 0", b, pre, ext);
        if ((int64_t)cu_ext[b + 1] - cu_ext[b] != ext)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: cu_ext[%d] - cu_ext[%d] = %lld but ext_len = %d", b, b + 1,
                       b, (long long)cu_ext[b + 1] - cu_ext[b], ext);
        if (cu_ext[b + 1] > total_tokens)
            return bad(MSGL_ERR_INVALID_ARG, "cu_ext[%d] = %d exceeds total_tokens %d", b + 1, cu_ext[b + 1],
                       total_tokens);
        if (ext > max_ext_len)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: ext_len %d exceeds max_ext_len %d", b, ext, max_ext_len);
        if ((int64_t)pre + ext > max_seq_len)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: prefix_len + ext_len = %lld exceeds max_seq_len %d", b,
                       (long long)pre + ext, max_seq_len);
        if (positions)
            for (int32_t i = 0; i < ext; ++i)
                if (positions[cu_ext[b] + i] != pre + i)
                    return bad(MSGL_ERR_INVALID_ARG, "request %d row %d: positions[%d] = %d, expected %d", b, i,
                               cu_ext[b] + i, positions[cu_ext[b] + i], pre + i);
        if ((rc = check_pages(num_pages, page_size, page_ids, stride, width, b, b, (int64_t)pre + ext))) return rc;
    }
    if (cu_ext[num_reqs] != total_tokens)
        return bad(MSGL_ERR_INVALID_ARG, "cu_ext[%d] = %d but total_tokens = %d", num_reqs, cu_ext[num_reqs],
                   total_tokens);
    return MSGL_OK;
}

msgl_status msgl_check_decode_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids, int32_t stride,
                                   int32_t width, const int32_t *seq_lens, int32_t num_reqs, int32_t max_seq_len) {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, page_ids, stride, width);
    if (rc) return rc;
    if (num_reqs < 0) return bad(MSGL_ERR_INVALID_ARG, "num_reqs must be >= 0");
    if (num_reqs > 0 && !seq_lens) return bad(MSGL_ERR_INVALID_ARG, "seq_lens is NULL");
    const int64_t num_pages = num_slots / page_size;
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t n = seq_lens[b];
        if (n < 1 || n > max_seq_len)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: seq_len %d is outside [1, max_seq_len = %d]", b, n,
                       max_seq_len);
        if ((rc = check_pages(num_pages, page_size, page_ids, stride, width, b, b, n))) return rc;
    }
    return MSGL_OK;
}

msgl_status msgl_check_step_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                                 int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                                 const int32_t *cached_lens, const int32_t *new_lens, int32_t num_reqs,
                                 const int32_t *free_pages, int32_t num_free, int32_t total_tokens) try {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, req_table, table_stride, table_width);
    if (rc) return rc;
    if (num_reqs < 0 || num_rows < 0 || num_free < 0 || total_tokens < 0) return bad(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_reqs > 0 && !cached_lens) return bad(MSGL_ERR_INVALID_ARG, "cached_lens is NULL");
    if (num_free > 0 && !free_pages) return bad(MSGL_ERR_INVALID_ARG, "free_pages is NULL");
    const int64_t num_pages = num_slots / page_size;
    std::unordered_set<int32_t> rows, used;
    int64_t tokens = 0, taken = 0;
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t row = req_rows ? req_rows[b] : b, cached = cached_lens[b], fresh = new_lens ? new_lens[b] : 1;
        if (row < 0 || row >= num_rows)
            return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: row %d is outside [0, %d)", b, row, num_rows);
        if (!rows.insert(row).second)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: row %d belongs to an earlier request too", b, row);
        if (cached < 0 || fresh < 0)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: cached_len %d and new_len %d must be >= 0", b, cached, fresh);
        if ((int64_t)cached + fresh > INT32_MAX)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: %lld tokens do not fit 32 bits", b, (long long)cached + fresh);
        const int64_t old_pages = ((int64_t)cached + page_size - 1) / page_size;
        const int64_t pages = ((int64_t)cached + fresh + page_size - 1) / page_size;
        if (pages > table_width)
            return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: %lld tokens need %lld pages but the table width is %d", b,
                       (long long)cached + fresh, (long long)pages, table_width);
        if ((rc = check_pages(num_pages, page_size, req_table, table_stride, table_width, b, row, cached))) return rc;
        for (int64_t p = 0; p < old_pages; ++p) used.insert(req_table[(int64_t)row * table_stride + p]);
        tokens += fresh;
        taken += pages - old_pages;
        if (tokens > total_tokens)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: %lld tokens so far but total_tokens = %d", b,
                       (long long)tokens, total_tokens);
        if (taken > num_free)
            return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: %lld pages so far but num_free = %d", b, (long long)taken,
                       num_free);
    }
    for (int64_t p = 0; p < taken; ++p) {
        if (free_pages[p] < 0 || free_pages[p] >= num_pages)
            return bad(MSGL_ERR_OUT_OF_RANGE, "free_pages[%lld] = %d is outside [0, %lld)", (long long)p, free_pages[p],
                       (long long)num_pages);
        if (!used.insert(free_pages[p]).second)
            return bad(MSGL_ERR_INVALID_ARG, "free_pages[%lld] = %d is in use", (long long)p, free_pages[p]);
    }
    return MSGL_OK;
} catch (const std::exception &) {
    return no_memory();
}

msgl_status msgl_check_groups_meta(int64_t num_slots, int32_t page_size, const int32_t *page_ids, int32_t stride,
                                   int32_t width, const int32_t *group_start, const int32_t *shared_lens,
                                   const int32_t *seq_lens, int32_t num_reqs, int32_t max_seq_len) {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, page_ids, stride, width);
    if (rc) return rc;
    if (num_reqs < 0) return bad(MSGL_ERR_INVALID_ARG, "num_reqs must be >= 0");
    if (num_reqs > 0 && (!group_start || !shared_lens || !seq_lens))
        return bad(MSGL_ERR_INVALID_ARG, "group_start, shared_lens and seq_lens must be non-NULL");
    const int64_t num_pages = num_slots / page_size;
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t first = group_start[b], n = seq_lens[b];
        if (n < 1 || n > max_seq_len)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: seq_len %d is outside [1, max_seq_len = %d]", b, n, max_seq_len);
        if (first != b && (b == 0 || first != group_start[b - 1]))
            return bad(MSGL_ERR_INVALID_ARG, "request %d: group_start %d is neither %d nor the row's before", b, first, b);
        const bool alone = first == b && (b + 1 == num_reqs || group_start[b + 1] != b);
        const int32_t shared = alone ? 0 : shared_lens[b];
        if (shared < 0 || shared > n)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: shared_len %d is outside [0, seq_len = %d]", b, shared, n);
        if (first != b && shared != shared_lens[first])
            return bad(MSGL_ERR_INVALID_ARG, "request %d: shared_len %d but its group's first has %d", b, shared,
                       shared_lens[first]);
        // shared keys on the first row's pages, the others on its own
        if (first == b && (rc = check_pages(num_pages, page_size, page_ids, stride, width, b, b, n))) return rc;
        if (((int64_t)n + page_size - 1) / page_size > width)
            return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: %d keys do not fit the table width %d", b, n, width);
        for (int64_t p = shared / page_size; p * page_size < n; ++p) {
            const int32_t id = page_ids[(int64_t)b * stride + p];
            if (id < 0 || id >= num_pages)
                return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: page_ids[%lld] = %d is outside [0, %lld)", b,
                           (long long)p, id, (long long)num_pages);
        }
    }
    return MSGL_OK;
}

msgl_status msgl_check_fork_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                                 int32_t table_stride, int32_t table_width, const int32_t *parent_rows,
                                 const int32_t *child_rows, const int32_t *lens, int32_t num_forks,
                                 const int32_t *free_pages, int32_t num_free) try {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, req_table, table_stride, table_width);
    if (rc) return rc;
    if (num_forks < 0 || num_rows < 0 || num_free < 0) return bad(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_forks > 0 && (!parent_rows || !child_rows || !lens))
        return bad(MSGL_ERR_INVALID_ARG, "parent_rows, child_rows and lens must be non-NULL");
    if (num_free > 0 && !free_pages) return bad(MSGL_ERR_INVALID_ARG, "free_pages is NULL");
    const int64_t num_pages = num_slots / page_size;
    std::unordered_set<int32_t> parents, children, used;
    int64_t taken = 0;
    auto none = [&](int32_t i) { return parent_rows[i] == -1 && child_rows[i] == -1; };
    for (int32_t i = 0; i < num_forks; ++i)
        if (!none(i)) parents.insert(parent_rows[i]);
    for (int32_t i = 0; i < num_forks; ++i) {
        if (none(i)) continue;
        for (const int32_t row : {parent_rows[i], child_rows[i]})
            if (row < 0 || row >= num_rows)
                return bad(MSGL_ERR_OUT_OF_RANGE, "fork %d: row %d is outside [0, %d)", i, row, num_rows);
        if (parents.count(child_rows[i]))
            return bad(MSGL_ERR_INVALID_ARG, "fork %d: row %d is a parent too", i, child_rows[i]);
        if (!children.insert(child_rows[i]).second)
            return bad(MSGL_ERR_INVALID_ARG, "fork %d: row %d is an earlier fork's child too", i, child_rows[i]);
        if (lens[i] < 0) return bad(MSGL_ERR_INVALID_ARG, "fork %d: length %d must be >= 0", i, lens[i]);
        if ((rc = check_pages(num_pages, page_size, req_table, table_stride, table_width, i, parent_rows[i], lens[i],
                              "fork")))
            return rc;
        for (int64_t p = 0; p * page_size < lens[i]; ++p)
            used.insert(req_table[(int64_t)parent_rows[i] * table_stride + p]);
        taken += lens[i] % page_size != 0;
        if (taken > num_free)
            return bad(MSGL_ERR_OUT_OF_RANGE, "fork %d: %lld pages so far but num_free = %d", i, (long long)taken, num_free);
    }
    for (int64_t p = 0; p < taken; ++p) {
        if (free_pages[p] < 0 || free_pages[p] >= num_pages)
            return bad(MSGL_ERR_OUT_OF_RANGE, "free_pages[%lld] = %d is outside [0, %lld)", (long long)p, free_pages[p],
                       (long long)num_pages);
        if (!used.insert(free_pages[p]).second)
            return bad(MSGL_ERR_INVALID_ARG, "free_pages[%lld] = %d is in use", (long long)p, free_pages[p]);
    }
    return MSGL_OK;
} catch (const std::exception &) {
    return no_memory();
}

msgl_status msgl_check_copy_meta(int64_t num_slots, int32_t page_size, const int32_t *src, const int32_t *dst,
                                 const int32_t *tokens, int32_t num_pairs) try {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, nullptr, 0, 0);
    if (rc) return rc;
    if (num_pairs < 0) return bad(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_pairs > 0 && (!src || !dst)) return bad(MSGL_ERR_INVALID_ARG, "src and dst must be non-NULL");
    const int64_t num_pages = num_slots / page_size;
    std::unordered_set<int32_t> read, written;
    for (int32_t i = 0; i < num_pairs; ++i) {
        if (src[i] == -1 && dst[i] == -1) continue;
        for (const int32_t page : {src[i], dst[i]})
            if (page < 0 || page >= num_pages)
                return bad(MSGL_ERR_OUT_OF_RANGE, "pair %d: page %d is outside [0, %lld)", i, page, (long long)num_pages);
        if (tokens && (tokens[i] < 0 || tokens[i] > page_size))
            return bad(MSGL_ERR_INVALID_ARG, "pair %d: %d tokens are outside [0, page_size = %d]", i, tokens[i], page_size);
        if (!written.insert(dst[i]).second)
            return bad(MSGL_ERR_INVALID_ARG, "pair %d: page %d is an earlier pair's dst too", i, dst[i]);
        if (src[i] != dst[i]) read.insert(src[i]);   // (a page onto itself stays what it is)
    }
    for (int32_t i = 0; i < num_pairs; ++i)
        if (dst[i] >= 0 && read.count(dst[i]))
            return bad(MSGL_ERR_INVALID_ARG, "pair %d: page %d is written and read", i, dst[i]);
    return MSGL_OK;
} catch (const std::exception &) {
    return no_memory();
}

msgl_status msgl_check_held_meta(int64_t num_slots, int32_t page_size, const int32_t *req_table, int32_t num_rows,
                                 int32_t table_stride, int32_t table_width, const int32_t *req_rows,
                                 const int32_t *lens, int32_t num_reqs) {
    msgl::set_last_error("");
    msgl_status rc = check_pool_scalars(num_slots, page_size, req_table, table_stride, table_width);
    if (rc) return rc;
    if (num_reqs < 0 || num_rows < 0) return bad(MSGL_ERR_INVALID_ARG, "negative size");
    if (num_reqs > 0 && !lens) return bad(MSGL_ERR_INVALID_ARG, "lens is NULL");
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t row = req_rows ? req_rows[b] : b;
        if (row == -1) continue;
        if (row < 0 || row >= num_rows)
            return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: row %d is outside [0, %d)", b, row, num_rows);
        if (lens[b] < 0) return bad(MSGL_ERR_INVALID_ARG, "request %d: length %d must be >= 0", b, lens[b]);
        if ((rc = check_pages(num_slots / page_size, page_size, req_table, table_stride, table_width, b, row, lens[b])))
            return rc;
    }
    return MSGL_OK;
}

msgl_status msgl_check_draft_meta(int32_t vocab, const int32_t *tokens, const int32_t *cu_ext, const float *accept_u,
                                  const float *sample_u, int32_t num_reqs, int32_t total_tokens) {
    msgl::set_last_error("");
    if (num_reqs < 0 || total_tokens < 0 || vocab <= 0)
        return bad(MSGL_ERR_INVALID_ARG, "num_reqs and total_tokens must be >= 0 and vocab > 0");
    if (num_reqs == 0) return MSGL_OK;
    if (!cu_ext || !sample_u || (total_tokens > 0 && (!tokens || !accept_u)))
        return bad(MSGL_ERR_INVALID_ARG, "tokens, cu_ext, accept_u and sample_u must be non-NULL");
    for (int32_t b = 0; b < num_reqs; ++b) {
        const int32_t first = cu_ext[b], end = cu_ext[b + 1];
        if (first < 0 || first > end || end > total_tokens)
            return bad(MSGL_ERR_INVALID_ARG, "request %d: rows [%d, %d) are not rows of [0, %d)", b, first, end, total_tokens);
        for (int32_t r = first; r + 1 < end; ++r) {
            if (tokens[r + 1] < 0 || tokens[r + 1] >= vocab)
                return bad(MSGL_ERR_OUT_OF_RANGE, "request %d: tokens[%d] = %d is outside [0, %d)", b, r + 1, tokens[r + 1],
                           vocab);
            if (!(accept_u[r] >= 0.f && accept_u[r] < 1.f))
                return bad(MSGL_ERR_INVALID_ARG, "request %d: accept_u[%d] = %g is outside [0, 1)", b, r, accept_u[r]);
        }
        if (first < end && !(sample_u[b] >= 0.f && sample_u[b] < 1.f))
            return bad(MSGL_ERR_INVALID_ARG, "request %d: sample_u = %g is outside [0, 1)", b, sample_u[b]);
    }
    return MSGL_OK;
}

}  // extern "C"
