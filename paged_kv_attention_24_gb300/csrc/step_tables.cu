// Block tables and slot maps of one step, from the request lengths.
//
// "不懂SGLang？从miniSGLang开始", §1.3 item 3: the page table and the positions
// locate each token's K/V; §1.2 item 3 and "Mini-SGLang 实战指南", §6.2: every
// request takes its pages from one pool.
//
// With P(x) = ceil(x / page_size), request b needs P(cached_b + new_b) -
// P(cached_b) new pages; its place in the list of free pages and its place among
// the step's tokens are sums over the requests before it.  Both sums are taken
// again by every block (a few kilobytes of lengths out of L2), which costs less
// than a pass of its own that the rest would wait for.
//
// Bound by latency: the lengths, then the table entries they lead to, then the
// stores.  One block per request and 2048 columns or tokens of it, so that a row
// of a few thousand entries is one round of independent loads; block num_reqs
// writes the totals and the padding behind the last token.  4 decoding requests:
// 4.0 us; 256 of up to 2047 tokens, page size 1: 5.7 us; 64 prefills of 1024
// tokens behind up to 16384: 6.1 us.
#include <limits.h>

#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kChunk = kThreads * kPerThread;

struct Request {
    int32_t cached, tokens, row;   // tokens: max(new, 0)
    int32_t old_pages, need;
    bool ok;                       // its own numbers are in range
};

__device__ __forceinline__ Request request_at(const StepTablesArgs &a, int i) {
    Request r;
    r.cached = __ldg(a.cached_lens + i);
    const int n = a.new_lens ? __ldg(a.new_lens + i) : 1;
    r.row = a.req_rows ? __ldg(a.req_rows + i) : i;
    r.tokens = max(n, 0);
    const long long s = (long long)r.cached + n;
    const long long ps1 = (1 << a.log2_ps) - 1;
    const long long pages = (s + ps1) >> a.log2_ps;
    r.ok = r.cached >= 0 && n >= 0 && s <= INT_MAX && pages <= a.max_pages && r.row >= 0 && r.row < a.num_rows;
    r.old_pages = r.ok ? (int)(((long long)r.cached + ps1) >> a.log2_ps) : 0;
    r.need = r.ok ? (int)pages - r.old_pages : 0;
    return r;
}

// Sums over the whole block; every thread gets both.
__device__ __forceinline__ void block_sum2(long long &x, long long &y) {
    __shared__ long long part[2][kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (lane == 0) { part[0][warp] = x; part[1][warp] = y; }
    __syncthreads();
    x = y = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) { x += part[0][w]; y += part[1][w]; }
}

__global__ void __launch_bounds__(kThreads) step_tables_kernel(const StepTablesArgs a) {
    const int b = blockIdx.x;
    const int at0 = blockIdx.y * kChunk + threadIdx.x;   // this thread's first column and token
    Request r{};
    if (b < a.num_reqs) {
        // a chunk behind the request's last column and token has nothing to do
        r = request_at(a, b);
        if (blockIdx.y > 0 && blockIdx.y * kChunk >= max(r.old_pages + r.need, r.tokens)) return;
    }
    long long cu = 0, off = 0;   // tokens and new pages of the requests before b
    for (int i = threadIdx.x; i < b; i += kThreads) {
        const Request x = request_at(a, i);
        cu += x.tokens;
        off += x.need;
    }
    block_sum2(cu, off);
    if (b == a.num_reqs) {
        // totals, and the padding behind the last token
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            a.cu_ext[b] = (int)min(cu, (long long)a.total_tokens);
            long long taken = off;
            if (off > a.num_free || cu > a.total_tokens) {
                // some request was refused: the pages up to the last one served
                long long c = 0, o = 0;
                taken = 0;
                for (int i = 0; i < b; ++i) {
                    const Request x = request_at(a, i);
                    c += x.tokens;
                    o += x.need;
                    if (x.need > 0 && c <= a.total_tokens && o <= a.num_free) taken = o;
                }
            }
            a.pages_taken[0] = (int)taken;
        }
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) {
            const long long t = (long long)at0 + u * kThreads;
            if (t >= cu && t < a.total_tokens) {
                a.positions[t] = 0;
                a.out_loc[t] = -1;
            }
        }
        return;
    }
    const bool fits = cu + r.tokens <= a.total_tokens;
    const bool paged = r.need == 0 || off + r.need <= a.num_free;
    const bool served = r.ok && fits && paged;
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        a.seq_lens[b] = served ? r.cached + r.tokens : 0;
        a.cu_ext[b] = (int)min(cu, (long long)a.total_tokens);
        if (!r.ok || !fits) report(a.status, MSGL_DEVERR_LENGTH);
        if (!paged) report(a.status, MSGL_DEVERR_NO_PAGES);
    }
    const int pages = served ? r.old_pages + r.need : 0;
    int32_t *mine = a.req_table + (long long)r.row * a.table_stride;
    int32_t *out = a.page_ids + (long long)b * a.stride;
    const int32_t *fresh = a.free_pages + off - r.old_pages;   // page p >= old_pages is fresh[p]
    int32_t id[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int p = at0 + u * kThreads;
        id[u] = p < pages ? (p < r.old_pages ? mine[p] : __ldg(fresh + p)) : -1;
    }
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int p = at0 + u * kThreads;
        if (p < pages) {
            out[p] = id[u];
            if (p >= r.old_pages) mine[p] = id[u];
        }
    }
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int i = at0 + u * kThreads;
        if (i >= r.tokens || cu + i >= a.total_tokens) break;
        const int pos = served ? r.cached + i : 0, p = pos >> a.log2_ps;
        int slot = -1;
        if (served) {
            const int page = p < r.old_pages ? mine[p] : __ldg(fresh + p);
            if (page >= 0 && page < a.num_pages)
                slot = (page << a.log2_ps) + (pos & ((1 << a.log2_ps) - 1));
            else
                bad = true;
        }
        a.positions[cu + i] = pos;
        a.out_loc[cu + i] = slot;
    }
    if (bad) report(a.status, MSGL_DEVERR_PAGE_RANGE);
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs &a, cudaStream_t stream) {
    const int most = max(max(a.total_tokens, a.max_pages), 1);
    const long long chunks = ((long long)most + kChunk - 1) / kChunk;
    step_tables_kernel<<<dim3(a.num_reqs + 1, (unsigned)chunks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace msgl
