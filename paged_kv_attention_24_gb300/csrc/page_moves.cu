// Requests that continue other requests on the same pages, and copies of pages.
//
// "Mini-SGLang 实战指南", §6.2 and §6.5: requests that begin alike hold the same pages of
// the one pool.  Whole pages are never written again, so a fork takes them over by
// id; the last, partly filled page would be written by both, so the fork gets a
// new one and a copy of what is in it.
//
// Both are copies: of table rows (latency: rows, lengths, ids, stores; 4 forks of 63 pages
// 2.3 us, 256 of up to 16384 4.8) and of pool rows (HBM: every byte read once and written once;
// 1024 pages of 16 slots in 4 layers, 537 MB, in 80 us, 6.7 TB/s).
#include <limits.h>

#include "kernels.h"

namespace msgl {

namespace {

// ---------------------------------------------------------------------- fork
//
// One block per fork and 4096 columns of its row, as in the step tables.  A fork
// needs one new page or none, so its place among the free pages is the number of
// earlier forks with a partly filled page, counted again by every block; the same
// loop sees whether its child's row is named by another fork.
constexpr int kForkThreads = 256;
constexpr int kPerThread = 16;
constexpr int kChunk = kForkThreads * kPerThread;

struct Fork {
    int32_t parent, child, tokens;
    int32_t full, tail;     // whole pages, tokens on the last one
    bool none, rows_ok, len_ok;
};

__device__ __forceinline__ Fork fork_at(const ForkArgs &a, int i) {
    Fork f;
    f.parent = __ldg(a.parent_rows + i);
    f.child = __ldg(a.child_rows + i);
    f.tokens = __ldg(a.lens + i);
    f.none = f.parent == -1 && f.child == -1;
    f.rows_ok = f.parent >= 0 && f.parent < a.num_rows && f.child >= 0 && f.child < a.num_rows;
    const int mask = (1 << a.log2_ps) - 1;
    f.full = f.tokens >> a.log2_ps;
    f.tail = f.tokens & mask;
    f.len_ok = f.tokens >= 0 && (int64_t)f.full + (f.tail > 0) <= a.table_width;
    if (f.none || !f.rows_ok || !f.len_ok) f.full = f.tail = 0;
    return f;
}

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkArgs a) {
    const int b = blockIdx.x, at0 = blockIdx.y * kChunk + (int)threadIdx.x;
    Fork f{};
    if (b < a.num_forks) {
        f = fork_at(a, b);
        if (blockIdx.y > 0 && blockIdx.y * kChunk > f.full) return;
    } else if (blockIdx.y > 0) {
        return;
    }
    // (f.full is 0 unless rows and length are in range, so these are read before the counts below are known)
    const int32_t *theirs = a.req_table + (int64_t)max(f.parent, 0) * a.table_stride;
    int32_t id[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int p = at0 + u * kForkThreads;
        if (p < f.full) id[u] = theirs[p];
    }
    const int32_t source = f.tail > 0 ? theirs[f.full] : -1;
    int n = 0;
    bool twice = false;
    for (int i = threadIdx.x; i < a.num_forks; i += kForkThreads) {
        const Fork x = fork_at(a, i);
        n += i < b && x.tail > 0;
        twice |= b < a.num_forks && (f.child == x.parent || (i != b && f.child == x.child));
    }
    __shared__ int part[kForkThreads / 32];
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
    const bool clash = __syncthreads_or(twice);
    int before = 0;
#pragma unroll
    for (int w = 0; w < kForkThreads / 32; ++w) before += part[w];
    if (b == a.num_forks) {
        if (threadIdx.x == 0) a.pages_taken[0] = min(before, a.num_free);
        return;
    }
    const bool rows_ok = f.rows_ok && !clash, paged = f.tail == 0 || before < a.num_free;
    bool served = !f.none && rows_ok && f.len_ok && paged, pages_ok = true;
    int32_t fresh = -1;
    if (served && f.tail > 0) {
        fresh = __ldg(a.free_pages + before);
        pages_ok = fresh >= 0 && fresh < a.num_pages && source >= 0 && source < a.num_pages;
        served = pages_ok;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        const bool copies = served && f.tail > 0;
        a.copy_src[b] = copies ? source : -1;
        a.copy_dst[b] = copies ? fresh : -1;
        a.copy_tokens[b] = copies ? f.tail : 0;
        if (!f.none) {
            if (!rows_ok) report(a.status, MSGL_DEVERR_ROW);
            else if (!f.len_ok) report(a.status, MSGL_DEVERR_LENGTH);
            else if (!paged) report(a.status, MSGL_DEVERR_NO_PAGES);
            else if (!pages_ok) report(a.status, MSGL_DEVERR_PAGE_RANGE);
        }
    }
    if (!served) return;
    int32_t *mine = a.req_table + (int64_t)f.child * a.table_stride;
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
        const int p = at0 + u * kForkThreads;
        if (p < f.full + (f.tail > 0)) mine[p] = p < f.full ? id[u] : fresh;
    }
}

// ---------------------------------------------------------------------- copy
//
// A warp takes 2 KB of one page's K or V in one pool, all its loads before its
// stores; the pools and their K and V are the grid's second axis, so that a
// block's addresses differ by the page only.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kPiece = 32 * kCopyUnroll;           // 16-byte vectors

template <int kBuffers>
struct CopyBuffers {
    void *at[kBuffers];
};

template <int kBuffers>
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const CopyPagesArgs a, const __grid_constant__ CopyBuffers<kBuffers> buffers) {
    const int lane = threadIdx.x & 31;
    uint4 *pool = static_cast<uint4 *>(buffers.at[blockIdx.y]);
    const int n = a.count ? min(max(__ldg(a.count), 0), a.num_pairs) : a.num_pairs;
    const int64_t units = ((int64_t)n + a.group - 1) / a.group * a.turns;
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    for (int64_t w = ((int64_t)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; w < units; w += warps) {
        // some pieces of each page of a group of pairs, looked up a lane each
        const int64_t first = w / a.turns * a.group;
        const int turn = (int)(w % a.turns), per = kPiece * a.span;
        int src = -1, dst = -1, tokens = 0;
        if (lane < a.group && first + lane < n) {
            src = __ldg(a.src + first + lane);
            dst = __ldg(a.dst + first + lane);
            tokens = a.tokens ? __ldg(a.tokens + first + lane) : a.page_size;
            uint32_t bad = 0;
            if (src != -1 || dst != -1) {
                if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) bad = MSGL_DEVERR_PAGE_RANGE;
                else if (tokens < 0 || tokens > a.page_size) bad = MSGL_DEVERR_LENGTH;
            }
            if (bad && turn == 0) report(a.status, bad);
            if (bad) src = -1;
        }
        for (uint32_t live = __ballot_sync(0xffffffffu, src != -1); live; live &= live - 1) {
            const int i = __ffs(live) - 1;
            const int all = __shfl_sync(0xffffffffu, tokens, i) * a.row_vecs, most = min(all, (turn + 1) * per);
            const uint4 *from = pool + (int64_t)__shfl_sync(0xffffffffu, src, i) * a.page_vecs;
            uint4 *to = pool + (int64_t)__shfl_sync(0xffffffffu, dst, i) * a.page_vecs;
            for (int at = turn * per + lane; at < most; at += kPiece) {
                uint4 r[kCopyUnroll];
#pragma unroll
                for (int u = 0; u < kCopyUnroll; ++u)
                    if (at + u * 32 < most) r[u] = ld_stream_16(from + at + u * 32);
#pragma unroll
                for (int u = 0; u < kCopyUnroll; ++u)
                    if (at + u * 32 < most) st_stream_16(to + at + u * 32, r[u]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream) {
    const long long chunks = ((long long)max(a.table_width, 1) + kChunk - 1) / kChunk;
    fork_kernel<<<dim3(a.num_forks + 1, (unsigned)chunks), kForkThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int kBuffers>
static cudaError_t launch_copy(const CopyPagesArgs &a, void *const *buffers, unsigned blocks, cudaStream_t stream) {
    CopyBuffers<kBuffers> b{};
    for (int i = 0; i < a.num_buffers; ++i) b.at[i] = buffers[i];
    copy_pages_kernel<kBuffers><<<dim3(blocks, a.num_buffers), kCopyThreads, 0, stream>>>(a, b);
    return cudaGetLastError();
}

cudaError_t launch_copy_pages(CopyPagesArgs a, void *const *buffers, cudaStream_t stream) {
    a.pieces = (int32_t)((a.page_vecs + kPiece - 1) / kPiece);
    // Pairs, and then pieces, by twos, fours, .. where there are more than 16 for every warp that runs at once: a list
    // that is padding for the most part (a compaction's, without its count) is then looked through quickly
    // (600000 entries and 36 pools: one by one 35 ms, in groups of 32 pairs 1.9 ms, and pages as a whole 0.14).
    const int64_t pieces = (int64_t)a.num_pairs * a.pieces * a.num_buffers, enough = (int64_t)sm_count() * 64 * 16;
    for (a.group = 1; a.group < 32 && pieces / (2 * a.group) >= enough;) a.group *= 2;
    for (a.span = 1; a.span < a.pieces && pieces / (2 * a.group * a.span) >= enough;) a.span *= 2;
    a.turns = (a.pieces + a.span - 1) / a.span;
    const int64_t blocks = (((int64_t)a.num_pairs + a.group - 1) / a.group * a.turns + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    // (more than run at once, up to 64 an SM: 1024 pages of 16 slots in 4 layers take 91.5 us with 4 an SM, 84 with 8,
    // 83 with 16, 80 with 64)
    const int64_t cap = ((int64_t)sm_count() * 64 + a.num_buffers - 1) / a.num_buffers;
    const unsigned n = (unsigned)(blocks < cap ? blocks : cap);
    // (2 KB of addresses cost a launch 0.7 us, so that few pools have a kernel of their own)
    return a.num_buffers <= 16 ? launch_copy<16>(a, buffers, n, stream) : launch_copy<2 * kMaxCopyPools>(a, buffers, n, stream);
}

}  // namespace msgl
