// The pages that no request holds, and the pages in use moved to the front of the pool.
//
// "Mini-SGLang 实战指南", §6.2: every request's pages come from the one pool; §6.5: several
// requests may hold the same page.  Which pages are in use follows from the tables
// and lengths of the running requests, so nothing is counted from step to step: a
// page is free when no request's table names it, whatever forks, rejected drafts
// and finished requests did before.
//
// One cluster of 8 blocks, one launch: every block takes its share of the table
// entries and marks their pages in a bitmap in its own shared memory; the blocks
// then join their bitmaps, an eighth of the pages each, count, and write what is
// theirs.  Pools of more pages than a bitmap has bits take a round for each part.
//
// Bound by latency up to some thousand entries (lengths, entries, two or three
// exchanges between the blocks, stores), by the 8 SMs' loads and stores beyond.
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kPerLane = 8;
constexpr int kUnit = 32 * kPerLane;                 // table entries of one warp's turn

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ uint32_t ld_peer(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void st_peer(uint32_t at, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

struct Shared {
    int32_t row[kThreads], pages[kThreads], unit[kThreads];   // requests of the present batch
    uint32_t warp[2][kWarps];
    uint32_t counts[2][2][kCluster];                          // exchanged, two numbers a block
};

// x summed over the warp's lanes up to this one.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    return x;
}

// f(entry's address in the table, its place in the output) for every table entry of a request, 8 to a lane.
template <class F>
__device__ __forceinline__ void for_entries(const PageMapArgs &a, Shared &s, bool tell, F f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = cluster_rank() * kWarps + warp;
    for (int b0 = 0; b0 < a.num_reqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int row = -1, pages = 0;
        if (b < a.num_reqs) {
            row = a.req_rows ? __ldg(a.req_rows + b) : b;
            const int len = __ldg(a.lens + b);
            const int64_t need = ((int64_t)len + (1 << a.log2_ps) - 1) >> a.log2_ps;
            const bool row_ok = row >= 0 && row < a.num_rows, len_ok = len >= 0 && need <= a.table_width;
            // a request of a length that cannot be keeps whatever its row names: nothing of it is given away
            pages = row_ok ? (len_ok ? (int)need : a.table_width) : 0;
            if (tell && row != -1 && !row_ok) report(a.status, MSGL_DEVERR_ROW);
            if (tell && row_ok && !len_ok) report(a.status, MSGL_DEVERR_LENGTH);
        }
        const uint32_t units = (pages + kUnit - 1) / kUnit, upto = warp_scan(units);
        __syncthreads();                                       // the batch before is done with
        if (lane == 31) s.warp[0][warp] = upto;
        s.row[threadIdx.x] = row;
        s.pages[threadIdx.x] = pages;
        __syncthreads();
        if (warp == 0) s.warp[1][lane] = warp_scan(s.warp[0][lane]);
        __syncthreads();
        s.unit[threadIdx.x] = (warp ? s.warp[1][warp - 1] : 0) + upto;   // units up to and with this request
        const int total = s.warp[1][kWarps - 1];
        __syncthreads();
        for (int u = first; u < total; u += kCluster * kWarps) {
            int lo = 0;                                        // the first request whose units pass u
#pragma unroll
            for (int step = kThreads / 2; step > 0; step >>= 1)
                if (s.unit[lo + step - 1] <= u) lo += step;
            const int col = (u - (lo ? s.unit[lo - 1] : 0)) * kUnit + lane, n = s.pages[lo];
            const int64_t at = (int64_t)s.row[lo] * a.table_stride + col;
            int32_t id[kPerLane];
#pragma unroll
            for (int k = 0; k < kPerLane; ++k)
                if (col + 32 * k < n) id[k] = a.table[at + 32 * k];
#pragma unroll
            for (int k = 0; k < kPerLane; ++k)
                if (col + 32 * k < n) f(id[k], (int64_t)s.row[lo] * a.out_stride + col + 32 * k);
        }
    }
}

// Bits of 32 pages from p0 on that something beside the requests holds.
__device__ __forceinline__ uint32_t held_word(const PageMapArgs &a, int64_t p0) {
    if (!a.held) return 0;
    uint32_t bits = 0;
    for (int i = 0; i < 32; ++i)
        if (p0 + i < a.num_pages && __ldg(a.held + p0 + i)) bits |= 1u << i;
    return bits;
}

// Marks the pages [p0, p0 + 32 * kCluster * slice) that the requests hold, and leaves this block's slice of
// them, joined, in bits[rank * slice ..].
__device__ __forceinline__ void mark(const PageMapArgs &a, Shared &s, uint32_t *bits, int slice, int64_t p0, bool tell) {
    for (int i = threadIdx.x; i < kCluster * slice; i += kThreads) bits[i] = 0;
    __syncthreads();
    for_entries(a, s, tell, [&](int32_t id, int64_t) {
        if (id < 0 || id >= a.num_pages) {
            if (tell) report(a.status, MSGL_DEVERR_PAGE_RANGE);
            return;
        }
        const int64_t at = id - p0;
        if (at >= 0 && at < 32ll * kCluster * slice) atomicOr(bits + (at >> 5), 1u << (at & 31));
    });
    cluster_sync();
    const int rank = cluster_rank();
    for (int i = threadIdx.x; i < slice; i += kThreads) {
        uint32_t *mine = bits + rank * slice + i, v = *mine;
#pragma unroll
        for (int k = 1; k < kCluster; ++k) v |= ld_peer(peer(mine, (rank + k) % kCluster));
        *mine = v;
    }
    __syncthreads();
}

// Sums of x and y over the block's warps before this one and over the blocks before this one; every block's
// totals.  which: two exchanges in a row use different places.
struct Places {
    uint32_t x, y, all_x, all_y;
};
__device__ __forceinline__ Places exchange(Shared &s, uint32_t x, uint32_t y, int which) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank();
    if (lane == 0) {
        s.warp[0][warp] = x;
        s.warp[1][warp] = y;
    }
    __syncthreads();
    const uint32_t wx = s.warp[0][lane], wy = s.warp[1][lane];
    Places p;
    p.x = __reduce_add_sync(0xffffffffu, lane < warp ? wx : 0);
    p.y = __reduce_add_sync(0xffffffffu, lane < warp ? wy : 0);
    if (warp == 0) {
        const uint32_t bx = __reduce_add_sync(0xffffffffu, wx), by = __reduce_add_sync(0xffffffffu, wy);
        if (lane < kCluster) {
            st_peer(peer(&s.counts[which][0][rank], lane), bx);
            st_peer(peer(&s.counts[which][1][rank], lane), by);
        }
    }
    cluster_sync();
    p.all_x = p.all_y = 0;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
        const uint32_t bx = s.counts[which][0][k], by = s.counts[which][1][k];
        if (k < rank) {
            p.x += bx;
            p.y += by;
        }
        p.all_x += bx;
        p.all_y += by;
    }
    return p;
}

// out[place + i] = the i-th page of the word's set bits, for the 32 words that a warp's lanes hold; most: entries
// from there on are not written.  Returns the place behind them.
__device__ __forceinline__ uint32_t write_bits(uint32_t word, int64_t page, uint32_t place, int32_t *out, uint32_t most) {
    const int lane = threadIdx.x & 31;
    const uint32_t n = __popc(word), upto = warp_scan(n);
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
        const uint32_t w = __shfl_sync(0xffffffffu, word, i), at = place + __shfl_sync(0xffffffffu, upto - n, i);
        const uint32_t to = at + __popc(w & ((1u << lane) - 1));
        if (w >> lane & 1 && to < most) out[to] = (int32_t)(page + 32 * i + lane);
    }
    return place + __shfl_sync(0xffffffffu, upto, 31);
}

__device__ __forceinline__ void fill(int32_t *out, int64_t from, int64_t to) {
    for (int64_t i = from + (int64_t)cluster_rank() * kThreads + threadIdx.x; i < to; i += kCluster * kThreads) out[i] = -1;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) free_pages_kernel(const PageMapArgs a, int slice) {
    extern __shared__ uint32_t bits[];
    __shared__ Shared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank();
    const int run = ((slice + kWarps - 1) / kWarps + 31) / 32 * 32;   // words of a warp
    uint32_t before = 0;
    int round = 0;
    for (int64_t p0 = 0; p0 < a.num_pages; p0 += 32ll * kCluster * slice, ++round) {
        mark(a, s, bits, slice, p0, round == 0);
        uint32_t *mine = bits + rank * slice;
        const int w0 = min(warp * run, slice), w1 = min(w0 + run, slice);
        uint32_t n = 0;
        for (int w = w0 + lane; w < w1; w += 32) {
            const int64_t page = p0 + 32ll * (rank * slice + w), left = a.num_pages - page;
            const uint32_t inside = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1 : 0;
            const uint32_t free = ~(mine[w] | held_word(a, page)) & inside;
            mine[w] = free;
            n += __popc(free);
        }
        const Places p = exchange(s, __reduce_add_sync(0xffffffffu, n), 0, round & 1);
        uint32_t place = before + p.x;
        for (int w = w0; w < w1; w += 32) {
            const uint32_t word = w + lane < w1 ? mine[w + lane] : 0;
            place = write_bits(word, p0 + 32ll * (rank * slice + w), place, a.pages_out, 0xffffffffu);
        }
        before += p.all_x;
        // (the next round clears bitmaps that a slower block may still be reading)
        cluster_sync();
    }
    fill(a.pages_out, before, a.num_pages);
    if (rank == 0 && threadIdx.x == 0) a.count_out[0] = (int32_t)before;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    compact_pages_kernel(const PageMapArgs a, int slice) {
    extern __shared__ uint32_t bits[];
    __shared__ Shared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank();
    uint32_t *stays = bits + kCluster * slice;                       // this block's slice: in use but not movable
    mark(a, s, bits, slice, 0, true);
    uint32_t *mine = bits + rank * slice;
    const int run = ((slice + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int w0 = min(warp * run, slice), w1 = min(w0 + run, slice);
    uint32_t n = 0;
    for (int w = w0 + lane; w < w1; w += 32) {
        stays[w] = held_word(a, 32ll * (rank * slice + w));
        n += __popc(mine[w] | stays[w]);
    }
    const uint32_t used = exchange(s, __reduce_add_sync(0xffffffffu, n), 0, 0).all_x;
    // the pages behind the first `used` ones go to the free pages among those, both in order
    auto below = [&](int w) -> uint32_t {                            // the word's pages in front of page `used`
        const int64_t left = (int64_t)used - 32ll * (rank * slice + w);
        return left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1 : 0;
    };
    auto holes = [&](int w) { return w < w1 ? ~(mine[w] | stays[w]) & below(w) : 0; };
    auto moves = [&](int w) { return w < w1 ? mine[w] & ~stays[w] & ~below(w) : 0; };
    uint32_t from = 0, to = 0;
    for (int w = w0 + lane; w < w1; w += 32) {
        from += __popc(moves(w));
        to += __popc(holes(w));
    }
    const Places p = exchange(s, __reduce_add_sync(0xffffffffu, from), __reduce_add_sync(0xffffffffu, to), 1);
    uint32_t src = p.x, dst = p.y;
    for (int w = w0; w < w1; w += 32) {
        const int64_t page = 32ll * (rank * slice + w);
        src = write_bits(moves(w + lane), page, src, a.src, p.all_x);
        dst = write_bits(holes(w + lane), page, dst, a.dst, p.all_x);
        const uint32_t all = w + lane < w1 ? mine[w + lane] | stays[w + lane] : 0, go = moves(w + lane);
        for (int i = 0; i < 32 && w + i < w1; ++i) {
            const uint32_t u = __shfl_sync(0xffffffffu, all, i), m = __shfl_sync(0xffffffffu, go, i);
            const int64_t at = page + 32 * i + lane;
            if (at < a.num_pages && !(m >> lane & 1)) a.pages_out[at] = u >> lane & 1 ? (int32_t)at : -1;
        }
    }
    fill(a.src, p.all_x, a.num_pages / 2);
    fill(a.dst, p.all_x, a.num_pages / 2);
    if (rank == 0 && threadIdx.x == 0) {
        a.count_out[0] = (int32_t)p.all_x;
        a.used_out[0] = (int32_t)used;
    }
    cluster_sync();
    for (uint32_t i = rank * kThreads + threadIdx.x; i < p.all_x; i += kCluster * kThreads)
        a.pages_out[__ldcg(a.src + i)] = __ldcg(a.dst + i);
    cluster_sync();
    // A page that did not move keeps its id, and so does one that this loop has already renamed (a row that is
    // named twice): its new id was free, so the map says -1 there.
    for_entries(a, s, false, [&](int32_t id, int64_t at) {
        const int32_t now = id >= (int32_t)used && id < a.num_pages ? __ldcg(a.pages_out + id) : -1;
        if (now >= 0) a.table_out[at] = now;
        else if (a.table_out != a.table) a.table_out[at] = id;
    });
}

// Bitmaps of at most this many words, 8 slices.
constexpr int kMostWords = kMaxMapPages / 32;
static_assert(kMostWords % (32 * kCluster) == 0, "slices of whole 32-word groups");

template <class K>
cudaError_t launch_map(K kernel, const PageMapArgs &a, bool with_stays, cudaStream_t stream) {
    const int64_t words = ((int64_t)a.num_pages + 31) / 32;
    const int64_t most = words < kMostWords ? words : kMostWords;
    const int slice = (int)((most + kCluster - 1) / kCluster);
    const size_t bytes = ((size_t)kCluster + with_stays) * slice * 4;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((kCluster + 1) * (size_t)(kMostWords / kCluster) * 4));
    if (e != cudaSuccess) return e;
    kernel<<<kCluster, kThreads, bytes, stream>>>(a, slice);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_free_pages(const PageMapArgs &a, cudaStream_t stream) {
    return launch_map(free_pages_kernel, a, false, stream);
}

cudaError_t launch_compact_pages(const PageMapArgs &a, cudaStream_t stream) {
    return launch_map(compact_pages_kernel, a, true, stream);
}

}  // namespace msgl
