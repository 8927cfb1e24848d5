// The pages that no request holds, and the pages in use moved to the front of the pool.
//
// "Mini-SGLang 实战指南", §6.2: every request's pages come from the one pool; §6.5: several
// requests may hold the same page.  Which pages are in use follows from the tables
// and lengths of the running requests, so nothing is counted from step to step: a
// page is free when no request's table names it, whatever forks, rejected drafts
// and finished requests did before.
//
// A bitmap of the pool, one bit a page, in the workspace: set from `held`, then every
// table entry marks its page, then each block lists its share of the pages, its place in the
// lists from a count of all bits before its own, for which a cluster of 8 blocks goes over the
// whole bitmap once (128 KB for a million pages, out of L2; each block by itself: compaction
// 17.9 us in place of 16.2).  The kernels follow each other by programmatic dependent
// launch; each waits for the one before, all of whose blocks did, before it touches
// what that one wrote.
//
// Bound by scattered atomics and the lists' stores (half a million entries, 740 thousand pages:
// free 13.3 us; 280 thousand and 550 thousand: compaction 14.6 to 15.7; some 4 us of each for the atomics, 120 to
// 130 a nanosecond, and 1 to 3 more or less by where the bitmap lies), which want many SMs: one cluster of 8
// blocks with the bitmap in shared memory took 32 and 63 us (16 blocks 23 and 44: a shared-memory
// atomic takes a cycle a lane).  A byte a page, written without atomics, is no faster to mark
// (10.9 against 8.5 us for half a million random pages, with the clearing of the map) and eight times as much to
// count.  Pools of up to 32 thousand pages under small tables are bound by latency and
// launches, and such a cluster does them in one launch (small_pool_kernel).
#include "cluster.cuh"
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBatch = kThreads;                     // requests looked at together
constexpr int kCluster = 8;                          // blocks that count together
constexpr int kPerLane = 8;
constexpr int kUnit = 32 * kPerLane;                 // table entries of one warp's turn

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// ----------------------------------------------------------- table entries

// The row and the number of table entries of request b.
__device__ __forceinline__ int entries_of(const PageMapArgs &a, int b, bool tell, int &row) {
    row = a.req_rows ? __ldg(a.req_rows + b) : b;
    const int len = __ldg(a.lens + b);
    const int64_t need = ((int64_t)len + (1 << a.log2_ps) - 1) >> a.log2_ps;
    const bool row_ok = row >= 0 && row < a.num_rows, len_ok = len >= 0 && need <= a.table_width;
    if (tell && row != -1 && !row_ok) report(a.status, MSGL_DEVERR_ROW);
    if (tell && row_ok && !len_ok) report(a.status, MSGL_DEVERR_LENGTH);
    // a request of a length that cannot be keeps whatever its row names: nothing of it is given away
    return row_ok ? (len_ok ? (int)need : a.table_width) : 0;
}

struct Batch {
    int32_t row[kBatch], pages[kBatch], unit[kBatch], warp[kWarps];
};

// The table entries of a row from column c0 on, kPerLane to a lane.
struct Unit {
    int row, c0, n;
    int32_t id[kPerLane];
    __device__ __forceinline__ void load(const PageMapArgs &a) {
        const int col = c0 + (int)(threadIdx.x & 31);
        const int64_t at = (int64_t)row * a.table_stride + col;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k)
            if (col + 32 * k < n) id[k] = a.table[at + 32 * k];
    }
    __device__ __forceinline__ bool has(int k) const { return c0 + (int)(threadIdx.x & 31) + 32 * k < n; }
    __device__ __forceinline__ int64_t place(const PageMapArgs &a, int k) const {   // in the output
        return (int64_t)row * a.out_stride + c0 + (int)(threadIdx.x & 31) + 32 * k;
    }
};

// f(unit) for all table entries of the requests, over all warps of the grid's first `blocks` blocks; ready(), once, by
// every thread (one without entries too: the grid's end then says that the grid before has ended), in front of the
// first f, but behind the first loads.  Where full rows would give a warp no more units than twice the batches of
// requests, it looks each unit's request up itself (20000 requests of 4 pages: 88 -> 11 us); else (rows much wider than
// what is in them) the rows' units are counted first, a batch of requests at a time, and dealt out evenly.
template <class R, class F>
__device__ __forceinline__ void for_entries(const PageMapArgs &a, Batch &s, int blocks, bool tell, R ready, F f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = max(1, (a.table_width + kUnit - 1) / kUnit);
    // (the chunks of a row, of which the last are often empty, to different blocks: free 13.8 -> 13.4 us; rows of one
    // chunk to warps that are neighbours, as their lengths are: 20000 of them 11.7 us, else 15.5)
    const int first = chunks > 1 ? warp * blocks + blockIdx.x : blockIdx.x * kWarps + warp, warps = blocks * kWarps;
    Unit x;
    x.n = 0;
    const int64_t rounds = ((int64_t)a.num_reqs * chunks + warps - 1) / warps;
    if (rounds <= 2 * ((a.num_reqs + kBatch - 1) / kBatch)) {
        auto look = [&](int u) {
            const int b = u / chunks;
            x.c0 = (u - b * chunks) * kUnit;
            x.n = u < a.num_reqs * chunks ? entries_of(a, b, tell && x.c0 == 0 && lane == 0, x.row) : 0;
            x.load(a);
        };
        look(first);
        ready();
        f(x);
        for (int u = first + warps; u < a.num_reqs * chunks; u += warps) {
            look(u);
            f(x);
        }
        return;
    }
    for (int b0 = 0; b0 < a.num_reqs; b0 += kBatch) {
        const int b = b0 + threadIdx.x;
        int row = -1, pages = 0;
        if (b < a.num_reqs) pages = entries_of(a, b, tell && blockIdx.x == 0, row);
        const uint32_t units = (pages + kUnit - 1) / kUnit, upto = warp_scan(units);
        __syncthreads();                                       // the batch before is done with
        if (lane == 31) s.warp[warp] = upto;
        s.row[threadIdx.x] = row;
        s.pages[threadIdx.x] = pages;
        __syncthreads();
        const uint32_t all = warp_scan(lane < kWarps ? s.warp[lane] : 0);
        const uint32_t before = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);
        s.unit[threadIdx.x] = (warp ? before : 0) + upto;      // units up to and with this request
        const int total = __shfl_sync(0xffffffffu, all, 31);
        __syncthreads();
        auto look = [&](int u) {
            int lo = 0;                                        // the first request whose units pass u
#pragma unroll
            for (int step = kBatch / 2; step > 0; step >>= 1)
                if (s.unit[lo + step - 1] <= u) lo += step;
            x.row = s.row[lo];
            x.c0 = (u - (lo ? s.unit[lo - 1] : 0)) * kUnit;
            x.n = u < total ? s.pages[lo] : 0;
            x.load(a);
        };
        look(first);
        if (b0 == 0) ready();
        f(x);
        for (int u = first + warps; u < total; u += warps) {
            look(u);
            f(x);
        }
    }
}

// -------------------------------------------------------------- the bitmaps

// Bits of 32 pages from p0 on (a multiple of 32) that something beside the requests holds.
__device__ __forceinline__ uint32_t held_word(const PageMapArgs &a, int64_t p0) {
    uint32_t bits = 0;
    if (!a.held) return 0;
    if (p0 + 32 <= a.num_pages && (reinterpret_cast<uintptr_t>(a.held) & 15) == 0) {
        const uint4 *h = reinterpret_cast<const uint4 *>(a.held + p0);
        const uint4 x = __ldg(h), y = __ldg(h + 1);
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) bits |= ((__vcmpne4(w[i], 0) & 0x08040201u) * 0x01010101u >> 24) << (4 * i);
        return bits;
    }
    for (int i = 0; i < 32 && p0 + i < a.num_pages; ++i)
        if (__ldg(a.held + p0 + i)) bits |= 1u << i;
    return bits;
}

// Words of the bitmap: whole 16-byte vectors.
__host__ __device__ __forceinline__ int64_t words_of(int32_t num_pages) { return ((int64_t)num_pages + 127) / 128 * 4; }

// stays = the pages that `held` names and the bits behind the last page, which nothing moves or gives away; used
// begins as the same.
__global__ void __launch_bounds__(256) begin_kernel(const PageMapArgs a) {
    let_next_start();
    const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (w >= words_of(a.num_pages)) return;
    const int64_t left = a.num_pages - 32 * w;
    const uint32_t bits = held_word(a, 32 * w) | (left >= 32 ? 0u : left > 0 ? 0xffffffffu << left : 0xffffffffu);
    a.used_bits[w] = bits;
    if (a.stay_bits) a.stay_bits[w] = bits;
}

// Marks the pages of a unit in a bitmap (in global or in shared memory).
__device__ __forceinline__ void mark_unit(const PageMapArgs &a, const Unit &x, uint32_t *bitmap) {
    bool bad = false;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const bool has = x.has(k), fine = has && x.id[k] >= 0 && x.id[k] < a.num_pages;
        bad |= has && !fine;
        // Neighbouring pages, as a list in ascending order hands them out, are bits of one word, and the atomics on a
        // word are taken one by one: where runs of lanes have a word in common, the first lane of a run marks for
        // all (256 requests over 2048 common pages in a row: 315 -> 16 us).
        const int word = fine ? x.id[k] >> 5 : -1 - lane;
        uint32_t bits = 1u << (x.id[k] & 31);
        bool marks = fine;
        const uint32_t heads = __ballot_sync(0xffffffffu, lane == 0 | word != __shfl_up_sync(0xffffffffu, word, 1));
        if (__popc(heads) <= 16) {
            const uint32_t later = heads & ~((2u << lane) - 1);
            const int end = later ? __ffs(later) - 1 : 32;   // of the lane's run
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_down_sync(0xffffffffu, bits, o);
                if (lane + o < end) bits |= y;
            }
            marks = fine && heads >> lane & 1;
        }
        if (marks) atomicOr(bitmap + word, bits);
    }
    if (bad) report(a.status, MSGL_DEVERR_PAGE_RANGE);
}

__global__ void __launch_bounds__(kThreads) mark_kernel(const PageMapArgs a) {
    __shared__ Batch s;
    for_entries(a, s, gridDim.x, true, [] { wait_for_last(); let_next_start(); }, [&](const Unit &x) { mark_unit(a, x, a.used_bits); });
}

// ----------------------------------------------------------------- the lists

// Sums over the whole block of up to three numbers; every thread gets them.  Not called twice without a barrier
// of the caller's between.
template <int W, int N>
__device__ __forceinline__ void block_sums(uint32_t (&x)[N], uint32_t (*part)[W]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __reduce_add_sync(0xffffffffu, x[i]);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[i][warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __reduce_add_sync(0xffffffffu, lane < W ? part[i][lane] : 0);
}

__device__ __forceinline__ uint32_t ones(const uint4 &x) { return __popc(x.x) + __popc(x.y) + __popc(x.z) + __popc(x.w); }

// out[place + i] = the i-th page of a word's set bits; most: entries from there on are not written.
__device__ __forceinline__ void write_bits(uint32_t word, int64_t page, uint32_t place, int32_t *out, uint32_t most) {
    const int lane = threadIdx.x & 31;
    const uint32_t to = place + __popc(word & ((1u << lane) - 1));
    if (word >> lane & 1 && to < most) out[to] = (int32_t)(page + lane);
}

// -1 in out[from, to), by all threads of the grid.
__device__ __forceinline__ void fill(int32_t *out, int64_t from, int64_t to, int threads) {
    const int64_t me = (int64_t)blockIdx.x * threads + threadIdx.x, all = (int64_t)gridDim.x * threads;
    const int64_t head = min(to, from + (-((reinterpret_cast<uintptr_t>(out) >> 2) + (uint64_t)from) & 3));
    const int64_t quads = (to - head) / 4, tail = head + 4 * quads;
    if (me < head - from) out[from + me] = -1;
    if (me < to - tail) out[tail + me] = -1;
    for (int64_t i = me; i < quads; i += all) *reinterpret_cast<int4 *>(out + head + 4 * i) = make_int4(-1, -1, -1, -1);
}

// A block's share of the words.  It goes over them a block of threads at a time: a thread looks at one, a scan says where
// its pages go, and then each warp writes every 16th word's.  (Every warp scanning for itself saves two barriers, but
// warps with the same scan keep the SM's issue slots busy: 6.7 against 5.7 us for the list of 740 thousand pages.)
struct Share {
    int64_t w0, w1, words, first;    // first: where the cluster's shares begin
};
__device__ __forceinline__ Share share_of(const PageMapArgs &a, int rank) {
    Share s;
    s.words = words_of(a.num_pages);
    const int64_t each = ((s.words + gridDim.x - 1) / gridDim.x + 31) / 32 * 32;
    s.w0 = min((int64_t)blockIdx.x * each, s.words);
    s.w1 = min(s.w0 + each, s.words);
    s.first = min((int64_t)(blockIdx.x - rank) * each, s.words);
    return s;
}

// The part of one or two bitmaps that a block counts for its cluster: an eighth of the vectors.  The first kHold a
// thread stay in its registers from count to count (all of them up to a million pages).
template <bool kBoth>
struct Slice {
    static constexpr int kHold = 2;
    const uint4 *x, *y;
    int64_t v0, v1;
    uint4 r[kHold], s[kHold];
    __device__ __forceinline__ uint4 at(const uint4 *from, int64_t v) const {
        return from && v < v1 ? __ldcg(from + v) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const uint32_t *x_, const uint32_t *y_, int64_t words, int rank) {
        x = reinterpret_cast<const uint4 *>(x_);
        y = kBoth ? reinterpret_cast<const uint4 *>(y_) : nullptr;
        const int64_t each = (words / 4 + kCluster - 1) / kCluster;
        v0 = min(rank * each, words / 4) + threadIdx.x;
        v1 = min((rank + 1) * each, words / 4);
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            r[i] = at(x, v0 + i * kThreads);
            if (kBoth) s[i] = at(y, v0 + i * kThreads);
        }
    }
    // f(first word, four words of x, four of y)
    template <class F>
    __device__ __forceinline__ void each(bool both, F f) const {
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (v0 + i * kThreads < v1) f(4 * (v0 + i * kThreads), r[i], s[i]);
        constexpr int kTogether = kBoth ? 2 : 4;
        for (int64_t v = v0 + kHold * kThreads; v < v1; v += kTogether * kThreads) {
            uint4 p[kTogether], q[kTogether];
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                p[i] = at(x, v + i * kThreads);
                if (kBoth) q[i] = at(both ? y : nullptr, v + i * kThreads);
            }
#pragma unroll
            for (int i = 0; i < kTogether; ++i)
                if (v + i * kThreads < v1) f(4 * (v + i * kThreads), p[i], q[i]);
        }
    }
};

// x summed over the threads before this one of a block of W warps; all: over the whole block.
template <int W>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t (&part)[W], uint32_t &all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t upto = warp_scan(x);
    if (lane == 31) part[warp] = upto;
    __syncthreads();
    const uint32_t w = lane < W ? part[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + upto - x;
}

// Up to four numbers of every block of the cluster, in all of them.  The blocks are known to run (cluster_started) before
// one writes into another's shared memory, and none is written to when it may have ended.
struct Peers {
    uint4 of[kCluster];
    __device__ __forceinline__ void put(int rank, const uint4 &x) {
        if (threadIdx.x >= kCluster) return;
        asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(peer_address(of + rank, threadIdx.x)),
                     "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                     : "memory");
    }
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2) free_list_kernel(const PageMapArgs a) {
    __shared__ uint32_t part[3][kWarps], words[kThreads], places[kThreads];
    __shared__ Peers peers;
    cluster_started();
    const int warp = threadIdx.x >> 5, rank = cluster_rank();
    const Share s = share_of(a, rank);
    wait_for_last();
    auto load = [&](int64_t w0) { return w0 + threadIdx.x < s.w1 ? ~__ldcg(a.used_bits + w0 + threadIdx.x) : 0u; };
    Slice<false> slice;
    slice.load(a.used_bits, nullptr, s.words, rank);
    uint32_t word = load(s.w0);
    uint32_t n[3] = {0, 0, (uint32_t)__popc(word)};   // free pages: of the slice before the cluster's shares, of all of it; of the share
    for (int64_t w0 = s.w0 + kThreads; w0 < s.w1; w0 += kThreads) n[2] += __popc(load(w0));
    slice.each(false, [&](int64_t w, const uint4 &x, const uint4 &) {
        const uint32_t free = 128 - ones(x);
        n[1] += free;
        if (w < s.first) n[0] += free;
    });
    block_sums<kWarps>(n, part);
    cluster_wait();
    peers.put(rank, make_uint4(n[0], n[1], n[2], 0));
    cluster_arrive();
    cluster_wait();
    uint32_t place = 0, total = 0, all;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
        const uint4 x = peers.of[k];
        place += x.x + (k < rank ? x.z : 0);
        total += x.y;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.count_out[0] = (int32_t)total;
    for (int64_t w0 = s.w0; w0 < s.w1; w0 += kThreads) {
        if (w0 > s.w0) word = load(w0);
        __syncthreads();
        const uint32_t before = block_scan<kWarps>(__popc(word), part[0], all);
        words[threadIdx.x] = word;
        places[threadIdx.x] = place + before;
        __syncthreads();
        const int mine = (int)min((int64_t)kThreads, s.w1 - w0);
        for (int i = warp; i < mine; i += kWarps) write_bits(words[i], 32 * (w0 + i), places[i], a.pages_out, 0xffffffffu);
        place += all;
    }
    fill(a.pages_out, total, a.num_pages, kThreads);
}

// The pages of word w in front of page `used`.
__device__ __forceinline__ uint32_t below(uint32_t used, int64_t w) {
    const int64_t left = (int64_t)used - 32 * w;
    return left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1 : 0;
}

// The moves: the movable pages from page `used` on go to the free pages in front of it, both in order.  Leaves for
// every word which of its pages move, and the number of moves before them.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2) moves_kernel(const PageMapArgs a) {
    __shared__ uint32_t part[5][kWarps], used_words[kThreads];
    __shared__ uint4 words[kThreads];
    __shared__ Peers peers[3];
    cluster_started();
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank();
    const Share s = share_of(a, rank);
    wait_for_last();
    uint32_t u, stays;
    auto load = [&](int64_t w) {
        u = w < s.w1 ? __ldcg(a.used_bits + w) : 0xffffffffu;
        stays = w < s.w1 ? __ldcg(a.stay_bits + w) : 0xffffffffu;
    };
    Slice<true> slice;
    slice.load(a.used_bits, a.stay_bits, s.words, rank);
    load(s.w0 + threadIdx.x);
    uint32_t n[1] = {0};
    slice.each(false, [&](int64_t, const uint4 &x, const uint4 &) { n[0] += ones(x); });
    block_sums<kWarps>(n, part);
    cluster_wait();
    peers[0].put(rank, make_uint4(n[0], 0, 0, 0));
    cluster_arrive();
    cluster_wait();
    uint32_t used = (uint32_t)a.num_pages - (uint32_t)(32 * s.words);
#pragma unroll
    for (int k = 0; k < kCluster; ++k) used += peers[0].of[k].x;
    // moves of the slice before the cluster's shares, holes there, all its moves; moves and holes of the share
    uint32_t m[5] = {0, 0, 0, 0, 0};
    slice.each(true, [&](int64_t w, const uint4 &x, const uint4 &y) {
        if (32 * (w + 4) <= used) {
            if (w < s.first) m[1] += 128 - ones(x);
            return;
        }
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t front = below(used, w + i), moves = __popc(xs[i] & ~ys[i] & ~front);
            m[2] += moves;
            if (w < s.first) {
                m[0] += moves;
                m[1] += __popc(~xs[i] & front);
            }
        }
    });
    uint32_t front, moves, holes;
    auto look = [&](int64_t w) {
        front = below(used, w);
        moves = u & ~stays & ~front;
        holes = ~u & front;
    };
    for (int64_t w = s.w0 + threadIdx.x + kThreads; w - threadIdx.x < s.w1; w += kThreads) {   // (large pools)
        const uint32_t u0 = u, stays0 = stays;
        load(w);
        look(w);
        m[3] += __popc(moves);
        m[4] += __popc(holes);
        u = u0, stays = stays0;
    }
    look(s.w0 + threadIdx.x);
    m[3] += __popc(moves);
    m[4] += __popc(holes);
    __syncthreads();
    block_sums<kWarps>(m, part);
    peers[1].put(rank, make_uint4(m[0], m[1], m[2], 0));
    peers[2].put(rank, make_uint4(m[3], m[4], 0, 0));
    cluster_arrive();
    cluster_wait();
    uint32_t from = 0, to = 0, total = 0, all_moves, all_holes;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
        const uint4 x = peers[1].of[k], y = peers[2].of[k];
        from += x.x + (k < rank ? y.x : 0);
        to += x.y + (k < rank ? y.y : 0);
        total += x.z;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.count_out[0] = (int32_t)total;
        a.used_out[0] = (int32_t)used;
    }
    for (int64_t w0 = s.w0; w0 < s.w1; w0 += kThreads) {
        const int64_t w = w0 + threadIdx.x;
        if (w0 > s.w0) {
            load(w);
            look(w);
        }
        __syncthreads();
        const uint32_t moved = from + block_scan<kWarps>(__popc(moves), part[0], all_moves),
                       filled = to + block_scan<kWarps>(__popc(holes), part[1], all_holes);
        if (w < s.w1) a.moves[w] = make_uint2(moves, moved);
        words[threadIdx.x] = make_uint4(moves, moved, holes, filled);
        used_words[threadIdx.x] = u;
        __syncthreads();
        const int mine = (int)min((int64_t)kThreads, s.w1 - w0);
        for (int i = warp; i < mine; i += kWarps) {
            const uint4 x = words[i];
            const int64_t page = 32 * (w0 + i) + lane;
            write_bits(x.x, page - lane, x.y, a.src, total);
            write_bits(x.z, page - lane, x.w, a.dst, total);
            if (page < a.num_pages && !(x.x >> lane & 1)) a.pages_out[page] = used_words[i] >> lane & 1 ? (int32_t)page : -1;
        }
        from += all_moves;
        to += all_holes;
    }
    fill(a.src, total, a.num_pages / 2, kThreads);
    fill(a.dst, total, a.num_pages / 2, kThreads);
}

// The new ids of a unit's pages: one that moves takes the place of its number among the moves (by words of 32 pages: which
// of them move, and the moves before them; in global or in shared memory).
__device__ __forceinline__ void rename_unit(const PageMapArgs &a, const Unit &x, const uint2 *moves) {
    // (an id that was given out here, in a row that is named twice, is of a page that does not move)
    int32_t to[kPerLane];                                      // the move's number, -1: none
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const int32_t id = x.has(k) ? x.id[k] : -1;
        const bool may = id >= 0 && id < a.num_pages;
        // (through L1: requests that share pages look up the same words)
        const uint2 m = may ? moves[id >> 5] : make_uint2(0, 0);
        const uint32_t bit = 1u << (id & 31);
        to[k] = m.x & bit ? (int32_t)(m.y + __popc(m.x & (bit - 1))) : -1;
    }
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
        if (to[k] >= 0) to[k] = a.dst[to[k]];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
        if (x.has(k) && (to[k] >= 0 || a.table_out != a.table)) a.table_out[x.place(a, k)] = to[k] >= 0 ? to[k] : x.id[k];
}

// The new ids: of all pages in the requests' tables (the first entry_blocks blocks), and of those that move in the
// map (the others).
__global__ void __launch_bounds__(kThreads) rename_kernel(const PageMapArgs a, int entry_blocks) {
    __shared__ Batch s;
    if (blockIdx.x >= entry_blocks) {
        wait_for_last();
        const int moves = __ldcg(a.count_out), blocks = gridDim.x - entry_blocks;
        for (int64_t i = (int64_t)(blockIdx.x - entry_blocks) * kThreads + threadIdx.x; i < moves; i += (int64_t)blocks * kThreads)
            a.pages_out[__ldcg(a.src + i)] = __ldcg(a.dst + i);
        return;
    }
    for_entries(a, s, entry_blocks, false, [] { wait_for_last(); }, [&](const Unit &x) { rename_unit(a, x, a.moves); });
}

// --------------------------------------------------------------- small pools

// All of it in one launch, for small pools and tables: a cluster of 8 blocks, each of which marks its share of the
// entries in a bitmap in its own shared memory, joins all 8 (so that each knows every page), and lists and renames
// its share.  Free pages of 64 requests in 15 thousand pages: 6.8 -> 4.8 us in a graph, launched one by one 8.7 ->
// 6.5; compaction of 32 requests in 13 thousand: 9.0 -> 7.9 and 12.3 -> 10.3.  At 32 thousand pages the three or
// four launches are level in a graph (free 5.9 to 7.4 against 5.2 to 6.7, compaction 9.3 to 10.6 against 9.4 to 11.2), at
// 60 thousand ahead (free 6.0 against 6.6).
constexpr int kSmallWords = 1024, kSmallUnits = 2 * kCluster * kWarps;
static_assert(kSmallWords == 2 * kThreads, "two words a thread");

// 8 bytes out of another block's shared memory.
__device__ __forceinline__ uint2 ld_peer(const void *p, int rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(peer_address(p, rank)) : "memory");
    return v;
}

template <bool kCompact>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) small_pool_kernel(const PageMapArgs a) {
    __shared__ __align__(16) uint32_t mine[kSmallWords], held[kSmallWords / kCluster], used[kSmallWords];
    __shared__ uint32_t places[kSmallWords];
    __shared__ uint2 moves[kCompact ? kSmallWords : 1];
    __shared__ uint32_t part[2][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank(), t2 = 2 * threadIdx.x;
    const int words = (int)words_of(a.num_pages), share = (words / 2 + kCluster - 1) / kCluster * 2;
    const int w0 = min(rank * share, words), w1 = min(w0 + share, words);
    const int chunks = max(1, (a.table_width + kUnit - 1) / kUnit), units = a.num_reqs * chunks;
    *reinterpret_cast<uint2 *>(mine + t2) = make_uint2(0, 0);
    // the pages held beside the requests' and the bits behind the last page: this block's share
    for (int w = w0 + threadIdx.x; w < w1; w += kThreads) {
        const int64_t left = (int64_t)a.num_pages - 32 * w;
        held[w - w0] = held_word(a, 32 * w) | (left >= 32 ? 0u : left > 0 ? 0xffffffffu << left : 0xffffffffu);
    }
    Unit x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = rank + kCluster * (warp + i * kWarps), b = u / chunks;
        x[i].c0 = (u - b * chunks) * kUnit;
        x[i].n = u < units ? entries_of(a, b, x[i].c0 == 0 && lane == 0, x[i].row) : 0;
        x[i].load(a);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (rank + kCluster * (warp + i * kWarps) < units) mark_unit(a, x[i], mine);
    cluster_arrive();
    cluster_wait();
    // two words a thread: of all blocks' marks, and of the block that looked up what is held there
    uint32_t u[2] = {}, st[2] = {0xffffffffu, 0xffffffffu};
    if (t2 < words) {
        const uint2 h = ld_peer(held + t2 % share, t2 / share);
        st[0] = h.x, st[1] = h.y;
        uint2 v[kCluster];
#pragma unroll
        for (int k = 0; k < kCluster; ++k) v[k] = ld_peer(mine + t2, k);
#pragma unroll
        for (int k = 0; k < kCluster; ++k) u[0] |= v[k].x, u[1] |= v[k].y;
    }
    // (no block leaves while another may still read its bitmap)
    cluster_arrive();
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] |= st[i];
    if constexpr (!kCompact) {
        uint32_t all, n = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) n += __popc(~u[i]);
        uint32_t place = block_scan<kWarps>(n, part[0], all);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            used[t2 + i] = u[i];
            places[t2 + i] = place;
            place += __popc(~u[i]);
        }
        __syncthreads();
        for (int w = w0 + warp; w < w1; w += kWarps) write_bits(~used[w], 32ll * w, places[w], a.pages_out, 0xffffffffu);
        fill(a.pages_out, all, a.num_pages, kThreads);
        if (rank == 0 && threadIdx.x == 0) a.count_out[0] = (int32_t)all;
        cluster_wait();
    } else {
        uint32_t n[1] = {0};
#pragma unroll
        for (int i = 0; i < 2; ++i) n[0] += __popc(u[i]);
        block_sums<kWarps>(n, part);
        const uint32_t total = n[0] - (uint32_t)(32 * kSmallWords - a.num_pages);
        uint32_t go = 0, to = 0, all_go, all_to;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t front = below(total, t2 + i);
            go += __popc(u[i] & ~st[i] & ~front);
            to += __popc(~u[i] & front);
        }
        __syncthreads();
        uint32_t from = block_scan<kWarps>(go, part[0], all_go), place = block_scan<kWarps>(to, part[1], all_to);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t front = below(total, t2 + i), go = u[i] & ~st[i] & ~front;
            used[t2 + i] = u[i];
            moves[t2 + i] = make_uint2(go, from);
            places[t2 + i] = place;
            from += __popc(go);
            place += __popc(~u[i] & front);
        }
        __syncthreads();
        for (int w = w0 + warp; w < w1; w += kWarps) {
            const uint2 m = moves[w];
            const int page = 32 * w + lane;
            write_bits(m.x, 32ll * w, m.y, a.src, all_go);
            write_bits(~used[w] & below(total, w), 32ll * w, places[w], a.dst, all_go);
            if (page < a.num_pages && !(m.x >> lane & 1)) a.pages_out[page] = used[w] >> lane & 1 ? page : -1;
        }
        fill(a.src, all_go, a.num_pages / 2, kThreads);
        fill(a.dst, all_go, a.num_pages / 2, kThreads);
        if (rank == 0 && threadIdx.x == 0) {
            a.count_out[0] = (int32_t)all_go;
            a.used_out[0] = (int32_t)total;
        }
        cluster_wait();
        // (the moves of all blocks are there)
        cluster_arrive();
        cluster_wait();
        for (uint32_t i = rank * kThreads + threadIdx.x; i < all_go; i += kCluster * kThreads)
            a.pages_out[__ldcg(a.src + i)] = __ldcg(a.dst + i);
#pragma unroll
        for (int i = 0; i < 2; ++i) rename_unit(a, x[i], moves);
    }
}

bool takes_small(const PageMapArgs &a) {
    const int64_t chunks = a.table_width > 0 ? (a.table_width + kUnit - 1) / kUnit : 1;
    return words_of(a.num_pages) <= kSmallWords && a.num_reqs * chunks <= kSmallUnits;
}

template <class... A>
cudaError_t launch_after(void (*kernel)(A...), int blocks, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Sets and marks the bitmaps; entry_blocks: for the kernels that go over the table entries.
cudaError_t launch_marks(const PageMapArgs &a, int entry_blocks, cudaStream_t stream) {
    begin_kernel<<<(unsigned)(words_of(a.num_pages) / 256 + 1), 256, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_after(mark_kernel, entry_blocks, kThreads, stream, a) : e;
}

// A block for every kWarps units that full rows would have, at most two an SM.  An odd number, so that the chunks of a
// long row do not all fall to the same blocks.
int entry_blocks(const PageMapArgs &a) {
    const int64_t chunks = a.table_width > 0 ? (a.table_width + kUnit - 1) / kUnit : 1;
    const int64_t want = ((int64_t)a.num_reqs * chunks + kWarps - 1) / kWarps, most = 2 * sm_count() - 1;
    return (int)(want < most ? want : most) | 1;
}

// A block for every 32 words, in whole clusters, at most 2 in a GPC (of 19 SMs on average): they start beside the blocks
// that still mark, where twice as many wait for room (740 thousand pages: free 13.4 against 15.1 us, compaction 14.6
// against 15.4).  Twice as many where a block would go over its share in several rounds (8 million pages: 15.7 against
// 21.7 and 40 against 51).
int list_blocks(const PageMapArgs &a) {
    const int64_t words = words_of(a.num_pages), want = (words + 32 * kCluster - 1) / (32 * kCluster);
    const int64_t gpcs = (sm_count() + 18) / 19, most = (words > 2 * gpcs * kCluster * kThreads ? 4 : 2) * gpcs;
    return kCluster * (int)(want < 1 ? 1 : want < most ? want : most);
}

// A thread for every four moves that there may be, at most a block an SM.
int move_blocks(const PageMapArgs &a) {
    const int64_t want = a.num_pages / 2 / (4 * kThreads) + 1;
    return (int)(want < sm_count() ? want : sm_count());
}

}  // namespace

size_t page_map_workspace_bytes(int32_t num_pages) {
    return ((size_t)words_of(num_pages) * 4 * 4 + 255) / 256 * 256;
}

static void set_workspace(PageMapArgs &a, void *workspace, bool compact) {
    a.used_bits = static_cast<uint32_t *>(workspace);
    a.stay_bits = compact ? a.used_bits + words_of(a.num_pages) : nullptr;
    a.moves = compact ? reinterpret_cast<uint2 *>(a.stay_bits + words_of(a.num_pages)) : nullptr;
}

cudaError_t launch_free_pages(PageMapArgs a, void *workspace, cudaStream_t stream) {
    if (takes_small(a)) {
        small_pool_kernel<false><<<kCluster, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    set_workspace(a, workspace, false);
    cudaError_t e = launch_marks(a, entry_blocks(a), stream);
    return e == cudaSuccess ? launch_after(free_list_kernel, list_blocks(a), kThreads, stream, a) : e;
}

cudaError_t launch_compact_pages(PageMapArgs a, void *workspace, cudaStream_t stream) {
    if (takes_small(a)) {
        small_pool_kernel<true><<<kCluster, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    set_workspace(a, workspace, true);
    const int blocks = entry_blocks(a);
    cudaError_t e = launch_marks(a, blocks, stream);
    if (e == cudaSuccess) e = launch_after(moves_kernel, list_blocks(a), kThreads, stream, a);
    return e == cudaSuccess ? launch_after(rename_kernel, blocks + move_blocks(a), kThreads, stream, a, blocks) : e;
}

}  // namespace msgl
