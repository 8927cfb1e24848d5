// Shared device helpers for libmsgl_attn (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/msgl_attn.h"

namespace msgl {

constexpr int kHeadDim = 128;          // the only head_dim the kernels are built for
constexpr int kMaxGroup = 64;          // largest q-heads-per-kv-head ratio supported
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// View of the pool as the kernels use it.
struct PoolView {
    const __nv_bfloat16 *k;
    const __nv_bfloat16 *v;
    int64_t num_slots;
    int32_t num_pages;   // num_slots / page_size
    int32_t log2_ps;     // page_size = 1 << log2_ps
    int32_t hkv;
};

struct PageView {
    const int32_t *ids;
    int32_t stride;
    int32_t width;
};

// Slot of key j of request b, or -1 (and *bad set) when the page index or id is out of range.
__device__ __forceinline__ int64_t slot_of(const PoolView &pool, const PageView &pt, int b, int j,
                                           bool &bad) {
    const int pidx = j >> pool.log2_ps;
    if (pidx >= pt.width) { bad = true; return -1; }
    const int pid = __ldg(pt.ids + (int64_t)b * pt.stride + pidx);
    if (pid < 0 || pid >= pool.num_pages) { bad = true; return -1; }
    return ((int64_t)pid << pool.log2_ps) + (j & ((1 << pool.log2_ps) - 1));
}

__device__ __forceinline__ void report(uint32_t *status, uint32_t bits) {
    if (status) atomicOr(status, bits);
}

__device__ __forceinline__ int seq_valid(const int32_t *seq_lens, int b, int max_seq) {
    const int s = __ldg(seq_lens + b);
    return (s >= 1 && s <= max_seq) ? s : 0;
}

// Keys per CTA range: an equal share, but at least two tiles, so that a small
// batch does not scatter into hundreds of tiny partials for the merge to fold.
constexpr long long kMinKeysPerCta = 32;
__host__ __device__ __forceinline__ long long keys_per_cta(long long total, long long ctas) {
    const long long share = (total + ctas - 1) / ctas;
    return share > kMinKeysPerCta ? share : kMinKeysPerCta;
}

// The same where requests may have a few keys each (behind a shared prefix): a request begun costs a
// range more than a tile, so the least share is the requests' average (37 requests of 1 key: 37 ranges
// in place of 2, 55 -> 24 us).
__device__ __forceinline__ long long grouped_keys_per_cta(long long total, long long ctas, int num_reqs) {
    const long long share = (total + ctas - 1) / ctas, least = min(kMinKeysPerCta, max(total / num_reqs, 1ll));
    return max(share, least);
}

// The rows of a shared-prefix decode.  A group's rows are cut into pairs of Q tiles of pair_rows / 2
// rows each (the tiles of its tensor-core kernel; pair_rows = 2 * floor(128 / G)).
struct GroupRows {
    const int32_t *seq_lens, *group_start, *shared_lens;
    int32_t num_reqs, max_seq_len, pair_rows;
};

constexpr int kPrefixTileKeys = 128;

// What the arrays say of row b (all loads at once: one after the other, as the rules below need them,
// they are most of the time that a CTA's count of the batch takes).
struct GroupRow {
    int32_t b, seq, lead, next, shared;   // next: the group of row b + 1, -1 behind the last row
};

__device__ __forceinline__ GroupRow group_row_at(const GroupRows &r, int b) {
    const int after = min(b + 1, r.num_reqs - 1);
    GroupRow x{b, __ldg(r.seq_lens + b), __ldg(r.group_start + b), __ldg(r.group_start + after), __ldg(r.shared_lens + b)};
    if (after == b) x.next = -1;
    return x;
}

__device__ __forceinline__ int valid_seq(const GroupRows &r, const GroupRow &x) {
    return x.seq >= 1 && x.seq <= r.max_seq_len ? x.seq : 0;
}

// The keys that only row x.b attends, and the first of them.  A request with a neighbour in its group
// starts behind the shared keys; entries that break the group rules give no keys (the merge reports
// them).
__device__ __forceinline__ int own_keys(const GroupRows &r, const GroupRow &x, int &first) {
    const int s = valid_seq(r, x);
    first = x.lead != x.b || x.next == x.b ? x.shared : 0;
    return first >= 0 && first <= s ? s - first : 0;
}

// All keys of row x.b where the shared ones are read through its group's first row; 0 when its
// entries are out of range.  from: the first key that is read through its own.
__device__ __forceinline__ int through_keys(const GroupRows &r, const GroupRow &x, int &from) {
    const int own = own_keys(r, x, from), s = valid_seq(r, x);
    return x.lead >= 0 && x.lead <= x.b && from >= 0 && own + from == s ? s : 0;
}

// 128-key tiles of shared keys of the pair that starts at row x.b; 0 when none does.  Whatever the
// group arrays hold, the entries used (group_start[b], shared_lens[b]) are in range.
__device__ __forceinline__ int pair_tiles(const GroupRows &r, const GroupRow &x) {
    const bool starts = x.lead >= 0 && x.lead <= x.b && (x.b - x.lead) % r.pair_rows == 0 &&
                        (x.lead != x.b || x.next == x.b);
    return starts && x.shared > 0 && x.shared <= r.max_seq_len ? (x.shared + kPrefixTileKeys - 1) / kPrefixTileKeys : 0;
}

// The status bits of row x.b: its length, the rules of group_start and shared_lens, and that the
// pair it belongs to can be worked on.  start: its first own key; pair: its pair's first row (-1:
// no shared keys).
__device__ __forceinline__ uint32_t group_row_errors(const GroupRows &r, const GroupRow &x, int &start, int &pair) {
    start = 0;
    pair = -1;
    if (valid_seq(r, x) == 0) return MSGL_DEVERR_LENGTH;
    const int b = x.b, lead = x.lead, s = x.shared;
    if (lead == b && x.next != b) return 0;   // alone
    if (lead < 0 || lead > b || s < 0 || s > x.seq) return MSGL_DEVERR_GROUP;
    const int half = r.pair_rows / 2, first = lead + (b - lead) / r.pair_rows * r.pair_rows;
    const int before = __ldg(r.group_start + max(b - 1, 0)), lead_lead = __ldg(r.group_start + lead),
              lead_shared = __ldg(r.shared_lens + lead), second = __ldg(r.group_start + min(first + half, b));
    const GroupRow p = group_row_at(r, first);
    if (lead != b && (before != lead || lead_lead != lead || lead_shared != s)) return MSGL_DEVERR_GROUP;
    start = s;
    if (s == 0) return 0;
    pair = first;
    if (p.lead != lead || p.shared != s || pair_tiles(r, p) == 0) return MSGL_DEVERR_GROUP;
    if (b - first >= half && second != lead) return MSGL_DEVERR_GROUP;
    return 0;
}

// What a batch asks for.
struct BatchSums {
    long long all, own;      // keys attended, and those of them that are not shared
    long long shared;        // shared keys, each group's once
    long long tiles;         // key tiles of all pairs, and (kPairShift) the pairs
};
constexpr int kPairShift = 44;
constexpr long long kTilesMask = (1ll << kPairShift) - 1;

__device__ __forceinline__ void add_row(const GroupRows &r, int i, BatchSums &s) {
    const GroupRow x = group_row_at(r, i);
    int from;
    s.own += own_keys(r, x, from);
    s.all += through_keys(r, x, from);
    const int t = pair_tiles(r, x);
    if (t > 0) {
        s.tiles += t + (1ll << kPairShift);
        if (x.lead == i) s.shared += x.shared;
    }
}

// What a call's kernels know of each other's cost (in whole numbers, so that all of them come to
// the same answer).  Measured: HBM gives 6.4 TB/s; a split CTA starts within 5 us, takes a 16-key tile
// of its heads in tile_ns out of L2 or HBM (0.93 us for page boxes of 8 heads, 0.5 us for per-key rows
// of one head and 0.1 us more for each further one) and 0.6 us more for every request it begins; a
// prefix CTA takes 8 us to its first scores and out of its last piece, 1.55 us for a key tile (2.35 us
// while the other SMs saturate HBM) and 2.5 us for every item it begins.
struct ShareModel {
    int32_t sms;               // CTAs of the prefix grid, one an SM
    int32_t gx, ngr;           // the split's grid: key ranges, groups of kv heads
    int32_t tile_ns;
    int32_t always;            // MSGL_SHARE_ALWAYS
};

// The SMs' shares: `prefix` of them take the groups' shared keys, the others the requests' own
// (`split` key ranges for each group of heads).  prefix = 0: the split takes all keys, the shared
// ones once a request.
struct Share {
    int32_t prefix, split;
};

// Sharing reads less but has two kernels to feed, so each gets SMs of its own: the split is bound
// by HBM with two thirds of them, and the prefix kernel's fixed cost is paid by the others only.
// Every lane prices some of the partitions; the cheapest one is taken, the one with fewer prefix
// CTAs (fewer pieces to join) among equals.
__device__ __forceinline__ Share share_plan(const BatchSums &s, const ShareModel &m, int hkv, int num_reqs) {
    const long long units = (s.tiles & kTilesMask) * hkv, items = (s.tiles >> kPairShift) * hkv;
    if (m.sms == 0 || units == 0) return Share{0, m.gx};
    // times in units of 64 ns (of SMs: up to 68 s)
    auto t64 = [](long long ns) -> uint32_t { return (uint32_t)min(ns >> 6, 1ll << 30); };
    const uint32_t hbm = t64((s.own + s.shared) * (hkv * kHeadDim * 4) / 6400);
    // (a request's own keys end in a tile that is half empty on average)
    const uint32_t own = t64((s.own / 16 + num_reqs / 2) * m.tile_ns + num_reqs * 600ll);
    const uint32_t all = t64((s.all / 16 + num_reqs / 2) * m.tile_ns + num_reqs * 600ll);
    const uint32_t pre = t64(units * 1550 + items * 2500), crowded = t64(units * 800);
    constexpr uint32_t kPrefixStart = 8000 / 64, kSplitStart = 5000 / 64, kJoin = 3000 / 64;
    // (32 candidates, closer together where there are few: a CTA more or less matters most there)
    uint32_t best = 0xffffffffu;   // the time, then the prefix CTAs
    const int lane = threadIdx.x & 31, most = m.sms - m.ngr;
    const int p = 1 + lane + max(most - 32, 0) * lane * lane / 961;
    if (p <= most) {
        const uint32_t k = min((m.sms - p) / m.ngr, m.gx);
        const uint32_t t = max(kPrefixStart + (pre + crowded / 100 * min(m.sms - p, 100)) / p,
                               kSplitStart + max(hbm, own / k));
        best = min(t, (1u << 23) - 1) << 8 | p;
    }
    best = __reduce_min_sync(0xffffffffu, best);
    const uint32_t through = kSplitStart + max(hbm, all / m.gx);
    // (kJoin: for the pieces that sharing adds to the join)
    if (best == 0xffffffffu || (!m.always && through <= (best >> 8) + kJoin))
        return m.always ? Share{m.sms, m.gx} : Share{0, m.gx};
    const int n = best & 255;
    return Share{n, min((m.sms - n) / m.ngr, m.gx)};
}

// A batch as one block sees it: thread i has rows [b0, b1) = [i * k, (i + 1) * k).  `before` counts
// the keys (all and own) and tiles of the rows before b0.  scratch: 4 entries per warp, not used
// again before the block's next barrier.
struct BatchScan {
    int b0, b1;
    BatchSums before, mine, total;
};

__device__ __forceinline__ void scan_batch(const GroupRows &r, long long (*scratch)[4], BatchScan &s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
    const int k = (r.num_reqs + threads - 1) / threads;
    s.b0 = min(r.num_reqs, (int)threadIdx.x * k);
    s.b1 = min(r.num_reqs, s.b0 + k);
    s.mine = BatchSums{0, 0, 0, 0};
    for (int b = s.b0; b < s.b1; ++b) add_row(r, b, s.mine);
    // (rolled loops: this runs at the start of every CTA, where each line of code not yet in the
    // instruction cache costs more than the loop)
    long long x[4] = {s.mine.all, s.mine.own, s.mine.tiles, s.mine.shared};
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long u = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += u;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 4; ++i) scratch[warp][i] = x[i];
    __syncthreads();
    long long total[4] = {0, 0, 0, 0};
    const int warps = threads >> 5;
#pragma unroll 1
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long y = scratch[w][i];
            total[i] += y;
            if (w < warp) x[i] += y;
        }
    s.before = BatchSums{x[0] - s.mine.all, x[1] - s.mine.own, 0, x[2] - s.mine.tiles};
    s.total = BatchSums{total[0], total[1], total[3], total[2]};
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint4 ld_stream_16(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

__device__ __forceinline__ void st_stream_16(void *p, uint4 r) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(r.x), "r"(r.y),
                 "r"(r.z), "r"(r.w)
                 : "memory");
}

}  // namespace msgl
