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

// Shared-prefix decode: the keys of request b that only it attends, and the first of them.  A
// request with a neighbour in its group starts behind the shared keys; entries that break the
// group rules give no keys (the merge reports them).
__device__ __forceinline__ int own_keys_shared(const int32_t *seq_lens, const int32_t *group_start,
                                               const int32_t *shared_lens, int num_reqs, int max_seq, int b,
                                               int &first) {
    const int s = seq_valid(seq_lens, b, max_seq);
    const bool grouped = __ldg(group_start + b) != b || (b + 1 < num_reqs && __ldg(group_start + b + 1) == b);
    first = grouped ? __ldg(shared_lens + b) : 0;
    return first >= 0 && first <= s ? s - first : 0;
}

// The rows of a shared-prefix decode.  A group's rows are cut into pairs of Q tiles of pair_rows / 2
// rows each (the tiles of its tensor-core kernel; pair_rows = 2 * floor(128 / G)).
struct GroupRows {
    const int32_t *seq_lens, *group_start, *shared_lens;
    int32_t num_reqs, max_seq_len, pair_rows;
};

constexpr int kPrefixTileKeys = 128;

// 128-key tiles of shared keys of the pair that starts at row b; 0 when none does.  Whatever the
// group arrays hold, the entries used (group_start[b], shared_lens[b]) are in range.
__device__ __forceinline__ int pair_tiles(const GroupRows &r, int b) {
    const int lead = __ldg(r.group_start + b), s = __ldg(r.shared_lens + b);
    const int next = b + 1 < r.num_reqs ? __ldg(r.group_start + b + 1) : -1;
    const bool starts = lead >= 0 && lead <= b && (b - lead) % r.pair_rows == 0 && (lead != b || next == b);
    return starts && s > 0 && s <= r.max_seq_len ? (s + kPrefixTileKeys - 1) / kPrefixTileKeys : 0;
}

// The status bits of row b: its length, the rules of group_start and shared_lens, and that the
// pair it belongs to can be worked on.  start: its first own key; pair: its pair's first row (-1:
// no shared keys).
__device__ __forceinline__ uint32_t group_row_errors(const GroupRows &r, int b, int &seq, int &start, int &pair) {
    seq = __ldg(r.seq_lens + b);
    start = 0;
    pair = -1;
    if (seq < 1 || seq > r.max_seq_len) return MSGL_DEVERR_LENGTH;
    const int lead = __ldg(r.group_start + b);
    if (lead == b && !(b + 1 < r.num_reqs && __ldg(r.group_start + b + 1) == b)) return 0;   // alone
    const int s = __ldg(r.shared_lens + b);
    if (lead < 0 || lead > b || s < 0 || s > seq) return MSGL_DEVERR_GROUP;
    if (lead != b && (__ldg(r.group_start + b - 1) != lead || __ldg(r.group_start + lead) != lead ||
                      __ldg(r.shared_lens + lead) != s))
        return MSGL_DEVERR_GROUP;
    start = s;
    if (s == 0) return 0;
    const int half = r.pair_rows / 2;
    pair = lead + (b - lead) / r.pair_rows * r.pair_rows;
    if (__ldg(r.group_start + pair) != lead || __ldg(r.shared_lens + pair) != s || pair_tiles(r, pair) == 0)
        return MSGL_DEVERR_GROUP;
    if (b - pair >= half && __ldg(r.group_start + pair + half) != lead) return MSGL_DEVERR_GROUP;
    return 0;
}

// All keys of row b where the shared ones are read through its group's first row; 0 when its
// entries are out of range.  from: the first key that is read through its own.
__device__ __forceinline__ int through_keys(const GroupRows &r, int b, int *from = nullptr) {
    int split;
    const int own = own_keys_shared(r.seq_lens, r.group_start, r.shared_lens, r.num_reqs, r.max_seq_len, b, split);
    const int lead = __ldg(r.group_start + b);
    if (from) *from = split;
    const int s = seq_valid(r.seq_lens, b, r.max_seq_len);
    return lead >= 0 && lead <= b && split >= 0 && own + split == s ? s : 0;
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
    int from;
    s.own += own_keys_shared(r.seq_lens, r.group_start, r.shared_lens, r.num_reqs, r.max_seq_len, i, from);
    s.all += through_keys(r, i);
    const int t = pair_tiles(r, i);
    if (t > 0) {
        s.tiles += t + (1ll << kPairShift);
        if (__ldg(r.group_start + i) == i) s.shared += __ldg(r.shared_lens + i);
    }
}

// Whether the kernel that reads shared keys once for their group pays (whole nanoseconds, so that
// every kernel of a call comes to the same answer).  Without it the split kernel reads them once a
// request, which after the first comes out of L2: the call takes what HBM needs for the keys in the
// pool or what L2 needs for all that are attended.  With it, HBM's time for the requests' own
// keys, a fixed part (start, first tile, pieces, join) and the tiles.  Measured: 6.4 TB/s from
// HBM, 10.5 TB/s from L2, 14 us, 1.5 us a tile and SM.
__device__ __forceinline__ bool prefix_pays(const BatchSums &s, int hkv, int sms) {
    const long long key = (long long)hkv * kHeadDim * 4;   // bytes
    const long long through = max((s.own + s.shared) * key / 6400, s.all * key / 10500);
    const long long prefix = s.own * key / 6400 + 14000 + (s.tiles & kTilesMask) * hkv * 1500 / sms;
    return prefix < through;
}

// A batch as one block sees it: thread i has rows [b0, b1) = [i * k, (i + 1) * k).  `before` counts
// the keys (all and own) and tiles of the rows before b0.  scratch: 4 entries per warp, not used
// again before the block's next barrier.
struct BatchScan {
    int b0, b1;
    BatchSums before, mine, total;
};

template <int kMaxWarps>
__device__ __forceinline__ void scan_batch(const GroupRows &r, long long (*scratch)[4], BatchScan &s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
    const int k = (r.num_reqs + threads - 1) / threads;
    s.b0 = min(r.num_reqs, (int)threadIdx.x * k);
    s.b1 = min(r.num_reqs, s.b0 + k);
    s.mine = BatchSums{0, 0, 0, 0};
    for (int b = s.b0; b < s.b1; ++b) add_row(r, b, s.mine);
    long long x[4] = {s.mine.all, s.mine.own, s.mine.tiles, s.mine.shared};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += u;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 4; ++i) scratch[warp][i] = x[i];
    __syncthreads();
    long long before[4], total[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        before[i] = x[i];
        total[i] = 0;
    }
    const int warps = threads >> 5;
#pragma unroll
    for (int w = 0; w < kMaxWarps; ++w)
        if (w < warps)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long y = scratch[w][i];
                total[i] += y;
                if (w < warp) before[i] += y;
            }
    s.before = BatchSums{before[0] - s.mine.all, before[1] - s.mine.own, 0, before[2] - s.mine.tiles};
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
