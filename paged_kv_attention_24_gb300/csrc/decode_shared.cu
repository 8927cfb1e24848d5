// Shared-prefix decode: one query row per request, groups of requests over one prefix.
//
// "Mini-SGLang 实战指南", §6.5 "Radix Cache": requests with a common prefix hold
// the same pages; §6.3 and §6.4: decode has its own kernels and is replayed
// under CUDA graphs, so every launch shape depends on host scalars only.
//
// A row's softmax over its keys is split in two: the keys its group shares and
// its own.  Each part gives (o, lse); o = sum w_i o_i / sum w_i with w_i =
// exp(lse_i - max lse) joins them, as it joins the pieces of each part.
//
// * Own keys: the decode's split kernel (decode.cu), its ranges laid over the
//   rows' own keys only.  Bound by HBM.
// * Shared keys: n rows x G q heads of one kv head against the same keys, a
//   matrix product with n * G rows per K/V byte, on the tensor cores
//   (prefix_tc_kernel).  The keys of a group are read once per 256 packed rows
//   (and from L2 after the first) instead of once per request.
// * The merge joins all pieces of a row.
//
// Each of the first two has SMs of its own (share_plan in common.cuh prices the
// partitions; every CTA counts the batch and comes to the same one).  The split
// is launched behind the prefix kernel with programmatic dependent launch, so
// its CTAs start on the SMs that the plan leaves free while the prefix kernel
// works on the others; its last CTA outwaits the prefix kernel, so that the merge
// behind it finds both done.
//
// Reading a shared key once a request is not much worse than it sounds: after the
// first it comes out of L2, and the split kernel takes 10 to 13 TB/s from there
// (0.73 to 0.93 us for a 64 KB tile and SM) against 6.4 from HBM.  So the plan also prices
// the split kernel alone, small batches skip the rest (kThroughBytes), and short
// requests take a kernel of a single launch (decode_short.cu).  Sharing pays when
// the groups are large: 256 requests over 32768 shared tokens, 64 q heads: 0.23 ms
// with, 2.5 ms without; 32 groups of 8 over up to 1024 (page size 1): 115 and 147 us;
// 64 requests over 2048 of about 5600: 161 us either way (floor 142).
#include <cuda.h>
#include <limits.h>
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"

namespace msgl {

namespace {

// ------------------------------------------------------------------ the rows
// A group's rows are cut into pairs of Q tiles: a tile packs R = 128 / G rows x the G q
// heads of a kv head, a pair 2R rows.  A unit of work is one 128-key tile for one pair and
// kv head; units are numbered pair by pair (in row order), head by head, tile by tile, and
// CTA c takes units [c * per, (c + 1) * per).  share_plan() says how many CTAs have any.

constexpr int kRows = 128;                 // rows per Q tile (MMA M)
constexpr int kKeys = kPrefixTileKeys;     // keys per K/V tile
constexpr int kMaxPrefixCtas = 160;        // bound on the grid, sizes the workspace

// ------------------------------------------------------------- prefix kernel
constexpr int kStages = 2;                 // K tiles in flight
constexpr int kVStages = 3;                // V tiles in flight (V is needed later than K)
constexpr int kLoadWarps = 4;              // they load and issue; 8 softmax warps behind them
constexpr int kThreads = 32 * (kLoadWarps + 8);
constexpr uint32_t kHalf = 16384;          // 128 rows x 128 bytes (64 bf16)
constexpr uint32_t kTile = 2 * kHalf;      // 128 x 128 bf16
constexpr uint32_t kVBlock = 4096, kVHalf = 2048;   // V in blocks of 16 keys (see extend.cu)
constexpr int kMaxSegs = 32;               // segments of one window of a CTA's units
constexpr int kBadRing = 8;                // segments the loaders can be ahead, rounded up

// One pair of Q tiles and one kv head against a run of key tiles.
struct Seg {
    int32_t row, lead, shared;             // pair's first row, group's first row, shared keys
    int32_t g2;                            // 2 * kv head + (the second Q tile has rows)
    int32_t t0, n;                         // first key tile, key tiles
};

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTile;
constexpr uint32_t kOffV = kOffK + kStages * kTile;
constexpr uint32_t kOffBar = kOffV + kVStages * kTile;
constexpr uint32_t kOffSegs = kOffBar + 256;
constexpr uint32_t kOffX = kOffSegs + kMaxSegs * sizeof(Seg);
constexpr uint32_t kSmemBytes = kOffX + kRows * 8 + 1024;   // + slack to align the base to 1024
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
static_assert(kOffX % 16 == 0, "alignment of the exchange");

// barrier slots
constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = 4, kVFull = 6, kVEmpty = 9, kSFull = 12, kPFull = 14,
              kOFull = 16, kXFull = 18, kDrain = 19, kNumBars = 20;

// What the merge needs to know of a row, written by the prefix kernel's last CTA (a plan kernel in
// front of everything cost 6 to 8 us more than counting the batch in every CTA).
struct RowPlan {
    int32_t err, start;                    // status bits; first own key
    int32_t in_pair;                       // row within its pair of Q tiles, -1: no shared keys
    int32_t own_pieces;                    // pieces of the split kernel's
    int64_t own_slot;                      // its first piece's row of the split's partials
    int64_t unit;                          // units before the row
    int64_t unit_of_pair;                  // units before its pair
};

struct PrefixArgs {
    PoolView pool;
    PageView pages;
    GroupRows rows;
    int32_t hq, group, rows_per_tile, q_box_rows, oob_row, box_rows, v_blocks;
    ShareModel share;
    float scale_log2;
    float *o, *lse;            // [num_reqs, hq, 128], [num_reqs, hq]: pieces that begin at the first key
    float *cont_o, *cont_lse;  // [CTA, 2, 128, 128], [CTA, 2, 128]: a CTA's piece that begins later
    RowPlan *plan;             // [num_reqs]
    int64_t *per_cta;          // [1]
    uint32_t *status;
};

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                              uint32_t *status) {
    if (ptx::mbar_wait(bar, parity)) return true;
    report(status, MSGL_DEVERR_TIMEOUT);
    *abort_flag = 1;
    return false;
}

// The two halves of the block run to this one from different places.
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// A warp's walk over a CTA's units, segment by segment.
struct Walk {
    int32_t row, tiles;       // the current pair's first row and key tiles
    int32_t off;              // next unit, counted from the pair's first
    long long left;           // units to go

    // The first pair at or behind row r; tiles = 0 when there is none.
    __device__ __forceinline__ void find(const GroupRows &rows, int r) {
        const int lane = threadIdx.x & 31;
        tiles = 0;
        for (; r < rows.num_reqs; r += 32) {
            const int t = r + lane < rows.num_reqs ? pair_tiles(rows, group_row_at(rows, r + lane)) : 0;
            const unsigned m = __ballot_sync(0xffffffffu, t > 0);
            if (m) {
                row = r + __ffs(m) - 1;
                tiles = __shfl_sync(0xffffffffu, t, __ffs(m) - 1);
                return;
            }
        }
    }
    // Stands on unit `at + skip`, where `at` units lie before row r.
    __device__ __forceinline__ void start(const GroupRows &rows, int hkv, int r, long long skip, long long units) {
        left = units;
        for (find(rows, r); tiles > 0; find(rows, row + 1)) {
            const long long here = (long long)tiles * hkv;
            if (skip < here) break;
            skip -= here;
        }
        off = (int)skip;
    }
    __device__ __forceinline__ bool next(const GroupRows &rows, int hkv, Seg &s) {
        if (left <= 0) return false;
        if (off == tiles * hkv) {
            find(rows, row + 1);
            off = 0;
        }
        if (tiles == 0) return false;   // (the lengths changed under the call)
        s.row = row;
        s.lead = __ldg(rows.group_start + row);
        s.shared = __ldg(rows.shared_lens + row);
        const int second = row + rows.pair_rows / 2;
        const int two = second < rows.num_reqs && __ldg(rows.group_start + second) == s.lead;
        const int g = off / tiles;
        s.g2 = 2 * g + two;
        s.t0 = off - g * tiles;
        s.n = (int)min((long long)(tiles - s.t0), left);
        off += s.n;
        left -= s.n;
        return true;
    }
    // The next segments, as many as fit.
    __device__ __forceinline__ int fill(const GroupRows &rows, int hkv, Seg *segs) {
        int n = 0;
        Seg s;
        while (n < kMaxSegs && next(rows, hkv, s)) {
            if ((threadIdx.x & 31) == 0) segs[n] = s;
            ++n;
        }
        return n;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap kt_map,
                     const __grid_constant__ CUtensorMap vt_map, const PrefixArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the split kernel may take the SMs that this grid leaves free
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool last_cta = blockIdx.x == gridDim.x - 1;

    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + kOffBar;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + kOffBar + 8 * kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 4);
    volatile int *num_segs = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 8);
    volatile int *more_segs = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 12);
    volatile int *bad_seg = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 16);   // [kBadRing]
    Walk *saved_walk = reinterpret_cast<Walk *>(smem + kOffBar + 8 * kNumBars + 16 + 4 * kBadRing);
    static_assert(8 * kNumBars + 16 + 4 * kBadRing + sizeof(Walk) <= 256, "barrier block");
    Seg *segs = reinterpret_cast<Seg *>(smem + kOffSegs);
    float2 *xchg = reinterpret_cast<float2 *>(smem + kOffX);            // (m, l) of stream 1's rows
    long long(*scratch)[4] = reinterpret_cast<long long(*)[4]>(smem + kOffX);   // of the block's scan

    const GroupRows &rows = a.rows;
    const int hkv = a.pool.hkv;
    const int R = a.rows_per_tile, G = a.group;

    // ---- this CTA's units; none when the split kernel takes the shared keys too
    BatchScan batch;
    scan_batch(rows, scratch, batch);
    const Share share = share_plan(batch.total, a.share, hkv, rows.num_reqs);
    const bool pays = share.prefix > 0;
    const long long before = (batch.before.tiles & kTilesMask) * hkv, mine = (batch.mine.tiles & kTilesMask) * hkv;
    const long long units = pays ? (batch.total.tiles & kTilesMask) * hkv : 0;
    const long long per = pays ? (units + share.prefix - 1) / share.prefix : 1;
    const long long u0 = per * blockIdx.x, u1 = min(units, u0 + per);
    // (a CTA with nothing to do frees its SM for the split as soon as it can; the last one lays out
    // the merge's plan)
    if (u0 >= u1 && !last_cta) return;

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(kQFull), 1);
        ptx::mbar_init(bar(kQEmpty), 1);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar(kKFull + s), 1);
            ptx::mbar_init(bar(kKEmpty + s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            ptx::mbar_init(bar(kVFull + s), 1);
            ptx::mbar_init(bar(kVEmpty + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bar(kSFull + t), 1);
            ptx::mbar_init(bar(kPFull + t), 4);
            ptx::mbar_init(bar(kOFull + t), 1);
        }
        ptx::mbar_init(bar(kXFull), 4);
        ptx::mbar_init(bar(kDrain), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (threadIdx.x < kBadRing) bad_seg[threadIdx.x] = 0;
    if (warp == 2) {
        ptx::tc_alloc(ptx::smem_u32((const void *)tmem_slot), 512);
        ptx::tc_relinquish();
    }
    if (warp == 3) {
        // zero the Q rows a TMA box does not cover (GQA padding rows)
        const int used = a.q_box_rows * G;
        const int pad_bytes = (kRows - used) * 128;
        for (int t = 0; t < 2; ++t)
            for (int h = 0; h < 2; ++h) {
                uint8_t *p = smem + kOffQ + t * kTile + h * kHalf + used * 128;
                for (int x = lane * 16; x < pad_bytes; x += 32 * 16)
                    *reinterpret_cast<uint4 *>(p + x) = make_uint4(0, 0, 0, 0);
            }
        ptx::fence_proxy_async_smem();
    }

    // the warp whose rows hold the first unit lays out the first segments
    const unsigned owner = __ballot_sync(0xffffffffu, u0 < u1 && before <= u0 && u0 < before + mine);
    if (owner) {
        const int l = __ffs(owner) - 1;
        Walk walk;
        walk.start(rows, hkv, __shfl_sync(0xffffffffu, batch.b0, l), __shfl_sync(0xffffffffu, u0 - before, l), u1 - u0);
        const int n = walk.fill(rows, hkv, segs);
        if (lane == 0) {
            *num_segs = n;
            *more_segs = walk.left > 0 && n > 0;
            *saved_walk = walk;
        }
    }

    if (last_cta) {
        // the rows' places among the pieces, for the merge
        const long long split_per = grouped_keys_per_cta(pays ? batch.total.own : batch.total.all, share.split, rows.num_reqs);
        long long at = pays ? batch.before.own : batch.before.all, unit = before;
        for (int b = batch.b0; b < batch.b1; ++b) {
            a.plan[b].unit = unit;
            unit += (long long)pair_tiles(rows, group_row_at(rows, b)) * hkv;
        }
        __threadfence_block();
        __syncthreads();
        for (int b = batch.b0; b < batch.b1; ++b) {
            int start, pair, first;
            const GroupRow x = group_row_at(rows, b);
            const int n = pays ? own_keys(rows, x, first) : through_keys(rows, x, first);
            const long long c0 = at / split_per;
            a.plan[b].err = (int32_t)group_row_errors(rows, x, start, pair);
            if (!pays) pair = -1;
            a.plan[b].start = start;
            a.plan[b].in_pair = pair >= 0 ? b - pair : -1;
            a.plan[b].own_pieces = n > 0 ? (int)((at + n - 1) / split_per - c0) + 1 : 0;
            a.plan[b].own_slot = b + c0;
            a.plan[b].unit_of_pair = pair >= 0 ? __ldcg(&a.plan[pair].unit) : 0;
            at += n;
        }
        if (threadIdx.x == 0) *a.per_cta = per;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (u0 >= u1) {
        if (warp == 2) ptx::tc_dealloc(tmem, 512);
        return;
    }

    // Every role counts segments and K/V tiles the same way.  A segment with rows in both Q
    // tiles runs them as two streams over the same key tiles; one with rows in the first only
    // runs the even and the odd key tiles as two streams, joined at its end.  Either way one
    // stream's softmax overlaps the other's products.
    const bool lsu = a.box_rows == 0;
    uint32_t seg = 0, tile0 = 0;
    bool ok = true;
    // When a list of segments is used up, warp 0 lays out the next; both halves of the block meet
    // before it and after.  False at the end, or when a role gave up (all agree: its flag was set
    // before the barrier).
    auto next_segs = [&]() -> bool {
        if (!*more_segs) return false;
        __syncwarp();   // (the barrier counts whole warps)
        block_sync();
        if (*abort_flag) return false;
        if (warp == 0) {
            Walk walk = *saved_walk;
            const int n = walk.fill(rows, hkv, segs);
            __syncwarp();
            if (lane == 0) {
                *num_segs = n;
                *more_segs = walk.left > 0 && n > 0;
                *saved_walk = walk;
            }
        }
        block_sync();
        return true;
    };

    // (registers: 128 x 104 + 256 x 200 = 384 x 168, what the block was launched with)
    if (warp < kLoadWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // MMA issuer: stages and parities of the next K, V and P to use
        uint32_t ks = 0, kpar = 0, vs = 0, vpar = 0, ppar0 = 0, ppar1 = 0;
        do {
            const int count = *num_segs;
            for (int e = 0; e < count && ok; ++e) {
                const Seg p = segs[e];
                const int g = p.g2 >> 1, n = p.n;
                const bool two = p.g2 & 1;
                if (warp == 2) {
                    // ---------------------------------------------------- Q loader
                    if (seg > 0)
                        ok = __all_sync(0xffffffffu, wait_or_abort(bar(kQEmpty), (seg & 1) ^ 1, abort_flag, a.status));
                    if (ok && lane == 0) {
                        const uint32_t box = 64u * G * a.q_box_rows * 2u;
                        ptx::mbar_arrive_expect_tx(bar(kQFull), box * (two ? 4u : 2u));
                        for (int t = 0; t < (two ? 2 : 1); ++t)
                            for (int h = 0; h < 2; ++h)
                                ptx::tma_load_3d(sbase + kOffQ + t * kTile + h * kHalf, &q_map, 64 * h, g * G,
                                                 p.row + t * R, bar(kQFull));
                    }
                }
                if (warp == 0 || warp == 3 || (lsu && warp == 2 && ok)) {
                    // ---------------------------------------------------- K/V loaders
                    const bool is_v = warp >= 3;
                    // Pool rows of tile j's keys, four consecutive keys per lane.  A key past the
                    // shared ones or behind a bad page id gets oob_row (zero fill).
                    auto key_rows = [&](int j, int (&kr)[4], bool &all_ok, int64_t &slot0) {
                        all_ok = true;
                        slot0 = 0;
                        bool bad = false;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int key = (p.t0 + j) * kKeys + 4 * lane + x;
                            kr[x] = a.oob_row;
                            bool badp = false;
                            const int64_t slot = key < p.shared ? slot_of(a.pool, a.pages, p.lead, key, badp) : -1;
                            if (slot >= 0) {
                                kr[x] = (int)(slot * hkv + g);
                                if (x == 0) slot0 = slot;
                            } else {
                                all_ok = false;
                            }
                            bad |= badp;
                        }
                        if (bad) bad_seg[seg % kBadRing] = (int)seg + 1;
                        __syncwarp();
                    };
                    int kr[4];
                    bool all_ok;
                    int64_t slot0;
                    if (lsu) {
                        // 16-byte cp.async copies into the SWIZZLE_128B K-major layout (see extend.cu).
                        // Warps 0 and 2 copy the K tiles of one stage each and hand a tile over when
                        // its copies have landed; warp 3 copies the V tiles and hands one over when its
                        // next has been issued.  Either way the copies of two tiles overlap.
                        const __nv_bfloat16 *pool = is_v ? a.pool.v : a.pool.k;
                        const int step = is_v ? 1 : 2;
                        const int first = is_v ? 0 : (int)((tile0 ^ (warp == 2 ? 1u : 0u)) & 1u);
                        const int hi = lane >> 4, c = lane & 15;
                        const uint32_t col_off = (uint32_t)(c >> 3) * kHalf;
                        if (first < n) key_rows(first, kr, all_ok, slot0);
                        for (int j = first; j < n && ok; j += step) {
                            const uint32_t gi = tile0 + j;
                            const uint32_t st = is_v ? gi % kVStages : gi % kStages;
                            const uint32_t round = is_v ? gi / kVStages : gi / kStages;
                            ok = __all_sync(0xffffffffu, !*abort_flag &&
                                                             wait_or_abort(bar((is_v ? kVEmpty : kKEmpty) + st),
                                                                           (round & 1) ^ 1, abort_flag, a.status));
                            if (!ok) break;
                            const uint32_t dst = sbase + (is_v ? kOffV : kOffK) + st * kTile;
#pragma unroll 16
                            for (int i = 0; i < 64; ++i) {
                                const int r0 = __shfl_sync(0xffffffffu, (i & 1) ? kr[2] : kr[0], i >> 1);
                                const int r1 = __shfl_sync(0xffffffffu, (i & 1) ? kr[3] : kr[1], i >> 1);
                                const int row = hi ? r1 : r0;
                                const int r = 2 * i + hi;
                                const bool valid = row < a.oob_row;
                                ptx::cp_async_16(
                                    dst + col_off + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4),
                                    pool + (valid ? (int64_t)row * kHeadDim + c * 8 : 0), valid ? 16u : 0u);
                            }
                            ptx::cp_async_commit();
                            if (j + step < n) key_rows(j + step, kr, all_ok, slot0);
                            if (is_v && j > 0) {
                                // all but the newest copies have landed: hand over the tile before
                                asm volatile("cp.async.wait_group 1;" ::: "memory");
                                ptx::fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) ptx::mbar_arrive(bar(kVFull + (gi + kVStages - 1) % kVStages));
                            }
                            if (!is_v || j == n - 1) {
                                ptx::cp_async_wait_all();
                                ptx::fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) ptx::mbar_arrive(bar((is_v ? kVFull : kKFull) + st));
                            }
                        }
                    } else {
                        // TMA: a page that is a contiguous run of pool rows and holds shared keys only
                        // arrives in tiled copies issued by its first lane; any other 4-key group is
                        // gathered four rows at a time.
                        const int BR = a.box_rows;
                        const int lanes_per_box = BR / 4;
                        const int box_lead = (lane / lanes_per_box) * lanes_per_box;
                        const unsigned box_bits =
                            lanes_per_box >= 32 ? 0xffffffffu : ((1u << lanes_per_box) - 1u) << box_lead;
                        const CUtensorMap *gm = is_v ? &v_map : &k_map;
                        const CUtensorMap *tm = is_v ? &vt_map : &kt_map;
                        for (int j = 0; j < n && ok; ++j) {
                            key_rows(j, kr, all_ok, slot0);
                            const unsigned ok_mask = __ballot_sync(0xffffffffu, all_ok);
                            const bool tiled = (ok_mask & box_bits) == box_bits;
                            const uint32_t gi = tile0 + j;
                            const uint32_t st = is_v ? gi % kVStages : gi % kStages;
                            const uint32_t round = is_v ? gi / kVStages : gi / kStages;
                            ok = __all_sync(0xffffffffu, !*abort_flag &&
                                                             wait_or_abort(bar((is_v ? kVEmpty : kKEmpty) + st),
                                                                           (round & 1) ^ 1, abort_flag, a.status));
                            if (!ok) break;
                            const uint32_t full = bar((is_v ? kVFull : kKFull) + st);
                            // this lane's four keys: rows 4 lane .. 4 lane + 3 (K), or their place in V's blocks
                            const uint32_t dst = is_v ? sbase + kOffV + st * kTile + (uint32_t)(lane >> 2) * kVBlock +
                                                            (uint32_t)(lane & 3) * 512u
                                                      : sbase + kOffK + st * kTile + lane * 512;
                            const uint32_t half_off = is_v ? kVHalf : kHalf;
                            if (lane == 0) ptx::mbar_arrive_expect_tx(full, kTile);
                            __syncwarp();
                            if (!tiled) {
                                ptx::tma_gather4(dst, gm, 0, kr[0], kr[1], kr[2], kr[3], full);
                                ptx::tma_gather4(dst + half_off, gm, 64, kr[0], kr[1], kr[2], kr[3], full);
                            } else if (lane == box_lead) {
                                if (is_v) {
                                    for (int x = 0; x < (BR > 32 ? BR / 32 : 1); ++x)
                                        ptx::tma_load_5d(dst + (uint32_t)x * 2u * kVBlock, tm, 0, g,
                                                         (int)slot0 + 32 * x, 0, 0, full);
                                } else {
                                    ptx::tma_load_3d(dst, tm, 0, g, (int)slot0, full);
                                    ptx::tma_load_3d(dst + kHalf, tm, 64, g, (int)slot0, full);
                                }
                            }
                        }
                    }
                } else if (warp == 1) {
                    // ---------------------------------------------------- MMA issuer
                    if (lane == 0) {
                        constexpr uint32_t idesc_s = ptx::umma_idesc_bf16(128, 128, false, false);
                        constexpr uint32_t idesc_o = ptx::umma_idesc_bf16(128, 128, false, true);
                        const uint64_t qdesc = ptx::umma_desc_sw128(sbase + kOffQ, 16, 1024);
                        const uint64_t kdesc = ptx::umma_desc_sw128(sbase + kOffK, 16, 1024);
                        const uint64_t vdesc = ptx::umma_desc_sw128(sbase + kOffV, a.v_blocks ? kVHalf : kHalf, 1024);
                        const uint32_t vstep = (a.v_blocks ? kVBlock : 16u * 128u) >> 4;   // MMA kk's 16 keys
                        // The issuing thread keeps the tensor pipe's pace: each group tests the barrier
                        // that the next one needs after its 4th MMA, so that the test's latency hides
                        // behind the MMAs still queued (see extend.cu).
                        auto s_group = [&](int t, int q, uint32_t pb, uint32_t pp) -> bool {
                            const uint64_t qd = qdesc + (uint64_t)(q * (kTile >> 4));
                            const uint64_t kd = kdesc + (uint64_t)(ks * (kTile >> 4));
                            bool r = false;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                                ptx::tc_mma_ss(tmem + 128 * t, qd + o, kd + o, idesc_s, kk > 0);
                                if (kk == 3 && pb) r = ptx::mbar_test_wait(pb, pp);
                            }
                            ptx::tc_commit(bar(kSFull + t));
                            return r;
                        };
                        auto pv_group = [&](int t, bool acc, uint32_t pb, uint32_t pp) -> bool {
                            const uint64_t vd = vdesc + (uint64_t)(vs * (kTile >> 4));
                            bool r = false;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                ptx::tc_mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + kk * 8,
                                               vd + (uint64_t)(kk * vstep), idesc_o, (acc || kk > 0) ? 1u : 0u);
                                if (kk == 3 && pb) r = ptx::mbar_test_wait(pb, pp);
                            }
                            return r;
                        };
                        auto need = [&](bool tested, uint32_t b, uint32_t parity) -> bool {
                            if (!tested && !wait_or_abort(b, parity, abort_flag, a.status)) ok = false;
                            ptx::tc_fence_after();
                            return ok;
                        };
                        auto k_bar = [&]() -> uint32_t { return bar(kKFull) + 8u * ks; };
                        auto v_bar = [&]() -> uint32_t { return bar(kVFull) + 8u * vs; };
                        auto k_next = [&]() {
                            ks ^= 1u;
                            kpar ^= ks == 0 ? 1u : 0u;
                        };
                        auto v_next = [&]() {
                            vs = vs == kVStages - 1 ? 0 : vs + 1;
                            vpar ^= vs == 0 ? 1u : 0u;
                        };
                        bool v_ok = false;   // V's barrier was seen complete
                        if (need(false, bar(kQFull), seg & 1) && need(false, k_bar(), kpar)) {
                            s_group(0, 0, 0, 0);
                            if (two) {
                                // Per key tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
                                v_ok = s_group(1, 1, v_bar(), vpar);
                                k_next();
                                for (int j = 0; j + 1 < n; ++j) {
                                    if (!need(v_ok, v_bar(), vpar) || !need(false, bar(kPFull + 0), ppar0)) break;
                                    const bool k_ok = pv_group(0, j > 0, k_bar(), kpar);
                                    if (!need(k_ok, k_bar(), kpar)) break;
                                    const bool p_ok = s_group(0, 0, bar(kPFull + 1), ppar1);
                                    if (!need(p_ok, bar(kPFull + 1), ppar1)) break;
                                    pv_group(1, j > 0, 0, 0);
                                    v_next();
                                    v_ok = s_group(1, 1, v_bar(), vpar);
                                    k_next();
                                    ppar0 ^= 1u;
                                    ppar1 ^= 1u;
                                }
                                if (ok && need(v_ok, v_bar(), vpar) && need(false, bar(kPFull + 0), ppar0)) {
                                    const bool p_ok = pv_group(0, n > 1, bar(kPFull + 1), ppar1);
                                    ptx::tc_commit(bar(kOFull + 0));
                                    if (need(p_ok, bar(kPFull + 1), ppar1)) {
                                        pv_group(1, n > 1, 0, 0);
                                        ptx::tc_commit(bar(kOFull + 1));
                                        v_next();
                                        ppar0 ^= 1u;
                                        ppar1 ^= 1u;
                                    }
                                }
                            } else {
                                // Key tile j belongs to stream j & 1: PV_t(j), S_t(j+2)
                                k_next();
                                if (n > 1 && need(false, k_bar(), kpar)) {
                                    v_ok = s_group(1, 0, v_bar(), vpar);
                                    k_next();
                                }
                                for (int j = 0; j < n && ok; ++j) {
                                    const int t = j & 1;
                                    const bool more = j + 2 < n;
                                    if (!need(v_ok, v_bar(), vpar) ||
                                        !need(false, bar(kPFull + t), t ? ppar1 : ppar0))
                                        break;
                                    const bool k_ok = pv_group(t, j > 1, more ? k_bar() : 0u, kpar);
                                    v_next();
                                    v_ok = false;
                                    if (t) ppar1 ^= 1u;
                                    else ppar0 ^= 1u;
                                    if (!more) {
                                        ptx::tc_commit(bar(kOFull + t));
                                    } else {
                                        if (!need(k_ok, k_bar(), kpar)) break;
                                        v_ok = s_group(t, 0, v_bar(), vpar);
                                        k_next();
                                    }
                                }
                            }
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
                tile0 += n;
                ++seg;
            }
        } while (next_segs());
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // -------------------------------------------------------------- softmax
        const int t = (warp - kLoadWarps) >> 2;                 // stream of this warpgroup
        const int quad = warp & 3;
        const int r = quad * 32 + lane;                // TMEM lane = tile row
        const int tok_l = r / G, jh = r - tok_l * G;
        uint32_t spar = 0, opar = 0, xpar = 0;         // parities of the next S, O and exchange
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = lane_base + 128 * t;
        const uint32_t tO = lane_base + 256 + 128 * t;
        do {
            const int count = *num_segs;
            for (int e = 0; e < count && ok; ++e) {
                const bool two = segs[e].g2 & 1;
                const int n = segs[e].n, step = two ? 1 : 2;
                const int first = two ? 0 : t;         // this stream's key tiles: first, first + step, ...
                if (first < n) {
                    const int visible0 = segs[e].shared - segs[e].t0 * kKeys;   // keys from the first tile on
                    const int tok = segs[e].row + (two ? t * R : 0) + tok_l;
                    const bool valid =
                        tok_l < R && tok < rows.num_reqs && __ldg(rows.group_start + tok) == segs[e].lead;
                    // a warp without rows of the group leaves its P as it is: its rows of O are not used
                    const bool idle = !__any_sync(0xffffffffu, valid);
                    // The K/V stages are released from here: S(j) done means the MMAs issued before it
                    // are, so K(j) and the V of the stream's tile before are free (see extend.cu).  Two
                    // Q tiles read each K and V: the second stream releases both.
                    const bool releaser = lane == 0 && quad == 0 && (!two || t == 1);
                    float m_ref = -INFINITY, l = 0.f;
                    for (int j = first; j < n; j += step) {
                        ok = __all_sync(0xffffffffu, wait_or_abort(bar(kSFull + t), spar, abort_flag, a.status));
                        if (!ok) break;
                        spar ^= 1u;
                        ptx::tc_fence_after();
                        if (releaser) {
                            ptx::mbar_arrive(bar(kKEmpty + (tile0 + j) % kStages));
                            if (j != first) ptx::mbar_arrive(bar(kVEmpty + (tile0 + j - step) % kVStages));
                            if (j == n - 1) ptx::mbar_arrive(bar(kQEmpty));
                        }
                        if (!idle) {
                            uint32_t v[128];
                            ptx::tc_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(v + 0));
                            ptx::tc_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                            ptx::tc_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(v + 64));
                            ptx::tc_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(v + 96));
                            ptx::tc_wait_ld();
                            const int visible = visible0 - j * kKeys;   // keys of this tile that exist
                            if (visible < kKeys) {
#pragma unroll
                                for (int i = 0; i < 128; ++i)
                                    if (i >= visible) v[i] = __float_as_uint(-INFINITY);
                            }
                            auto row_max = [&]() -> float {
                                float mxa = -INFINITY, mxb = -INFINITY, mxc = -INFINITY, mxd = -INFINITY;
#pragma unroll
                                for (int i = 0; i < 128; i += 8) {
                                    mxa = ptx::max3(mxa, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                                    mxb = ptx::max3(mxb, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                                    mxc = ptx::max3(mxc, __uint_as_float(v[i + 4]), __uint_as_float(v[i + 5]));
                                    mxd = ptx::max3(mxd, __uint_as_float(v[i + 6]), __uint_as_float(v[i + 7]));
                                }
                                return fmaxf(fmaxf(mxa, mxb), fmaxf(mxc, mxd)) * a.scale_log2;
                            };
                            // The first tile's row max is the reference; it moves only when a row sum
                            // shows a score 2^8 above it (every p stays below 2^8; see extend.cu).
                            if (j == first) m_ref = fmaxf(m_ref, row_max());
                            float ls = 0.f;
#pragma unroll 1
                            for (int pass = 0;; ++pass) {
                                // P = 2^(s * scale_log2 - m_ref) (masked scores are -inf -> 0), back over S
                                // as bf16: at most half a step, 2^-8, of each weight, while the row sum
                                // takes the unrounded ones
                                const uint64_t sc2 = ptx::f2_pack(a.scale_log2, a.scale_log2);
                                const uint64_t nm2 = ptx::f2_pack(-m_ref, -m_ref);
                                uint64_t l2 = ptx::f2_pack(0.f, 0.f);
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    uint32_t pk[16];
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const int x = 32 * c + 2 * i;
                                        const uint64_t x2 = ptx::f2_fma(
                                            ptx::f2_pack(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sc2, nm2);
                                        float x0, x1;
                                        ptx::f2_unpack(x2, x0, x1);
                                        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
                                        l2 = ptx::f2_add(l2, ptx::f2_pack(p0, p1));
                                        pk[i] = ptx::pack_bf16(p0, p1);
                                    }
                                    ptx::tc_st16(tS + 16 * c, pk);
                                }
                                float la, lb;
                                ptx::f2_unpack(l2, la, lb);
                                ls = la + lb;
                                if (pass == 1 || j == first || __all_sync(0xffffffffu, ls < 256.f)) break;
                                const float m_new = fmaxf(m_ref, row_max());
                                const bool moves = m_new > m_ref + 8.f;
                                if (!__any_sync(0xffffffffu, moves)) break;
                                const float alpha = moves ? ptx::ex2(m_ref - m_new) : 1.f;
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    uint32_t o32[32];
                                    ptx::tc_ld32(tO + 32 * c, o32);
                                    ptx::tc_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        o32[i] = __float_as_uint(__uint_as_float(o32[i]) * alpha);
                                    ptx::tc_st32(tO + 32 * c, o32);
                                }
                                ptx::tc_wait_st();
                                l *= alpha;
                                if (moves) m_ref = m_new;
                            }
                            l += ls;
                            ptx::tc_wait_st();
                        }
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(kPFull + t));
                    }
                    if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kOFull + t), opar, abort_flag, a.status));
                    if (!ok) break;
                    opar ^= 1u;
                    ptx::tc_fence_after();
                    if (releaser)   // the V of this stream's last tile
                        ptx::mbar_arrive(bar(kVEmpty + (tile0 + first + (n - 1 - first) / step * step) % kVStages));
                    const bool join = !two && n > 1;   // the even and odd key tiles' streams are one piece
                    if (join && t == 1) {
                        // Stream 0 reads these rows' O from TMEM.  (No product overwrites them before
                        // stream 0 is through: the next segment's first PV waits for its P.)
                        xchg[r] = make_float2(m_ref, l);
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(kXFull));
                    } else {
                        float f0, f1 = 0.f;
                        if (join) {
                            ok = __all_sync(0xffffffffu, wait_or_abort(bar(kXFull), xpar, abort_flag, a.status));
                            if (!ok) break;
                            xpar ^= 1u;
                            ptx::tc_fence_after();
                            const float2 other = xchg[r];
                            const float m = fmaxf(m_ref, other.x);
                            f0 = ptx::ex2(m_ref - m);
                            f1 = ptx::ex2(other.x - m);
                            l = l * f0 + other.y * f1;
                            m_ref = m;
                            f0 /= l;
                            f1 /= l;
                        } else {
                            f0 = 1.f / l;
                        }
                        // this piece's o / l and lse, fp32
                        if (!idle) {
                            const bool bad = bad_seg[seg % kBadRing] == (int)seg + 1;
                            const int head = (segs[e].g2 >> 1) * G + jh;
                            const bool begins = segs[e].t0 == 0;
                            const long long at = begins ? (long long)tok * a.hq + head
                                                        : ((long long)blockIdx.x * 2 + t) * kRows + r;
                            float *dst = (begins ? a.o : a.cont_o) + at * kHeadDim;
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t o32[32];
                                ptx::tc_ld32(tO + 32 * c, o32);
                                ptx::tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o32[i] = __float_as_uint(__uint_as_float(o32[i]) * f0);
                                if (join) {
                                    uint32_t p32[32];
                                    ptx::tc_ld32(tO + 128 + 32 * c, p32);
                                    ptx::tc_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        o32[i] = __float_as_uint(fmaf(__uint_as_float(p32[i]), f1,
                                                                      __uint_as_float(o32[i])));
                                }
                                if (valid) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i) ptx::st_v8(dst + 32 * c + 8 * i, o32 + 8 * i);
                                }
                            }
                            // NaN marks a piece that met a bad page
                            if (valid)
                                (begins ? a.lse : a.cont_lse)[at] =
                                    bad || !(l > 0.f) ? __int_as_float(0x7fc00000) : (m_ref + log2f(l)) * kLn2;
                            if (bad && t == 0 && quad == 0 && lane == 0) report(a.status, MSGL_DEVERR_PAGE_RANGE);
                            ptx::tc_fence_before();
                        }
                    }
                }
                tile0 += n;
                ++seg;
            }
        } while (next_segs());
    }

    if (warp == 1 && lane == 0) {
        // every MMA issued above has completed once this fires
        ptx::tc_commit(bar(kDrain));
        ptx::mbar_wait(bar(kDrain), 0, 400000000LL);
    }
    if (*abort_flag) {
        // a wait gave up: leave time for the copies in flight to land before shared memory goes away
        if (lsu) ptx::cp_async_wait_all();
        const long long t_end = clock64() + 400000000LL;
        while (clock64() < t_end) __nanosleep(1000);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tc_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------- merge
// One warp per (request, q head), each lane 4 of the 128 dims.  A row's pieces are taken kAtOnce at
// a time (their lse and values loaded together), with a running maximum and sum.  Bound by latency and
// the rows in flight.  Large batches: four pieces, one round for most rows, four blocks an SM.  (With the
// next four pieces loaded while these are joined, three blocks fit: +1 to 1.5 us a call.  Six blocks
// spill: +3 us.)  256 requests of 64 q heads, 30 MB of pieces: 10 us of the call's 227.

constexpr int kMergeThreads = 256;

struct MergeArgs {
    int32_t hq, group, rows_per_tile;
    const RowPlan *plan;
    const int64_t *per_cta;                  // units per prefix CTA
    const float *part_o, *part_lse;          // own keys: rows of hq heads
    const float *pre_o, *pre_lse, *cont_o, *cont_lse;
    __nv_bfloat16 *o;
    float *lse;
    uint32_t *status;
};

__device__ __forceinline__ long long div_units(long long a, long long b) {
    return ((a | b) >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

template <int kAtOnce>
__global__ void __launch_bounds__(kMergeThreads, kAtOnce > 4 ? 1 : 4) shared_merge_kernel(const MergeArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int h = blockIdx.x * (kMergeThreads / 32) + warp;
    if (h >= a.hq) return;
    const long long row = (long long)b * a.hq + h;
    __nv_bfloat16 *orow = a.o + row * kHeadDim + lane * 4;
    // the plan and the pieces are complete and visible after this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RowPlan p = a.plan[b];
    if (p.err) {
        if (h == 0 && lane == 0) report(a.status, (uint32_t)p.err);
        *reinterpret_cast<uint2 *>(orow) = make_uint2(0u, 0u);
        if (lane == 0) a.lse[row] = -INFINITY;
        return;
    }
    // prefix pieces: the first where the item begins, then one per CTA that continues it
    int np = 0;
    long long cont0 = 0;   // the row of the first continuing piece (one CTA, 2 * kRows rows, further each)
    if (p.in_pair >= 0) {
        const int g = h / a.group;
        const int tiles = (p.start + kKeys - 1) / kKeys;
        const long long per = *a.per_cta;
        const long long u = p.unit_of_pair + (long long)g * tiles;
        const long long cta0 = div_units(u, per);
        np = (int)(div_units(u + tiles - 1, per) - cta0) + 1;
        const int t = p.in_pair / a.rows_per_tile;
        cont0 = ((cta0 + 1) * 2 + t) * kRows + (p.in_pair - t * a.rows_per_tile) * a.group + (h - g * a.group);
    }
    const int n = np + p.own_pieces;
    const float *own_lse = a.part_lse + p.own_slot * a.hq + h;
    const float *own_o = a.part_o + (p.own_slot * a.hq + h) * kHeadDim + lane * 4;
    auto load = [&](int i, float &x, float4 &v) {
        x = -INFINITY;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= n) return;
        const float *l, *o;
        if (i >= np) {
            l = own_lse + (long long)(i - np) * a.hq;
            o = own_o + (long long)(i - np) * a.hq * kHeadDim;
        } else if (i == 0) {
            l = a.pre_lse + row;
            o = a.pre_o + row * kHeadDim + lane * 4;
        } else {
            const long long at = cont0 + (long long)(i - 1) * 2 * kRows;
            l = a.cont_lse + at;
            o = a.cont_o + at * kHeadDim + lane * 4;
        }
        x = *l;
        v = *reinterpret_cast<const float4 *>(o);
    };
    float M = -INFINITY, L = 0.f, acc0 = 0.f, acc1 = 0.f, acc2 = 0.f, acc3 = 0.f;
    bool failed = false;
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
        float x[kAtOnce];
        float4 v[kAtOnce];
        float m = M;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) load(i0 + k, x[k], v[k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            failed |= isnan(x[k]);
            m = fmaxf(m, x[k]);
        }
        if (m > -INFINITY) {
            const float al = __expf(M - m);
            L *= al;
            acc0 *= al;
            acc1 *= al;
            acc2 *= al;
            acc3 *= al;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float w = __expf(x[k] - m);
                L += w;
                acc0 += w * v[k].x;
                acc1 += w * v[k].y;
                acc2 += w * v[k].z;
                acc3 += w * v[k].w;
            }
            M = m;
        }
    }
    const bool none = failed || !(L > 0.f);
    const float inv = none ? 0.f : 1.f / L;
    *reinterpret_cast<uint2 *>(orow) =
        none ? make_uint2(0u, 0u)
             : make_uint2(ptx::pack_bf16(acc0 * inv, acc1 * inv), ptx::pack_bf16(acc2 * inv, acc3 * inv));
    if (lane == 0) a.lse[row] = none ? -INFINITY : M + logf(L);
}

// Up to this many bytes of K/V to attend (by the host's bounds), the split kernel alone needs 14 to
// 22 us, and the prefix kernel would take longer than that for its start, one tile and the join.
constexpr long long kThroughBytes = 140ll << 20;

// Where the one-launch kernel of short requests is taken instead of the split and merge (by
// "never", and by "auto" up to kThroughBytes).  Up to 128 keys its blocks are small enough to keep
// several on an SM (about 128 keys, page size 1: 16/8 heads 64 requests 12.3 against 16.0 us, 2000
// requests 163 against 172, 256 to 600 requests 28 to 55 against 26 to 47; 64/8 and 16/2 heads ahead at
// every size, 35 against 41 and 15 against 23 us for 300 requests).  Batches of that kind beyond
// kThroughBytes go by the device's plan in three launches: 40 us in place of 55 for 600 requests of 16/8
// heads, 42 in place of 35 for 300 of 64/8, 76 in place of 54 for 2000 of 16/2.  Longer requests have an SM to themselves, or nearly: ahead as long as
// there are at most two a SM (512 keys, 8 kv heads: 8 requests 8.2 against 11.5 us at page size 1 and
// 13.8 at 16, 32 requests 13 against 17, 64 requests 23 against 21; 1024 keys: 16 requests 13.4 against
// 17, but 2 requests 12.6 against 11.9 at page size 1), and the split's many CTAs win on the longest.
bool takes_short(const DecodeArgs &d) {
    if (d.num_reqs > 65535) return false;
    const long long blocks = (long long)d.num_reqs * d.pool.hkv * ((d.hq / d.pool.hkv + 7) / 8);
    if (d.max_seq_len <= 128) return true;
    return blocks <= (d.max_seq_len <= 512 ? 2 : d.max_seq_len <= 1024 ? 1 : 0) * (long long)sm_count();
}

// Where each part of the workspace begins.
struct Layout {
    size_t pre_o, pre_lse, cont_o, cont_lse, plan, total;
};

Layout layout_of(int32_t num_reqs, int32_t hq, int32_t hkv) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)num_reqs * hq, cont = (size_t)kMaxPrefixCtas * 2 * kRows;
    Layout l;
    l.pre_o = plan_decode(num_reqs, hq, hkv, 1).workspace;
    l.pre_lse = l.pre_o + rows * kHeadDim * sizeof(float);
    l.cont_o = up(l.pre_lse + rows * sizeof(float));
    l.cont_lse = l.cont_o + cont * kHeadDim * sizeof(float);
    l.plan = up(l.cont_lse + cont * sizeof(float));   // units per CTA, then a RowPlan for each row
    l.total = up(l.plan + 256 + (size_t)num_reqs * sizeof(RowPlan));
    return l;
}

}  // namespace

size_t decode_shared_workspace_bytes(int32_t num_reqs, int32_t hq, int32_t hkv) {
    return layout_of(num_reqs, hq, hkv).total;
}

cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream) {
    DecodeArgs d = a.dec;
    const int hkv = d.pool.hkv, G = d.hq / hkv, R = kRows / G;
    const DecodePlan plan = plan_decode(d.num_reqs, d.hq, hkv, d.max_seq_len);
    d.pair_rows = 2 * R;
    const bool small =
        d.num_reqs == 1 || (long long)d.num_reqs * d.max_seq_len * hkv * kHeadDim * 4 <= kThroughBytes;
    if (a.sharing == MSGL_SHARE_NEVER || (a.sharing == MSGL_SHARE_AUTO && small))
        return takes_short(d) ? launch_decode_short(d, stream) : launch_decode(d, plan, stream);
    d.share = decode_split_model(d.hq, d.pool);
    d.share.sms = sm_count() < kMaxPrefixCtas ? sm_count() : kMaxPrefixCtas;
    d.share.always = a.sharing == MSGL_SHARE_ALWAYS;
    const Layout l = layout_of(d.num_reqs, d.hq, hkv);
    char *ws = static_cast<char *>(a.workspace);
    AttnMaps m;
    cudaError_t e = encode_attn_maps(d.pool, d.q, d.hq, d.num_reqs, R, m);
    if (e != cudaSuccess) return e;
    static bool attr_set[64];   // per device; idempotent, racing setters write the same value
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }

    PrefixArgs p{};
    p.pool = d.pool;
    p.pages = d.pages;
    p.rows = GroupRows{d.seq_lens, d.group_start, d.shared_lens, d.num_reqs, d.max_seq_len, 2 * R};
    p.hq = d.hq;
    p.group = G;
    p.rows_per_tile = R;
    p.q_box_rows = m.q_box_rows;
    p.oob_row = m.oob_row;
    p.box_rows = m.box_rows;
    p.v_blocks = m.v_blocks;
    p.share = d.share;
    p.scale_log2 = d.scale * kLog2e;
    p.o = reinterpret_cast<float *>(ws + l.pre_o);
    p.lse = reinterpret_cast<float *>(ws + l.pre_lse);
    p.cont_o = reinterpret_cast<float *>(ws + l.cont_o);
    p.cont_lse = reinterpret_cast<float *>(ws + l.cont_lse);
    p.per_cta = reinterpret_cast<int64_t *>(ws + l.plan);
    p.plan = reinterpret_cast<RowPlan *>(ws + l.plan + 256);
    p.status = d.status;
    const int ctas = d.share.sms;
    prefix_tc_kernel<<<ctas, kThreads, kSmemBytes, stream>>>(m.q, m.k, m.v, m.kt, m.vt, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_decode(d, plan, stream, DecodePhase::kSplit);
    if (e != cudaSuccess) return e;

    MergeArgs g{};
    g.hq = d.hq;
    g.group = G;
    g.rows_per_tile = R;
    g.plan = p.plan;
    g.per_cta = p.per_cta;
    g.part_o = d.part_o;
    g.part_lse = d.part_lse;
    g.pre_o = p.o;
    g.pre_lse = p.lse;
    g.cont_o = p.cont_o;
    g.cont_lse = p.cont_lse;
    g.o = d.o;
    g.lse = d.lse;
    g.status = d.status;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3((d.hq + kMergeThreads / 32 - 1) / (kMergeThreads / 32), d.num_reqs);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    // (the pieces of a few rows are many each)
    const bool few = (long long)cfg.gridDim.x * cfg.gridDim.y <= 2ll * sm_count();
    return cudaLaunchKernelEx(&cfg, few ? shared_merge_kernel<16> : shared_merge_kernel<4>, g);
}

}  // namespace msgl
