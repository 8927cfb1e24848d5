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
// The prefix kernel is launched behind the split with programmatic dependent
// launch: its CTAs take each SM as the split's range there ends, and its last
// CTA outwaits the split, so that the merge behind it finds both done.
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
// CTA c takes units [c * per, (c + 1) * per).

constexpr int kRows = 128;                 // rows per Q tile (MMA M)
constexpr int kKeys = 128;                 // keys per K/V tile
constexpr int kMaxPrefixCtas = 160;        // bound on the grid, sizes the workspace
constexpr int kMinUnits = 2;               // K/V tiles per CTA at least: fewer pieces to join

struct Rows {
    const int32_t *seq_lens, *group_start, *shared_lens;
    int32_t num_reqs, max_seq_len;
    int32_t pair_rows;                     // 2R
};

// K/V tiles of the pair that starts at row b; 0 when none does.  Whatever the group arrays
// hold, the entries used (group_start[b], shared_lens[b]) are in range.
__device__ __forceinline__ int pair_tiles(const Rows &r, int b) {
    const int lead = __ldg(r.group_start + b), s = __ldg(r.shared_lens + b);
    const int next = b + 1 < r.num_reqs ? __ldg(r.group_start + b + 1) : -1;
    const bool starts = lead >= 0 && lead <= b && (b - lead) % r.pair_rows == 0 && (lead != b || next == b);
    return starts && s > 0 && s <= r.max_seq_len ? (s + kKeys - 1) / kKeys : 0;
}

__host__ __device__ __forceinline__ long long units_per_cta(long long units, long long ctas) {
    const long long share = (units + ctas - 1) / ctas;
    return share > kMinUnits ? share : kMinUnits;
}

// ------------------------------------------------------------- prefix kernel
constexpr int kStages = 2;                 // K tiles in flight
constexpr int kVStages = 3;                // V tiles in flight (V is needed later than K)
constexpr int kThreads = 384;              // 12 warps
constexpr uint32_t kHalf = 16384;          // 128 rows x 128 bytes (64 bf16)
constexpr uint32_t kTile = 2 * kHalf;      // 128 x 128 bf16
constexpr uint32_t kVBlock = 4096, kVHalf = 2048;   // V in blocks of 16 keys (see extend.cu)
constexpr int kMaxPairs = 64;              // pairs of one window of a CTA's units
constexpr int kBadRing = 8;                // segments the loaders can be ahead, rounded up

struct Pair {
    long long unit;                        // its first unit
    int32_t row, lead, shared, two;        // first row, group's first row, keys, second tile has rows
};

constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTile;
constexpr uint32_t kOffV = kOffK + kStages * kTile;
constexpr uint32_t kOffBar = kOffV + kVStages * kTile;
constexpr uint32_t kOffPairs = kOffBar + 256;
constexpr uint32_t kSmemBytes = kOffPairs + kMaxPairs * sizeof(Pair) + 1024;   // + slack to align the base
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

// barrier slots
constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kKEmpty = 4, kVFull = 6, kVEmpty = 9, kSFull = 12, kPFull = 14,
              kOFull = 16, kDrain = 18, kNumBars = 19;

struct PrefixArgs {
    PoolView pool;
    PageView pages;
    Rows rows;
    int32_t hq, group, rows_per_tile, q_box_rows, oob_row, box_rows, v_blocks;
    float scale_log2;
    float *o, *lse;            // [num_reqs, hq, 128], [num_reqs, hq]: pieces that begin at the first key
    float *cont_o, *cont_lse;  // [CTA, 2, 128, 128], [CTA, 2, 128]: a CTA's piece that begins later
    uint32_t *status;
};

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                              uint32_t *status) {
    if (ptx::mbar_wait(bar, parity)) return true;
    report(status, MSGL_DEVERR_TIMEOUT);
    *abort_flag = 1;
    return false;
}

// Exclusive prefix sum of v over the block; total gets the sum.  scratch: 12 entries.
__device__ __forceinline__ long long block_excl_scan(long long v, long long *scratch, long long &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    __syncthreads();
    return before + x - v;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap kt_map,
                     const __grid_constant__ CUtensorMap vt_map, const PrefixArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The grid may start before the split kernel in front of it has finished.  The last CTA
    // waits for that kernel, so this grid does not complete before it: what runs next sees
    // the partials of both.
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");

    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + kOffBar;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + kOffBar + 8 * kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 4);
    volatile int *num_pairs = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 8);
    volatile int *bad_seg = reinterpret_cast<volatile int *>(smem + kOffBar + 8 * kNumBars + 16);   // [kBadRing]
    Pair *pairs = reinterpret_cast<Pair *>(smem + kOffPairs);
    long long *scratch = reinterpret_cast<long long *>(pairs);   // of the block's scans, between windows

    // ---- this CTA's units: thread i counts rows [i * k, (i + 1) * k)
    const Rows &rows = a.rows;
    const int hkv = a.pool.hkv;
    const int per_thread = (rows.num_reqs + kThreads - 1) / kThreads;
    const int b0 = min(rows.num_reqs, (int)threadIdx.x * per_thread);
    const int b1 = min(rows.num_reqs, b0 + per_thread);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += pair_tiles(rows, b);
    long long units;
    const long long before = block_excl_scan(mine, scratch, units) * hkv;
    units *= hkv;
    const long long per = units_per_cta(units, gridDim.x);
    const long long u0 = per * blockIdx.x, u1 = min(units, u0 + per);
    if (u0 >= u1) return;

    const int R = a.rows_per_tile, G = a.group;
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
        ptx::mbar_init(bar(kDrain), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (threadIdx.x < kBadRing) bad_seg[threadIdx.x] = 0;
    if (warp == 2) {
        ptx::tc_alloc(ptx::smem_u32((const void *)tmem_slot), 512);
        ptx::tc_relinquish();
    }
    if (warp == 2 || warp == 3) {
        // zero the Q rows a TMA box does not cover (GQA padding rows)
        const int used = a.q_box_rows * G;
        const int pad_bytes = (kRows - used) * 128;
        for (int t = 0; t < 2; ++t)
            for (int h = 0; h < 2; ++h) {
                uint8_t *p = smem + kOffQ + t * kTile + h * kHalf + used * 128;
                for (int x = (threadIdx.x - 64) * 16; x < pad_bytes; x += 64 * 16)
                    *reinterpret_cast<uint4 *>(p + x) = make_uint4(0, 0, 0, 0);
            }
        ptx::fence_proxy_async_smem();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool lsu = a.box_rows == 0;

    // What every role counts the same way: segments (one pair, one kv head, a run of key
    // tiles) and K/V tiles done so far; tiles of each Q tile's S and P.
    uint32_t seg = 0, tile0 = 0, s_done0 = 0, s_done1 = 0, two_segs = 0;
    bool ok = true;

    // ---- windows: the pairs that the next units belong to, at most kMaxPairs at a time
    for (long long w0 = u0; w0 < u1;) {
        {
            // every pair that intersects [w0, u1), in order; its index is the count of such
            // pairs before it
            long long at = before;
            int n = 0;
            for (int b = b0; b < b1; ++b) {
                const long long here = (long long)pair_tiles(rows, b) * hkv;
                if (here > 0 && at + here > w0 && at < u1) ++n;
                at += here;
            }
            long long n_all;
            int idx = (int)block_excl_scan(n, scratch, n_all);
            at = before;
            for (int b = b0; b < b1 && n > 0 && idx < kMaxPairs; ++b) {
                const long long here = (long long)pair_tiles(rows, b) * hkv;
                if (here > 0 && at + here > w0 && at < u1 && idx < kMaxPairs) {
                    Pair p;
                    p.unit = at;
                    p.row = b;
                    p.lead = __ldg(rows.group_start + b);
                    p.shared = __ldg(rows.shared_lens + b);
                    p.two = b + R < rows.num_reqs && __ldg(rows.group_start + b + R) == p.lead;
                    pairs[idx++] = p;
                }
                at += here;
            }
            if (threadIdx.x == 0) *num_pairs = (int)min(n_all, (long long)kMaxPairs);
            __syncthreads();
        }
        const int np = *num_pairs;
        if (np == 0) break;   // (the lengths changed under the call)
        const Pair last = pairs[np - 1];
        const long long w1 = min(u1, last.unit + (long long)((last.shared + kKeys - 1) / kKeys) * hkv);

        // One segment: pair e, kv head g, key tiles [t0, t0 + n).
        int e = 0;
        for (long long u = w0; u < w1 && ok;) {
            const Pair p = pairs[e];
            const int nkt = (p.shared + kKeys - 1) / kKeys;
            const long long off = u - p.unit;
            const int g = (int)(off / nkt);
            const int t0 = (int)(off - (long long)g * nkt);
            const int n = (int)min((long long)(nkt - t0), w1 - u);
            const bool two = p.two != 0;

            if (warp == 0 || warp == 3 || (lsu && warp == 2)) {
                // -------------------------------------------------------- K/V loaders
                const bool is_v = warp == 3;
                if (warp == 0) {
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
                // Pool rows of tile j's keys, four consecutive keys per lane.  A key past the
                // shared ones or behind a bad page id gets oob_row (zero fill).
                auto key_rows = [&](int j, int (&kr)[4], bool &all_ok, int64_t &slot0) {
                    all_ok = true;
                    slot0 = 0;
                    bool bad = false;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = (t0 + j) * kKeys + 4 * lane + x;
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
                    // 16-byte cp.async copies into the SWIZZLE_128B K-major layout (see extend.cu);
                    // warp 0 copies the even K tiles (counted over the segments), warp 2 the odd
                    const __nv_bfloat16 *pool = is_v ? a.pool.v : a.pool.k;
                    const int step = is_v ? 1 : 2;
                    const int first = is_v ? 0 : (int)((tile0 ^ (warp == 2 ? 1u : 0u)) & 1u);
                    const int hi = lane >> 4, c = lane & 15;
                    const uint32_t col_off = (uint32_t)(c >> 3) * kHalf;
                    int next[4] = {0, 0, 0, 0};
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
#pragma unroll
                        for (int i = 0; i < 64; ++i) {
                            const int e0 = (i & 1) * 2;
                            const int r0 = __shfl_sync(0xffffffffu, kr[e0], i >> 1);
                            const int r1 = __shfl_sync(0xffffffffu, kr[e0 + 1], i >> 1);
                            const int row = hi ? r1 : r0;
                            const int r = 2 * i + hi;
                            const bool valid = row < a.oob_row;
                            ptx::cp_async_16(dst + col_off + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4),
                                             pool + (valid ? (int64_t)row * kHeadDim + c * 8 : 0), valid ? 16u : 0u);
                        }
                        ptx::cp_async_commit();
                        if (j + step < n) key_rows(j + step, next, all_ok, slot0);
                        ptx::cp_async_wait_all();
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar((is_v ? kVFull : kKFull) + st));
#pragma unroll
                        for (int x = 0; x < 4; ++x) kr[x] = next[x];
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
                                    ptx::tma_load_5d(dst + (uint32_t)x * 2u * kVBlock, tm, 0, g, (int)slot0 + 32 * x, 0,
                                                     0, full);
                            } else {
                                ptx::tma_load_3d(dst, tm, 0, g, (int)slot0, full);
                                ptx::tma_load_3d(dst + kHalf, tm, 64, g, (int)slot0, full);
                            }
                        }
                    }
                }
            } else if (warp == 1) {
                // -------------------------------------------------------- MMA issuer
                if (lane == 0) {
                    constexpr uint32_t idesc_s = ptx::umma_idesc_bf16(128, 128, false, false);
                    constexpr uint32_t idesc_o = ptx::umma_idesc_bf16(128, 128, false, true);
                    const uint64_t qdesc = ptx::umma_desc_sw128(sbase + kOffQ, 16, 1024);
                    const uint64_t kdesc = ptx::umma_desc_sw128(sbase + kOffK, 16, 1024);
                    const uint64_t vdesc = ptx::umma_desc_sw128(sbase + kOffV, a.v_blocks ? kVHalf : kHalf, 1024);
                    const uint32_t vstep = (a.v_blocks ? kVBlock : 16u * 128u) >> 4;   // MMA kk's 16 keys
                    // Each group tests the next one's barrier after its 4th MMA, so that the test's
                    // latency hides behind the MMAs still queued (see extend.cu).
                    auto s_group = [&](int t, uint32_t gi, uint32_t pb, uint32_t pp) -> bool {
                        const uint64_t qd = qdesc + (uint64_t)(t * (kTile >> 4));
                        const uint64_t kd = kdesc + (uint64_t)((gi % kStages) * (kTile >> 4));
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
                    auto pv_group = [&](int t, uint32_t gi, bool acc, uint32_t pb, uint32_t pp) -> bool {
                        const uint64_t vd = vdesc + (uint64_t)((gi % kVStages) * (kTile >> 4));
                        bool r = false;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            ptx::tc_mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + kk * 8, vd + (uint64_t)(kk * vstep),
                                           idesc_o, (acc || kk > 0) ? 1u : 0u);
                            if (kk == 3 && pb) r = ptx::mbar_test_wait(pb, pp);
                        }
                        return r;
                    };
                    auto need = [&](bool tested, uint32_t b, uint32_t parity) -> bool {
                        if (!ok) return false;
                        if (!tested && !wait_or_abort(b, parity, abort_flag, a.status)) ok = false;
                        ptx::tc_fence_after();
                        return ok;
                    };
                    // Order per K/V tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
                    bool v_ok = false;
                    need(false, bar(kQFull), seg & 1);
                    if (need(false, bar(kKFull + tile0 % kStages), (tile0 / kStages) & 1)) {
                        s_group(0, tile0, 0, 0);
                        if (two) s_group(1, tile0, 0, 0);
                    }
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t gi = tile0 + j, gn = gi + 1;
                        const bool more = j + 1 < n;
                        if (!need(v_ok, bar(kVFull + gi % kVStages), (gi / kVStages) & 1)) break;
                        if (!need(false, bar(kPFull + 0), (s_done0 + j) & 1)) break;
                        const uint32_t kb = bar(kKFull + gn % kStages), kp = (gn / kStages) & 1;
                        const bool k_ok = pv_group(0, gi, j > 0, more ? kb : 0u, kp);
                        if (!more) ptx::tc_commit(bar(kOFull + 0));
                        bool p_ok = false;
                        v_ok = false;
                        const uint32_t vb = more ? bar(kVFull + gn % kVStages) : 0u, vp = (gn / kVStages) & 1;
                        const uint32_t pb = bar(kPFull + 1), pp = (s_done1 + j) & 1;
                        if (more) {
                            if (!need(k_ok, kb, kp)) break;
                            const bool r = s_group(0, gn, two ? pb : vb, two ? pp : vp);
                            if (two) p_ok = r;
                            else v_ok = r;
                        }
                        if (two) {
                            if (!need(p_ok, pb, pp)) break;
                            pv_group(1, gi, j > 0, 0, 0);
                            if (!more) ptx::tc_commit(bar(kOFull + 1));
                            else v_ok = s_group(1, gn, vb, vp);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
            } else if (warp >= 4) {
                // -------------------------------------------------------- softmax
                const int t = (warp - 4) >> 2;                 // Q tile of this warpgroup
                if (t == 0 || two) {
                    const int quad = warp & 3;
                    const int r = quad * 32 + lane;            // TMEM lane = tile row
                    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
                    const uint32_t tS = tmem + lane_base + 128 * t;
                    const uint32_t tO = tmem + lane_base + 256 + 128 * t;
                    const uint32_t s_done = t ? s_done1 : s_done0;
                    float m_ref = -INFINITY, l = 0.f;
                    // The K/V stages are released from here: the last tile's S(j) done means every
                    // MMA issued before it is, so K(j) and V(j-1) are free (see extend.cu).
                    const bool releaser = lane == 0 && warp == (two ? 8 : 4);
                    for (int j = 0; j < n; ++j) {
                        const uint32_t gi = tile0 + j;
                        ok = __all_sync(0xffffffffu,
                                        wait_or_abort(bar(kSFull + t), (s_done + j) & 1, abort_flag, a.status));
                        if (!ok) break;
                        ptx::tc_fence_after();
                        if (releaser) {
                            ptx::mbar_arrive(bar(kKEmpty + gi % kStages));
                            if (j > 0) ptx::mbar_arrive(bar(kVEmpty + (gi - 1) % kVStages));
                            if (j == n - 1) ptx::mbar_arrive(bar(kQEmpty));
                        }
                        uint32_t v[128];
                        ptx::tc_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(v + 0));
                        ptx::tc_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                        ptx::tc_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(v + 64));
                        ptx::tc_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(v + 96));
                        ptx::tc_wait_ld();
                        const int visible = p.shared - (t0 + j) * kKeys;   // keys of this tile that exist
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
                        // The first tile's row max is the reference; it moves only when a row sum shows
                        // a score 2^8 above it (every p stays below 2^8; see extend.cu).
                        if (j == 0) m_ref = fmaxf(m_ref, row_max());
                        float ls = 0.f;
#pragma unroll 1
                        for (int pass = 0;; ++pass) {
                            // P = 2^(s * scale_log2 - m_ref) (masked scores are -inf -> 0), back over S
                            // as bf16: a relative rounding of 2^-9 of each weight, while the row sum takes
                            // the unrounded ones
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
                            if (pass == 1 || j == 0 || __all_sync(0xffffffffu, ls < 256.f)) break;
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
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(kPFull + t));
                    }
                    // this piece's o / l and lse, fp32
                    const uint32_t o_parity = (t ? two_segs : seg) & 1;
                    if (ok)
                        ok = __all_sync(0xffffffffu, wait_or_abort(bar(kOFull + t), o_parity, abort_flag, a.status));
                    if (ok) {
                        ptx::tc_fence_after();
                        if (releaser) ptx::mbar_arrive(bar(kVEmpty + (tile0 + n - 1) % kVStages));
                        const int tok_l = r / G, jh = r - tok_l * G;
                        const int tok = p.row + t * R + tok_l;
                        const bool store = tok_l < R && tok < rows.num_reqs && __ldg(rows.group_start + tok) == p.lead;
                        const bool bad = bad_seg[seg % kBadRing] == (int)seg + 1;
                        const float inv = l > 0.f ? 1.f / l : 0.f;
                        const long long at = t0 == 0 ? (long long)tok * a.hq + g * G + jh
                                                     : ((long long)blockIdx.x * 2 + t) * kRows + r;
                        float *dst = (t0 == 0 ? a.o : a.cont_o) + at * kHeadDim;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o32[32];
                            ptx::tc_ld32(tO + 32 * c, o32);
                            ptx::tc_wait_ld();
                            if (store) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o32[i] = __float_as_uint(__uint_as_float(o32[i]) * inv);
#pragma unroll
                                for (int i = 0; i < 4; ++i) ptx::st_v8(dst + 32 * c + 8 * i, o32 + 8 * i);
                            }
                        }
                        // NaN marks a piece that met a bad page
                        if (store)
                            (t0 == 0 ? a.lse : a.cont_lse)[at] =
                                bad || !(l > 0.f) ? __int_as_float(0x7fc00000) : (m_ref + log2f(l)) * kLn2;
                        if (bad && t == 0 && threadIdx.x == 128) report(a.status, MSGL_DEVERR_PAGE_RANGE);
                        ptx::tc_fence_before();
                    }
                }
            }
            s_done0 += n;
            if (two) {
                s_done1 += n;
                ++two_segs;
            }
            tile0 += n;
            ++seg;
            u += n;
            if (u - p.unit == (long long)nkt * hkv) ++e;
        }
        w0 = w1;
        if (__syncthreads_or(!ok)) break;
    }

    if (warp == 1 && lane == 0) {
        // every MMA issued above has completed once this fires
        ptx::tc_commit(bar(kDrain));
        ptx::mbar_wait(bar(kDrain), 0, 400000000LL);
    }
    if (*abort_flag) {
        // Let issued copies land before shared memory goes away: each loader waits, with a
        // limit, for the full barriers of the stages it may have filled last.
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
// One warp per (request, q head), its pieces found by the same arithmetic that gave them
// out; a request's two sums (own keys, units of the rows before it) are taken by its block.

constexpr int kMergeThreads = 256;
constexpr int kMaxDecodeCtas = 512;
constexpr int kMaxPieces = kMaxPrefixCtas + 1 + kMaxDecodeCtas + 1;

struct MergeArgs {
    Rows rows;
    int32_t hq, hkv, rows_per_tile, split_ctas, prefix_ctas;
    const float *part_o, *part_lse;          // own keys: row b + CTA
    const float *pre_o, *pre_lse, *cont_o, *cont_lse;
    __nv_bfloat16 *o;
    float *lse;
    uint32_t *status;
};

// The rules of group_start and shared_lens for row b, and that its pair was worked on.
__device__ __forceinline__ uint32_t row_errors(const Rows &r, int rows_per_tile, int b, int &seq, int &start, int &pair) {
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
    pair = lead + (b - lead) / r.pair_rows * r.pair_rows;
    if (__ldg(r.group_start + pair) != lead || __ldg(r.shared_lens + pair) != s || pair_tiles(r, pair) == 0)
        return MSGL_DEVERR_GROUP;
    if (b - pair >= rows_per_tile && __ldg(r.group_start + pair + rows_per_tile) != lead) return MSGL_DEVERR_GROUP;
    return 0;
}

__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const MergeArgs a) {
    __shared__ long long s_part[kMergeThreads / 32][4];
    __shared__ float s_w[kMergeThreads / 32][kMaxPieces];
    const Rows &rows = a.rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    int seq, start, pair;
    const uint32_t err = row_errors(rows, a.rows_per_tile, b, seq, start, pair);
    // own keys of all rows and of those before b; K/V tiles of all pairs and of those before b's
    long long sums[4] = {0, 0, 0, 0};
    for (int i = threadIdx.x; i < rows.num_reqs; i += kMergeThreads) {
        int first;
        const int own = own_keys_shared(rows.seq_lens, rows.group_start, rows.shared_lens, rows.num_reqs,
                                        rows.max_seq_len, i, first);
        const int tiles = pair_tiles(rows, i);
        sums[0] += own;
        sums[2] += tiles;
        if (i < b) sums[1] += own;
        if (i < pair) sums[3] += tiles;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sums[k] += __shfl_xor_sync(0xffffffffu, sums[k], o);
        if (lane == 0) s_part[warp][k] = sums[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        sums[k] = 0;
#pragma unroll
        for (int w = 0; w < kMergeThreads / 32; ++w) sums[k] += s_part[w][k];
    }
    const int h = blockIdx.x * (kMergeThreads / 32) + warp;
    if (h >= a.hq) return;
    const long long row = (long long)b * a.hq + h;
    __nv_bfloat16 *orow = a.o + row * kHeadDim + lane * 4;
    // the pieces are complete and visible after this point (and the caller's outputs free to write)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (err) {
        if (h == 0 && lane == 0) report(a.status, err);
        *reinterpret_cast<uint2 *>(orow) = make_uint2(0u, 0u);
        if (lane == 0) a.lse[row] = -INFINITY;
        return;
    }
    // prefix pieces: the first where the item begins, then one per CTA that continues it
    int np = 0;
    long long cta0 = 0, cont_row = 0;
    if (pair >= 0) {
        const int G = a.hq / a.hkv, g = h / G;
        const int tiles = (start + kKeys - 1) / kKeys;
        const long long per = units_per_cta(sums[2] * a.hkv, a.prefix_ctas);
        const long long u = sums[3] * a.hkv + (long long)g * tiles;
        cta0 = u / per;
        np = (int)((u + tiles - 1) / per - cta0) + 1;
        const int i = b - pair, t = i / a.rows_per_tile;
        cont_row = t * kRows + (i - t * a.rows_per_tile) * G + (h - g * G);
    }
    // own pieces: one per split CTA whose range touches the row's own keys
    int ns = 0;
    long long split0 = 0;
    if (seq > start) {
        const long long per = keys_per_cta(sums[0], a.split_ctas);
        split0 = sums[1] / per;
        ns = (int)((sums[1] + (seq - start) - 1) / per - split0) + 1;
    }
    const int n = np + ns;
    auto at = [&](int i, const float *&o, const float *&l) {
        if (i >= np) {
            const long long x = (b + split0 + (i - np)) * a.hq + h;
            o = a.part_o + x * kHeadDim;
            l = a.part_lse + x;
        } else if (i == 0) {
            o = a.pre_o + row * kHeadDim;
            l = a.pre_lse + row;
        } else {
            const long long x = (cta0 + i) * 2 * kRows + cont_row;
            o = a.cont_o + x * kHeadDim;
            l = a.cont_lse + x;
        }
    };
    float M = -INFINITY;
    bool failed = false;
    for (int i = lane; i < n; i += 32) {
        const float *o, *l;
        at(i, o, l);
        const float x = *l;
        s_w[warp][i] = x;
        failed |= isnan(x);
        M = fmaxf(M, x);
    }
    failed = __any_sync(0xffffffffu, failed);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const bool none = failed || M == -INFINITY;
    float L = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float w = none ? 0.f : expf(s_w[warp][i] - M);
        s_w[warp][i] = w;
        L += w;
    }
    L = warp_sum(L);
    __syncwarp();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (!none) {
        for (int i0 = 0; i0 < n; i0 += 4) {
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *o, *l;
                at(min(i0 + k, n - 1), o, l);
                v[k] = *reinterpret_cast<const float4 *>(o + lane * 4);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float w = i0 + k < n ? s_w[warp][i0 + k] : 0.f;
                acc[0] += w * v[k].x;
                acc[1] += w * v[k].y;
                acc[2] += w * v[k].z;
                acc[3] += w * v[k].w;
            }
        }
    }
    const float inv = none ? 0.f : 1.f / L;
    *reinterpret_cast<uint2 *>(orow) =
        make_uint2(ptx::pack_bf16(acc[0] * inv, acc[1] * inv), ptx::pack_bf16(acc[2] * inv, acc[3] * inv));
    if (lane == 0) a.lse[row] = none ? -INFINITY : M + logf(L);
}

// Where each part of the workspace begins.
struct Layout {
    size_t pre_o, pre_lse, cont_o, cont_lse, total;
};

Layout layout_of(int32_t num_reqs, int32_t hq, int32_t hkv) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)num_reqs * hq, cont = (size_t)kMaxPrefixCtas * 2 * kRows;
    Layout l;
    l.pre_o = plan_decode(num_reqs, hq, hkv, 1).workspace;
    l.pre_lse = l.pre_o + rows * kHeadDim * sizeof(float);
    l.cont_o = up(l.pre_lse + rows * sizeof(float));
    l.cont_lse = l.cont_o + cont * kHeadDim * sizeof(float);
    l.total = up(l.cont_lse + cont * sizeof(float));
    return l;
}

}  // namespace

size_t decode_shared_workspace_bytes(int32_t num_reqs, int32_t hq, int32_t hkv) {
    return layout_of(num_reqs, hq, hkv).total;
}

cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream) {
    const DecodeArgs &d = a.dec;
    const int hkv = d.pool.hkv, G = d.hq / hkv, R = kRows / G;
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
    e = launch_decode(d, plan_decode(d.num_reqs, d.hq, hkv, d.max_seq_len), stream, DecodePhase::kSplit);
    if (e != cudaSuccess) return e;

    PrefixArgs p{};
    p.pool = d.pool;
    p.pages = d.pages;
    p.rows = Rows{d.seq_lens, d.group_start, d.shared_lens, d.num_reqs, d.max_seq_len, 2 * R};
    p.hq = d.hq;
    p.group = G;
    p.rows_per_tile = R;
    p.q_box_rows = m.q_box_rows;
    p.oob_row = m.oob_row;
    p.box_rows = m.box_rows;
    p.v_blocks = m.v_blocks;
    p.scale_log2 = d.scale * kLog2e;
    p.o = reinterpret_cast<float *>(ws + l.pre_o);
    p.lse = reinterpret_cast<float *>(ws + l.pre_lse);
    p.cont_o = reinterpret_cast<float *>(ws + l.cont_o);
    p.cont_lse = reinterpret_cast<float *>(ws + l.cont_lse);
    p.status = d.status;
    const int ctas = sm_count() < kMaxPrefixCtas ? sm_count() : kMaxPrefixCtas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    e = cudaLaunchKernelEx(&cfg, prefix_tc_kernel, m.q, m.k, m.v, m.kt, m.vt, p);
    if (e != cudaSuccess) return e;

    MergeArgs g{};
    g.rows = p.rows;
    g.hq = d.hq;
    g.hkv = hkv;
    g.rows_per_tile = R;
    g.split_ctas = decode_split_ctas(d.hq, hkv);
    g.prefix_ctas = ctas;
    g.part_o = d.part_o;
    g.part_lse = d.part_lse;
    g.pre_o = p.o;
    g.pre_lse = p.lse;
    g.cont_o = p.cont_o;
    g.cont_lse = p.cont_lse;
    g.o = d.o;
    g.lse = d.lse;
    g.status = d.status;
    cfg.gridDim = dim3((d.hq + kMergeThreads / 32 - 1) / (kMergeThreads / 32), d.num_reqs);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, shared_merge_kernel, g);
}

}  // namespace msgl
